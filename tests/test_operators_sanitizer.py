"""The entry points of the stand-alone operators, built as host code with
AddressSanitizer and UndefinedBehaviorSanitizer and driven with extreme
descriptors: no overflow on the way to a refusal, nothing launched by a rejected
call, nothing outside the documented limits handed to a launcher."""
from __future__ import annotations

import os

import pytest

import mixture_experts_ffn_05_amd as moe
from tests.test_sanitizers import ENV, ROOT, SAN, _run, pytestmark  # noqa: F401


def test_operator_validation_under_sanitizers(tmp_path):
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("HIP headers not installed")
    csrc = os.path.join(ROOT, "mixture_experts_ffn_05_amd/csrc")
    inc = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + csrc, "-I" + os.path.join(ROOT, "include")]
    objs = []
    for src in (os.path.join(csrc, "ops_api.hip"), os.path.join(ROOT, "tests/sanitize/operators_driver.cpp")):
        o = str(tmp_path / (os.path.basename(src) + ".o"))
        _run(["g++", "-std=c++17", *SAN, *inc, "-c", "-x", "c++", src, "-o", o])
        objs.append(o)
    exe = str(tmp_path / "operators_asan")
    _run(["g++", *SAN, *objs, "-o", exe])
    assert _run([exe], env=ENV).strip() == "ok"


def test_items_of_a_4_bit_product_are_counted_in_32_bits():
    """Sizes whose work items could pass 32 bits are refused before a launch."""
    many = moe.w4(1 << 22, 1 << 16, 32, 256, group=32)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_w4_matvec(many, 4096, 4096, None, 4096, 4096, None, None, 4096, 0)
    assert e.value.code == moe.MOE_ERR_UNSUPPORTED
