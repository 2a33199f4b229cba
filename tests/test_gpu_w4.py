"""moe_w4_matvec against its 64-bit form: every group size, zero points and
none, partial groups and chunks, more groups than one table holds, one row to
several passes, SwiGLU, segments and pairs as the layer makes them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref
from tests.test_gpu_grouped_mm import DT, _put, _segments

pytestmark = pytest.mark.gpu

SHAPES = {
    # T, k, E, N, K; no offsets where E = 1 and dense is set
    "smallest": dict(T=1, k=1, E=1, N=2, K=32, dense=True),
    "one_token": dict(T=1, k=4, E=16, N=70, K=96, empty=tuple(range(0, 12))),
    "one_token_wide": dict(T=1, k=2, E=3, N=34, K=2880, empty=(1,)),
    "dense_rows": dict(T=13, k=1, E=1, N=130, K=352, dense=True),
    "dense_64": dict(T=64, k=1, E=1, N=96, K=512, dense=True),
    "decode": dict(T=16, k=4, E=32, N=64, K=320, empty=(3, 4, 30)),
    "several_passes": dict(T=40, k=2, E=20, N=48, K=288, empty=tuple(range(2, 20))),
    "long_rows": dict(T=3, k=1, E=2, N=32, K=9248),
    "rows_outside": dict(T=9, k=2, E=3, N=40, K=160, lead=3, behind=4),
    "bad_pairs": dict(T=12, k=2, E=3, N=40, K=160, bad=True),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_w4(name, group, dtype):
    print(f"w4 {name} group {group} {dtype}", flush=True)
    c = dict(SHAPES[name])
    T, k, E, N, K = (c[x] for x in "TkENK")
    M, G, dt = T * k, -(-K // group), DT[dtype]
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    x = torch.randn(T, K, generator=g).to(dt)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand(E, N, G, generator=g) * 0.05 + 0.001).to(dt)
    zeros = torch.randint(0, 16, (E, N, G), generator=g, dtype=torch.uint8)
    bias = torch.randn(E, N, generator=g).to(dt)
    off = None if c.get("dense") else torch.from_numpy(_segments(rng, M, E, c.get("empty", ()), c.get("lead", 0), c.get("behind", 0)))
    pairs = None if c.get("dense") else torch.from_numpy(rng.permutation(M).astype(np.int32))
    if c.get("bad"):
        pairs[2], pairs[9] = M, -1
    for swiglu, z, use_bias, out in ((False, zeros, True, dtype), (False, None, False, "f32"), (True, zeros, True, dtype),
                                     (True, None, False, "f32")):
        cols = N // 2 if swiglu else N
        y = torch.full((M, cols), 7.0, dtype=DT[out], device="cuda")
        d = moe.w4(M, N, K, E, T=T, k=k, group=group, dtype=moe.DTYPE[dt], out_dtype=moe.DTYPE[DT[out]],
                   act=moe.MOE_ACT_SWIGLU if swiglu else moe.MOE_ACT_NONE)
        moe.moe_w4_matvec(d, _put(x), _put(off), _put(pairs), _put(codes), _put(scales), _put(z),
                          _put(bias) if use_bias else None, y)
        torch.cuda.synchronize()
        want, bound, inside = ref.w4_product(x, off if off is not None else [0, M], pairs, k, codes, scales, z,
                                             bias if use_bias else None, group, swiglu, DT[out], M)
        y = y.cpu()
        ref.assert_within(y[inside], want[inside], bound[inside], f"{name} group {group} swiglu {swiglu} {dtype}->{out}")
        assert (y[~inside] == 7).all()


def test_every_code_and_zero_is_exact():
    """x picks one column at a time: y is scale * (code - zero) itself."""
    K, N = 64, 256
    x = torch.zeros(K, K, dtype=torch.bfloat16)
    x[torch.arange(K), torch.arange(K)] = 1
    n, i = torch.arange(N)[:, None], torch.arange(K)[None]
    code = ((n + 3 * i) % 16).to(torch.uint8)
    zero = (n // 16 % 16).expand(N, 2).to(torch.uint8)
    codes = (code[:, 0::2] | code[:, 1::2] << 4).contiguous()
    scales = torch.full((N, 2), 0.375, dtype=torch.bfloat16)
    y = torch.empty(K, N, dtype=torch.float32, device="cuda")
    d = moe.w4(K, N, K, 1, group=32, out_dtype=moe.MOE_DT_F32)
    moe.moe_w4_matvec(d, _put(x), None, None, _put(codes), _put(scales), _put(zero.contiguous()), None, y)
    torch.cuda.synchronize()
    want = 0.375 * (code.double() - zero[:, :1].double())
    assert torch.equal(y.cpu().double(), want.t())


def test_nan_row_stays_alone():
    M, N, K = 9, 48, 160
    g = torch.Generator().manual_seed(6)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    x[4, 77] = float("inf")
    codes = torch.randint(0, 256, (1, N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.ones(1, N, 5, dtype=torch.bfloat16)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_matvec(moe.w4(M, N, K, 1, group=32), _put(x), None, None, _put(codes), _put(scales), None, None, y)
    torch.cuda.synchronize()
    fine = torch.isfinite(y.cpu())
    assert fine[torch.arange(M) != 4].all() and not fine[4].all()
