"""moe_w4_matvec where a wave streams items of its own (thousands of 32-row
pieces of weights): every count of rows per item, group size, even and odd counts
of column chunks, partial groups, empty experts, rows outside the segments."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref
from tests.test_gpu_grouped_mm import DT, _put, _segments

pytestmark = pytest.mark.gpu

E, N = 6, 8210  # 257 pieces of 32 rows, the last one short


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,dtype", [(5, 608, "bf16"), (5, 352, "f16"), (12, 608, "bf16"), (12, 96, "bf16"), (30, 608, "f16"),
                                      (30, 1312, "bf16")])
def test_streaming(T, K, dtype, group):
    print(f"w4 streaming T {T} K {K} group {group} {dtype}", flush=True)
    k, dt = 2, DT[dtype]
    M, G = T * k, -(-K // group)
    rng, g = np.random.default_rng(9), torch.Generator().manual_seed(9)
    x = torch.randn(T, K, generator=g).to(dt)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand(E, N, G, generator=g) * 0.05 + 0.001).to(dt)
    zeros = torch.randint(0, 16, (E, N, G), generator=g, dtype=torch.uint8)
    bias = torch.randn(E, N, generator=g).to(dt)
    off = torch.from_numpy(_segments(rng, M, E, (1,), 1, 2))
    pairs = torch.from_numpy(rng.permutation(M).astype(np.int32))
    pairs[3] = -1
    for swiglu, z in ((False, zeros), (False, None), (True, zeros), (True, None)):
        cols = N // 2 if swiglu else N
        y = torch.full((M, cols), 7.0, dtype=dt, device="cuda")
        d = moe.w4(M, N, K, E, T=T, k=k, group=group, dtype=moe.DTYPE[dt],
                   act=moe.MOE_ACT_SWIGLU if swiglu else moe.MOE_ACT_NONE)
        args = (d, _put(x), _put(off), _put(pairs), _put(codes), _put(scales), _put(z), _put(bias))
        moe.moe_w4_matvec(*args, y)
        again = torch.full_like(y, 7.0)
        moe.moe_w4_matvec(*args, again)
        torch.cuda.synchronize()
        want, bound, inside = ref.w4_product(x, off, pairs, k, codes, scales, z, bias, group, swiglu, dt, M)
        assert torch.equal(y, again)
        y = y.cpu()
        ref.assert_within(y[inside], want[inside], bound[inside], f"swiglu {swiglu} zeros {z is not None}")
        assert (y[~inside] == 7).all()
