"""Offsets that pass 32 bits: more than 2^31 elements of weights, of rows and of
gradients, 2^32 bytes of 4-bit codes.  Parts near the end are compared with
their 64-bit forms."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _randn(*shape, seed=1, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF) * scale


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [1, 3])
def test_weights(rows):
    """rows 1: only three experts have rows (the decode form); 3: all of them."""
    E, N, K = 130, 4096, 4224
    print(f"weights of {E * N * K} elements, {rows} rows an expert", flush=True)
    b = _randn(E, N, K, scale=0.1)
    assert b.numel() > 1 << 31
    used = [0, 127, 129] if rows == 1 else list(range(E))
    count = [rows if e in used else 0 for e in range(E)]
    off = torch.tensor([0] + count, dtype=torch.int32).cumsum(0).to(torch.int32)
    M = int(off[-1])
    a, dc = _randn(M, K, seed=2), _randn(M, N, seed=3)
    y, da = torch.zeros(M, N, dtype=BF, device="cuda"), torch.zeros(M, K, dtype=BF, device="cuda")
    g = moe.gmm(M, N, K, E)
    moe.moe_grouped_mm(g, a, off.cuda(), None, b, None, y)
    moe.moe_grouped_mm_dgrad(g, dc, off.cuda(), b, da)
    torch.cuda.synchronize()
    ac, dcc, y, da = a.cpu(), dc.cpu(), y.cpu(), da.cpu()
    for e in (0, 127, 129):
        lo, hi = int(off[e]), int(off[e + 1])
        w = b[e:e + 1].cpu()
        want, bound, _ = ref.product(ac[lo:hi], [0, hi - lo], None, 1, w, None, BF, hi - lo)
        ref.assert_within(y[lo:hi], want, bound, f"forward of expert {e}")
        want, bound, _ = ref.product_dgrad(dcc[lo:hi], [0, hi - lo], w, BF, hi - lo)
        ref.assert_within(da[lo:hi], want, bound, f"data gradient of expert {e}")
    del b
    d = moe.gmm(M, N, K, E, out_dtype=moe.MOE_DT_F32)
    n = moe.moe_grouped_mm_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    db, dbias = torch.full((E, N, K), 7.0, device="cuda"), torch.empty(E, N, device="cuda")
    moe.moe_grouped_mm_wgrad(d, a, off.cuda(), None, dc, db, dbias, ws, n)
    torch.cuda.synchronize()
    for e in (0, 126, 127, 129):
        lo, hi = int(off[e]), int(off[e + 1])
        want, bound, wb, bb = ref.product_wgrad(ac[lo:hi], [0, hi - lo], None, 1, dcc[lo:hi], 1, torch.float32, hi - lo)
        ref.assert_within(db[e], want[0], bound[0], f"weight gradient of expert {e}")
        ref.assert_within(dbias[e], wb[0], bb[0], f"bias gradient of expert {e}")


def test_rows_of_products():
    T, N, K = 1_050_000, 64, 2056
    print(f"{T * K} elements of rows", flush=True)
    a, b, dc = _randn(T, K), _randn(1, N, K, seed=2, scale=0.1), _randn(T, N, seed=3)
    assert a.numel() > 1 << 31
    g = moe.gmm(T, N, K, 1)
    y = torch.empty(T, N, dtype=BF, device="cuda")
    moe.moe_grouped_mm(g, a, None, None, b, None, y)
    part = slice(T - 70, T)
    torch.cuda.synchronize()
    want, bound, _ = ref.product(a[part].cpu(), [0, 70], None, 1, b.cpu(), None, BF, 70)
    ref.assert_within(y[part], want, bound, "forward")
    d = moe.gmm(T, N, K, 1, out_dtype=moe.MOE_DT_F32)
    n = moe.moe_grouped_mm_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    db = torch.empty(1, N, K, device="cuda")
    moe.moe_grouped_mm_wgrad(d, a, None, None, dc, db, None, ws, n)
    v, s = torch.zeros(N, K, dtype=torch.float64, device="cuda"), torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for r in range(0, T, 50_000):
        p, q = dc[r:r + 50_000].double().t().contiguous(), a[r:r + 50_000].double()
        v += p @ q
        s += p.abs() @ q.abs()
    torch.cuda.synchronize()
    # the rows' sum in at most 64 ranges, one rounding a product and a partial sum
    ref.assert_within(db[0], v.cpu(), (T + 70) * 2 * ref.U * s.cpu() + ref.U * v.abs().cpu(), "weight gradient")
    del y
    da = torch.empty(T, K, dtype=BF, device="cuda")
    moe.moe_grouped_mm_dgrad(g, dc, None, b, da)
    torch.cuda.synchronize()
    want, bound, _ = ref.product_dgrad(dc[part].cpu(), [0, 70], b.cpu(), BF, 70)
    ref.assert_within(da[part], want, bound, "data gradient")


def test_rows_of_norms():
    T, H = 1_050_000, 2056
    print(f"norms over {T * H} elements", flush=True)
    x, dy, w = _randn(T, H), _randn(T, H, seed=2), _randn(H, seed=3).float()
    d = moe.norm(T, H, moe.MOE_DT_BF16, moe.MOE_DT_F32, moe.MOE_NORM_RMS, 1e-5)
    y, dx, o = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(3))
    n = moe.moe_norm_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dw = torch.empty(H, device="cuda")
    moe.moe_norm_in(d, x, w, None, y)
    moe.moe_norm_out(d, x, dy, w, None, None, None, o)
    moe.moe_norm_in_backward(d, x, w, dy, None, dx, dw, None, ws, n)
    torch.cuda.synchronize()
    for part in (slice(0, 5), slice(T - 9, T)):
        xc, dc, eps = x[part].cpu(), dy[part].cpu(), float(d.eps)
        want, bound, _ = ref.norm_in(xc, w.cpu(), None, "rms", eps, BF)
        ref.assert_within(y[part], want, bound, "norm_in")
        keep = torch.ones(xc.shape, dtype=torch.bool)
        want, bound = ref.norm_out(xc, dc, w.cpu(), None, None, keep, 1.0, 1.0, "rms", eps, BF)
        ref.assert_within(o[part], want, bound, "norm_out")
        gx, ex, *_ = ref.norm_grads(xc, w.cpu(), None, dc.double(), torch.zeros(xc.shape, dtype=torch.float64), "rms", eps, BF)
        ref.assert_within(dx[part], gx, 1.01 * (ex + ref.half_step(BF) * gx.abs() + ref.floor_of(BF)), "norm_in backward")


def test_codes():
    E, N, K, group = 130, 8192, 8192, 64
    print(f"{E * N * K // 2} bytes of codes", flush=True)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 32
    scales = (torch.rand(E, N, K // group, device="cuda") * 0.01).to(BF)
    zeros = torch.randint(0, 16, (E, N, K // group), dtype=torch.uint8, device="cuda")
    count = [0] * E
    count[0], count[127], count[129] = 2, 1, 3
    off = torch.tensor([0] + count, dtype=torch.int32).cumsum(0).to(torch.int32)
    x = _randn(6, K)
    y = torch.empty(6, N, dtype=BF, device="cuda")
    moe.moe_w4_matvec(moe.w4(6, N, K, E, group=group), x, off.cuda(), None, codes, scales, zeros, None, y)
    torch.cuda.synchronize()
    xc, y = x.cpu(), y.cpu()
    for e in (0, 127, 129):
        lo, hi = int(off[e]), int(off[e + 1])
        for cols in (slice(0, 40), slice(N - 64, N)):
            part = [t[e:e + 1, cols].cpu() for t in (codes, scales, zeros)]
            want, bound, _ = ref.w4_product(xc[lo:hi], [0, hi - lo], None, 1, *part, None, group, False, BF, hi - lo)
            ref.assert_within(y[lo:hi, cols], want, bound, f"expert {e}")
