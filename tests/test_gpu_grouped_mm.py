"""moe_grouped_mm and its gradients against their 64-bit forms.

Sizes sit where the kernels change: the decode form (at most 64 rows), the
128 x 64 and 256 x 256 tiles, tails of every tile and of the contracted length,
widths and strides that rule out the direct loads, empty experts, rows outside
every segment, pairs out of range, weight gradients cut into row ranges."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _segments(rng, M, E, empty, lead=0, behind=0):
    """Random offsets over rows lead .. M - behind; experts in `empty` get none."""
    share = rng.random(E) + 0.05
    share[list(empty)] = 0
    cut = np.floor(np.cumsum(share) / share.sum() * (M - lead - behind) + 1e-9).astype(np.int64)
    return np.concatenate([[lead], lead + cut]).astype(np.int32)


def _strided(t, ld):
    """The same rows with `ld` elements from one to the next, the rest NaN."""
    if not ld:
        return t
    full = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype)
    full[:, :t.shape[1]] = t
    return full


def _case(seed, dtype, T, k, E, N, K, gather, empty=(), lead=0, behind=0, bad_pairs=False):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    M = T * k
    dt = DT[dtype]
    a = torch.randn(T if gather else M, K, generator=g).to(dt)
    b = (torch.randn(E, N, K, generator=g) * 0.1).to(dt)
    bias = torch.randn(E, N, generator=g).to(dt)
    dc = torch.randn(M, N, generator=g).to(dt)
    offsets = torch.from_numpy(_segments(rng, M, E, empty, lead, behind))
    pairs = None
    if gather:
        pairs = torch.from_numpy(rng.permutation(M).astype(np.int32))
        if bad_pairs:
            pairs[M // 2], pairs[M // 3] = -5, M + 7
    return a, b, bias, dc, offsets, pairs, M


SHAPES = {
    # name: T, k, E, N, K, gather, extra
    "one_row": dict(T=1, k=1, E=1, N=1, K=1, gather=False),
    "one_token": dict(T=1, k=4, E=8, N=96, K=160, gather=True, empty=(1, 2, 5, 7)),
    "decode": dict(T=16, k=4, E=32, N=200, K=328, gather=True, empty=(0, 31, 13)),
    "decode_dense": dict(T=61, k=1, E=1, N=97, K=136, gather=False),
    "decode_two_passes": dict(T=25, k=2, E=24, N=64, K=64, gather=True, empty=tuple(range(2, 24))),
    "decode_odd_width": dict(T=7, k=2, E=3, N=31, K=45, gather=True),
    "tiny": dict(T=64, k=2, E=8, N=512, K=256, gather=True),
    "small_tile_tails": dict(T=90, k=3, E=5, N=136, K=72, gather=True, empty=(2,), bad_pairs=True),
    "odd_widths": dict(T=77, k=3, E=5, N=333, K=250, gather=True, empty=(4,)),
    "odd_widths_rows": dict(T=150, k=1, E=3, N=33, K=35, gather=False),
    "large_tile_tails": dict(T=700, k=1, E=3, N=264, K=104, gather=True, empty=(1,)),
    "large_tile_rows": dict(T=560, k=2, E=2, N=520, K=320, gather=False),
    "rows_outside": dict(T=200, k=1, E=3, N=72, K=40, gather=True, lead=9, behind=21),
    "rows_outside_decode": dict(T=30, k=2, E=3, N=72, K=40, gather=True, lead=5, behind=8),
    "all_empty": dict(T=40, k=2, E=4, N=48, K=40, gather=True, lead=80),
    "many_experts": dict(T=130, k=4, E=256, N=40, K=48, gather=True),
}


def _put(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_forward(name, dtype):
    print(f"grouped forward {name} {dtype}", flush=True)
    c = dict(SHAPES[name])
    a, b, bias, _, off, pairs, M = _case(11, dtype, **c)
    for use_bias, out in ((True, dtype), (False, "f32")):
        y = torch.full((M, c["N"]), 7.0, dtype=DT[out], device="cuda")
        d = moe.gmm(M, c["N"], c["K"], c["E"], T=c["T"], k=c["k"], dtype=moe.DTYPE[DT[dtype]], out_dtype=moe.DTYPE[DT[out]])
        moe.moe_grouped_mm(d, _put(a), _put(off), _put(pairs), _put(b), _put(bias) if use_bias else None, y)
        torch.cuda.synchronize()
        want, bound, inside = ref.product(a, off, pairs, c["k"], b, bias if use_bias else None, DT[out], M)
        y = y.cpu()
        ref.assert_within(y[inside], want[inside], bound[inside], f"{name} {dtype}->{out}")
        assert (y[~inside] == 7).all(), f"{name}: rows outside the segments were written"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_data_gradient(name, dtype):
    print(f"grouped dgrad {name} {dtype}", flush=True)
    c = dict(SHAPES[name])
    _, b, _, dc, off, _, M = _case(12, dtype, **c)
    for out in (dtype, "f32"):
        da = torch.full((M, c["K"]), 7.0, dtype=DT[out], device="cuda")
        d = moe.gmm(M, c["N"], c["K"], c["E"], dtype=moe.DTYPE[DT[dtype]], out_dtype=moe.DTYPE[DT[out]])
        moe.moe_grouped_mm_dgrad(d, _put(dc), _put(off), _put(b), da)
        torch.cuda.synchronize()
        want, bound, inside = ref.product_dgrad(dc, off, b, DT[out], M)
        da = da.cpu()
        ref.assert_within(da[inside], want[inside], bound[inside], f"{name} {dtype}->{out}")
        assert (da[~inside] == 7).all()


WGRAD_ONLY = {
    # few tiles and many rows: the segments are cut into row ranges
    "split_dense": dict(T=3000, k=1, E=1, N=72, K=136, gather=False),
    "split_gather": dict(T=1700, k=2, E=2, N=40, K=64, gather=True),
    "split_odd": dict(T=2600, k=1, E=2, N=33, K=35, gather=True, empty=(0,)),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(SHAPES) + sorted(WGRAD_ONLY))
def test_weight_gradient(name, dtype):
    print(f"grouped wgrad {name} {dtype}", flush=True)
    c = dict({**SHAPES, **WGRAD_ONLY}[name])
    a, _, _, dc, off, pairs, M = _case(13, dtype, **c)
    E, N, K = c["E"], c["N"], c["K"]
    for out, accumulate in (("f32", False), ("f32", True), (dtype, False)):
        d = moe.gmm(M, N, K, E, T=c["T"], k=c["k"], dtype=moe.DTYPE[DT[dtype]], out_dtype=moe.DTYPE[DT[out]],
                    accumulate=accumulate)
        n = moe.moe_grouped_mm_workspace_size(d)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        db = torch.full((E, N, K), 0.5, dtype=DT[out], device="cuda")
        dbias = torch.full((E, N), 0.25, dtype=torch.float32, device="cuda")
        moe.moe_grouped_mm_wgrad(d, _put(a), _put(off), _put(pairs), _put(dc), db, dbias, ws, n)
        torch.cuda.synchronize()
        want, bound, wbias, bbias = ref.product_wgrad(a, off, pairs, c["k"], dc, E, DT[out], M)
        if accumulate:
            want, wbias = want + 0.5, wbias + 0.25
            bound, bbias = bound + ref.U * (want.abs() + 0.5), bbias + ref.U * (wbias.abs() + 0.25)
        ref.assert_within(db, want, bound, f"{name} db {out} accumulate {accumulate}")
        ref.assert_within(dbias, wbias, bbias, f"{name} dbias accumulate {accumulate}")
        db2 = torch.full_like(db, 0.5)
        moe.moe_grouped_mm_wgrad(d, _put(a), _put(off), _put(pairs), _put(dc), db2, None, ws, n)
        torch.cuda.synchronize()
        assert torch.equal(db, db2), "the same call gives other bits"


@pytest.mark.parametrize("M_scale", [1, 9])
@pytest.mark.parametrize("lda,ldc", [(48, 80), (43, 75)])
def test_strides(lda, ldc, M_scale):
    """Rows with room behind them (NaN there): read and written where they are."""
    T, k, E, N, K = 30 * M_scale, 2, 3, 72, 40
    a, b, bias, dc, off, pairs, M = _case(14, "bf16", T, k, E, N, K, True)
    d = moe.gmm(M, N, K, E, T=T, k=k, lda=lda, ldc=ldc)
    y = torch.full((M, ldc), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm(d, _strided(a, lda).cuda(), _put(off), _put(pairs), _put(b), _put(bias), y)
    da = torch.full((M, lda), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm_dgrad(d, _strided(dc, ldc).cuda(), _put(off), _put(b), da)
    d.out_dtype = moe.MOE_DT_F32
    db = torch.empty(E, N, K, device="cuda")
    dbias = torch.empty(E, N, device="cuda")
    n = moe.moe_grouped_mm_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_mm_wgrad(d, _strided(a, lda).cuda(), _put(off), _put(pairs), _strided(dc, ldc).cuda(), db, dbias, ws, n)
    torch.cuda.synchronize()
    want, bound, inside = ref.product(a, off, pairs, k, b, bias, torch.bfloat16, M)
    ref.assert_within(y[:, :N].cpu()[inside], want[inside], bound[inside], "strided forward")
    assert (y[:, N:] == 7).all()
    want, bound, inside = ref.product_dgrad(dc, off, b, torch.bfloat16, M)
    ref.assert_within(da[:, :K].cpu()[inside], want[inside], bound[inside], "strided dgrad")
    assert (da[:, K:] == 7).all()
    want, bound, wbias, bbias = ref.product_wgrad(a, off, pairs, k, dc, E, torch.float32, M)
    ref.assert_within(db, want, bound, "strided wgrad")
    ref.assert_within(dbias, wbias, bbias, "strided dbias")


@pytest.mark.parametrize("rows", [40, 600])
def test_unaligned_bases(rows):
    """Operands that start one element behind a 16-byte boundary."""
    T, k, E, N, K = rows, 1, 2, 64, 64
    a, b, _, dc, off, pairs, M = _case(15, "f16", T, k, E, N, K, True)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1).cuda()
        return buf[1:].view(t.shape)

    d = moe.gmm(M, N, K, E, T=T, k=k, dtype=moe.MOE_DT_F16)
    y, da = shifted(torch.zeros(M, N, dtype=torch.float16)), shifted(torch.zeros(M, K, dtype=torch.float16))
    moe.moe_grouped_mm(d, shifted(a), _put(off), _put(pairs), shifted(b), None, y)
    moe.moe_grouped_mm_dgrad(d, shifted(dc), _put(off), shifted(b), da)
    torch.cuda.synchronize()
    want, bound, inside = ref.product(a, off, pairs, k, b, None, torch.float16, M)
    ref.assert_within(y.cpu()[inside], want[inside], bound[inside], "unaligned forward")
    want, bound, inside = ref.product_dgrad(dc, off, b, torch.float16, M)
    ref.assert_within(da.cpu()[inside], want[inside], bound[inside], "unaligned dgrad")


def test_nan_stays_in_its_row():
    """A NaN in one input row, and in one expert's weights, reaches only the
    outputs that use it, across tile and contraction tails."""
    T, k, E, N, K = 150, 1, 3, 72, 40
    a, b, bias, dc, off, pairs, M = _case(16, "bf16", T, k, E, N, K, False)
    off = torch.tensor([0, 40, 90, 150], dtype=torch.int32)
    a[3], b[2, 5] = float("nan"), float("inf")
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm(moe.gmm(M, N, K, E), _put(a), _put(off), None, _put(b), _put(bias), y)
    db = torch.zeros(E, N, K, device="cuda")
    d = moe.gmm(M, N, K, E, out_dtype=moe.MOE_DT_F32)
    n = moe.moe_grouped_mm_workspace_size(d)
    moe.moe_grouped_mm_wgrad(d, _put(a), _put(off), None, _put(dc), db, None, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y.cpu())
    want = torch.zeros(M, N, dtype=torch.bool)
    want[3] = True
    want[90:, 5] = True
    assert torch.equal(bad, want)
    assert torch.isnan(db[0]).all() and torch.isfinite(db[1:]).all()


def test_no_rows_zero_gradients():
    d = moe.gmm(0, 24, 40, 3, out_dtype=moe.MOE_DT_F32)
    db, dbias = torch.full((3, 24, 40), 7.0, device="cuda"), torch.full((3, 24), 7.0, device="cuda")
    moe.moe_grouped_mm_wgrad(d, None, None, None, None, db, dbias, None, 0)
    torch.cuda.synchronize()
    assert (db == 0).all() and (dbias == 0).all()
    db.fill_(7)
    d.accumulate = 1
    moe.moe_grouped_mm_wgrad(d, None, None, None, None, db, dbias, None, 0)
    torch.cuda.synchronize()
    assert (db == 7).all()


def test_offsets_out_of_range_are_clamped():
    """Offsets past the rows, negative or decreasing read as clamped segments."""
    T, E, N, K = 100, 4, 40, 32
    a, b, _, _, _, _, M = _case(17, "bf16", T, 1, E, N, K, False)
    off = torch.tensor([-7, 30, 20, 60, 1 << 30], dtype=torch.int32)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm(moe.gmm(M, N, K, E), _put(a), _put(off), None, _put(b), None, y)
    torch.cuda.synchronize()
    v = a.double()
    want = torch.empty(M, N, dtype=torch.float64)
    want[:30], want[60:] = v[:30] @ b[0].double().t(), v[60:] @ b[3].double().t()
    want[30:60] = v[30:60] @ b[2].double().t()  # rows 20..29 belong to two segments and are not compared
    s = v.abs().sum(1, keepdim=True) * b.double().abs().max()
    keep = torch.tensor([i < 20 or i >= 30 for i in range(M)])
    bound = ref.half_step(torch.bfloat16) * want.abs() + (K + 2) * 2 * ref.U * s
    ref.assert_within(y.cpu()[keep], want[keep], bound[keep], "clamped")


def test_gradients_against_differences():
    """The two gradients of sum(dc * forward) against central differences of
    the forward in 64 bits, on sampled entries."""
    T, k, E, N, K = 20, 2, 3, 24, 40
    a, b, _, dc, off, pairs, M = _case(18, "f16", T, k, E, N, K, True)
    d = moe.gmm(M, N, K, E, T=T, k=k, dtype=moe.MOE_DT_F16, out_dtype=moe.MOE_DT_F32)
    da, db = torch.empty(M, K, device="cuda"), torch.empty(E, N, K, device="cuda")
    n = moe.moe_grouped_mm_workspace_size(d)
    moe.moe_grouped_mm_dgrad(d, _put(dc), _put(off), _put(b), da)
    moe.moe_grouped_mm_wgrad(d, _put(a), _put(off), _put(pairs), _put(dc), db, None,
                             torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    torch.cuda.synchronize()

    def loss(a64, b64):
        rows = a64[torch.div(pairs.long(), k, rounding_mode="floor")]
        v = torch.cat([rows[lo:hi] @ b64[e].t() for e, lo, hi in ref.segments(off, M)])
        return (v * dc.double()).sum().item()

    rng, h = np.random.default_rng(1), 1e-3
    a64, b64 = a.double(), b.double()
    dtok = torch.zeros(T, K, dtype=torch.float64).index_add_(0, torch.div(pairs.long(), k, rounding_mode="floor"), da.double().cpu())
    for _ in range(12):
        i, j, e, q = rng.integers(T), rng.integers(K), rng.integers(E), rng.integers(N)
        for t, at, got in ((a64, (i, j), dtok[i, j]), (b64, (e, q, j), db[e, q, j].item())):
            keep = t[at].item()
            t[at] = keep + h
            up = loss(a64, b64)
            t[at] = keep - h
            down = loss(a64, b64)
            t[at] = keep
            # the loss is linear in each: differences are exact up to 64-bit rounding
            assert abs((up - down) / (2 * h) - got) <= 1e-4 * (1 + abs(got))
