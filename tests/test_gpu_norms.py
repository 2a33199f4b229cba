"""moe_norm_in, moe_norm_out and their backward against 64-bit forms: widths of
one to several vectors per thread, odd and even, every gate, dropout drawn again
in the backward, rows of zeros, infinities under the dropout, buffers in place."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref
from tests.test_gpu_grouped_mm import DT, _put

pytestmark = pytest.mark.gpu

EPS = 1e-5
KIND = {"none": moe.MOE_NORM_NONE, "rms": moe.MOE_NORM_RMS, "layer": moe.MOE_NORM_LAYER}
GATE = {"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL, "token": moe.MOE_GATE_TOKEN, "full": moe.MOE_GATE_FULL}
SEED, OFFSET = 0x9E3779B97F4A7C15 >> 1, (5 << 32) + 77

# (T, H): one column, less than a vector, one wave's vectors and tails of them,
# each kernel form's edges, more rows than workgroups take at once
SIZES = [(1, 1), (3, 7), (5, 64), (2, 513), (9, 1439), (1, 2880), (33, 2880), (7, 4096), (6, 4104), (3, 8199), (2, 16384),
         (2100, 40)]


def _inputs(T, H, dtype, wdtype, kind, gate, seed=3):
    g = torch.Generator().manual_seed(seed + T + H)
    t = {"x": torch.randn(T, H, generator=g) * 2, "res": torch.randn(T, H, generator=g), "dy": torch.randn(T, H, generator=g),
         "dres": torch.randn(T, H, generator=g)}
    t = {n: v.to(DT[dtype]) for n, v in t.items()}
    t["w"] = (1 + 0.3 * torch.randn(H, generator=g)).to(DT[wdtype]) if kind != "none" else None
    t["b"] = (0.3 * torch.randn(H, generator=g)).to(DT[wdtype]) if kind == "layer" else None
    shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[gate]
    t["gate"] = torch.randn(*shape, generator=g).to(DT[dtype]) if shape else None
    if kind != "none" and T > 2:
        t["x"][1] = 0  # a row of zeros: n = 0, r = 1 / sqrt(eps)
    return t


def _desc(T, H, dtype, wdtype, kind, gate="none", res_scale=1.0, p=0.0):
    return moe.norm(T, H, moe.DTYPE[DT[dtype]], moe.DTYPE[DT[wdtype]], KIND[kind], EPS, GATE[gate], res_scale, p)


def _eps(d):
    return float(d.eps)  # as the kernel has it, in fp32


def _rng(p):
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda") if p else None


def _keep(T, H, p):
    return ref.philox_keep(T, H, p, SEED, OFFSET) if p else (torch.ones(T, H, dtype=torch.bool), 1.0)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_in(T, H, kind, dtype, wdtype):
    print(f"norm_in {T}x{H} {kind} {dtype}/{wdtype}", flush=True)
    t = _inputs(T, H, dtype, wdtype, kind, "none")
    d = _desc(T, H, dtype, wdtype, kind)
    y = torch.empty(T, H, dtype=DT[dtype], device="cuda")
    moe.moe_norm_in(d, _put(t["x"]), _put(t["w"]), _put(t["b"]), y)
    torch.cuda.synchronize()
    want, bound, _ = ref.norm_in(t["x"], t["w"], t["b"], kind, _eps(d), DT[dtype])
    ref.assert_within(y, want, bound, f"norm_in {T}x{H} {kind} {dtype}")


CASES = [("rms", "channel", 0.1, "bf16", "f32"), ("layer", "token", 0.25, "f16", "f16"), ("rms", "full", 0.0, "f32", "f32"),
         ("layer", "channel", 0.5, "bf16", "bf16"), ("none", "none", 0.1, "bf16", "bf16"), ("none", "full", 0.0, "f16", "f16"),
         ("rms", "none", 0.0, "f16", "f32"), ("layer", "full", 0.3, "f32", "f32"), ("rms", "token", 0.0, "bf16", "bf16")]


@pytest.mark.parametrize("kind,gate,p,dtype,wdtype", CASES)
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_out(T, H, kind, gate, p, dtype, wdtype):
    print(f"norm_out {T}x{H} {kind} {gate} p {p} {dtype}/{wdtype}", flush=True)
    t = _inputs(T, H, dtype, wdtype, kind, gate)
    d = _desc(T, H, dtype, wdtype, kind, gate, 0.75, p)
    keep, ks = _keep(T, H, p)
    out = torch.empty(T, H, dtype=DT[dtype], device="cuda")
    args = (_put(t["w"]), _put(t["b"]), _put(t["gate"]), _rng(p))
    moe.moe_norm_out(d, _put(t["x"]), _put(t["res"]), *args, out)
    torch.cuda.synchronize()
    want, bound = ref.norm_out(t["x"], t["res"], t["w"], t["b"], t["gate"], keep, ks, 0.75, kind, _eps(d), DT[dtype])
    ref.assert_within(out, want, bound, f"norm_out {T}x{H} {kind} {gate}")
    inplace = _put(t["res"])
    moe.moe_norm_out(d, _put(t["x"]), inplace, *args, inplace)
    alone = torch.empty_like(out)
    moe.moe_norm_out(d, _put(t["x"]), None, *args, alone)
    torch.cuda.synchronize()
    assert torch.equal(inplace, out)
    want, bound = ref.norm_out(t["x"], None, t["w"], t["b"], t["gate"], keep, ks, 0.75, kind, _eps(d), DT[dtype])
    ref.assert_within(alone, want, bound, f"norm_out without a residual {T}x{H} {kind} {gate}")
    if p and gate == "none":
        assert (alone.cpu()[~keep] == 0).all()


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_in_backward(T, H, kind, dtype, wdtype):
    print(f"norm_in_backward {T}x{H} {kind} {dtype}/{wdtype}", flush=True)
    t = _inputs(T, H, dtype, wdtype, kind, "none")
    d = _desc(T, H, dtype, wdtype, kind, res_scale=0.75)
    n = moe.moe_norm_workspace_size(d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    dx = torch.empty(T, H, dtype=DT[dtype], device="cuda")
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm_in_backward(d, _put(t["x"]), _put(t["w"]), _put(t["dy"]), _put(t["dres"]), dx, dw, db, ws, n)
    torch.cuda.synchronize()
    zero = torch.zeros(T, H, dtype=torch.float64)
    gx, ex, gw, ew, gb, eb = ref.norm_grads(t["x"], t["w"], t["b"], t["dy"].double(), zero, kind, _eps(d), DT[dtype])
    want = gx + 0.75 * t["dres"].double()
    bound = ex + 2 * ref.U * (want.abs() + t["dres"].double().abs()) + ref.half_step(DT[dtype]) * want.abs() + ref.floor_of(DT[dtype])
    ref.assert_within(dx, want, 1.01 * bound, f"dx {T}x{H} {kind}")
    ref.assert_within(dw, gw, ew, "dweight")
    ref.assert_within(db, gb, eb, "dbias")
    # without the optional parts, and over the residual's gradient in place
    only, same = torch.empty_like(dx), _put(t["dres"])
    moe.moe_norm_in_backward(d, _put(t["x"]), _put(t["w"]), _put(t["dy"]), None, only, None, None, ws, n)
    moe.moe_norm_in_backward(d, _put(t["x"]), _put(t["w"]), _put(t["dy"]), same, same, dw, None, ws, n)
    torch.cuda.synchronize()
    ref.assert_within(only, gx, 1.01 * (ex + ref.half_step(DT[dtype]) * gx.abs() + ref.floor_of(DT[dtype])), "dx alone")
    assert torch.equal(same, dx)
    ref.assert_within(dw, gw, ew, "dweight again")


@pytest.mark.parametrize("kind,gate,p,dtype,wdtype", CASES)
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_out_backward(T, H, kind, gate, p, dtype, wdtype):
    print(f"norm_out_backward {T}x{H} {kind} {gate} p {p} {dtype}/{wdtype}", flush=True)
    t = _inputs(T, H, dtype, wdtype, kind, gate)
    d = _desc(T, H, dtype, wdtype, kind, gate, 0.75, p)
    keep, ks = _keep(T, H, p)
    n = moe.moe_norm_workspace_size(d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    df = torch.empty(T, H, dtype=DT[dtype], device="cuda")
    dw = torch.empty(H, device="cuda") if kind != "none" else None
    db = torch.empty(H, device="cuda") if kind == "layer" else None
    dgate = None
    if gate != "none":
        dgate = torch.empty(t["gate"].shape, dtype=DT[dtype] if gate == "full" else torch.float32, device="cuda")
    moe.moe_norm_out_backward(d, _put(t["x"]), _put(t["w"]), _put(t["b"]), _put(t["gate"]), _rng(p), _put(t["dy"]), df, dw,
                              db, dgate, ws, n)
    torch.cuda.synchronize()
    dk = t["dy"].double() * keep.double() * ks
    g = t["gate"].double() if t["gate"] is not None else torch.ones(1, 1, dtype=torch.float64)
    dn = dk * g
    gx, ex, gw, ew, gb, eb = ref.norm_grads(t["x"], t["w"], t["b"], dn, 3 * ref.U * dn.abs(), kind, _eps(d), DT[dtype])
    ref.assert_within(df, gx, 1.01 * (ex + ref.half_step(DT[dtype]) * gx.abs() + ref.floor_of(DT[dtype])), f"df {T}x{H} {kind} {gate}")
    if dw is not None:
        ref.assert_within(dw, gw, ew, "dweight")
    if db is not None:
        ref.assert_within(db, gb, eb, "dbias")
    if dgate is None:
        return
    nv, _, en = ref.norm_in(t["x"], t["w"], t["b"], kind, _eps(d), torch.float32)
    dg, eg = dk * nv, dk.abs() * en + 3 * ref.U * (dk * nv).abs()
    if gate == "channel":
        dg, eg = dg.sum(0, keepdim=True), eg.sum(0, keepdim=True) + (T + 40) * ref.U * dg.abs().sum(0, keepdim=True)
    elif gate == "token":
        # taken as r sum(dk c w) + sum(dk b): c w and b apart, 90 roundings each, r off by 90 of its own
        b = t["b"].double() if t["b"] is not None else 0.0
        parts = (dk * (nv - b)).abs() + (dk * b).abs() if t["b"] is not None else dg.abs()
        dg, eg = dg.sum(1, keepdim=True), (eg + 200 * ref.U * parts).sum(1, keepdim=True)
    else:
        eg = eg + ref.half_step(DT[dtype]) * dg.abs() + ref.floor_of(DT[dtype])
    ref.assert_within(dgate, dg, 1.01 * eg + 1e-30, f"dgate {gate}")


def test_backward_is_the_same_every_time():
    T, H = 700, 2880
    t = _inputs(T, H, "bf16", "f32", "rms", "channel")
    d = _desc(T, H, "bf16", "f32", "rms", "channel", 1.0, 0.1)
    n = moe.moe_norm_workspace_size(d)
    got = []
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(H, device="cuda"), torch.empty(1, H, device="cuda")]
        moe.moe_norm_out_backward(d, _put(t["x"]), _put(t["w"]), None, _put(t["gate"]), _rng(0.1), _put(t["dy"]), out[0],
                                  out[1], None, out[2], ws, n)
        torch.cuda.synchronize()
        got.append(out)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_dropped_values_leave_no_trace():
    """Infinities and NaN in dropped places (no norm, so that they stay there)
    reach neither the output nor the gate's gradient."""
    T, H, p = 40, 200, 0.5
    t = _inputs(T, H, "f32", "f32", "none", "channel")
    d = _desc(T, H, "f32", "f32", "none", "channel", 0.75, p)
    keep, ks = _keep(T, H, p)
    clean, dirty = t["x"].clone(), t["x"].clone()
    dirty[~keep] = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(int((~keep).sum())) % 3]
    n = moe.moe_norm_workspace_size(d)
    got = []
    for f in (clean, dirty):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        o, df, dg = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda"), torch.empty(1, H, device="cuda")
        moe.moe_norm_out(d, _put(f), _put(t["res"]), None, None, _put(t["gate"]), _rng(p), o)
        moe.moe_norm_out_backward(d, _put(f), None, None, _put(t["gate"]), _rng(p), _put(t["dy"]), df, None, None, dg, ws, n)
        torch.cuda.synchronize()
        got.append((o, df, dg))
    for a, b in zip(*got):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_dropout_rate_and_streams():
    """The share kept, and other masks for other seeds, offsets, rows."""
    T, H, p = 512, 1024, 0.3
    f = torch.ones(T, H, device="cuda")
    d = _desc(T, H, "f32", "f32", "none", "none", 1.0, p)
    masks = []
    for seed, off in ((1, 0), (1, 1), (2, 0)):
        o = torch.empty(T, H, device="cuda")
        moe.moe_norm_out(d, f, None, None, None, None, torch.tensor([seed, off], dtype=torch.int64, device="cuda"), o)
        torch.cuda.synchronize()
        keep, ks = ref.philox_keep(T, H, p, seed, off)
        assert torch.equal(o.cpu() != 0, keep)
        masks.append(keep)
    for m in masks:  # 6 standard deviations of a binomial share
        assert abs(m.double().mean().item() - 0.7) < 6 * (0.21 / (T * H)) ** 0.5 + 2 ** -16
    for a, b in ((0, 1), (0, 2)):
        both = (masks[a] & masks[b]).double().mean().item()
        assert abs(both - 0.49) < 6 * (0.49 * 0.51 / (T * H)) ** 0.5 + 2 ** -14


@pytest.mark.parametrize("kind,gate", [("rms", "channel"), ("layer", "token"), ("layer", "full")])
def test_gradients_against_differences(kind, gate):
    """Against central differences of the whole block's norms in 64 bits."""
    T, H, p = 4, 24, 0.25
    t = _inputs(T, H, "f32", "f32", kind, gate)
    t["x"][1] = torch.randn(H, generator=torch.Generator().manual_seed(9))
    d = _desc(T, H, "f32", "f32", kind, gate, 0.75, p)
    keep, ks = _keep(T, H, p)
    n = moe.moe_norm_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    df, dw, db = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    dg = torch.empty(t["gate"].shape, device="cuda")
    moe.moe_norm_out_backward(d, _put(t["x"]), _put(t["w"]), _put(t["b"]), _put(t["gate"]), _rng(p), _put(t["dy"]), df, dw,
                              db if kind == "layer" else None, dg, ws, n)
    torch.cuda.synchronize()
    v = {n_: t[n_].double() for n_ in ("x", "w", "b", "gate") if t[n_] is not None}

    def loss():
        o, _ = ref.norm_out(v["x"], None, v["w"], v.get("b"), v["gate"], keep, ks, 0.75, kind, _eps(d), torch.float64)
        return (o * t["dy"].double()).sum().item()

    got = {"x": df, "w": dw, "b": db, "gate": dg}
    h = 1e-5
    for name, val in v.items():
        flat, grad = val.reshape(-1), got[name].double().cpu().reshape(-1)
        for i in range(0, flat.numel(), 7):
            keep0 = flat[i].item()
            flat[i] = keep0 + h
            up = loss()
            flat[i] = keep0 - h
            down = loss()
            flat[i] = keep0
            # differences: h^2 of the third derivative and 1e-16 / h; the gradient: fp32
            assert abs((up - down) / (2 * h) - grad[i].item()) <= 1e-4 * (1 + abs(grad[i].item())), (name, i)


def test_no_rows():
    d = _desc(0, 40, "bf16", "f32", "layer", "channel", 1.0, 0.0)
    dw, db, dg = (torch.full((40,), 7.0, device="cuda") for _ in range(3))
    moe.moe_norm_out_backward(d, None, None, None, None, None, None, None, dw, db, dg, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all() and (dg == 0).all()
    dw.fill_(7)
    moe.moe_norm_in_backward(d, None, None, None, None, None, dw, None, None, 0)
    moe.moe_norm_in(d, None, None, None, None)
    torch.cuda.synchronize()
    assert (dw == 0).all()
