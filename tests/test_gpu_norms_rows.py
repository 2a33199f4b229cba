"""The norms and their backward over thousands of rows (many rows a workgroup,
next rows in flight, long column sums) and over more columns than a wave holds,
against their 64-bit forms."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref
from tests.test_gpu_grouped_mm import DT, _put
from tests.test_gpu_norms import _desc, _eps, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,kind,dtype,wdtype", [(4101, 2500, "rms", "bf16", "f32"), (4700, 2049, "layer", "f16", "f16"),
                                                  (6200, 4096, "layer", "bf16", "f32")])
def test_many_rows(T, H, kind, dtype, wdtype):
    print(f"norms over many rows {T}x{H} {kind} {dtype}", flush=True)
    dt = DT[dtype]
    t = _inputs(T, H, dtype, wdtype, kind, "channel")
    d_in, d_out = _desc(T, H, dtype, wdtype, kind), _desc(T, H, dtype, wdtype, kind, "channel")
    n = moe.moe_norm_workspace_size(d_in)
    assert n == moe.moe_norm_workspace_size(d_out)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    layer = kind == "layer"
    y, dx, df = (torch.empty(T, H, dtype=dt, device="cuda") for _ in range(3))
    dw, db, dw2, db2, dgate = (torch.empty(H, device="cuda") for _ in range(5))
    x, w, b, gate, dy = (_put(t[v]) for v in ("x", "w", "b", "gate", "dy"))
    moe.moe_norm_in(d_in, x, w, b, y)
    moe.moe_norm_in_backward(d_in, x, w, dy, None, dx, dw, db if layer else None, ws, n)
    moe.moe_norm_out_backward(d_out, x, w, b, gate, None, dy, df, dw2, db2 if layer else None, dgate, ws, n)
    torch.cuda.synchronize()
    eps = _eps(d_in)
    want, bound, en = ref.norm_in(t["x"], t["w"], t["b"], kind, eps, dt)
    ref.assert_within(y, want, bound, "y")
    half, floor = ref.half_step(dt), ref.floor_of(dt)
    dk = t["dy"].double()
    for what, dn, edn, gx_, gw_, gb_ in (("norm_in", dk, torch.zeros_like(dk), dx, dw, db),
                                         ("norm_out", dk * t["gate"].double(), 3 * ref.U * (dk * t["gate"].double()).abs(), df, dw2, db2)):
        gx, ex, gw, ew, gb, eb = ref.norm_grads(t["x"], t["w"], t["b"], dn, edn, kind, eps, dt)
        ref.assert_within(gx_, gx, 1.01 * (ex + half * gx.abs() + floor), f"{what}: dx")
        ref.assert_within(gw_, gw, ew, f"{what}: dweight")
        if layer:
            ref.assert_within(gb_, gb, eb, f"{what}: dbias")
    dg, eg = dk * want, dk.abs() * en + 3 * ref.U * (dk * want).abs()
    ref.assert_within(dgate, dg.sum(0), 1.01 * (eg.sum(0) + (T + 40) * ref.U * dg.abs().sum(0)) + 1e-30, "dgate")
