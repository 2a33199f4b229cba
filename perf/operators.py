"""Timed cases of the library's stand-alone operators, with their plain forms.

Four operators, each a call (or a forward/backward pair of calls) of
include/moe.h:

* ``product``       moe_grouped_mm: rows times their expert's matrix, ragged
                    segments (the expert FFN's two products taken alone);
* ``product_grad``  moe_grouped_mm_dgrad and moe_grouped_mm_wgrad: its gradients;
* ``w4``            moe_w4_matvec: the same product with 4-bit weights and a
                    scale per group, for decoding (optional SwiGLU epilogue);
* ``norms``         moe_norm_in and moe_norm_out: the norm before a block, and
                    after it the norm, dropout, gate and scaled residual;
* ``norms_grad``    their backward.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, through the library.  ``exact`` computes them in 64 bits from
the definitions, by another route (masks and gathers instead of segments, a
host-side generator for the dropout).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the products of the smallest layer the tests use: 64 tokens, 2 of 8 experts; latency
        dict(name="product_tiny", op="product", dtype="bf16", T=64, k=2, E=8, N=512, K=256, gather=True, bias=True,
             skew=0.0),
        # one decode step of 16 sequences through the 20b layer's gate/up product: weights are the traffic
        dict(name="product_decode16", op="product", dtype="bf16", T=16, k=4, E=32, N=5760, K=2880, gather=True,
             bias=True, skew=0.0),
        # prefill of 8192 tokens, skewed expert popularity, token rows gathered: matrix-core bound
        dict(name="product_prefill_zipf", op="product", dtype="bf16", T=8192, k=4, E=32, N=5760, K=2880, gather=True,
             bias=False, skew=1.1),
        # gradients at odd widths in fp16: rows that are not aligned to a vector load
        dict(name="product_grad_odd", op="product_grad", dtype="f16", T=77, k=3, E=5, N=333, K=250, gather=True,
             bias=True, skew=0.0),
        # one micro-batch of training through the 20b layer's down product
        dict(name="product_grad_prefill_zipf", op="product_grad", dtype="bf16", T=8192, k=4, E=32, N=2880, K=2880,
             gather=False, bias=True, skew=1.1),
        # a single decoded token, gate/up with SwiGLU, groups of 32
        dict(name="w4_one_token_swiglu", op="w4", dtype="bf16", T=1, k=4, E=32, N=5760, K=2880, group=32, zeros=False,
             bias=False, swiglu=True),
        # 16 streams through the 128-expert layer, gate/up with SwiGLU, zero points, groups of 64
        dict(name="w4_decode16_swiglu", op="w4", dtype="bf16", T=16, k=4, E=128, N=5760, K=2880, group=64, zeros=True,
             bias=True, swiglu=True),
        # a dense projection at 64 rows, groups of 128, fp16
        dict(name="w4_dense64", op="w4", dtype="f16", T=64, k=1, E=1, N=2880, K=2880, group=128, zeros=True, bias=True,
             swiglu=False),
        # the norms around one decoded token's block: latency
        dict(name="norms_one_token", op="norms", dtype="bf16", T=1, H=2880, kind="rms", gate="none", p=0.0, scale=1.0),
        # the norms around a training block: gate per channel, dropout
        dict(name="norms_prefill", op="norms", dtype="bf16", T=8192, H=2880, kind="rms", gate="channel", p=0.1,
             scale=0.5),
        # gradients at an odd width, layer norm, a gate per token, fp16
        dict(name="norms_grad_odd", op="norms_grad", dtype="f16", T=1025, H=1439, kind="layer", gate="token", p=0.2,
             scale=0.7),
        # gradients around a training block
        dict(name="norms_grad_prefill", op="norms_grad", dtype="bf16", T=8192, H=2880, kind="rms", gate="channel",
             p=0.1, scale=0.5),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["product", "product_grad", "w4", "norms", "norms_grad"])
    if op in ("product", "product_grad"):
        top = 2.0 * 32768 * 2880 * (5760 if op == "product" else 2880)
        while True:
            step = rng.choice([1, 2, 8, 32, 32, 64])
            c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]), T=_logint(rng, 1, 8192), k=rng.randint(1, 4),
                     E=_logint(rng, 4, 128), N=step * _logint(rng, max(1, 64 // step), 5760 // step),
                     K=step * _logint(rng, max(1, 64 // step), 2880 // step), gather=rng.random() < 0.5,
                     bias=rng.random() < 0.5, skew=rng.choice([0.0, 0.0, 1.1]))
            if c["E"] * c["N"] * c["K"] <= 32 * 5760 * 2880 and 2.0 * c["T"] * c["k"] * c["N"] * c["K"] <= top:
                return c
    if op == "w4":
        while True:
            swiglu = rng.random() < 0.5
            dense = rng.random() < 0.4
            E = 1 if dense else _logint(rng, 4, 128)
            c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), T=_logint(rng, 1, 64), k=1 if dense else rng.randint(1, 4),
                     E=E, N=(2 if swiglu else 1) * _logint(rng, 64, 2880), K=32 * _logint(rng, 2, 90),
                     group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, bias=rng.random() < 0.5, swiglu=swiglu)
            if min(c["T"] * c["k"], E) * c["N"] * c["K"] <= 64 * 5760 * 2880:
                return c
    while True:
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), T=_logint(rng, 1, 16384),
                 H=rng.choice([1, 8, 8, 32]) * 1, kind=rng.choice(["rms", "rms", "layer"]),
                 gate=rng.choice(["none", "channel", "token", "full"]), p=rng.choice([0.0, 0.1, 0.25]),
                 scale=rng.choice([1.0, 0.5, 0.22]))
        c["H"] *= _logint(rng, max(1, 64 // c["H"]), 8192 // c["H"])
        if c["T"] * c["H"] * (2 if c["dtype"] == "f32" else 1) * (2 if c["gate"] == "full" else 1) <= 8192 * 2880:
            return c


# ------------------------------------------------------------------ inputs


def _routing(c, g):
    """k distinct experts per token, Zipf(skew) popularity: offsets, the pairs
    sorted by expert, and the segment lengths."""
    pop = torch.arange(1, c["E"] + 1, device=DEV, dtype=torch.float32).pow(-c.get("skew", 0.0))
    noise = -torch.log(-torch.log(torch.rand(c["T"], c["E"], device=DEV, generator=g).clamp(1e-9, 1 - 1e-7)))
    idx = (pop.log() + noise).topk(c["k"], dim=1).indices.reshape(-1)
    counts = torch.bincount(idx, minlength=c["E"])
    offsets = torch.zeros(c["E"] + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return idx, offsets, torch.sort(idx, stable=True).indices.to(torch.int32), counts.tolist()


def _randn(g, *shape, dtype, std=1.0):
    return torch.randn(*shape, device=DEV, dtype=dtype, generator=g) * std


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("product", "product_grad"):
        M = c["T"] * c["k"]
        s["expert"], s["offsets"], s["pairs"], s["counts"] = _routing(c, g)
        s["a"] = _randn(g, c["T"] if c["gather"] else M, c["K"], dtype=dt)
        s["b"] = _randn(g, c["E"], c["N"], c["K"], dtype=dt, std=0.02)
        s["bias"] = _randn(g, c["E"], c["N"], dtype=dt, std=0.1) if c["bias"] else None
        if c["op"] == "product":
            s["c"] = torch.empty(M, c["N"], dtype=dt, device=DEV)
        else:
            s["dc"] = _randn(g, M, c["N"], dtype=dt)
            s["da"] = torch.empty(M, c["K"], dtype=dt, device=DEV)
            s["db"] = torch.empty(c["E"], c["N"], c["K"], dtype=torch.float32, device=DEV)
            s["dbias"] = torch.empty(c["E"], c["N"], dtype=torch.float32, device=DEV) if c["bias"] else None
            s["ws"] = {}
    elif c["op"] == "w4":
        M, G = c["T"] * c["k"], -(-c["K"] // c["group"])
        s["expert"], s["offsets"], s["pairs"], s["counts"] = _routing(c, g)
        s["x"] = _randn(g, c["T"], c["K"], dtype=dt)
        s["codes"] = torch.randint(0, 256, (c["E"], c["N"], c["K"] // 2), dtype=torch.uint8, device=DEV, generator=g)
        s["scales"] = (torch.rand(c["E"], c["N"], G, device=DEV, generator=g) * 0.008 + 0.001).to(dt)
        s["zeros"] = torch.randint(5, 11, (c["E"], c["N"], G), dtype=torch.uint8, device=DEV, generator=g) if c["zeros"] else None
        s["bias"] = _randn(g, c["E"], c["N"], dtype=dt, std=0.1) if c["bias"] else None
        s["y"] = torch.empty(M, c["N"] // (2 if c["swiglu"] else 1), dtype=dt, device=DEV)
    else:
        T, H = c["T"], c["H"]
        s["x"] = _randn(g, T, H, dtype=dt, std=2.0)      # the residual stream, read by the block
        s["f"] = _randn(g, T, H, dtype=dt)               # what the block gave
        s["w_in"] = 1 + _randn(g, H, dtype=torch.float32, std=0.1)
        s["w_out"] = 1 + _randn(g, H, dtype=torch.float32, std=0.1)
        layer = c["kind"] == "layer"
        s["b_in"] = _randn(g, H, dtype=torch.float32, std=0.1) if layer else None
        s["b_out"] = _randn(g, H, dtype=torch.float32, std=0.1) if layer else None
        shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[c["gate"]]
        s["gate"] = _randn(g, *shape, dtype=dt, std=0.5) if shape else None
        s["rng"] = torch.randint(0, 1 << 62, (2,), device=DEV, generator=g, dtype=torch.int64) if c["p"] else None
        if c["op"] == "norms":
            s["y"], s["o"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        else:
            s["dy"], s["do"] = _randn(g, T, H, dtype=dt), _randn(g, T, H, dtype=dt)
            s["dx"], s["df"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            f32 = dict(dtype=torch.float32, device=DEV)
            s["dw_in"], s["dw_out"] = torch.empty(H, **f32), torch.empty(H, **f32)
            s["db_in"] = torch.empty(H, **f32) if layer else None
            s["db_out"] = torch.empty(H, **f32) if layer else None
            # one gate for all rows or all channels gathers its gradient in 32 bits
            s["dgate"] = None if shape is None else torch.empty(shape, dtype=dt if c["gate"] == "full" else torch.float32, device=DEV)
            s["ws"] = {}
    return s


# ------------------------------------------------------------------ plain forms


def _segments(c, rows, counts):
    """(expert, its rows) of every expert that has some."""
    return [(e, r) for e, r in enumerate(torch.split(rows, counts)) if r.shape[0]]


def _plain_product(s):
    c = s["case"]
    a = s["a"].float()
    if c["gather"]:
        a = a[s["pairs"].long() // c["k"]]
    out = torch.empty_like(s["c"])
    at = 0
    for e, r in _segments(c, a, s["counts"]):
        v = r @ s["b"][e].float().t()
        out[at:at + r.shape[0]] = (v + s["bias"][e].float() if c["bias"] else v).to(out.dtype)
        at += r.shape[0]
    return out


def _plain_product_grad(s):
    c = s["case"]
    a, dc = s["a"].float(), s["dc"].float()
    if c["gather"]:
        a = a[s["pairs"].long() // c["k"]]
    da, db = torch.empty_like(s["da"]), torch.zeros_like(s["db"])
    dbias = torch.zeros_like(s["dbias"]) if c["bias"] else None
    at = 0
    for e, r in _segments(c, dc, s["counts"]):
        to = at + r.shape[0]
        da[at:to] = (r @ s["b"][e].float()).to(da.dtype)
        torch.mm(r.t(), a[at:to], out=db[e])
        if c["bias"]:
            dbias[e] = r.sum(0)
        at = to
    return [da, db, dbias]


def _plain_w4(s):
    c = s["case"]
    x = s["x"].float()[s["pairs"].long() // c["k"]]
    out = torch.empty(x.shape[0], c["N"], device=DEV)
    at = 0
    for e, r in _segments(c, x, s["counts"]):
        q = torch.stack([s["codes"][e] & 15, s["codes"][e] >> 4], -1).reshape(c["N"], c["K"]).float()
        z = (s["zeros"][e].float() if c["zeros"] else torch.full_like(s["scales"][e], 8, dtype=torch.float32))
        w = (q - z.repeat_interleave(c["group"], 1)[:, :c["K"]]) * s["scales"][e].float().repeat_interleave(c["group"], 1)[:, :c["K"]]
        v = r @ w.t()
        out[at:at + r.shape[0]] = v + s["bias"][e].float() if c["bias"] else v
        at += r.shape[0]
    if c["swiglu"]:
        g, u = out.chunk(2, 1)
        out = g / (1 + torch.exp(-g)) * u
    return out.to(s["y"].dtype)


def _mulhilo(a, m):
    p = a * m  # the low 64 bits of the product, whatever its sign
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _plain_keep(c, rng):
    """The dropout's kept elements, scaled: Philox4x32-10 at counter (column / 8,
    row, offset), key seed; 16 bits for each of 8 neighbouring columns."""
    T, V = c["T"], -(-c["H"] // 8)
    seed, off = rng[0], rng[1]
    c0 = torch.arange(V, device=DEV).expand(T, V)
    c1 = torch.arange(T, device=DEV)[:, None].expand(T, V)
    c2, c3 = (off & 0xFFFFFFFF).expand(T, V), ((off >> 32) & 0xFFFFFFFF).expand(T, V)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    w = torch.stack([c0, c1, c2, c3], -1)
    bits = torch.stack([w & 0xFFFF, w >> 16], -1).reshape(T, V * 8)[:, :c["H"]]
    return (bits >= round(c["p"] * 65536)).float() / (1 - round(c["p"] * 65536) / 65536)


EPS = 1e-5


def _normalised(c, x):
    if c["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_norms(s):
    c = s["case"]
    x, f = s["x"].float(), s["f"].float()
    y = _normalised(c, x)[0] * s["w_in"]
    n = _normalised(c, f)[0] * s["w_out"]
    if c["kind"] == "layer":
        y, n = y + s["b_in"], n + s["b_out"]
    if c["p"]:
        n = n * _plain_keep(c, s["rng"])
    if s["gate"] is not None:
        n = n * s["gate"].float()
    return [y.to(s["y"].dtype), (c["scale"] * x + n).to(s["o"].dtype)]


def _norm_grad(c, x, w, dn):
    """dx, dw, db of n(x) w + b for the gradient dn."""
    xh, r = _normalised(c, x)
    t = dn * w
    dx = t - xh * (t * xh).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - t.mean(-1, keepdim=True)
    return dx * r, (dn * xh).sum(0), dn.sum(0) if c["kind"] == "layer" else None


def _plain_norms_grad(s):
    c = s["case"]
    x, f, dy, do = s["x"].float(), s["f"].float(), s["dy"].float(), s["do"].float()
    n = _normalised(c, f)[0] * s["w_out"]
    if c["kind"] == "layer":
        n = n + s["b_out"]
    dgate, dn = None, do
    if c["p"]:
        keep = _plain_keep(c, s["rng"])
        n, dn = n * keep, dn * keep
    if s["gate"] is not None:
        dgate = do * n
        dgate = {"channel": lambda: dgate.sum(0, keepdim=True), "token": lambda: dgate.sum(1, keepdim=True),
                 "full": lambda: dgate}[c["gate"]]().to(s["dgate"].dtype)
        dn = dn * s["gate"].float()
    df, dw_out, db_out = _norm_grad(c, f, s["w_out"], dn)
    dx, dw_in, db_in = _norm_grad(c, x, s["w_in"], dy)
    dx = c["scale"] * do + dx
    return [dx.to(s["dx"].dtype), dw_in, db_in, df.to(s["df"].dtype), dw_out, db_out, dgate]


PLAIN = {"product": _plain_product, "product_grad": _plain_product_grad, "w4": _plain_w4, "norms": _plain_norms,
         "norms_grad": _plain_norms_grad}


# ------------------------------------------------------------------ the library's calls


def _moe():
    import mixture_experts_ffn_05_amd as moe
    return moe


def _workspace(s, name, size):
    """A workspace that the program keeps, made at its first use."""
    if name not in s["ws"]:
        s["ws"][name] = torch.empty(max(size(), 256), dtype=torch.uint8, device=DEV)
    return s["ws"][name]


def _gmm(moe, c):
    return moe.gmm(M=c["T"] * c["k"], N=c["N"], K=c["K"], E=c["E"], T=c["T"], k=c["k"], dtype=moe.DTYPE[DTYPES[c["dtype"]]])


def _own_product(s):
    moe, c = _moe(), s["case"]
    moe.moe_grouped_mm(_gmm(moe, c), s["a"], s["offsets"], s["pairs"] if c["gather"] else None, s["b"], s["bias"], s["c"])
    return s["c"]


def _own_product_grad(s):
    moe, c = _moe(), s["case"]
    d = _gmm(moe, c)
    moe.moe_grouped_mm_dgrad(d, s["dc"], s["offsets"], s["b"], s["da"])
    d.out_dtype = moe.MOE_DT_F32
    ws = _workspace(s, "wgrad", lambda: moe.moe_grouped_mm_workspace_size(d))
    moe.moe_grouped_mm_wgrad(d, s["a"], s["offsets"], s["pairs"] if c["gather"] else None, s["dc"], s["db"], s["dbias"], ws, ws.numel())
    return [s["da"], s["db"], s["dbias"]]


def _own_w4(s):
    moe, c = _moe(), s["case"]
    d = moe.w4(M=c["T"] * c["k"], N=c["N"], K=c["K"], E=c["E"], T=c["T"], k=c["k"], group=c["group"],
               dtype=moe.DTYPE[DTYPES[c["dtype"]]], act=moe.MOE_ACT_SWIGLU if c["swiglu"] else moe.MOE_ACT_NONE)
    moe.moe_w4_matvec(d, s["x"], s["offsets"], s["pairs"], s["codes"], s["scales"], s["zeros"], s["bias"], s["y"])
    return s["y"]


def _norm_descs(moe, c):
    kind = {"rms": moe.MOE_NORM_RMS, "layer": moe.MOE_NORM_LAYER}[c["kind"]]
    gate = {"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL, "token": moe.MOE_GATE_TOKEN,
            "full": moe.MOE_GATE_FULL}[c["gate"]]
    dt = moe.DTYPE[DTYPES[c["dtype"]]]
    return (moe.norm(c["T"], c["H"], dt, moe.MOE_DT_F32, kind, EPS, res_scale=c["scale"]),
            moe.norm(c["T"], c["H"], dt, moe.MOE_DT_F32, kind, EPS, gate=gate, res_scale=c["scale"], dropout_p=c["p"]))


def _own_norms(s):
    moe = _moe()
    d_in, d_out = _norm_descs(moe, s["case"])
    moe.moe_norm_in(d_in, s["x"], s["w_in"], s["b_in"], s["y"])
    moe.moe_norm_out(d_out, s["f"], s["x"], s["w_out"], s["b_out"], s["gate"], s["rng"], s["o"])
    return [s["y"], s["o"]]


def _own_norms_grad(s):
    moe = _moe()
    d_in, d_out = _norm_descs(moe, s["case"])
    ws = _workspace(s, "norms", lambda: moe.moe_norm_workspace_size(d_out))
    moe.moe_norm_out_backward(d_out, s["f"], s["w_out"], s["b_out"], s["gate"], s["rng"], s["do"], s["df"], s["dw_out"],
                              s["db_out"], s["dgate"], ws, ws.numel())
    moe.moe_norm_in_backward(d_in, s["x"], s["w_in"], s["dy"], s["do"], s["dx"], s["dw_in"], s["db_in"], ws, ws.numel())
    return [s["dx"], s["dw_in"], s["db_in"], s["df"], s["dw_out"], s["db_out"], s["dgate"]]


OWN = {"product": _own_product, "product_grad": _own_product_grad, "w4": _own_w4, "norms": _own_norms,
       "norms_grad": _own_norms_grad}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}[c["dtype"]]
    if c["op"] in ("product", "product_grad", "w4"):
        M, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
        # experts that some token chose, in expectation over an even routing
        used = E if c.get("skew") and c["T"] > 64 else E * (1 - (1 - c["k"] / E) ** c["T"])
        rows_in = c["T"] * K if c["op"] == "w4" or c["gather"] else M * K
        flops = 2.0 * M * N * K
        if c["op"] == "product":
            return {"bytes": size * (rows_in + used * N * (K + c["bias"]) + M * N), "flops": flops}
        if c["op"] == "product_grad":
            return {"bytes": size * (rows_in + used * N * K + M * N + M * K) + 4.0 * E * N * (K + c["bias"]), "flops": 2 * flops}
        G = -(-K // c["group"])
        weights = used * N * (K / 2 + G * (size + c["zeros"]) + size * c["bias"])
        return {"bytes": weights + size * (rows_in + M * N / (2 if c["swiglu"] else 1)), "flops": flops}
    T, H = c["T"], c["H"]
    layer = 2 if c["kind"] == "layer" else 1
    gate = {"none": 0, "channel": H, "token": T, "full": T * H}[c["gate"]]
    if c["op"] == "norms":  # x, f in; y, o out
        return {"bytes": size * (4.0 * T * H + gate) + 8 * H * layer, "flops": 20.0 * T * H}
    dgate = gate * (size if c["gate"] == "full" else 4)
    return {"bytes": size * (6.0 * T * H + gate) + dgate + 4 * H * (3 + 2 * layer), "flops": 40.0 * T * H}


# ------------------------------------------------------------------ in 64 bits


def _exact_rows(c, s, x):
    """The sorted rows' inputs in 64 bits, and each row's expert."""
    order = torch.argsort(s["expert"], stable=True)
    x = x.double()
    return (x[torch.div(order, c["k"], rounding_mode="floor")] if x.shape[0] == c["T"] and (c["op"] == "w4" or c["gather"]) else x), s["expert"][order]


def _exact_keep(c, rng):
    seed, off = (int(v) & (1 << 64) - 1 for v in rng.tolist())
    T, V = c["T"], -(-c["H"] // 8)
    u = np.uint64
    lo = u(0xFFFFFFFF)
    ctr = [np.broadcast_to(np.arange(V, dtype=u), (T, V)), np.broadcast_to(np.arange(T, dtype=u)[:, None], (T, V)),
           np.full((T, V), off & 0xFFFFFFFF, u), np.full((T, V), off >> 32, u)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(b >> u(32)) ^ ctr[1] ^ u(key[0]), b & lo, (a >> u(32)) ^ ctr[3] ^ u(key[1]), a & lo]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    words = np.stack(ctr, -1).astype(np.uint32)
    bits = words.view(np.uint16).reshape(T, V * 8)[:, :c["H"]]  # little-endian: the low half first
    t = round(c["p"] * 65536)
    return torch.from_numpy((bits >= t).astype(np.float64) * (65536.0 / (65536 - t))).to(DEV)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] in ("product", "product_grad", "w4"):
        rows, expert = _exact_rows(c, s, s["x"] if c["op"] == "w4" else s["a"])
        outs = None
        for e in expert.unique().tolist():
            at = (expert == e).nonzero()[:, 0]
            r = rows[at]
            if c["op"] == "product_grad":
                if outs is None:
                    outs = [torch.zeros(s["da"].shape, dtype=torch.float64, device=DEV),
                            torch.zeros(s["db"].shape, dtype=torch.float64, device=DEV),
                            torch.zeros(s["dbias"].shape, dtype=torch.float64, device=DEV) if c["bias"] else None]
                d = s["dc"][at].double()
                outs[0][at] = torch.matmul(s["b"][e].double().t().contiguous(), d.t().contiguous()).t()
                outs[1][e] = torch.matmul(r.t().contiguous(), d).t()
                if c["bias"]:
                    outs[2][e] = torch.matmul(torch.ones(1, len(at), dtype=torch.float64, device=DEV), d)[0]
                continue
            if c["op"] == "w4":
                b = s["codes"][e].long()
                q = torch.zeros(c["N"], c["K"], dtype=torch.float64, device=DEV)
                q[:, 0::2], q[:, 1::2] = (b % 16).double(), (b // 16).double()
                col = torch.arange(c["K"], device=DEV) // c["group"]
                w = s["scales"][e].double()[:, col] * (q - (s["zeros"][e].double()[:, col] if c["zeros"] else 8.0))
            else:
                w = s["b"][e].double()
            v = torch.matmul(w, r.t().contiguous()).t()
            if s["bias"] is not None:
                v = v + s["bias"][e].double()
            if c.get("swiglu"):
                h = c["N"] // 2
                v = v[:, :h] * torch.sigmoid(v[:, :h]) * v[:, h:]
            if outs is None:
                outs = torch.zeros(rows.shape[0], v.shape[1], dtype=torch.float64, device=DEV)
            outs[at] = v
        return outs

    layer = c["kind"] == "layer"
    keep = _exact_keep(c, s["rng"]) if c["p"] else 1.0
    gate = s["gate"].double() if s["gate"] is not None else 1.0
    if c["op"] == "norms":
        x, f = s["x"].double(), s["f"].double()

        def normed(v, w, b):
            if layer:
                var, mean = torch.var_mean(v, dim=1, unbiased=False, keepdim=True)
                return (v - mean) / (var + EPS).sqrt() * w.double() + b.double()
            return v / (v.pow(2).mean(1, keepdim=True) + EPS).sqrt() * w.double()

        return [normed(x, s["w_in"], s["b_in"]), c["scale"] * x + gate * keep * normed(f, s["w_out"], s["b_out"])]

    # the gradients through autograd of the definition, in 64 bits
    leaf = lambda t: None if t is None else t.double().requires_grad_()  # noqa: E731
    x, f, w1, w2, b1, b2 = (leaf(s[n]) for n in ("x", "f", "w_in", "w_out", "b_in", "b_out"))
    gl = leaf(s["gate"])

    def normed(v, w, b):
        if layer:
            v = v - v.mean(1, keepdim=True)
        y = v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * w
        return y + b if layer else y

    out = c["scale"] * x + (1.0 if gl is None else gl) * keep * normed(f, w2, b2)
    loss = (out * s["do"].double()).sum() + (normed(x, w1, b1) * s["dy"].double()).sum()
    loss.backward()
    grad = lambda t: None if t is None else t.grad  # noqa: E731
    return [grad(x), grad(w1), grad(b1), grad(f), grad(w2), grad(b2), grad(gl)]
