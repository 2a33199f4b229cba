"""Plain 64-bit forms of the stand-alone operators, with the error bounds the
tests hold the kernels to.

Bounds count roundings.  U = 2^-24 is half a step of fp32 relative to a value
(torch.finfo(float32).eps / 2); an output rounded to `dtype` adds
finfo(dtype).eps / 2 of the value.  A sum of n products that are exact (16-bit
times 16-bit) is off by at most n * 2U * sum |terms| whatever its order: one
rounding a step, and a factor 2 because the matrix cores may truncate.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def floor_of(dtype) -> float:
    """Half the spacing of the subnormals: what a rounding may lose next to 0."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound elementwise, and non-finite values where ref has them."""
    got = got.double().cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} for {tuple(ref.shape)}"
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - ref).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, (f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, worst by {worst:.3e} "
                        f"at {divmod(int(over.argmax()), over.shape[-1] if over.dim() else 1)}")


# ------------------------------------------------------------------ grouped products


def segments(offsets, M):
    o = [min(max(int(v), 0), M) for v in offsets]
    return [(e, o[e], max(o[e], o[e + 1])) for e in range(len(o) - 1)]


def gathered(a, pairs, k, M):
    a = a.double()
    if pairs is None:
        return a[:M]
    r = torch.div(pairs.long(), k, rounding_mode="floor")
    ok = (pairs.long() >= 0) & (r < a.shape[0])
    return torch.where(ok[:, None], a[r.clamp(0, a.shape[0] - 1)], torch.zeros((), dtype=torch.float64))


def product(a, offsets, pairs, k, b, bias, out_dtype, M):
    """(values, bound, rows that belong to a segment)."""
    rows, b = gathered(a, pairs, k, M), b.double()
    N = b.shape[1]
    v, s = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    inside = torch.zeros(M, dtype=torch.bool)
    for e, lo, hi in segments(offsets, M):
        v[lo:hi] = rows[lo:hi] @ b[e].t()
        s[lo:hi] = rows[lo:hi].abs() @ b[e].abs().t()
        if bias is not None:
            v[lo:hi] += bias[e].double()
            s[lo:hi] += bias[e].double().abs()
        inside[lo:hi] = True
    return v, half_step(out_dtype) * v.abs() + floor_of(out_dtype) + (b.shape[2] + 2) * 2 * U * s, inside


def product_dgrad(dc, offsets, b, out_dtype, M):
    v, bound, inside = product(dc, offsets, None, 1, b.transpose(1, 2), None, out_dtype, M)
    return v, bound, inside


def product_wgrad(a, offsets, pairs, k, dc, E, out_dtype, M):
    rows, d = gathered(a, pairs, k, M), dc.double()[:M]
    N, K = d.shape[1], rows.shape[1]
    db, s = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    dbias, sb = torch.zeros(E, N, dtype=torch.float64), torch.zeros(E, N, dtype=torch.float64)
    for e, lo, hi in segments(offsets, M):
        db[e], s[e] = d[lo:hi].t() @ rows[lo:hi], d[lo:hi].abs().t() @ rows[lo:hi].abs()
        dbias[e], sb[e] = d[lo:hi].sum(0), d[lo:hi].abs().sum(0)
    bound = half_step(out_dtype) * db.abs() + floor_of(out_dtype) + (M + 70) * 2 * U * s  # 64 partial sums at most
    return db, bound, dbias, (M + 40) * 2 * U * sb + U * dbias.abs()


# ------------------------------------------------------------------ 4-bit products


def w4_weights(codes, scales, zeros, group):
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2).double()
    col = torch.arange(q.shape[-1]) // group
    z = zeros[..., col].double() if zeros is not None else 8.0
    return q, z, scales.double()[..., col]


def w4_product(x, offsets, pairs, k, codes, scales, zeros, bias, group, swiglu, out_dtype, M):
    rows = gathered(x, pairs, k, M)
    N = codes.shape[1]
    v, s = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    inside = torch.zeros(M, dtype=torch.bool)
    for e, lo, hi in segments(offsets, M):
        q, z, sc = w4_weights(codes[e], scales[e], None if zeros is None else zeros[e], group)
        v[lo:hi] = rows[lo:hi] @ ((q - z) * sc).t()
        # the kernel sums (16 + q) x and (16 + z) x before it subtracts them
        s[lo:hi] = rows[lo:hi].abs() @ ((32 + q + z) * sc.abs()).t()
        if bias is not None:
            v[lo:hi] += bias[e].double()
            s[lo:hi] += bias[e].double().abs()
        inside[lo:hi] = True
    err = (group + x.shape[1] / group + 8) * 2 * U * s
    if not swiglu:
        return v, half_step(out_dtype) * v.abs() + floor_of(out_dtype) + err, inside
    g, u = v.chunk(2, 1)
    eg, eu = err.chunk(2, 1)
    y = g * torch.sigmoid(g) * u
    # |silu'| <= 1.1; exp, divide and two products in fp32 (exp is good to 2 steps plus 2U |g|)
    bound = (half_step(out_dtype) * y.abs() + floor_of(out_dtype) + 1.1 * eg * (u.abs() + eu) +
             (g * torch.sigmoid(g)).abs() * eu + (12 + 4 * g.abs()) * U * y.abs() + 1e-30)
    return y, bound, inside


# ------------------------------------------------------------------ norms


def philox_keep(T, H, p, seed, offset):
    """Kept elements and their scale, in Python integers of 32 bits."""
    import numpy as np
    V, u, lo = -(-H // 8), np.uint64, np.uint64(0xFFFFFFFF)
    c = [np.broadcast_to(np.arange(V, dtype=u), (T, V)), np.broadcast_to(np.arange(T, dtype=u)[:, None], (T, V)),
         np.full((T, V), offset & 0xFFFFFFFF, u), np.full((T, V), offset >> 32, u)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & lo, (a >> u(32)) ^ c[3] ^ u(k1), a & lo]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    w = np.stack(c, -1).astype(np.uint32)
    bits = np.stack([w & 0xFFFF, w >> 16], -1).reshape(T, V * 8)[:, :H].astype(np.int64)
    q = round(p * 65536)
    return torch.from_numpy(bits >= q), 65536.0 / (65536 - q)


def normalised(x, kind, eps):
    """xh, r, and the error of xh per element: the row's sums are taken over at
    most 64 columns a thread, 6 steps in a wave and 8 waves (<= 80 roundings)."""
    x = x.double()
    if kind == "none":
        return x, torch.ones(x.shape[0], 1, dtype=torch.float64), torch.zeros_like(x)
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(x.shape[0], 1, dtype=torch.float64)
    c = x - mean
    r = (c.square().mean(1, keepdim=True) + eps).rsqrt()
    ec = (80 * U * x.abs().mean(1, keepdim=True) + U * c.abs()) if kind == "layer" else torch.zeros_like(x)
    rel_r = 90 * U + (ec * c.abs()).mean(1, keepdim=True) * r.square() * 2
    return c * r, r, ec * r + (c * r).abs() * rel_r + U * (c * r).abs()


def norm_in(x, w, b, kind, eps, out_dtype):
    xh, _, exh = normalised(x, kind, eps)
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else b.double()
    n = xh * w + b
    en = exh * w.abs() + 2 * U * ((xh * w).abs() + b.abs())
    return n, half_step(out_dtype) * n.abs() + floor_of(out_dtype) + 1.01 * en, en


def norm_out(f, res, w, b, gate, keep, ks, res_scale, kind, eps, out_dtype):
    n, _, en = norm_in(f, w, b, kind, eps, out_dtype)
    g = torch.ones(1, 1, dtype=torch.float64) if gate is None else gate.double()
    d = keep.double() * ks
    o = g * d * n
    eo = (g * d).abs() * en + 3 * U * o.abs()
    if res is not None:
        o = o + res_scale * res.double()
        eo = eo + 2 * U * ((res_scale * res.double()).abs() + o.abs())
    return o, half_step(out_dtype) * o.abs() + floor_of(out_dtype) + 1.01 * eo


def norm_grads(x, w, b, dn, edn, kind, eps, out_dtype):
    """dx, dw, db of n(x) w + b for its gradient dn (off by edn), each with its bound."""
    T, H = x.shape
    xh, r, exh = normalised(x, kind, eps)
    w = torch.ones(H, dtype=torch.float64) if w is None else w.double()
    t, et = dn * w, edn * w.abs() + U * (dn * w).abs()
    m1 = (t * xh).mean(1, keepdim=True) if kind != "none" else torch.zeros(T, 1, dtype=torch.float64)
    m2 = t.mean(1, keepdim=True) if kind == "layer" else torch.zeros(T, 1, dtype=torch.float64)
    dx = r * (t - xh * m1 - m2)
    em1 = (et * xh.abs() + t.abs() * exh).mean(1, keepdim=True) + 90 * U * (t * xh).abs().mean(1, keepdim=True)
    em2 = et.mean(1, keepdim=True) + 90 * U * t.abs().mean(1, keepdim=True)
    size = r * (t.abs() + (xh * m1).abs() + m2.abs())
    edx = r * (et + exh * m1.abs() + xh.abs() * em1 + (em2 if kind == "layer" else 0)) + 100 * U * size
    dw, edw = (dn * xh).sum(0), (edn * xh.abs() + dn.abs() * exh).sum(0) + (T + 40) * U * (dn * xh).abs().sum(0)
    db, edb = dn.sum(0), edn.sum(0) + (T + 40) * U * dn.abs().sum(0)
    return dx, edx, dw, 1.01 * edw + 1e-30, db, 1.01 * edb + 1e-30
