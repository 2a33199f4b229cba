"""The stand-alone operators as a model uses them: a mixture-of-experts block
with its norms around the layer's own router, permutation and combine, forward
and backward, in 16-bit and with 4-bit weights; captured into a graph; on two
streams at once.

Each step is held to the 64-bit form of what it was given (the buffers that the
step before it wrote), so every bound is that of one operator.
"""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_05_amd as moe
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu

BF, EPS, GROUP = torch.bfloat16, 1e-5, 32
SEED, OFFSET, P_DROP = 12345, 7, 0.125


class Block:
    """o = x + gate * drop(norm(experts(norm(x)))), and its gradients."""

    def __init__(self, T, H, E, k, I, seed, w4=False):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.H, self.E, self.k, self.I, self.M, self.w4 = T, H, E, k, I, T * k, w4
        dev = lambda t: t.cuda()  # noqa: E731
        self.x, self.w_router = dev(r(T, H).to(BF)), dev(r(E, H).to(BF))
        self.w_in, self.w_out = dev(1 + 0.1 * r(H)), dev(1 + 0.1 * r(H))
        self.gate = dev(r(1, H).to(BF))
        self.b1, self.b2 = dev((0.1 * r(E, 2 * I)).to(BF)), dev((0.1 * r(E, H)).to(BF))
        if w4:
            self.c1 = dev(torch.randint(0, 256, (E, 2 * I, H // 2), generator=g, dtype=torch.uint8))
            self.c2 = dev(torch.randint(0, 256, (E, H, I // 2), generator=g, dtype=torch.uint8))
            self.s1 = dev((0.01 * torch.rand(E, 2 * I, -(-H // GROUP), generator=g) + 0.001).to(BF))
            self.s2 = dev((0.01 * torch.rand(E, H, -(-I // GROUP), generator=g) + 0.001).to(BF))
        else:
            self.w1, self.w2 = dev((r(E, 2 * I, H) * H ** -0.5).to(BF)), dev((r(E, H, I) * I ** -0.5).to(BF))
        self.rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")
        e = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        i32, f32 = torch.int32, torch.float32
        self.n, self.idx, self.tw = e(T, H), e(T, k, dt=i32), e(T, k, dt=f32)
        self.off, self.pairs, self.rank = e(E + 1, dt=i32), e(self.M, dt=i32), e(self.M, dt=i32)
        self.u, self.h, self.v = e(self.M, 2 * I), e(self.M, I), e(self.M, H)
        self.f, self.o = e(T, H), e(T, H)
        self.do = dev(r(T, H).to(BF))
        self.ones = torch.ones(T, k, device="cuda")
        self.df, self.dv, self.dh, self.du = e(T, H), e(self.M, H), e(self.M, I), e(self.M, 2 * I)
        self.dns, self.dn, self.dx = e(self.M, H), e(T, H), e(T, H)
        self.dw_out, self.dgate, self.dw_in = e(H, dt=f32), e(1, H, dt=f32), e(H, dt=f32)
        self.dw1, self.db1 = e(E, 2 * I, H, dt=f32), e(E, 2 * I, dt=f32)
        self.dw2, self.db2 = e(E, H, I, dt=f32), e(E, H, dt=f32)
        self.dims = moe.dims(T, H, E, k, I, moe.MOE_WFMT_BF16)
        norm = lambda **kw: moe.norm(T, H, moe.MOE_DT_BF16, moe.MOE_DT_F32, moe.MOE_NORM_RMS, EPS, **kw)  # noqa: E731
        self.d_in = norm()
        self.d_out = norm(gate=moe.MOE_GATE_CHANNEL, dropout_p=P_DROP)
        self.g1, self.g2 = moe.gmm(self.M, 2 * I, H, E, T=T, k=k), moe.gmm(self.M, H, I, E)
        f32o = dict(out_dtype=moe.MOE_DT_F32)
        self.g1w, self.g2w = moe.gmm(self.M, 2 * I, H, E, T=T, k=k, **f32o), moe.gmm(self.M, H, I, E, **f32o)
        self.q1 = moe.w4(self.M, 2 * I, H, E, T=T, k=k, group=GROUP, act=moe.MOE_ACT_SWIGLU)
        self.q2 = moe.w4(self.M, H, I, E, group=GROUP)
        n = max(moe.moe_workspace_size(self.dims), moe.moe_grouped_mm_workspace_size(self.g1w),
                moe.moe_grouped_mm_workspace_size(self.g2w), moe.moe_norm_workspace_size(self.d_in),
                moe.moe_norm_workspace_size(self.d_out))
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def forward(self):
        ws, n = self.ws, self.ws.numel()
        moe.moe_norm_in(self.d_in, self.x, self.w_in, None, self.n)
        moe.moe_route(self.dims, self.n, self.w_router, self.idx, self.tw, ws, n)
        moe.moe_permute(self.dims, self.idx, self.off, self.pairs, self.rank, ws, n)
        if self.w4:
            moe.moe_w4_matvec(self.q1, self.n, self.off, self.pairs, self.c1, self.s1, None, self.b1, self.h)
            moe.moe_w4_matvec(self.q2, self.h, self.off, None, self.c2, self.s2, None, self.b2, self.v)
        else:
            moe.moe_grouped_mm(self.g1, self.n, self.off, self.pairs, self.w1, self.b1, self.u)
            a, b = self.u.float().chunk(2, 1)
            self.h.copy_(a * torch.sigmoid(a) * b)
            moe.moe_grouped_mm(self.g2, self.h, self.off, None, self.w2, self.b2, self.v)
        moe.moe_combine(self.dims, self.v, self.rank, self.tw, self.f)
        moe.moe_norm_out(self.d_out, self.f, self.x, self.w_out, None, self.gate, self.rng, self.o)

    def backward(self):
        """The routing's weights are taken as given."""
        ws, n = self.ws, self.ws.numel()
        moe.moe_norm_out_backward(self.d_out, self.f, self.w_out, None, self.gate, self.rng, self.do, self.df, self.dw_out,
                                  None, self.dgate, ws, n)
        p = self.pairs.long()
        self.dv.copy_(self.df.float()[p // self.k] * self.tw.view(-1)[p].unsqueeze(1))
        moe.moe_grouped_mm_wgrad(self.g2w, self.h, self.off, None, self.dv, self.dw2, self.db2, ws, n)
        moe.moe_grouped_mm_dgrad(self.g2, self.dv, self.off, self.w2, self.dh)
        a, b = self.u.float().chunk(2, 1)
        s, dh = torch.sigmoid(a), self.dh.float()
        self.du.copy_(torch.cat([dh * b * (s + a * s * (1 - s)), dh * a * s], 1))
        moe.moe_grouped_mm_wgrad(self.g1w, self.n, self.off, self.pairs, self.du, self.dw1, self.db1, ws, n)
        moe.moe_grouped_mm_dgrad(self.g1, self.du, self.off, self.w1, self.dns)
        moe.moe_combine(self.dims, self.dns, self.rank, self.ones, self.dn)  # a token's k gradients
        moe.moe_norm_in_backward(self.d_in, self.x, self.w_in, self.dn, self.do, self.dx, self.dw_in, None, ws, n)

    def run(self):
        self.forward()
        if not self.w4:
            self.backward()

    def results(self):
        names = ["n", "idx", "tw", "off", "pairs", "rank", "h", "v", "f", "o"]
        if not self.w4:
            names += ["u", "df", "dv", "dh", "du", "dns", "dn", "dx", "dw_out", "dgate", "dw_in", "dw1", "db1", "dw2", "db2"]
        return {n: getattr(self, n) for n in names}


BLOCKS = {
    # T, H, E, k, I; w4
    "one_token": (1, 128, 4, 2, 64, False),
    "decode": (13, 256, 8, 2, 96, False),
    "rows": (300, 256, 5, 3, 160, False),
    "w4_one_token": (1, 128, 4, 2, 64, True),
    "w4_decode": (13, 256, 8, 2, 96, True),
}


def _block(name, seed=2):
    *sizes, w4 = BLOCKS[name]
    return Block(*sizes, seed=seed, w4=w4)


def _combined(y, rank, w, T, k):
    terms = y.double()[rank.long()].view(T, k, -1) * w.double().unsqueeze(2)
    v = terms.sum(1)
    return v, ref.half_step(BF) * v.abs() + ref.floor_of(BF) + (k + 1) * 2 * ref.U * terms.abs().sum(1)


@pytest.mark.parametrize("name", sorted(BLOCKS))
def test_each_step_of_the_block(name):
    print(f"block {name}", flush=True)
    b = _block(name)
    b.run()
    torch.cuda.synchronize()
    c = {n: t.cpu() for n, t in vars(b).items() if torch.is_tensor(t)}
    T, H, E, k, M, off, pairs = b.T, b.H, b.E, b.k, b.M, c["off"], c["pairs"]
    eps = float(b.d_in.eps)
    # the routing is a permutation of the pairs into the experts' segments
    assert sorted(pairs.tolist()) == list(range(M)) and off[0] == 0 and off[-1] == M
    for e in range(E):
        assert (c["idx"].view(-1)[pairs[off[e]:off[e + 1]].long()] == e).all()
    assert (pairs[c["rank"].long()] == torch.arange(M)).all()

    want, bound, _ = ref.norm_in(c["x"], c["w_in"], None, "rms", eps, BF)
    ref.assert_within(c["n"], want, bound, "norm_in")
    if b.w4:
        want, bound, _ = ref.w4_product(c["n"], off, pairs, k, c["c1"], c["s1"], None, c["b1"], GROUP, True, BF, M)
        ref.assert_within(c["h"], want, bound, "gate-up, 4 bits")
        want, bound, _ = ref.w4_product(c["h"], off, None, 1, c["c2"], c["s2"], None, c["b2"], GROUP, False, BF, M)
        ref.assert_within(c["v"], want, bound, "down, 4 bits")
    else:
        want, bound, _ = ref.product(c["n"], off, pairs, k, c["w1"], c["b1"], BF, M)
        ref.assert_within(c["u"], want, bound, "gate-up")
        want, bound, _ = ref.product(c["h"], off, None, 1, c["w2"], c["b2"], BF, M)
        ref.assert_within(c["v"], want, bound, "down")
    ref.assert_within(c["f"], *_combined(c["v"], c["rank"], c["tw"], T, k), "combine")
    keep, ks = ref.philox_keep(T, H, P_DROP, SEED, OFFSET)
    want, bound = ref.norm_out(c["f"], c["x"], c["w_out"], None, c["gate"], keep, ks, 1.0, "rms", eps, BF)
    ref.assert_within(c["o"], want, bound, "norm_out")
    if b.w4:
        return

    # ---- backward
    half, floor = ref.half_step(BF), ref.floor_of(BF)
    dk = c["do"].double() * keep.double() * ks
    dn = dk * c["gate"].double()
    gx, ex, gw, ew, _, _ = ref.norm_grads(c["f"], c["w_out"], None, dn, 3 * ref.U * dn.abs(), "rms", eps, BF)
    ref.assert_within(c["df"], gx, 1.01 * (ex + half * gx.abs() + floor), "df")
    ref.assert_within(c["dw_out"], gw, ew, "dw_out")
    nv, _, en = ref.norm_in(c["f"], c["w_out"], None, "rms", eps, torch.float32)
    dg, eg = dk * nv, dk.abs() * en + 3 * ref.U * (dk * nv).abs()
    ref.assert_within(c["dgate"], dg.sum(0, keepdim=True),
                      1.01 * (eg.sum(0, keepdim=True) + (T + 40) * ref.U * dg.abs().sum(0, keepdim=True)) + 1e-30, "dgate")
    for what, a, pr, kk, dc, dw, db, w, dn_, N in (("down", "h", None, 1, "dv", "dw2", "db2", "w2", "dh", H),
                                                 ("gate-up", "n", pairs, k, "du", "dw1", "db1", "w1", "dns", 2 * b.I)):
        want, bound, wantb, boundb = ref.product_wgrad(c[a], off, pr, kk, c[dc], E, torch.float32, M)
        ref.assert_within(c[dw], want, bound, f"{what}: weight gradient")
        ref.assert_within(c[db], wantb, boundb, f"{what}: bias gradient")
        want, bound, _ = ref.product_dgrad(c[dc], off, c[w], BF, M)
        ref.assert_within(c[dn_], want, bound, f"{what}: data gradient")
    ref.assert_within(c["dn"], *_combined(c["dns"], c["rank"], torch.ones(T, k), T, k), "dn")
    gx, ex, gw, ew, _, _ = ref.norm_grads(c["x"], c["w_in"], None, c["dn"].double(), torch.zeros(T, H, dtype=torch.float64),
                                          "rms", eps, BF)
    want = gx + c["do"].double()
    ref.assert_within(c["dx"], want, 1.01 * (ex + 2 * ref.U * (want.abs() + c["do"].double().abs()) + half * want.abs() + floor),
                      "dx")
    ref.assert_within(c["dw_in"], gw, ew, "dw_in")


def _snapshot(b):
    return {n: t.clone() for n, t in b.results().items()}


def _same(b, want, what):
    for n, t in b.results().items():
        assert torch.equal(t, want[n]), f"{what}: {n} differs"


@pytest.mark.parametrize("name", ["rows", "decode", "w4_one_token", "w4_decode"])
def test_graph_replays_match_eager(name):
    """Captured once, replayed with two inputs by turns (their routing differs),
    with eager calls on the same buffers and workspace between the replays."""
    print(f"graph {name}", flush=True)
    b = _block(name)
    xs = [b.x.clone(), (b.x.float().flip(1) * 0.5).to(BF)]
    rngs = [b.rng.clone(), b.rng + 1]
    wants = []
    for x, rng in zip(xs, rngs):
        b.x.copy_(x)
        b.rng.copy_(rng)
        b.run()
        torch.cuda.synchronize()
        wants.append(_snapshot(b))
    assert not torch.equal(wants[0]["idx"], wants[1]["idx"])
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            b.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for rep in range(4):
        i = rep % 2
        b.x.copy_(xs[i])
        b.rng.copy_(rngs[i])
        for t in b.results().values():
            t.zero_()
        b.ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _same(b, wants[i], f"replay {rep}")
        b.x.copy_(xs[1 - i])
        b.rng.copy_(rngs[1 - i])
        b.run()
        torch.cuda.synchronize()
        _same(b, wants[1 - i], f"eager after replay {rep}")


def test_two_streams_at_once():
    """Blocks of different sizes, each with its own workspace, on two streams
    without a synchronisation between them: bit for bit what each gives alone."""
    blocks = [_block("rows", 3), _block("w4_decode", 4), _block("decode", 5)]
    wants = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        wants.append(_snapshot(b))
        for t in b.results().values():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [[] for _ in blocks]
    for _ in range(3):
        for i, (b, s) in enumerate(zip(blocks, streams)):
            with torch.cuda.stream(s):
                b.run()
                got[i].append(_snapshot(b))
    torch.cuda.synchronize()
    for i in range(len(blocks)):
        for rep, g in enumerate(got[i]):
            for n in g:
                assert torch.equal(g[n], wants[i][n]), f"block {i} repeat {rep}: {n} differs from the block run alone"


def test_explicit_stream_argument():
    """The stream is the call's own, whatever the current one is."""
    b = _block("decode", 6)
    b.run()
    torch.cuda.synchronize()
    want = b.n.clone()
    b.n.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    moe.moe_norm_in(b.d_in, b.x, b.w_in, None, b.n, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(b.n, want)
