"""The whole layer for a few tokens against its 64-bit definition, element by
element within what the roundings allow; graph replays, streams, repeated calls."""
import pytest
import torch

import _few_ref as ref
from _helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    return m


class Case:
    """Inputs and outputs of one call, with the call itself."""

    def __init__(self, xm, T, d, E, k, h, hs=0, dt=BF, mx8=False, bias=False, seed=0, tau=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 * seed + T + d + E)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.xm, self.T, self.d, self.E, self.k, self.h, self.hs, self.dt, self.mx8, self.tau = xm, T, d, E, k, h, hs, dt, mx8, tau
        self.x = r(T, d).to(dt)
        self.wg = (1.5 * d ** -0.5 * r(d, E)).to(dt)
        self.lb = 0.4 * r(E) if bias else None
        self.sb = 0.4 * r(E) if bias else None
        w = lambda n, K, N: (K ** -0.5 * r(n, K, N)).to(dt)
        self.plain = [w(E, d, h), w(E, d, h), w(E, h, d)]
        self.splain = [w(1, d, hs), w(1, d, hs), w(1, hs, d)] if hs else None
        if mx8:
            self.xq = torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda")
            self.xs = torch.empty(xm.mx8_scale_shape(T, d), dtype=torch.uint8, device="cuda")
            xm.xmoe_mx8_quantize(self.x, self.xq, self.xs)
            self.w = [self._q(t) for t in self.plain]
            self.s = [self._q(t) for t in self.splain] if hs else [None] * 3
        else:
            self.w = self.plain
            self.s = [t[0] for t in self.splain] if hs else [None] * 3
        self.ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        self.p = torch.full((T, k), float("nan"), device="cuda")
        self.z = torch.full((T, E), float("nan"), device="cuda")
        self.y = torch.full((T, d), float("nan"), dtype=dt, device="cuda")

    def _q(self, w):
        n, K, N = w.shape
        q = torch.empty((n, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((n,) + self.xm.mx8_scale_shape(N, K), dtype=torch.uint8, device="cuda")
        self.xm.xmoe_mx8_quantize_weights(w, q, s)
        return q, s

    def need(self):
        a = (self.T, self.d, self.E, self.k, self.h, self.hs)
        return self.xm.xmoe_layer_few_mx8_workspace_size(*a) if self.mx8 else self.xm.xmoe_layer_few_workspace_size(*a, self.dt)

    def run(self, **kw):
        rest = dict(inv_temperature=self.tau, logit_bias=self.lb, select_bias=self.sb, s1=self.s[0], s3=self.s[1], s2=self.s[2])
        out = (self.k, self.ids, self.p, self.z, self.y)
        if self.mx8:
            self.xm.xmoe_layer_few_mx8(self.x, self.xq, self.xs, self.wg, *self.w, *out, **{**rest, **kw})
        else:
            self.xm.xmoe_layer_few(self.x, self.wg, *self.w, *out, **{**rest, **kw})
        return self

    def outs(self):
        return [t.clone() for t in (self.ids, self.p, self.z, self.y)]

    def check(self, name=""):
        D = torch.float64
        T = self.T
        if self.mx8:
            of = lambda w, e: tuple(ref.mx8_weights(q[e], s[e]) for q, s in w)
            xe = ref.mx8_values(self.xq, self.xs)
            act_half = None
        else:
            of = lambda w, e: tuple(t[e].to(D) for t in w)
            xe = self.x.to(D)
            act_half = 2.0 ** -16 if self.dt == torch.bfloat16 else 2.0 ** -24
        shared = None
        if self.hs:
            shared = of(self.s, 0) if self.mx8 else tuple(t.to(D) for t in self.s)
        ids = self.ids.long()
        assert int(ids.min()) >= 0 and int(ids.max()) < self.E, name
        assert all(len(set(r)) == self.k for r in ids.tolist()), name
        z, dz, p, dp, y, dy = ref.layer(self.x.to(D), xe, self.wg.to(D), lambda e: of(self.w, e), shared, ids, tau=self.tau,
                                        lbias=self.lb, out_half=ref.half_step(self.dt), act_half=act_half)
        assert ref.chosen_well(z, dz, self.sb, self.ids), name
        for what, got, want, tol in (("logits", self.z, z, dz + 2.0 ** -24 * z.abs()),
                                     ("topk_w", self.p, torch.gather(p, 1, ids), torch.gather(dp, 1, ids)),
                                     ("y", self.y, y, dy)):
            err = (got.to(D) - want).abs()
            assert bool((err <= tol).all()), f"{name} {what}: {float((err - tol).max()):.2e} past the bound"
        # and as a whole far inside it: a row or column in the wrong place shows here.  Roundings
        # of both signs add as their root: a bf16 or 8-bit act leaves under 2^-6 of y's norm
        # (8-bit bytes that round the other way are a few in a thousand), fp32 under 2^-16
        lim = 2.0 ** -16 if self.dt == F32 else 2.0 ** -6
        assert float((self.y.to(D) - y).norm()) <= lim * float(y.norm()), name
        return self


SIZES = [
    # T, d, E, k, h, hs
    (1, 64, 8, 1, 32, 0),
    (1, 2048, 64, 6, 1408, 2816),
    (2, 96, 16, 16, 64, 32),          # every expert
    (3, 1056, 40, 5, 288, 96),
    (15, 128, 8, 2, 96, 64),
    (16, 160, 24, 3, 224, 0),
    (17, 160, 24, 3, 224, 160),
    (31, 288, 64, 8, 96, 0),
    (33, 512, 8, 3, 544, 256),
    (64, 256, 136, 7, 128, 320),
    (64, 128, 8, 8, 1056, 0),         # every row on every expert
    (5, 2080, 1024, 4, 32, 0),
    (64, 64, 1024, 16, 32, 64),       # every expert chosen, many with one row
]


@pytest.mark.parametrize("T,d,E,k,h,hs", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_layer_few(xm, T, d, E, k, h, hs, kind):
    c = Case(xm, T, d, E, k, h, hs, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8", bias=T % 2 == 1, tau=0.7 if T % 2 else 1.0)
    c.run().check(kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,h,hs", [(7, 200, 16, 3, 136, 72), (40, 1000, 8, 2, 24, 8), (4, 8, 8, 2, 8, 8),
                                          (20, 8, 16, 2, 1400, 0), (9, 1016, 32, 6, 8, 0)])
def test_sizes_that_are_multiples_of_eight_only(xm, T, d, E, k, h, hs, kind):
    Case(xm, T, d, E, k, h, hs, dt=F32 if kind == "f32" else BF, bias=True).run().check(kind)


@pytest.mark.parametrize("E,k", [(1, 1), (3, 2), (30, 5), (65, 65), (257, 3), (1023, 2)])
def test_f32_takes_any_number_of_experts(xm, E, k):
    Case(xm, 6, 72, E, k, 40, 16, dt=F32, bias=True).run().check()


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_all_tokens_on_the_same_experts(xm, kind):
    c = Case(xm, 64, 128, 32, 4, 96, 0, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8")
    c.sb = torch.zeros(32, device="cuda")
    c.sb[[3, 9, 30, 31]] = 100.0
    c.run().check(kind)
    assert all(sorted(r) == [3, 9, 30, 31] for r in c.ids.tolist())


def test_ties_go_to_the_lowest_index(xm):
    c = Case(xm, 9, 64, 136, 5, 32)
    c.x.zero_()
    c.run()
    torch.cuda.synchronize()
    assert c.ids.tolist() == [[0, 1, 2, 3, 4]] * 9
    assert float((c.p - 1 / 136).abs().max()) < 1e-7 and not c.y.any()


def test_masked_experts_and_bad_logits_keep_ids_valid(xm):
    c = Case(xm, 4, 64, 72, 6, 32)
    c.lb = torch.full((72,), -float("inf"), device="cuda")
    c.lb[[70, 2, 40]] = torch.tensor([0.0, 1.0, 2.0], device="cuda")
    c.run()
    assert all(set(r[:3]) == {2, 40, 70} for r in c.ids.tolist())       # the rest weigh nothing
    assert all(len(set(r)) == 6 and max(r) < 72 for r in c.ids.tolist())
    assert not c.p[:, 3:].any() and torch.isfinite(c.y).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        c.lb.fill_(bad)
        c.run()
        assert all(len(set(r)) == 6 and 0 <= min(r) and max(r) < 72 for r in c.ids.tolist()), bad
    # one token's NaN leaves the others' rows as they are
    c = Case(xm, 5, 64, 16, 3, 32, 32)
    clean = c.run().outs()
    c.x[2, 7] = float("nan")
    c.run()
    keep = [0, 1, 3, 4]
    assert torch.equal(c.y[keep], clean[3][keep]) and torch.equal(c.ids[keep], clean[0][keep])
    assert torch.isnan(c.y[2]).all()


def test_infinite_weights_reach_only_their_column(xm):
    """Also where K ends inside a step and the next expert's rows follow."""
    for dt in (BF, F32):
        c = Case(xm, 3, 72, 8, 8, 40, dt=dt)
        clean = c.run().outs()
        c.w[2][7, 39, 5] = float("inf")   # the last expert's last row, and one between two experts
        c.w[2][3, 39, 6] = float("inf")
        c.run()
        other = [i for i in range(72) if i not in (5, 6)]
        assert torch.equal(c.y[:, other], clean[3][:, other])
        assert not torch.isfinite(c.y[:, 5:7]).any()


def test_no_tokens(xm):
    c = Case(xm, 0, 64, 8, 2, 32, 32)
    c.run()
    c = Case(xm, 0, 64, 8, 2, 32, 32, mx8=True)
    c.run()
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("T", [1, 40])
def test_repeats_graphs_and_streams(xm, kind, T):
    """The same bits on every call: eager, on another stream, and in a graph that is
    replayed between eager calls on other workspaces; a workspace full of NaNs changes
    nothing, and nothing is written past its needed bytes."""
    c = Case(xm, T, 256, 64, 6, 160, 320, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8", bias=True)
    n = c.need()
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    want = c.run(workspace=ws).check(kind).outs()
    assert bool((ws[n:] == 255).all())
    other = Case(xm, T, 256, 64, 6, 160, 320, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8", seed=3)
    s = torch.cuda.Stream()
    for t in (c.ids, c.p, c.z, c.y):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c.outs()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(workspace=ws)
    for i in range(4):
        for t in (c.ids, c.p, c.z, c.y):
            t.zero_()
        other.run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, c.outs())), i
        ws.fill_(255)
    # new tokens in the same graph
    c.x.copy_(other.x)
    if kind == "mx8":
        c.xq.copy_(other.xq)
        c.xs.copy_(other.xs)
    g.replay()
    c.check("new tokens")


def test_two_streams_at_once(xm):
    cs = [Case(xm, 12, 512, 64, 6, 224, 96, seed=i, mx8=i % 2 == 1) for i in range(4)]
    want = [c.run().outs() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [torch.empty(c.need(), dtype=torch.uint8, device="cuda") for c in cs]
    for _ in range(5):
        for c, s, w in zip(cs, streams, ws):
            c.run(stream=s, workspace=w)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert all(torch.equal(a, b) for a, b in zip(w, c.outs()))


@pytest.mark.parametrize("mx8", [False, True])
def test_a_tokens_row_hardly_depends_on_the_batch(xm, mx8):
    """Tokens alone and together: what differs is the order of fp32 sums, and for 8-bit
    activations a byte that rounds the other way."""
    c = Case(xm, 24, 512, 64, 6, 256, 128, mx8=mx8)
    c.run().check()
    for t in (0, 13, 23):
        one = Case(xm, 1, 512, 64, 6, 256, 128, mx8=mx8)
        one.wg, one.w, one.s, one.x = c.wg, c.w, c.s, c.x[t:t + 1].clone()
        if mx8:
            one.xm.xmoe_mx8_quantize(one.x, one.xq, one.xs)
        one.run().check()
        assert torch.equal(one.ids[0], c.ids[t])
        assert float((one.y[0].double() - c.y[t].double()).norm()) <= 2.0 ** -6 * float(c.y[t].double().norm())
