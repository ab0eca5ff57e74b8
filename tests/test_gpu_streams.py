"""Calls on streams that are not the current one: whose memory their workspaces
are, and the results of two callers at once."""
import pytest
import torch

import _block_ref as br
from _helpers import need_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.fixture
def taken(xm, monkeypatch):
    """(address, bytes) of every workspace that a call allocates."""
    seen, inner = [], xm._workspace

    def spy(ws, need, like, stream=None):
        t, n = inner(ws, need, like, stream)
        if ws is None:
            seen.append((t.data_ptr(), n))
        return t, n

    monkeypatch.setattr(xm, "_workspace", spy)
    return seen


def _freed(need):
    """Address of a block of `need` bytes that was just freed on the current stream,
    and that the next allocation there is given."""
    a = torch.empty(need, dtype=torch.uint8, device="cuda")
    at = a.data_ptr()
    del a
    b = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert b.data_ptr() == at
    return at


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_workspaces_on_another_stream(xm, taken, handle):
    """A call on another stream does not take the block that the current stream gave
    back, and has the bits of the call on the current one."""
    T, d, E, k = 4096, 2048, 64, 6
    g = _gen(1)
    s, dy = (torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rstd = torch.rsqrt(s.float().square().mean(1) + EPS)
    logits = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.topk(logits, k, 1).indices.to(torch.int32)
    st = torch.cuda.Stream()
    out = []
    for stream in (None, st.cuda_stream if handle else st):
        dx, dg = torch.empty_like(s), torch.empty(d, device="cuda")
        loss, counts = torch.empty(1, device="cuda"), torch.empty((1, E), dtype=torch.int32, device="cuda")
        coef = torch.empty((1, E), device="cuda")
        calls = (
            (xm.xmoe_add_rmsnorm_bwd_workspace_size(T, d, s.dtype),
             lambda: xm.xmoe_add_rmsnorm_bwd(dy, None, s, gamma, rstd, dx, dg, stream=stream)),
            (xm.xmoe_balance_loss_workspace_size(T, E),
             lambda: xm.xmoe_balance_loss(logits, ids, 0.1, loss, counts, coef, stream=stream)))
        torch.cuda.synchronize()
        for need, call in calls:
            at = _freed(need)
            del taken[:]
            call()
            (ws, n), = taken
            assert n >= need
            if stream is not None:
                assert ws + n <= at or at + need <= ws, "took the current stream's block"
        torch.cuda.synchronize()
        out.append((dx, dg, loss, counts, coef))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def _serving(seed=0):
    import workloads
    wl = workloads.Workload("streams8", "bf16", T=40, d=512, E=64, h=1408, k=6, n_shared=1, h_shared=512, backward=True)
    inp = {k: v.cuda() for k, v in workloads.generate(wl).items() if v is not None}
    w = {k: inp[k] for k in ("wg", "w1", "w3", "w2", "s1", "s3", "s2")}
    w["norm"] = torch.ones(wl.d, dtype=torch.bfloat16, device="cuda")
    return wl, w, inp["x"]


def _busy(ms=10):
    """Work of some milliseconds queued on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    for _ in range(ms):
        a @ a


def test_a_forward_on_another_stream_behind_the_quantization(xm):
    """Constructed, or refreshed, behind queued work on one stream, and run at once on
    another: the bits of a block that is waited for."""
    from padding_free_expert_amd.layer import MoEBlock8
    wl, w, x = _serving()
    want = MoEBlock8(w, wl.T, wl.k).forward(x)[0].clone()
    st, rt = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy()
    block = MoEBlock8(w, wl.T, wl.k)
    out, _ = block.forward(x, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for n in ("w1", "w3", "w2", "s1", "s3", "s2"):
        w[n].mul_(0.5)
    want = MoEBlock8(w, wl.T, wl.k).forward(x)[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(rt):
        _busy()
        block.refresh_weights()
    out, _ = block.forward(x, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_two_callers_at_once(xm):
    """Calls that allocate their workspaces, on two streams with no order between
    them, each on inputs and outputs of its own: the bits each has alone."""
    T, d, E, k, S = 4096, 2048, 64, 6, 3
    off = torch.tensor([0, 1000, 1001, T - 5], dtype=torch.int32, device="cuda")
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")

    class Caller:
        def __init__(self, seed):
            g = _gen(seed)
            self.s, self.dy = (torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            self.rstd = torch.rsqrt(self.s.float().square().mean(1) + EPS)
            self.logits = torch.randn((T, E), generator=g, device="cuda")
            self.ids = torch.topk(self.logits, k, 1).indices.to(torch.int32)
            self.out = self.buffers()

        @staticmethod
        def buffers():
            return dict(dx=torch.empty((T, d), dtype=torch.bfloat16, device="cuda"), dg=torch.empty(d, device="cuda"),
                        loss=torch.empty(1, device="cuda"), counts=torch.empty((S, E), dtype=torch.int32, device="cuda"),
                        coef=torch.empty((S, E), device="cuda"))

        def call(self, o, stream=None):
            xm.xmoe_add_rmsnorm_bwd(self.dy, None, self.s, gamma, self.rstd, o["dx"], o["dg"], stream=stream)
            xm.xmoe_balance_loss(self.logits, self.ids, 0.1, o["loss"], o["counts"], o["coef"], off, stream=stream)

    callers, ss = [Caller(1), Caller(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for c in callers:
        alone.append(c.buffers())
        c.call(alone[-1])
        torch.cuda.synchronize()
    assert not torch.equal(alone[0]["coef"], alone[1]["coef"])
    _busy(2)     # what the current stream gives back meanwhile stays its own
    for _ in range(10):
        for c, st in zip(callers, ss):
            c.call(c.out, stream=st)
    torch.cuda.synchronize()
    for c, a in zip(callers, alone):
        for n, t in c.out.items():
            assert torch.equal(t, a[n]), n


@pytest.mark.parametrize("S", [1, 3, 70])
def test_workspaces_of_captured_calls_on_a_forked_stream(xm, S):
    """Calls that allocate their workspaces, captured on a stream forked from the
    capture's: every replay on new inputs has the bits of eager calls, with eager
    work and synchronizations between the replays."""
    T, d, E, k = 2500, 512, 160, 6
    g = _gen(S)
    off = None if S == 1 else torch.linspace(0, T - 3, S + 1, device="cuda").to(torch.int32)
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    s, dy = (torch.empty((T, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rstd, logits = torch.empty(T, device="cuda"), torch.empty((T, E), device="cuda")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")

    def fill():
        s.copy_(torch.randn((T, d), generator=g, device="cuda"))
        dy.copy_(torch.randn((T, d), generator=g, device="cuda"))
        rstd.copy_(torch.rsqrt(s.float().square().mean(1) + EPS))
        logits.copy_(torch.randn((T, E), generator=g, device="cuda"))
        ids.copy_(torch.topk(logits, k, 1).indices)

    def buffers():
        return (torch.empty_like(s), torch.empty(d, device="cuda"), torch.empty(1, device="cuda"),
                torch.empty((S, E), dtype=torch.int32, device="cuda"), torch.empty((S, E), device="cuda"))

    def call(o, stream=None):
        xm.xmoe_add_rmsnorm_bwd(dy, None, s, gamma, rstd, o[0], o[1], stream=stream)
        xm.xmoe_balance_loss(logits, ids, 0.1, o[2], o[3], o[4], off, stream=stream)

    fill()
    got, want = buffers(), buffers()
    call(got)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        call(got, side)
        main.wait_stream(side)
    for i in range(5):
        fill()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        call(want)
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, n)
