"""Norm, gate with balance loss and experts run together, as a transformer block
uses them: the training block against autograd in 64 bits, the serving block
with 8-bit experts against its 64-bit definition, both captured as graphs and on
other streams.

Tolerances are the layer's: normwise 1e-4 in fp32 and 2e-2 in bf16 (and for the
8-bit block, whose act bytes may round the other way where the sums differ in
the last bits).  The references take the GPU's expert choice (a choice between
near ties is checked by the gate's own tests)."""
import pytest
import torch

import _block_ref as br
import workloads
from _helpers import need_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6
ALPHA = 0.5


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    return m


def _near(got, ref, rtol, name):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    n = float(ref.norm())
    err = float((got - ref).norm())
    assert err <= rtol * n + 1e-30, f"{name}: off by {err / max(n, 1e-300):.2e} of its norm"


def _inputs(wl, seed=0):
    inp = {k: v.cuda() for k, v in workloads.generate(wl, backward=True).items() if v is not None}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    dt = inp["x"].dtype
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    weights = {k: inp[k] for k in ("wg", "w1", "w3", "w2", "s1", "s3", "s2", "logit_bias", "select_bias") if k in inp}
    weights["norm"] = (1 + 0.2 * rnd(wl.d)).to(dt)
    return inp, weights, (2 * rnd(wl.T, wl.d)).to(dt), rnd(wl.T, wl.d).to(dt), g


def _reference(wl, weights, x, res, dout, dsum, ids, off, mask, up):
    """Autograd in 64 bits on the CPU, the expert choice given."""
    leaf = {k: v.double().cpu().requires_grad_() for k, v in weights.items() if k not in ("select_bias", "logit_bias")}
    x64 = x.double().cpu().requires_grad_()
    s = x64 + res.double().cpu()
    # the stored sum's rounding, passed through
    s = s + (s.detach().to(x.dtype).double() - s.detach())
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * leaf["norm"]
    z = y @ leaf["wg"] * wl.inv_tau
    if "logit_bias" in weights:
        z = z + weights["logit_bias"].double().cpu()
    p = torch.softmax(z, 1)
    ids = ids.cpu().long()
    out = torch.zeros_like(y)
    silu = torch.nn.functional.silu
    for e in range(wl.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            f = (silu(y[t] @ leaf["w1"][e]) * (y[t] @ leaf["w3"][e])) @ leaf["w2"][e]
            out = out.index_add(0, t, f * p[t, e][:, None])
    if "s1" in leaf:
        out = out + (silu(y @ leaf["s1"]) * (y @ leaf["s3"])) @ leaf["s2"]
    pick = br.sequences(wl.T, off.cpu() if off is not None else None, mask.cpu() if mask is not None else None, "cpu")
    some = max(1, sum(len(i) > 0 for i in pick))
    loss = torch.zeros((), dtype=torch.float64)
    for i in pick:
        if len(i):
            c = torch.bincount(ids[i].flatten(), minlength=wl.E).double()
            loss = loss + ALPHA / some * (wl.E * c / (wl.k * len(i)) * p[i].mean(0)).sum()
    total = (out * dout.double().cpu()).sum() + (s * dsum.double().cpu()).sum() + up * loss
    total.backward()
    return out, s, loss, x64.grad, leaf


CASES = {
    "f32": workloads.Workload("block_f32", "f32", T=75, d=96, E=12, h=40, k=3, n_shared=1, h_shared=56, backward=True),
    "bf16": workloads.Workload("block_bf16", "bf16", T=300, d=256, E=16, h=200, k=6, n_shared=2, h_shared=200,
                               backward=True),
    "bf16_many": workloads.Workload("block_many", "bf16", T=150, d=128, E=160, h=64, k=8, inv_tau=0.5, zipf_s=1.1,
                                    backward=True),
}


@pytest.mark.parametrize("seqs", [False, True], ids=["batch", "sequences"])
@pytest.mark.parametrize("name", list(CASES))
def test_training_block(xm, name, seqs):
    from padding_free_expert_amd.layer import MoEBlock
    wl = CASES[name]
    inp, weights, res, dsum, g = _inputs(wl)
    off = torch.tensor([0, wl.T // 3, wl.T // 3, wl.T - 7], dtype=torch.int32, device="cuda") if seqs else None
    mask = (torch.rand(wl.T, generator=g, device="cuda") < 0.8) if seqs else None
    up = torch.tensor([1.5], device="cuda")
    rtol = 1e-4 if wl.dtype == "f32" else 2e-2
    for kw in (dict(), dict(overlap=False), dict(lean=True)):
        block = MoEBlock(weights, wl.T, wl.k, EPS, inv_tau=wl.inv_tau, balance_alpha=ALPHA, n_seq=3 if seqs else 1, **kw)
        out, s = block.forward(inp["x"], res, seq_offsets=off, token_mask=mask)
        dx = block.backward(inp["dy"], dsum, dloss=up)
        torch.cuda.synchronize()
        m = block.moe
        ro, rs, rl, rdx, leaf = _reference(wl, weights, inp["x"], res, inp["dy"], dsum, m.topk_ids, off, mask, 1.5)
        _near(s, rs, 0.0, "sum")
        for got, ref, what in ((out, ro, "out"), (m.loss, rl.reshape(1), "loss"), (dx, rdx, "dx"),
                               (block.dgamma, leaf["norm"].grad, "dgamma"), (m.dwg, leaf["wg"].grad, "dwg"),
                               (m.dw1, leaf["w1"].grad, "dw1"), (m.dw3, leaf["w3"].grad, "dw3"),
                               (m.dw2, leaf["w2"].grad, "dw2")):
            _near(got, ref, rtol, f"{what} {kw}")
        live = torch.ones(wl.T, dtype=torch.bool, device="cuda") if mask is None else mask.clone()
        if seqs:
            live[wl.T - 7:] = False
        assert int(m.counts.sum()) == int(live.sum()) * wl.k


def test_the_loss_leaves_the_rest_of_the_layer_as_it_was(xm):
    """With alpha 0 the layer is the one without the loss, bit for bit; with the
    loss, everything but the gate's gradient (and dx) is."""
    from padding_free_expert_amd.layer import PaddingFreeMoE
    wl = CASES["bf16"]
    inp, weights, _, _, _ = _inputs(wl)
    a, b = PaddingFreeMoE(weights, wl.T, wl.k), PaddingFreeMoE(weights, wl.T, wl.k, balance_alpha=ALPHA)
    for m in (a, b):
        m.forward(inp["x"])
        m.backward(inp["dy"])
    torch.cuda.synchronize()
    assert torch.equal(a.y, b.y) and torch.equal(a.dw1, b.dw1) and torch.equal(a.dw2, b.dw2)
    assert not torch.equal(a.dwg, b.dwg)
    zero = torch.zeros(1, device="cuda")
    b.backward(inp["dy"], dloss=zero)
    torch.cuda.synchronize()
    assert torch.equal(a.dwg, b.dwg) and torch.equal(a.dx, b.dx)


def test_training_block_as_a_graph(xm):
    """Forward and backward captured; every replay on new inputs equals the eager
    step on them, with eager work and synchronizations between replays."""
    from padding_free_expert_amd.layer import MoEBlock
    wl = CASES["bf16"]
    inp, weights, res, dsum, g = _inputs(wl)
    off = torch.tensor([0, 100, 290], dtype=torch.int32, device="cuda")
    kw = dict(balance_alpha=ALPHA, n_seq=2)
    block, eager = MoEBlock(weights, wl.T, wl.k, EPS, **kw), MoEBlock(weights, wl.T, wl.k, EPS, **kw)
    x, r, dy = inp["x"].clone(), res.clone(), inp["dy"].clone()
    up = torch.ones(1, device="cuda")
    cs = torch.cuda.Stream()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        block.forward(x, r, seq_offsets=off)
        block.backward(dy, dsum, dloss=up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cs):
        block.forward(x, r, seq_offsets=off)
        block.backward(dy, dsum, dloss=up)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(x.dtype))
        up.fill_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        eager.forward(x, r, seq_offsets=off)
        eager.backward(dy, dsum, dloss=up)
        torch.cuda.synchronize()
        for name in ("y", "dwg", "dx", "loss", "counts"):
            assert torch.equal(getattr(block.moe, name), getattr(eager.moe, name)), (i, name)
        assert torch.equal(block.dx, eager.dx) and torch.equal(block.dgamma, eager.dgamma), i


def _serve_reference(wl, weights, x, res, ids, wq):
    """The serving block in 64 bits with the quantized weights given."""
    s, _, y = br.norm_ref(x, res, weights["norm"], EPS)
    yb = y.to(torch.bfloat16).double()
    z = yb @ weights["wg"].double() * wl.inv_tau
    p = torch.softmax(z, 1)

    def q(v):
        return br.mx8_round(v, br.mx8_bytes(v))

    def ffn(v, a, b, c):
        h1, h3 = v @ a.t(), v @ b.t()
        return q(h1 * torch.sigmoid(h1) * h3) @ c.t()

    yq = q(y)
    out = torch.zeros_like(y)
    for e in range(wl.E):
        t, _ = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            out[t] += ffn(yq[t], *(br.mx8_values(a[e], b[e]) for a, b in wq[:3])) * p[t, e][:, None]
    if len(wq) > 3:
        out += ffn(yq, *(br.mx8_values(a[0], b[0]) for a, b in wq[3:]))
    return out, s


SERVE = {
    "1 token": workloads.Workload("serve1", "bf16", T=1, d=256, E=64, h=96, k=6, n_shared=1, h_shared=160, backward=True),
    "decode": workloads.Workload("serve24", "bf16", T=24, d=512, E=16, h=224, k=4, backward=True),
    "prompt": workloads.Workload("serve700", "bf16", T=700, d=256, E=8, h=416, k=3, n_shared=2, h_shared=96,
                                 backward=True),
    "many experts": workloads.Workload("serve160", "bf16", T=90, d=160, E=160, h=64, k=8, backward=True),
}


@pytest.mark.parametrize("name", list(SERVE))
def test_serving_block(xm, name):
    from padding_free_expert_amd.layer import MoEBlock8
    wl = SERVE[name]
    inp, weights, res, _, _ = _inputs(wl)
    for overlap in (True, False):
        block = MoEBlock8(weights, wl.T, wl.k, wl.inv_tau, EPS, overlap=overlap)
        out, s = block.forward(inp["x"], res)
        torch.cuda.synchronize()
        wq = [block.w1q, block.w3q, block.w2q] + ([block.s1q, block.s3q, block.s2q] if block.shared else [])
        ref, rs = _serve_reference(wl, weights, inp["x"], res, block.topk_ids, wq)
        assert torch.equal(s, rs)
        _near(out, ref, 2e-2, f"out {name}")


def test_serving_block_on_another_stream_and_as_a_graph(xm):
    from padding_free_expert_amd.layer import MoEBlock8
    wl = SERVE["1 token"]
    inp, weights, res, _, g = _inputs(wl)
    block, eager = MoEBlock8(weights, 1, wl.k, eps=EPS), MoEBlock8(weights, 1, wl.k, eps=EPS)
    x, r = inp["x"].clone(), res.clone()
    want = [t.clone() for t in eager.forward(x, r)]
    cs = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = block.forward(x, r, stream=cs)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cs):
        block.forward(x, r)
    for i in range(5):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = eager.forward(x, r)
        torch.cuda.synchronize()
        assert torch.equal(block.out, want[0]) and torch.equal(block.sum, want[1]), i


def test_calls_on_two_streams_at_once(xm):
    """Two callers with buffers of their own, on two streams, no order between
    them: each has the bits it has alone."""
    from padding_free_expert_amd.layer import MoEBlock8
    wl = SERVE["prompt"]
    inp, weights, res, _, g = _inputs(wl)
    xs = [inp["x"], torch.randn((wl.T, wl.d), generator=g, device="cuda").to(torch.bfloat16)]
    blocks = [MoEBlock8(weights, wl.T, wl.k, eps=EPS) for _ in xs]
    alone = []
    for b, x in zip(blocks, xs):
        alone.append(b.forward(x, res)[0].clone())
    ss = [torch.cuda.Stream() for _ in xs]
    logits = torch.randn((4096, 64), generator=g, device="cuda")
    ids = torch.topk(logits, 6, 1).indices.to(torch.int32)
    loss = [torch.empty(1, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, x, st, l in zip(blocks, xs, ss, loss):
            b.forward(x, res, stream=st)
            # workspaces allocated in the call, on a stream that is not the current one
            xm.xmoe_balance_loss(logits, ids, 0.1, l, torch.empty((1, 64), dtype=torch.int32, device="cuda"),
                                 torch.empty((1, 64), device="cuda"), stream=st)
    torch.cuda.synchronize()
    for b, a in zip(blocks, alone):
        assert torch.equal(b.out, a)
    assert torch.equal(loss[0], loss[1])
