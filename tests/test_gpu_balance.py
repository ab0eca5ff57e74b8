"""Balance loss, counts and gradient against the 64-bit definition.

Bounds.  p: the argument of exp carries |s - max| times 2.25 * 2^-24 (the
difference, log2(e) in fp32 and the product), at most 24 times here (draws of
1.5 normal + normal) or nothing of a p, exp, the denominator and the division
ten halves more: 64 * 2^-24 = 2^-18 relative.  A
sum of p has positive terms, at most 128 / 4 in sequence in a lane and a tree
above it, then 64-bit sums: 2^-18 more.  coef is formed in 64 bits from
alpha, rounded to fp32 by the call, and rounded once itself: (1 + 2^-24)^2 - 1,
just above 2^-23."""
import pytest
import torch

import _block_ref as br
from _helpers import need_gpu

pytestmark = pytest.mark.gpu
P = 2.0 ** -18


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    return m


def _case(T, E, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits = 1.5 * torch.randn((T, E), generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(logits, k, 1).indices.to(torch.int32).contiguous()
    return logits, ids, g


def _run(xm, logits, ids, alpha, off, mask, dloss=None):
    T, E = logits.shape
    S = 1 if off is None else off.shape[0] - 1
    G = br.Guarded()
    loss, counts = G.empty((1,), torch.float32), G.empty((S, E), torch.int32)
    coef, dz = G.empty((S, E), torch.float32), G.empty((T, E), torch.float32)
    ws = G.empty((xm.xmoe_balance_loss_workspace_size(T, E, S),), torch.uint8)
    xm.xmoe_balance_loss(logits, ids, alpha, loss, counts, coef, off, mask, ws)
    xm.xmoe_balance_loss_bwd(logits, coef, dz, off, mask, dloss)
    G.check()
    return loss, counts, coef, dz


def _check(xm, logits, ids, k, off, mask, alpha=0.01, up=None):
    dloss = None if up is None else torch.tensor([up], device="cuda")
    loss, counts, coef, dz = _run(xm, logits, ids, alpha, off, mask, dloss)
    rl, rc, rf, p = br.balance_ref(logits, ids, k, off, mask, alpha)
    assert torch.equal(counts.long(), rc)
    br.close(coef, rf, 2.0 ** -23 + 2.0 ** -48, name="coef")
    br.close(loss, torch.tensor([rl], device="cuda"), 2 * P, name="loss")
    g, mag = br.balance_grad_ref(p, rf, off, mask)
    u = 1.0 if up is None else up
    br.close(dz, g * u, 0.0, 2 * P * abs(u) * mag, "dlogits")
    # deterministic, whatever order the blocks run in
    again = _run(xm, logits, ids, alpha, off, mask, dloss)
    for a, b in zip((loss, counts, coef, dz), again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (15, 8, 8), (16, 64, 6), (17, 33, 3), (100, 100, 5), (512, 160, 8),
                                   (1000, 129, 1), (4096, 64, 6), (8193, 256, 8), (70000, 24, 2), (300, 513, 7),
                                   (257, 1024, 64), (33, 1021, 8), (16391, 50, 3), (16384, 97, 2), (20001, 192, 8),
                                   (16399, 250, 4)])
def test_one_sequence(xm, T, E, k):
    print(f"[balance] T={T} E={E} k={k}", flush=True)
    logits, ids, g = _case(T, E, k, seed=T + E)
    _check(xm, logits, ids, k, None, None)
    mask = torch.rand(T, generator=g, device="cuda") < 0.6
    _check(xm, logits, ids, k, None, mask, alpha=1.0, up=-3.0)


@pytest.mark.parametrize("T,E,k,off", [
    (40, 16, 2, [0, 40]), (40, 16, 2, [0, 0, 40, 40]), (40, 16, 2, [3, 10, 10, 10, 33]),
    (300, 64, 6, [0, 16, 32, 33, 300]), (1000, 40, 4, [0, 1, 2, 3, 900, 901, 1000]),
    (2000, 160, 8, [100, 100]), (129, 512, 3, [0, 128, 129]), (17000, 72, 6, [5, 9000, 9000, 16003, 16999])])
def test_sequences(xm, T, E, k, off):
    print(f"[balance] T={T} E={E} off={off}", flush=True)
    logits, ids, g = _case(T, E, k, seed=T)
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    _check(xm, logits, ids, k, off, None, up=0.5)
    mask = torch.rand(T, generator=g, device="cuda") < 0.5
    mask[: T // 3] = False
    _check(xm, logits, ids, k, off, mask.to(torch.uint8))


@pytest.mark.parametrize("T,S", [(5000, 4096), (9000, 1025), (4097, 65), (600, 600)])
def test_many_short_sequences(xm, T, S):
    g = torch.Generator()
    g.manual_seed(S)
    cut = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g)).values
    off = torch.cat([torch.tensor([0]), cut, torch.tensor([T - 3])]).sort().values.to(torch.int32).cuda()
    logits, ids, _ = _case(T, 16, 2, seed=S)
    _check(xm, logits, ids, 2, off, None)


def test_nothing_counts(xm):
    logits, ids, _ = _case(64, 16, 2, seed=1)
    logits[:] = float("nan")     # nothing of it may reach the outputs
    mask = torch.zeros(64, dtype=torch.bool, device="cuda")
    loss, counts, coef, dz = _run(xm, logits, ids, 0.1, None, mask)
    for t in (loss, counts, coef, dz):
        assert bool((t == 0).all())
    e = torch.empty((0, 16), device="cuda")
    loss, counts, coef, dz = _run(xm, e, torch.empty((0, 2), dtype=torch.int32, device="cuda"), 0.1, None, None)
    assert float(loss) == 0 and bool((counts == 0).all()) and bool((coef == 0).all())


def test_masked_tokens_may_hold_anything(xm):
    T, E, k = 90, 40, 4
    logits, ids, g = _case(T, E, k, seed=2)
    mask = torch.rand(T, generator=g, device="cuda") < 0.5
    off = torch.tensor([0, 30, 80], dtype=torch.int32, device="cuda")
    want = _run(xm, logits, ids, 0.1, off, mask)
    dead = ~mask
    dead[80:] = True
    logits[dead] = float("nan")
    ids[dead] = 1 << 30
    got = _run(xm, logits, ids, 0.1, off, mask)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_excluded_experts_and_odd_ids(xm):
    """-infinity excludes an expert; ids outside [0, E) are not counted; an id
    twice in a token counts twice."""
    T, E, k = 50, 24, 3
    logits, ids, _ = _case(T, E, k, seed=3)
    logits[:, 5] = float("-inf")
    ids[0] = torch.tensor([7, 7, 7], device="cuda")
    ids[1] = torch.tensor([-1, E, 2], device="cuda")
    _check(xm, logits, ids, k, None, None)


def test_rows_of_lowest_values(xm):
    """Masks of the type's lowest value: a row with nothing else is uniform, and
    large logits stay finite."""
    big = torch.finfo(torch.float32).max
    for T, E, k in ((40, 24, 3), (70, 33, 2), (64, 160, 8)):
        logits, ids, _ = _case(T, E, k, seed=4)
        logits[0] = -big
        logits[1, 1:] = -big
        logits[2] = big
        logits[3, ::2] = -big
        logits[4] = -big
        logits[4, E - 1] = big
        logits[5] += 1e9
        logits[6] = -3e30
        logits[7, : E // 2] = float("-inf")
        logits[7, E // 2:] = -big
        _check(xm, logits, ids, k, None, None, alpha=1.0)


def test_gradient_against_differences(xm):
    """d loss / d logits against central differences of the loss with the counts
    held (they carry no gradient): step 2^-6 leaves 2^-12 relative, the loss's
    own rounding 2^-24 loss / 2^-6."""
    T, E, k = 8, 6, 2
    logits, ids, _ = _case(T, E, k, seed=5)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    loss, _, _, dz = _run(xm, logits, ids, 1.0, off, None)
    h = 2.0 ** -6
    for t, e in ((0, 0), (2, 5), (3, 1), (7, 4)):
        d = torch.zeros_like(logits)
        d[t, e] = h
        up = _run(xm, logits + d, ids, 1.0, off, None)[0].double()
        dn = _run(xm, logits - d, ids, 1.0, off, None)[0].double()
        br.close(dz[t, e].reshape(1), (up - dn) / (2 * h), 2.0 ** -8, 2.0 ** -15 * float(loss), f"dz[{t},{e}]")


@pytest.mark.parametrize("dtype,T,d,E,k,S,mask", [("f32", 60, 40, 12, 3, 1, False), ("f32", 200, 64, 33, 4, 5, True),
                                                  ("bf16", 300, 256, 64, 6, 3, True), ("bf16", 700, 128, 160, 8, 1, False)])
def test_gate_backward_with_the_loss(xm, dtype, T, d, E, k, S, mask):
    """dx and dwg of the gate with the loss's gradient: both gradients' sum.
    Tolerances as the gate's backward elsewhere: bf16 rounds dz to bf16 once."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    logits, ids, g = _case(T, E, k, seed=9)
    x = torch.randn((T, d), generator=g, device="cuda").to(dt)
    wg = (torch.randn((d, E), generator=g, device="cuda") * d ** -0.5).to(dt)
    dw = torch.randn((T, k), generator=g, device="cuda")
    off = None if S == 1 else torch.linspace(0, T - 2, S + 1, device="cuda").to(torch.int32)
    m = (torch.rand(T, generator=g, device="cuda") < 0.7) if mask else None
    alpha, tau, up = 50.0, 0.7, torch.tensor([2.0], device="cuda")
    loss, counts, coef, _ = _run(xm, logits, ids, alpha, off, m)
    ws = torch.empty(xm.xmoe_route_bwd_workspace_size(T, d, E, dt), dtype=torch.uint8, device="cuda")
    dx, dwg = torch.zeros_like(x), torch.empty((d, E), device="cuda")
    xm.xmoe_route_bwd_balance(x, wg, logits, ids, dw, coef, dx, dwg, ws, tau, accumulate=False, seq_offsets=off,
                              token_mask=m, dloss=up)
    _, _, rf, p = br.balance_ref(logits, ids, k, off, m, alpha)
    g2 = torch.zeros_like(p).scatter_(1, ids.long(), dw.double())
    for s, i in enumerate(br.sequences(T, off, m, "cuda")):
        g2[i] += 2.0 * rf[s]
    c = (p * g2).sum(1, keepdim=True)
    dz, mag = p * (g2 - c) * tau, p * (g2.abs() + c.abs()) * tau
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17
    W, X = wg.double(), x.double()
    # each term of a product carries dz's error; the result its own rounding
    br.close(dx, dz @ W.t(), br.half_step(dt) * 1.01, 1.01 * eps * (mag @ W.abs().t()), "dx")
    br.close(dwg, X.t() @ dz, 2.0 ** -24, 1.01 * eps * (X.abs().t() @ mag), "dwg")
    # without the loss's coefficients: the gate's own backward, bit for bit
    a, b = torch.empty_like(dx), torch.empty_like(dwg)
    xm.xmoe_route_bwd(x, wg, logits, ids, dw, a, b, ws, tau, accumulate=False)
    zero = torch.zeros_like(coef)
    xm.xmoe_route_bwd_balance(x, wg, logits, ids, dw, zero, dx, dwg, ws, tau, accumulate=False, seq_offsets=off,
                              token_mask=m)
    assert torch.equal(a, dx) and torch.equal(b, dwg)
