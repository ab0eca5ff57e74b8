"""The fp32 tile product's two heights: calls of 512 tiles of 64 rows and more take these,
smaller ones 32 rows.  Every sum runs in ascending k on both, so that a large call gives
the bits of calls on its parts; and the large one is held to the 64-bit definition."""
import pytest
import torch

from _helpers import need_gpu

pytestmark = pytest.mark.gpu
F32, F64, I32 = torch.float32, torch.float64, torch.int32


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    return m


def _randn(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


def _tiles(rows, groups, cols):
    return (-(-rows // 64) + groups) * -(-cols // 64)


def test_router(xm):
    """Logits: each sum off by at most d 2^-24 of its products' magnitudes, then a
    product and an addition of 2^-24 each."""
    T, d, E, k = 8200, 200, 250, 3
    assert _tiles(T, 1, E) >= 512 > _tiles(1100, 1, E)
    r = _randn(1)
    x, wg, lb = r(T, d), r(d, E) * d ** -0.5, r(E)

    def run(x):
        n = x.shape[0]
        ids, w, z = torch.empty((n, k), dtype=I32, device="cuda"), torch.empty((n, k), device="cuda"), torch.empty((n, E), device="cuda")
        xm.xmoe_route(x, wg, k, ids, w, z, 0.7, lb)
        return ids, w, z

    whole = run(x)
    tau = torch.tensor(0.7).double().item()  # as the call has it, in fp32
    dot = x.to(F64) @ wg.to(F64)
    want = dot * tau + lb.to(F64)
    tol = d * 2.0 ** -24 * (x.abs().to(F64) @ wg.abs().to(F64)) * tau * 1.01 + 2.0 ** -23 * (dot.abs() * tau + want.abs())
    assert bool(((whole[2].to(F64) - want).abs() <= tol).all())
    for r0 in range(0, T, 1100):
        for a, b in zip(whole, run(x[r0:r0 + 1100].contiguous())):
            assert torch.equal(a[r0:r0 + 1100], b), r0


def test_swiglu_backward(xm):
    """dA off by d 2^-24 of its products' magnitudes; a sigmoid by 2^-20 + 2^-23 |a| of
    itself (exp2 of a product in fp32, and the instructions' own last bits)."""
    counts, d, h = [333, 1, 0, 790, 420], 72, 1288
    off, E = [0], len(counts)
    for c in counts:
        off.append(off[-1] + c)
    R = off[-1]
    assert _tiles(R, E, h) >= 512 > _tiles(790, 1, h)
    r = _randn(2)
    dy, w2, h13 = r(R, d), r(E, h, d) * h ** -0.5, r(R, 2 * h) * 2
    tok = torch.arange(R, device="cuda").flip(0).to(I32)
    wt = r(R).abs()

    def run(rows, e0, e1, offs):
        dh = torch.full((rows.stop - rows.start, 2 * h), 3.0, device="cuda")
        xm.xmoe_expert_ffn_bwd_dact_gather(dy, tok[rows].contiguous(), wt[rows].contiguous(), w2[e0:e1], h13[rows].contiguous(),
                                           torch.tensor(offs, dtype=I32, device="cuda"), dh)
        return dh

    whole = run(slice(0, R), 0, E, off)
    D = lambda t: t.to(F64)
    for e in range(E):
        i = slice(off[e], off[e + 1])
        if counts[e] == 0:
            continue
        rows, w = D(dy[tok[i].long()]), D(w2[e]).t().contiguous()
        da, dda = rows @ w, d * 2.0 ** -24 * (rows.abs() @ w.abs())
        v, h1, h3 = D(wt[i])[:, None], D(h13[i, :h]), D(h13[i, h:])
        sg = torch.sigmoid(h1)
        slope, rel = sg + h1 * sg * (1 - sg), 2.0 ** -20 + 2.0 ** -23 * h1.abs()
        s1 = slope.abs() + 2 * rel * sg * (1 + 2 * h1.abs())
        tol1 = rel * (v * da * h3 * slope).abs() + v * h3.abs() * s1 * dda * 1.01 + v * (da * h3).abs() * 2 * rel * sg * (1 + 2 * h1.abs()) + 1e-37
        tol3 = (2.0 ** -23 + rel) * (v * da * h1 * sg).abs() + v * (h1 * sg).abs() * dda * 1.01 + 1e-37
        assert bool(((D(whole[i, :h]) - v * da * h3 * slope).abs() <= tol1).all()), e
        assert bool(((D(whole[i, h:]) - v * da * h1 * sg).abs() <= tol3).all()), e
        assert torch.equal(whole[i], run(i, e, e + 1, [0, counts[e]])), e


def test_gate_gradient_added_to_dx(xm):
    """dx + dz . wg^T: E 2^-24 of the products' magnitudes, and the addition."""
    T, d, E, k = 2100, 1000, 27, 4
    assert _tiles(T, 1, d) >= 512 > _tiles(700, 1, d)
    r = _randn(3)
    x, wg, z, g, base = r(T, d), r(d, E) * d ** -0.5, r(T, E), r(T, k), r(T, d)
    ids = torch.topk(r(T, E), k, 1).indices.to(I32)

    def run(i, accumulate):
        n = i.stop - i.start
        dx, dwg = base[i].clone(), torch.empty((d, E), device="cuda")
        ws = torch.empty(max(xm.xmoe_route_bwd_workspace_size(n, d, E, F32), 16), dtype=torch.uint8, device="cuda")
        c = lambda t: t[i].contiguous()
        xm.xmoe_route_bwd(c(x), wg, c(z), c(ids), c(g), dx, dwg, ws, 0.7, accumulate=accumulate)
        return dx

    added, alone = run(slice(0, T), True), run(slice(0, T), False)
    p = torch.softmax(z.to(F64), 1)
    gp = torch.zeros_like(p).scatter_(1, ids.long(), g.to(F64))
    tau = torch.tensor(0.7).double().item()
    dz = p * (gp - (p * gp).sum(1, keepdim=True)) * tau
    # dz: p off by E 2^-24 (its sum) and 2^-20 (exp, division), each sum of E terms by as much
    ddz = (E * 2.0 ** -24 + 2.0 ** -20) * 3 * p * (gp.abs() + (p * gp.abs()).sum(1, keepdim=True)) * tau
    w = wg.to(F64).t().contiguous()
    want, tol = dz @ w, ddz @ w.abs() + E * 2.0 ** -24 * (dz.abs() @ w.abs()) * 1.01
    assert bool(((alone.to(F64) - want).abs() <= tol + 2.0 ** -24 * want.abs()).all())
    want = want + base.to(F64)
    assert bool(((added.to(F64) - want).abs() <= tol + 2.0 ** -24 * want.abs() + 2.0 ** -24 * tol).all())
    for r0 in range(0, T, 700):
        i = slice(r0, r0 + 700)
        assert torch.equal(added[i], run(i, True)) and torch.equal(alone[i], run(i, False)), r0
