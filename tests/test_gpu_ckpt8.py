"""Pre-activations kept in 8 bits: the up-projection that stores them, the backward that
reads them, and the training layer with them, against 64-bit definitions.

Bounds.  Quantizing given fp32 sums is exact arithmetic and one rounding; where the sums
are whole numbers below 2^24 the bytes must be equal, else each value is within half a
step of the stored scale of a sum that is off by at most K 2^-24 of its products'
magnitudes.  The backward is fp32 arithmetic on exact values: dA off by d 2^-24 of its
products' magnitudes, a few roundings and the exp's and reciprocal's own error, and the output's
half step.  exp(-a) is exp2 of the fp32 product a log2(e): that product, at most 1.45 |a|,
is off by 2^-24 of itself for its rounding and 2^-25 for the constant's, so exp by ln 2
times that, under 1.5 |a| 2^-24 relative; for negative a the sigmoid is off by as much.
With the instructions' own last bits (2^-20 in all) a sigmoid's relative error is at most
2^-20 + 2^-23 |a|."""
import pytest
import torch

import _ckpt8_ref as ref
import workloads
from _block_ref import half_step
from _helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, F64, I32, U8, I8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8, torch.int8


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


def _offsets(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


# counts, d, h, T (None: not gathered), spare rows: every tile height and choice of
# tiles (large tiles from 1024 rows an expert, or a well filled last tile), widths that
# end inside a block of 32, of 128 and of a tile
CASES = {
    "one row": ([1], 8, 8, None, 0),
    "empty experts": ([0, 5, 0, 0, 33, 0], 72, 40, 9, 0),
    "all empty": ([0, 0, 0], 64, 32, 4, 3),
    "ragged": ([31, 0, 64, 1, 127, 128, 129, 3], 200, 136, 77, 5),
    "narrow": ([70, 3], 64, 24, 30, 0),
    "two column tiles": ([40, 90], 96, 264, None, 11),
    "wide": ([130, 17], 40, 1048, 60, 0),
    "256 wide": ([300, 200], 128, 512, 90, 0),
    "large tiles": ([1100, 1500], 64, 16384, 700, 0),
    "large tiles, few columns": ([5000], 136, 6664, None, 0),
    "well filled tile": ([384] * 16, 160, 4160, 500, 0),
}


def _case(name, dt, seed=0, whole=False):
    counts, d, h, T, spare = CASES[name]
    g = _gen(seed + len(name))
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    E, off = len(counts), _offsets(counts)
    R = off[-1] + spare
    n = T or R
    if whole:  # sums of whole numbers: below 2^24, exact in any order
        i = lambda lo, *s: torch.randint(-lo, lo + 1, s, generator=g, device="cuda").to(dt)
        x, w = i(9, n, d), lambda *s: i(5, *s)
    else:
        x, w = r(n, d).to(dt), lambda *s: (r(*s) * s[1] ** -0.5).to(dt)
    tok = None
    if T:
        tok = torch.randint(0, T, (R,), generator=g, device="cuda").to(I32)
    return dict(E=E, off=off, offsets=torch.tensor(off, dtype=I32, device="cuda"), R=R, d=d, h=h, x=x, tok=tok,
                w1=w(E, d, h), w3=w(E, d, h), w2=(r(E, h, d) * h ** -0.5).to(dt), dy=r(n, d).to(dt), g=g, spare=spare,
                weights=torch.rand(R, generator=g, device="cuda"), perm=torch.randperm(R, generator=g, device="cuda"))


def _up(xm, c, dt, **kw):
    R, h = c["R"], c["h"]
    act = torch.full((R, h), 3.0, dtype=dt, device="cuda")
    hq = torch.full((R, 2 * h), 77, dtype=I8, device="cuda")
    hs = torch.full(xm.ckpt8_scale_shape(R, h), 99, dtype=U8, device="cuda")
    xm.xmoe_expert_ffn_up_ckpt8(c["x"], c["w1"], c["w3"], c["offsets"], act, hq, hs, token_ids=c["tok"], **kw)
    return act, hq, hs


def _sums(c):
    """float64 H1, H3 and the magnitudes of their products."""
    n = c["off"][-1]
    rows = (c["x"] if c["tok"] is None else c["x"][c["tok"].long()]).to(F64)
    out = [torch.empty((n, c["h"]), dtype=F64, device="cuda") for _ in range(4)]
    for e in range(c["E"]):
        i = slice(c["off"][e], c["off"][e + 1])
        for b, w in enumerate((c["w1"][e].to(F64), c["w3"][e].to(F64))):
            out[b][i] = rows[i] @ w
            out[2 + b][i] = rows[i].abs() @ w.abs()
    return out


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name", CASES)
def test_up_stores_what_it_summed(xm, name, dt):
    c = _case(name, dt)
    act, hq, hs = _up(xm, c, dt)
    n, h = c["off"][-1], c["h"]
    want = torch.full_like(act, 3.0)
    if c["tok"] is None:
        xm.xmoe_expert_ffn_up(c["x"], c["w1"], c["w3"], c["offsets"], want)
    else:
        xm.xmoe_expert_ffn_up_gather(c["x"], c["tok"], c["w1"], c["w3"], c["offsets"], want)
    assert torch.equal(act, want), "act"
    assert bool((hq[n:] == 77).all()) and bool((hs[:, :, n:] == 99).all()) and bool((act[n:] == 3).all())
    h1, h3, m1, m3 = _sums(c)
    for b, (v, m) in enumerate(((h1, m1), (h3, m3))):
        byte, pad = ref.half(hs[:, :, :n], h, b)
        assert bool((pad == 127).all()), "bytes past h"
        err = c["d"] * 2.0 ** -24 * m
        a, top = ref.blocks(v).abs().amax(-1), ref.blocks(err).amax(-1)
        s = ref.scale(byte)
        assert bool((127 * s + top >= a).all()) and bool(((63.5 * s <= a + top) | (a == 0)).all()), "scale"
        got = hq[:n, b * h:(b + 1) * h].to(F64) * s.repeat_interleave(32, 1)[:, :h]
        tol = 0.5 * s.repeat_interleave(32, 1)[:, :h] + err
        assert bool(((got - v).abs() <= tol).all()), "values"
    val = torch.cat(ref.values(hq[:n], hs[:, :, :n]), 1)
    for out in (torch.full((c["R"], 2 * h), 5.0, dtype=t, device="cuda") for t in (BF, F32)):
        xm.xmoe_ckpt8_dequantize(hq, hs, out)
        assert torch.equal(out[:n].to(F64), val), "dequantized"


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name", [n for n in CASES if CASES[n][1] * 45 < 2 ** 24])
def test_exact_sums_give_exact_bytes(xm, name, dt):
    c = _case(name, dt, whole=True)
    c["x"][0] = 0  # zero blocks
    _, hq, hs = _up(xm, c, dt)
    n, h = c["off"][-1], c["h"]
    for b, v in enumerate(_sums(c)[:2]):
        q, byte, _ = ref.round8(v)
        assert torch.equal(ref.half(hs[:, :, :n], h, b)[0], byte) and torch.equal(hq[:n, b * h:(b + 1) * h], q)


@pytest.mark.parametrize("dt", [BF, F32])
def test_extremes(xm, dt):
    """A unit row picks W's rows: zeros, the borders of a scale, ties, subnormals, large
    values, infinities and NaN."""
    one = torch.finfo(BF).smallest_normal
    rows = [[0.0] * 32, [127.0] + [0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5] * 4 + [1.0] * 3, [127.5, 1.0] + [0.25] * 30,
            [254.0, -253.0] + [1.0] * 30, [63.5, 0.25] + [0.75] * 30, [one] + [one * 2.0 ** -5] * 31,
            [3e38] + [1e30] * 31, [float("inf")] + [1.0] * 31, [float("nan")] + [2.0] * 31, [-128.0] + [0.5] * 31]
    E, h = 1, 32 * len(rows) + 8
    w = torch.zeros((1, 8, h), device="cuda")
    w[0, 0, :-8] = torch.tensor(rows, device="cuda").flatten()
    w[0, 0, -8:] = 7.0
    w = w.to(dt)
    x = torch.zeros((2, 8), dtype=dt, device="cuda")
    x[0, 0] = 1.0
    c = dict(R=2, h=h, x=x, w1=w, w3=w.flip(2).contiguous(), offsets=torch.tensor([0, 2], dtype=I32, device="cuda"), tok=None)
    # products with the zeros of x are NaN where W is not finite: row 1 and those columns
    _, hq, hs = _up(xm, c, dt)
    for b, m in enumerate((c["w1"], c["w3"])):
        v = m[0, 0].to(F64)[None]
        q, byte, val = ref.round8(v)
        got, pad = ref.half(hs, h, b)
        assert torch.equal(got[:1], byte), (got[:1] - byte)
        keep = torch.isfinite(val)
        assert torch.equal(hq[:1, b * h:(b + 1) * h][keep], q[keep])
    out = torch.empty((2, 2 * h), device="cuda")
    xm.xmoe_ckpt8_dequantize(hq, hs, out)
    bad = ~torch.isfinite(ref.blocks(c["w1"][0, :1].to(F64))).all(-1)[0].repeat_interleave(32)[:h]
    assert torch.equal(torch.isnan(out[0, :h]), bad)


def _dact(xm, c, dt, hq, hs, weighted=True, order=True, dots=True, **kw):
    R, h = c["R"], c["h"]
    dh = torch.full((R, 2 * h), 3.0, dtype=dt, device="cuda")
    act = torch.full((R, h), 3.0, dtype=dt, device="cuda")
    dw = torch.full((R,), 3.0, device="cuda") if dots else None
    s2r = c["perm"].to(I32) if order and dots else None
    xm.xmoe_expert_ffn_bwd_dact_ckpt8(c["dy"], c["w2"], hq, hs, c["offsets"], dh, act, token_ids=c["tok"],
                                      row_weights=c["weights"] if weighted else None, slot_to_row=s2r, dweights=dw, **kw)
    return dh, act, dw


def _kept(c, dt):
    g, R, h = c["g"], c["R"], c["h"]
    h1 = torch.randn((R, h), generator=g, device="cuda", dtype=F64)
    h3 = torch.randn((R, h), generator=g, device="cuda", dtype=F64)
    h1[:, ::7] *= 6.0
    return ref.pack(h1, h3)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name", CASES)
def test_backward_from_kept_values(xm, name, dt):
    c = _case(name, dt)
    hq, hs = _kept(c, dt)
    n, h = c["off"][-1], c["h"]
    h1, h3 = ref.values(hq, hs)
    for weighted, order in ((True, True), (False, False)):
        dh, act, dw = _dact(xm, c, dt, hq, hs, weighted, order)
        g1, g3, a, dots, da, mag = ref.backward(c["dy"], c["tok"], c["w2"], h1, h3, c["weights"] if weighted else None, c["off"])
        eps = half_step(dt)
        w = c["weights"].to(F64)[:, None] if weighted else torch.ones((c["R"], 1), dtype=F64, device="cuda")
        dda = c["d"] * 2.0 ** -24 * mag
        sg = torch.sigmoid(h1)
        rel = 2.0 ** -20 + 2.0 ** -23 * h1.abs()
        s1 = (sg + h1 * sg * (1 - sg)).abs() + 2 * rel * sg * (1 + 2 * h1.abs())  # the slope, and what cancels in it
        for what, got, want, per in (("dH1", dh[:, :h], g1, h3.abs() * s1), ("dH3", dh[:, h:], g3, (h1 * sg).abs())):
            slope = w * da.abs() * h3.abs() * 2 * rel * sg * (1 + 2 * h1.abs()) if what == "dH1" else 0.0
            tol = (eps + rel) * want.abs() + w * per * dda * 1.01 + slope + 1e-37
            assert bool(((got[:n].to(F64) - want[:n]).abs() <= tol[:n]).all()), what
        assert bool(((act[:n].to(F64) - a[:n]).abs() <= (eps + rel[:n]) * a[:n].abs() + 1e-37).all()), "act"
        raw = (h1 * sg * h3).abs()
        tol = (raw * dda).sum(1) * 1.01 + ((rel + h * 2.0 ** -24) * raw * da.abs()).sum(1)
        rows = c["perm"] if order else torch.arange(c["R"], device="cuda")
        live = rows < n
        assert bool(((dw.to(F64) - dots[rows]).abs() <= tol[rows])[live].all()), "dweights"
        assert bool((dw[~live] == 3).all()) and bool((dh[n:] == 3).all()) and bool((act[n:] == 3).all())
    alone = _dact(xm, c, dt, hq, hs, True, True, dots=False)
    both = _dact(xm, c, dt, hq, hs, True, True)
    assert torch.equal(alone[0], both[0]) and torch.equal(alone[1], both[1])


def test_the_formula_is_the_gradient():
    """The 64-bit definition against autograd and central differences."""
    torch.manual_seed(3)
    R, d, h = 3, 8, 40
    w2, dy, w = torch.randn(1, h, d, dtype=F64), torch.randn(R, d, dtype=F64), torch.rand(R, dtype=F64)
    h1, h3 = (torch.randn(R, h, dtype=F64, requires_grad=True) for _ in range(2))
    wt = w.clone().requires_grad_()
    f = lambda a, b, v: (v[:, None] * ((a * torch.sigmoid(a) * b) @ w2[0]) * dy).sum()
    f(h1, h3, wt).backward()
    g1, g3, act, dots, _, _ = ref.backward(dy, None, w2, h1.detach(), h3.detach(), w, [0, R])
    assert torch.allclose(g1, h1.grad, rtol=1e-12, atol=1e-13) and torch.allclose(g3, h3.grad, rtol=1e-12, atol=1e-13)
    assert torch.allclose(dots, wt.grad, rtol=1e-12, atol=1e-13)
    step = 1e-6
    for r, c in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros(R, h, dtype=F64)
        e[r, c] = step
        a, b = h1.detach(), h3.detach()
        assert abs((f(a + e, b, w) - f(a - e, b, w)) / (2 * step) - g1[r, c]) < 1e-7
        assert abs((f(a, b + e, w) - f(a, b - e, w)) / (2 * step) - g3[r, c]) < 1e-7


@pytest.mark.parametrize("dt", [BF, F32])
def test_nan_blocks_reach_their_columns_only(xm, dt):
    c = _case("ragged", dt)
    hq, hs = _kept(c, dt)
    clean = _dact(xm, c, dt, hq, hs)
    hs[0, 0, 40, 1] = 255    # H1 of row 40, columns 32..63
    dh, act, dw = _dact(xm, c, dt, hq, hs)
    h = c["h"]
    cols = torch.zeros(2 * h, dtype=torch.bool, device="cuda")
    cols[32:64] = True
    cols[h + 32:h + 64] = True
    assert torch.isnan(dh[40][cols]).all() and torch.equal(dh[40][~cols], clean[0][40][~cols])
    keep = torch.arange(c["R"], device="cuda") != 40
    assert torch.equal(dh[keep], clean[0][keep]) and torch.equal(act[keep], clean[1][keep])
    assert torch.equal(torch.isnan(dw), c["perm"] == 40)


@pytest.mark.parametrize("dt", [BF, F32])
def test_repeats_graphs_and_streams(xm, dt):
    c = _case("ragged", dt)
    want = _up(xm, c, dt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _up(xm, c, dt)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = torch.full((xm.xmoe_expert_ffn_bwd_dact_ckpt8_workspace_size(c["R"], c["h"]) + 64,), 255, dtype=U8, device="cuda")
    _, hq, hs = want
    back = _dact(xm, c, dt, hq, hs, workspace=ws)
    assert bool((ws[-64:] == 255).all())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        fwd = _up(xm, c, dt)
        bwd = _dact(xm, c, dt, fwd[1], fwd[2], workspace=ws)
    for _ in range(3):
        for t in (*fwd, *bwd):
            t.fill_(3 if t.dtype != I8 else 77)
        fwd[2].fill_(99)
        ws.fill_(255)
        g.replay()
        _dact(xm, c, dt, hq, hs)
        torch.cuda.synchronize()
        n = c["off"][-1]
        assert all(torch.equal(a, b) for a, b in zip(want, fwd)) and all(torch.equal(a, b) for a, b in zip(back, bwd))


def _layer(wl, **kw):
    from padding_free_expert_amd.layer import PaddingFreeMoE
    inp = {k: v.cuda() for k, v in workloads.generate(wl, backward=True).items() if v is not None}
    weights = {k: inp[k] for k in ("wg", "w1", "w3", "w2", "s1", "s3", "s2", "logit_bias", "select_bias") if k in inp}
    return inp, weights, PaddingFreeMoE(weights, wl.T, wl.k, wl.inv_tau, **kw)


def _reference(wl, layer, w, x, dy):
    """The layer's gradients in 64 bits, taken at the kept pre-activations."""
    D = lambda t: t.detach().double().cpu()
    pft = {k: v.cpu() for k, v in layer.pft.fields().items()}
    tok, off, s2r = pft["token_ids"].long(), pft["expert_offsets"].tolist(), pft["slot_to_row"].long()
    E, k, kc, d = layer.E, layer.k, layer.kc, layer.d
    h1, h3 = ref.values(layer.hq.cpu(), layer.hscale.cpu())
    W1, W3, W2 = D(layer.W1), D(layer.W3), D(layer.W2)
    wr = pft["combine_weights"].double()
    g1, g3, act, dots, _, _ = ref.backward(D(dy), tok, W2, h1, h3, wr, off)
    out = {"dw1": [], "dw3": [], "dw2": []}
    dxs = torch.empty(len(tok), d, dtype=F64)
    X, DY = D(x), D(dy)
    for e in range(layer.Ec):
        i = slice(off[e], off[e + 1])
        out["dw1"].append(X[tok[i]].t() @ g1[i])
        out["dw3"].append(X[tok[i]].t() @ g3[i])
        out["dw2"].append(act[i].t() @ DY[tok[i]])
        dxs[i] = g1[i] @ W1[e].t() + g3[i] @ W3[e].t()
    out = {n: torch.stack(v)[:E] for n, v in out.items()}
    dtw = dots[s2r].view(wl.T, kc)[:, :k]
    z, ids = D(layer.logits), layer.topk_ids.cpu().long()
    p = torch.softmax(z, 1)
    g = torch.zeros_like(p).scatter_(1, ids, dtw)
    dz = p * (g - (p * g).sum(1, keepdim=True)) * wl.inv_tau
    dx = torch.zeros(wl.T, d, dtype=F64).index_add(0, tok, dxs) + dz @ D(w["wg"]).t()
    out["dwg"] = X.t() @ dz
    if layer.side_shared:
        a, b = ref.values(layer.sh_hq.cpu(), layer.sh_hscale.cpu())
        u1, u3, sact, _, _, _ = ref.backward(DY, None, D(w["s2"])[None], a, b, None, [0, wl.T])
        dx += u1 @ D(w["s1"]).t() + u3 @ D(w["s3"]).t()
        out.update(ds1=X.t() @ u1, ds3=X.t() @ u3, ds2=sact.t() @ DY)
    out.update(dx=dx, dtopk_w=dtw)
    return out


@pytest.mark.parametrize("name", ["tiny_f32", "dsmoe16b", "long_batch"])
@pytest.mark.parametrize("merge", [False, True])
@pytest.mark.parametrize("overlap", [False, True])
def test_training_layer(xm, name, merge, overlap):
    """The layer with kept pre-activations: the forward bit for bit the plain layer's, the
    gradients those at the kept values (normwise, the layer's tolerances: 1e-4 in fp32,
    2e-2 in bf16), near those of the plain layer."""
    wl = workloads.WORKLOADS[name] if name == "tiny_f32" else workloads.small(name)
    if merge and not wl.n_shared:
        pytest.skip("no shared experts to merge")
    inp, weights, layer = _layer(wl, ckpt8=True, merge_shared=merge, overlap=overlap)
    _, _, plain = _layer(wl, merge_shared=merge, overlap=overlap)
    x, dy = inp["x"], inp["dy"]
    y = layer.forward(x).clone()
    assert torch.equal(y, plain.forward(x))
    layer.act.fill_(float("nan"))   # neither is read by the backward
    layer.ye.fill_(float("nan"))
    layer.backward(dy)
    plain.backward(dy)
    rtol = 1e-4 if wl.dtype == "f32" else 2e-2
    got = layer.grads()
    for n, want in _reference(wl, layer, weights, x, dy).items():
        v = got[n].double().cpu().reshape(want.shape)
        assert torch.isfinite(v).all(), n
        err = float((v - want).norm() / want.norm())
        assert err <= rtol, f"{n}: off by {err:.2e} of its norm"
        # 8 bits: a value off by half a step, at most 1/127 of its block's largest.  The
        # product of the factors that carry it is off by under 2^-4 of its norm here
        far = float((v - plain.grads()[n].double().cpu().reshape(want.shape)).norm() / want.norm())
        assert far <= 2.0 ** -4 + rtol, f"{n}: {far:.2e} from the plain layer's"
    first = {n: v.clone() for n, v in got.items()}
    layer.forward(x)
    layer.backward(dy)
    assert all(torch.equal(first[n], v) for n, v in layer.grads().items())
    assert layer.saved_bytes() < 0.45 * plain.saved_bytes()


def test_training_layer_as_a_graph_and_in_a_block(xm):
    from padding_free_expert_amd.layer import MoEBlock
    wl = workloads.small("dsmoe16b")
    inp, weights, _ = _layer(wl)
    weights = dict(weights, norm=torch.ones(wl.d, dtype=inp["x"].dtype, device="cuda"))
    off = torch.tensor([0, 100, 290], dtype=I32, device="cuda")
    block = MoEBlock(weights, wl.T, wl.k, inv_tau=wl.inv_tau, ckpt8=True, balance_alpha=0.1, n_seq=2)
    res = inp["x"].flip(0).contiguous()

    def step():
        out, s = block.forward(inp["x"], res, seq_offsets=off)
        return out, s, block.backward(inp["dy"], s)

    want = [t.clone() for t in step()] + [v.clone() for v in block.moe.grads().values()] + [block.dgamma.clone()]
    assert all(torch.isfinite(t).all() for t in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(3):
        for t in (*outs, *block.moe.grads().values(), block.dgamma):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = list(outs) + list(block.moe.grads().values()) + [block.dgamma]
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_layer_refuses(xm):
    wl = workloads.small("dsmoe16b")
    for kw in (dict(ckpt8=True, lean=True), dict(ckpt8=True, backward=False)):
        with pytest.raises(ValueError, match="ckpt8"):
            _layer(wl, **kw)


@pytest.mark.parametrize("counts", [[34000], [17000, 120, 16880], [150] * 227])
def test_results_past_the_caches_are_those_of_parts(xm, counts):
    """Results of more than 256 MB take another way to memory: the same bits as calls on
    the single experts' rows, whose results do not (every expert alone for the ends, the
    last rows of a segment among them)."""
    d, h, off = 32, 1368, _offsets(counts)
    R, E = off[-1], len(counts)
    assert R * h * 6 > 2 ** 28
    g = _gen(9)
    dy = torch.randn((R, d), device="cuda", generator=g).to(BF)
    w2 = (torch.randn((E, h, d), device="cuda", generator=g) * h ** -0.5).to(BF)
    hq = torch.randint(-127, 128, (R, 2 * h), device="cuda", generator=g, dtype=I8)
    hs = torch.randint(118, 124, xm.ckpt8_scale_shape(R, h), device="cuda", generator=g, dtype=U8)
    wt = torch.rand((R,), device="cuda", generator=g)

    def run(r0, r1, e0, e1):
        n = r1 - r0
        o = torch.tensor([v - r0 for v in off[e0:e1 + 1]], dtype=I32, device="cuda") if e1 - e0 > 1 else \
            torch.tensor([0, n], dtype=I32, device="cuda")
        dh, act = torch.full((n, 2 * h), 3.0, dtype=BF, device="cuda"), torch.full((n, h), 3.0, dtype=BF, device="cuda")
        dw = torch.full((n,), 3.0, device="cuda")
        xm.xmoe_expert_ffn_bwd_dact_ckpt8(dy[r0:r1], w2[e0:e1], hq[r0:r1], hs[:, :, r0:r1].contiguous(), o, dh, act,
                                          row_weights=wt[r0:r1], dweights=dw)
        return dh, act, dw

    whole = run(0, R, 0, E)
    for e in sorted({0, E // 2, E - 1}):
        for r0 in range(off[e], off[e + 1], 8192):
            r1 = min(r0 + 8192, off[e + 1])
            for a, b in zip(whole, run(r0, r1, e, e + 1)):
                assert torch.equal(a[r0:r1], b), (e, r0)
