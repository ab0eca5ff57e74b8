"""Timed passes of the expert layer at its two ends: the whole layer for a few
tokens (gate, top-k, experts, shared experts, combine), with the layer's own
weights and with 8-bit weights; and the training pass whose pre-activations are
kept in 8 bits, forward (the up-projection that stores them) and backward (the
product and SwiGLU gradient that read them).

`own` chooses between the plain form (elementary torch operations) and the
calls of padding_free_expert_amd.

8-bit weights and rows are e4m3 with one power-of-two scale (a byte b stands for
2^(b - 127)) for each 32 consecutive elements of the summed axis; scales of n
rows of K elements lie as [ceil(K / 128), n, 4], the unused bytes of the last
group being 127.  Kept pre-activations are whole numbers of -127..127 times such
a scale, [rows, 2h] with scales [2, ceil(h / 128), rows, 4] (H1's, then H3's).
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence's next token, straight from the training weights (sampling between steps)
        dict(name="few 1 token", op="few", T=1, d=2048, h=1408, E=64, k=6, hs=2816, dtype="bf16", bias=False),
        # a small decode batch on uneven experts that a selection bias balances
        dict(name="few 12 tokens", op="few", T=12, d=2048, h=768, E=128, k=8, hs=0, dtype="bf16", bias=True),
        # the largest batch of the call: nearly every expert of a wide layer is read
        dict(name="few 64 tokens", op="few", T=64, d=4096, h=1024, E=160, k=8, hs=0, dtype="bf16", bias=False),
        # ragged fp32 sizes: the parity runs of a small model
        dict(name="few f32 ragged", op="few", T=5, d=1000, h=200, E=30, k=3, hs=328, dtype="f32", bias=True),
        # single-token serving with 8-bit weights
        dict(name="few8 1 token", op="few8", T=1, d=2048, h=1408, E=64, k=6, hs=2816, bias=False),
        # a handful of sequences on the widest experts here
        dict(name="few8 4 tokens", op="few8", T=4, d=7168, h=2048, E=256, k=8, hs=0, bias=True),
        # a decode batch, a row or two for each expert
        dict(name="few8 32 tokens", op="few8", T=32, d=2048, h=768, E=128, k=8, hs=0, bias=False),
        # a training micro-batch's up-projection that keeps H1 and H3 in 8 bits
        dict(name="ckpt up train", op="up", T=4096, d=2048, h=1408, E=64, k=6, dtype="bf16"),
        # ragged fp32 rows, blocks of 32 that end inside h
        dict(name="ckpt up f32 ragged", op="up", T=300, d=448, h=136, E=32, k=8, dtype="f32"),
        # its backward: dA, the SwiGLU gradient, the rebuilt activations and the routing weights' gradient
        dict(name="ckpt back train", op="back", T=4096, d=2048, h=1408, E=64, k=6, dtype="bf16"),
        # the same for shared experts side by side: one expert, every row, no routing weights
        dict(name="ckpt back shared", op="back", T=4096, d=2048, h=2816, E=1, k=0, dtype="bf16"),
        # a long batch on wide experts
        dict(name="ckpt back long", op="back", T=32768, d=4096, h=1024, E=160, k=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "few8", "up", "back"])
    if op == "few":
        E = rng.choice([8, 16, 40, 64, 128])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            E = rng.randint(2, 70)
        h = 8 * _log(rng, 4, 160)
        return dict(op=op, T=_log(rng, 1, 64), d=8 * _log(rng, 8, 512), h=h, E=E, k=rng.randint(1, min(8, E)),
                    hs=rng.choice([0, 0, h, 2 * h]), dtype=dtype, bias=rng.random() < 0.5)
    if op == "few8":
        E = rng.choice([8, 16, 40, 64, 128])
        h = 32 * _log(rng, 2, 56)
        return dict(op=op, T=_log(rng, 1, 64), d=32 * _log(rng, 4, 128), h=h, E=E, k=rng.randint(1, min(8, E)),
                    hs=rng.choice([0, 0, h, 2 * h]), bias=rng.random() < 0.5)
    E = rng.choice([1, 4, 16, 40, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d, h = 8 * _log(rng, 16, 320), 8 * _log(rng, 8, 176)
    T = _log(rng, 1, 8000 if dtype == "bf16" else 600)
    return dict(op=op, T=T, d=d, h=h, E=E, k=0 if E == 1 and op == "back" else rng.randint(1, min(8, E)), dtype=dtype)


# ------------------------------------------------------------------ inputs

def _dt(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _quantize(v):
    """fp32 [..., K] -> e4m3 [..., K] and scale bytes [..., K / 32]: the least
    power of two that brings the block's largest magnitude to at most 448."""
    b = v.unflatten(-1, (-1, 32))
    m, x = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, x - 9 + (m > 0.875).to(x.dtype), 0).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _quantize_int(v):
    """fp32 [..., h] -> whole numbers int8 [..., h] and exponents [..., ceil(h / 32)]: the
    least power of two that brings the block's largest magnitude to at most 127."""
    h = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -h % 32)).unflatten(-1, (-1, 32))
    m, x = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, x - 7 + (m > 127 / 128).to(x.dtype), 0).clamp(-127, 127)
    return torch.round(torch.ldexp(b, -e.unsqueeze(-1))).flatten(-2)[..., :h].to(torch.int8), e


def _groups(s):
    """Scale bytes [..., n, blocks] -> [..., ceil(blocks / 4), n, 4]."""
    s = torch.nn.functional.pad(s, (0, -s.shape[-1] % 4), value=127)
    return s.unflatten(-1, (-1, 4)).transpose(-3, -2).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    op, T, d, h, E, k, dt = case["op"], case["T"], case["d"], case["h"], case["E"], case["k"], _dt(case)
    s = dict(op=op, T=T, d=d, h=h, E=E, k=k, dt=dt)
    # rows as a norm leaves them, a few channels larger
    gain = 1.0 + 2.0 * (torch.rand(d, generator=g, device="cuda") > 0.99)

    def weights(n, K, N):
        w = torch.empty((n, K, N), dtype=dt, device="cuda")
        for e in range(0, n, 16):
            m = min(16, n - e)
            w[e:e + m] = randn(m, K, N) * K ** -0.5
        return w

    def weights8(n, N, K):
        q = torch.empty((n, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty((n, -(-K // 128), N, 4), dtype=torch.uint8, device="cuda")
        for e in range(0, n, 16):
            m = min(16, n - e)
            a, b = _quantize(randn(m, N, K) * K ** -0.5)
            q[e:e + m], sc[e:e + m] = a, _groups(b)
        return q, sc

    if op in ("few", "few8"):
        hs = case["hs"]
        s["x"] = (randn(T, d) * gain).to(dt)
        s["wg"] = (1.5 * d ** -0.5 * randn(d, E)).to(dt)
        s["lbias"] = 0.3 * randn(E) if case["bias"] else None
        s["sbias"] = 0.3 * randn(E) if case["bias"] else None
        s["tau"] = 1.0 if not case["bias"] else 0.5
        if op == "few":
            s["w1"], s["w3"], s["w2"] = weights(E, d, h), weights(E, d, h), weights(E, h, d)
            if hs:
                s["s1"], s["s3"], s["s2"] = weights(1, d, hs)[0], weights(1, d, hs)[0], weights(1, hs, d)[0]
        else:
            xq, xs = _quantize(s["x"].float())
            s["xq"], s["xs"] = xq, _groups(xs)
            s["w1"], s["w3"], s["w2"] = weights8(E, h, d), weights8(E, h, d), weights8(E, d, h)
            if hs:
                s["s1"], s["s3"], s["s2"] = weights8(1, hs, d), weights8(1, hs, d), weights8(1, d, hs)
        if not hs:
            s["s1"] = s["s3"] = s["s2"] = None
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, k), device="cuda")
        s["logits"] = torch.empty((T, E), device="cuda")
        s["y"] = torch.empty((T, d), dtype=dt, device="cuda")
        s["hs"] = hs
        return s

    # a routing on slightly uneven experts, its rows sorted by expert
    R = T * max(k, 1)
    key = randn(T, E) - 0.3 * torch.log1p(torch.arange(E, device="cuda"))
    top, choice = torch.topk(key, max(k, 1), 1)
    ids = choice.flatten()
    order = torch.argsort(ids, stable=True)
    n = torch.bincount(ids, minlength=E)
    s["offsets"] = torch.cat([torch.zeros(1, device="cuda"), torch.cumsum(n, 0)]).to(torch.int32)
    s["cap"] = int(n.max())
    s["expert"] = ids[order]
    s["place"] = torch.arange(R, device="cuda") - s["offsets"][s["expert"]].long()
    s["tokens"] = (order // max(k, 1)).to(torch.int32)
    s["act"] = torch.empty((R, h), dtype=dt, device="cuda")
    if op == "up":
        s["x"] = (randn(T, d) * gain).to(dt)
        s["w1"], s["w3"] = weights(E, d, h), weights(E, d, h)
        s["hq"] = torch.empty((R, 2 * h), dtype=torch.int8, device="cuda")
        s["hs"] = torch.empty((2, -(-h // 128), R, 4), dtype=torch.uint8, device="cuda")
        s["h13"] = torch.empty((R, 2 * h), dtype=torch.bfloat16, device="cuda")  # holds seven bits and a power of two exactly
        return s
    s["dy"] = (0.1 * randn(T, d)).to(dt)
    s["w2"] = weights(E, h, d)
    s["hq"] = torch.empty((R, 2 * h), dtype=torch.int8, device="cuda")
    s["hs"] = torch.empty((2, -(-h // 128), R, 4), dtype=torch.uint8, device="cuda")
    wide = 1.0 + 3.0 * (torch.rand(2, h, generator=g, device="cuda") > 0.99)
    for b in range(2):
        q, e = _quantize_int(randn(R, h) * wide[b])
        s["hq"][:, b * h:(b + 1) * h] = q
        s["hs"][b] = _groups((e + 127).to(torch.uint8))
    s["dh13"] = torch.empty((R, 2 * h), dtype=dt, device="cuda")
    if k:
        s["weights"] = torch.softmax(top, 1).flatten()[order].contiguous()
        s["rows"] = torch.empty(R, dtype=torch.int32, device="cuda")
        s["rows"][order] = torch.arange(R, dtype=torch.int32, device="cuda")
        s["dw"] = torch.empty((T, k), device="cuda")
    else:
        s["tokens"] = s["weights"] = s["rows"] = s["dw"] = None
    return s


# -------------------------------------------------------------- plain forms

def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _rows8(v):
    """The values that fp32 rows [..., K] stand for in 8 bits."""
    q, s = _quantize(v)
    return torch.ldexp(q.float().unflatten(-1, (-1, 32)), s.int().unsqueeze(-1) - 127).flatten(-2)


def _value8(q, s):
    """The fp32 values [..., n, K] of e4m3 rows and their scale groups."""
    K = q.shape[-1]
    s = s.transpose(-3, -2).flatten(-2)[..., : K // 32]
    return (q.float().unflatten(-1, (-1, 32)) * torch.exp2(s.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _pick8(w, sel):
    """[n, K, N] in fp32 of the chosen experts (None: all) of 8-bit weights."""
    q, s = w
    if sel is not None:
        q, s = q.view(torch.uint8)[sel].view(torch.float8_e4m3fn), s[sel]
    return _value8(q, s).transpose(1, 2)


def _pick(w, sel):
    return (w if sel is None else w[sel]).float()


def _plain_few(s):
    T, k, E = s["T"], s["k"], s["E"]
    # next to a border between two experts the choice needs 64 bits
    z = (s["x"].double() @ s["wg"].double()) * s["tau"]
    if s["lbias"] is not None:
        z = z + s["lbias"].double()
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    sel = z if s["sbias"] is None else z + s["sbias"].double()
    ids = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, ids).float()
    eight = s["op"] == "few8"
    pick, act8 = (_pick8, _rows8) if eight else (_pick, lambda v: v)
    x = _value8(s["xq"], s["xs"]) if eight else s["x"].float()
    if T * k <= E:
        # every slot with its expert's weights
        e = ids.flatten()
        rows = x.repeat_interleave(k, 0).unsqueeze(1)
        a = act8(_silu(torch.matmul(rows, pick(s["w1"], e))) * torch.matmul(rows, pick(s["w3"], e)))
        ye = torch.matmul(a, pick(s["w2"], e)).view(T, k, -1)
        y = (ye * w.unsqueeze(2)).sum(1)
    else:
        # every expert on every token
        gate = torch.zeros((T, E), device="cuda").scatter_(1, ids, w)
        rows = x.expand(E, -1, -1)
        a = act8(_silu(torch.matmul(rows, pick(s["w1"], None))) * torch.matmul(rows, pick(s["w3"], None)))
        ye = torch.matmul(a, pick(s["w2"], None))
        y = (ye * gate.t().unsqueeze(2)).sum(0)
    if s["s1"] is not None:
        one = (lambda v: pick(v, None)[0]) if eight else (lambda v: v.float())
        y = y + torch.matmul(act8(_silu(torch.matmul(x, one(s["s1"]))) * torch.matmul(x, one(s["s3"]))), one(s["s2"]))
    return {"y": y.to(s["dt"]), "ids": ids.to(torch.int32), "w": w, "logits": z.float()}


def _by_expert(s, rows):
    """Rows [R, K] laid out [E, cap, K], zeros behind an expert's own."""
    out = torch.zeros((s["E"], s["cap"], rows.shape[1]), device="cuda")
    out[s["expert"], s["place"]] = rows
    return out


def _plain_up(s):
    xe = _by_expert(s, s["x"].float()[s["tokens"].long()])
    a = torch.matmul(xe, s["w1"].float())[s["expert"], s["place"]]
    b = torch.matmul(xe, s["w3"].float())[s["expert"], s["place"]]
    out = []
    for v in (a, b):
        q, e = _quantize_int(v)
        out.append(torch.ldexp(q.float(), e.repeat_interleave(32, -1)[:, : s["h"]]))
    return {"act": (_silu(a) * b).to(s["dt"]), "h13": torch.cat(out, 1).to(torch.bfloat16)}


def _kept(s):
    """H1 and H3 [R, h] in fp32 from their 8 bits."""
    h = s["h"]
    e = s["hs"].transpose(1, 2).flatten(2)[..., : -(-h // 32)].float() - 127.0
    v = torch.exp2(e).repeat_interleave(32, 2)[..., :h]
    return s["hq"][:, :h].float() * v[0], s["hq"][:, h:].float() * v[1]


def _plain_back(s):
    h1, h3 = _kept(s)
    dy = s["dy"].float()
    rows = _by_expert(s, dy if s["tokens"] is None else dy[s["tokens"].long()])
    da = torch.matmul(rows, s["w2"].float().transpose(1, 2).contiguous())[s["expert"], s["place"]]
    sg = 1.0 / (1.0 + torch.exp(-h1))
    act = h1 * sg * h3
    out = {}
    if s["weights"] is not None:
        out["dw"] = (da * act).sum(1)[s["rows"].long()].view(s["T"], s["k"])
        w = s["weights"].unsqueeze(1)
        da, act = da * w, act * w
    out["dh13"] = torch.cat([da * h3 * sg * (1.0 + h1 * (1.0 - sg)), da * h1 * sg], 1).to(s["dt"])
    out["act"] = act.to(s["dt"])
    return out


# --------------------------------------------------------- the framework's

def _workspace(s, need):
    """A program's workspace for calls of these sizes, kept."""
    if "ws" not in s:
        s["ws"] = torch.empty(need(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_few(s):
    import padding_free_expert_amd as xm
    sizes = (s["T"], s["d"], s["E"], s["k"], s["h"], s["hs"])
    ws = _workspace(s, lambda: xm.xmoe_layer_few_workspace_size(*sizes, s["dt"]) if s["op"] == "few" else
                    xm.xmoe_layer_few_mx8_workspace_size(*sizes))
    rest = dict(inv_temperature=s["tau"], logit_bias=s["lbias"], select_bias=s["sbias"], s1=s["s1"], s3=s["s3"],
                s2=s["s2"], workspace=ws)
    if s["op"] == "few":
        xm.xmoe_layer_few(s["x"], s["wg"], s["w1"], s["w3"], s["w2"], s["k"], s["ids"], s["w"], s["logits"], s["y"], **rest)
    else:
        xm.xmoe_layer_few_mx8(s["x"], s["xq"], s["xs"], s["wg"], s["w1"], s["w3"], s["w2"], s["k"], s["ids"], s["w"],
                              s["logits"], s["y"], **rest)
    return {n: s[n] for n in ("y", "ids", "w", "logits")}


def _own_up(s):
    import padding_free_expert_amd as xm
    xm.xmoe_expert_ffn_up_ckpt8(s["x"], s["w1"], s["w3"], s["offsets"], s["act"], s["hq"], s["hs"], token_ids=s["tokens"])
    xm.xmoe_ckpt8_dequantize(s["hq"], s["hs"], s["h13"])
    return {"act": s["act"], "h13": s["h13"]}


def _own_back(s):
    import padding_free_expert_amd as xm
    ws = None if s["dw"] is None else _workspace(
        s, lambda: xm.xmoe_expert_ffn_bwd_dact_ckpt8_workspace_size(s["act"].shape[0], s["h"]))
    xm.xmoe_expert_ffn_bwd_dact_ckpt8(s["dy"], s["w2"], s["hq"], s["hs"], s["offsets"], s["dh13"], s["act"],
                                      token_ids=s["tokens"], row_weights=s["weights"], slot_to_row=s["rows"],
                                      dweights=s["dw"], workspace=ws)
    out = {"dh13": s["dh13"], "act": s["act"]}
    if s["dw"] is not None:
        out["dw"] = s["dw"]
    return out


def run(state):
    op = state["op"]
    if own:
        return {"few": _own_few, "few8": _own_few, "up": _own_up, "back": _own_back}[op](state)
    return {"few": _plain_few, "few8": _plain_few, "up": _plain_up, "back": _plain_back}[op](state)


# ------------------------------------------------------------------- work

def work(case):
    op, T, d, h, E, k = (case[n] for n in ("op", "T", "d", "h", "E", "k"))
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op in ("few", "few8"):
        hs = case["hs"]
        active = E * (1.0 - (1.0 - k / E) ** T)
        per = 33 / 32 if op == "few8" else es
        return {"bytes": (active * h + hs) * 3 * d * per + d * E * es + 2 * T * d * es + 4 * T * (E + 2 * k),
                "flops": 2.0 * T * d * (E + 3 * (k * h + hs))}
    R = T * max(k, 1)
    if op == "up":
        # x and the weights in; act and the two kept halves out, and these read once more as values
        return {"bytes": T * d * es + 2 * E * d * h * es + R * h * es + 2 * R * h * (2 * 33 / 32 + 2), "flops": 4.0 * R * d * h}
    return {"bytes": T * d * es + E * d * h * es + 2 * R * h * 33 / 32 + 3 * R * h * es + (12 * R if k else 0),
            "flops": 2.0 * R * d * h}


# ---------------------------------------------------- the definition, 64 bits

def _round64(v, top, eight):
    """float64 [..., K] rounded to 8 bits with a power-of-two scale for each 32 (K may
    end inside a block): e4m3 (top = 448) or whole numbers (top = 127)."""
    K = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -K % 32)).unflatten(-1, (-(-K // 32), 32))
    a = b.abs().max(dim=-1, keepdim=True).values
    e = torch.ceil(torch.log2(torch.where(a > 0, a / top, torch.ones_like(a))))
    e = torch.where(top * torch.exp2(e - 1) >= a, e - 1, e)  # log2's own rounding at a border
    e = torch.where(top * torch.exp2(e) < a, e + 1, e)
    e = torch.where(a > 0, e, torch.zeros_like(e)).clamp(-127, 127)
    r = b * torch.exp2(-e)
    step = torch.exp2((torch.frexp(r).exponent.to(torch.float64) - 1).clamp(min=-6) - 3) if eight else 1.0
    return (torch.round(r / step) * step * torch.exp2(e)).flatten(-2)[..., :K]


def _scale64(s, blocks):
    """Scale groups [groups, n, 4] -> float64 [n, 32 * blocks]."""
    e = s.permute(1, 0, 2).flatten(1)[:, :blocks].to(torch.float64) - 127
    return torch.exp2(e).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    f64, op, T, E, k, h = torch.float64, case["op"], case["T"], case["E"], case["k"], case["h"]
    if op in ("few", "few8"):
        eight = op == "few8"

        def mat(w):
            """[K, N] of one expert's (q, scale), or of its weights."""
            return (w[0].to(f64) * _scale64(w[1], w[0].shape[1] // 32)).t() if eight else w.to(f64)

        def ffn(v, a, b, c):
            u = v @ mat(a)
            u = u * torch.sigmoid(u) * (v @ mat(b))
            return (_round64(u, 448.0, True) if eight else u) @ mat(c)

        def of(w, e):
            return (w[0][e], w[1][e]) if eight else w[e]

        z = s["x"].to(f64) @ s["wg"].to(f64) * s["tau"]
        if s["lbias"] is not None:
            z = z + s["lbias"].to(f64)
        p = torch.softmax(z, dim=1)
        order = z if s["sbias"] is None else z + s["sbias"].to(f64)
        ids = torch.argsort(-order, dim=1, stable=True)[:, :k]
        x = s["xq"].to(f64) * _scale64(s["xs"], case["d"] // 32) if eight else s["x"].to(f64)
        y = torch.zeros_like(x)
        for e in torch.unique(ids).tolist():
            t = torch.nonzero((ids == e).any(1)).flatten()
            y[t] += p[t, e, None] * ffn(x[t], of(s["w1"], e), of(s["w3"], e), of(s["w2"], e))
        if s["s1"] is not None:
            y += ffn(x, *[(w[0][0], w[1][0]) if eight else w for w in (s["s1"], s["s3"], s["s2"])])
        return {"y": y, "ids": ids.to(torch.int32), "w": torch.gather(p, 1, ids), "logits": z}
    off = s["offsets"].tolist()
    R = off[-1]
    tok = torch.arange(R, device="cuda") if s["tokens"] is None else s["tokens"].long()
    if op == "up":
        act, h13 = torch.empty((R, h), dtype=f64, device="cuda"), torch.empty((R, 2 * h), dtype=f64, device="cuda")
        x = s["x"].to(f64)
        for e in range(E):
            i = slice(off[e], off[e + 1])
            xe = x[tok[i]]
            a, b = xe @ s["w1"][e].to(f64), xe @ s["w3"][e].to(f64)
            act[i] = a * torch.sigmoid(a) * b
            h13[i] = torch.cat([_round64(a, 127.0, False), _round64(b, 127.0, False)], 1)
        return {"act": act, "h13": h13}
    dh, act = torch.empty((R, 2 * h), dtype=f64, device="cuda"), torch.empty((R, h), dtype=f64, device="cuda")
    dots = torch.empty(R, dtype=f64, device="cuda")
    dy, blocks = s["dy"].to(f64), -(-h // 32)
    for e in range(E):
        i = slice(off[e], off[e + 1])
        a = s["hq"][i, :h].to(f64) * _scale64(s["hs"][0][:, i], blocks)[:, :h]
        b = s["hq"][i, h:].to(f64) * _scale64(s["hs"][1][:, i], blocks)[:, :h]
        da = dy[tok[i]] @ s["w2"][e].to(f64).t().contiguous()
        sg = torch.sigmoid(a)
        dots[i] = (da * a * sg * b).sum(1)
        w = 1.0 if s["weights"] is None else s["weights"][i].to(f64)[:, None]
        act[i] = w * a * sg * b
        dh[i, :h] = w * da * b * (sg + a * sg * (1 - sg))
        dh[i, h:] = w * da * a * sg
    out = {"dh13": dh, "act": act}
    if s["dw"] is not None:
        out["dw"] = dots[s["rows"].long()].view(T, k)
    return out
