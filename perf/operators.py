"""Timed passes of the operators around the expert layer: the residual addition
with the root-mean-square norm (forward, with an output in 8 bits, and
backward), the balance loss of the gate with its counts and gradient, and the
experts' feed-forward on 8-bit rows and weights.

`own` chooses between the plain form (elementary torch operations) and the
calls of padding_free_expert_amd.  8-bit values are e4m3 with one power-of-two
scale (a byte b stands for 2^(b - 127)) for each 32 consecutive elements of the
summed axis; scales of n rows of K elements lie as [ceil(K / 128), n, 4], the
unused bytes of the last group being 127.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a serving loop: residual added, normed, handed to 8-bit experts
        dict(name="norm8 1 token", op="norm", T=1, d=2048, dtype="bf16", res=True, out="q"),
        # the pre-norm of a training step, gate and experts reading y
        dict(name="norm train", op="norm", T=4096, d=2048, dtype="bf16", res=True, out="y"),
        # a long prompt in front of 8-bit experts; the gate reads y, the experts q
        dict(name="norm8 prompt", op="norm", T=8192, d=7168, dtype="bf16", res=True, out="yq"),
        # its backward in a long-batch training step, with the gradient that arrives on the residual path
        dict(name="norm back", op="norm_bwd", T=32768, d=4096, dtype="bf16", res=True),
        # ragged fp32 rows, no residual: the parity runs of a small model
        dict(name="norm back f32 ragged", op="norm_bwd", T=1021, d=1000, dtype="f32", res=False),
        # a training micro-batch's loss, counts and gradient, all tokens one batch
        dict(name="balance batch", op="balance", T=4096, E=64, k=6, S=1, masked=False),
        # packed sequences of a long batch, padding masked, a tail behind the last sequence
        dict(name="balance sequences", op="balance", T=32768, E=160, k=8, S=24, masked=True),
        # single-token serving: the chosen experts' weights are all that is read
        dict(name="experts8 1 token", op="experts", T=1, d=2048, h=1408, E=64, k=6, skew=0.0),
        # a decode batch: a few rows for each expert
        dict(name="experts8 decode", op="experts", T=96, d=2048, h=1408, E=64, k=6, skew=0.0),
        # a prompt on uneven experts
        dict(name="experts8 skewed", op="experts", T=2000, d=2048, h=768, E=128, k=8, skew=0.6),
        # a prompt of a training-sized batch
        dict(name="experts8 prompt", op="experts", T=4096, d=2048, h=1408, E=64, k=6, skew=0.0),
        # the widest experts of the workloads here, a large prefill
        dict(name="experts8 large", op="experts", T=16384, d=4096, h=1024, E=96, k=8, skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "balance", "experts", "experts"])
    if op in ("norm", "norm_bwd"):
        out = rng.choice(["y", "q", "yq"]) if op == "norm" else "y"
        step = 32 if "q" in out else 8
        d = step * max(1, _log(rng, 64, 8192) // step)
        T = _log(rng, 1, max(2, min(40000, 100_000_000 // d)))
        case = dict(op=op, T=T, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), res=rng.random() < 0.7)
        if op == "norm":
            case["out"] = out
        return case
    if op == "balance":
        E = rng.choice([8, 24, 64, 100, 160, 256, 512])
        T = _log(rng, 1, 30000)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=_log(rng, 1, min(T, 40)) if rng.random() < 0.6 else 1,
                    masked=rng.random() < 0.5)
    E = rng.choice([4, 8, 16, 40, 64])
    d, h = 32 * _log(rng, 4, 96), 32 * _log(rng, 2, 56)
    T = _log(rng, 1, 12000)
    return dict(op=op, T=T, d=d, h=h, E=E, k=rng.randint(1, min(8, E)), skew=rng.choice([0.0, 0.5]))


# ------------------------------------------------------------------ inputs

def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantize(v):
    """fp32 [..., K] -> e4m3 [..., K] and scale bytes [..., K / 32]: the least
    power of two that brings the block's largest magnitude to at most 448."""
    b = v.unflatten(-1, (-1, 32))
    m, x = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, x - 9 + (m > 0.875).to(x.dtype), 0).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _scale_groups(s):
    """Scale bytes [..., n, K / 32] -> [..., ceil(K / 128), n, 4]."""
    pad = -s.shape[-1] % 4
    s = torch.nn.functional.pad(s, (0, pad), value=127)
    return s.unflatten(-1, (-1, 4)).transpose(-3, -2).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op in ("norm", "norm_bwd"):
        T, d, dt = case["T"], case["d"], _dt(case)
        # a residual stream with a few large channels; rows of different size
        chan = 1.0 + 8.0 * (torch.rand(d, generator=g, device="cuda") > 0.995)
        a = (randn(T, d) * chan * torch.exp(0.5 * randn(T, 1))).to(dt)
        s = dict(op=op, gamma=(1.0 + 0.2 * randn(d)).to(dt), x=a)
        if op == "norm":
            s["out"] = case["out"]
            s["res"] = (2.0 * randn(T, d) * chan).to(dt) if case["res"] else None
            s["sum"] = torch.empty_like(a) if case["res"] else None
            s["y"] = torch.empty_like(a) if "y" in case["out"] else None
            s["q"] = torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda") if "q" in case["out"] else None
            s["qs"] = torch.empty((-(-d // 128), T, 4), dtype=torch.uint8, device="cuda") if "q" in case["out"] else None
            s["deq"] = torch.empty((T, d), dtype=torch.bfloat16, device="cuda") if "q" in case["out"] else None
        else:
            s["rstd"] = 1.0 / torch.sqrt(a.float().square().mean(1) + EPS)
            s["dy"] = randn(T, d).to(dt)
            s["dsum"] = randn(T, d).to(dt) if case["res"] else None
            s["dx"] = torch.empty_like(a)
            s["dgamma"] = torch.empty(d, device="cuda")
        return s
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        logits = 1.5 * randn(T, E) + 0.5 * randn(E)
        s = dict(op=op, logits=logits, ids=torch.topk(logits, k, 1).indices.to(torch.int32), k=k, S=S, E=E,
                 dloss=torch.ones(1, device="cuda"), mask=None, off=None)
        if S > 1:
            cut = torch.rand(S, generator=g, device="cuda") ** 2 + 0.02
            cut = torch.cumsum(cut, 0) / (cut.sum() * 1.03)  # a tail of tokens behind the last sequence
            s["off"] = torch.cat([torch.zeros(1, device="cuda"), cut * T]).to(torch.int32)
        if case["masked"]:
            s["mask"] = torch.rand(T, generator=g, device="cuda") < 0.85
        s["loss"] = torch.empty(1, device="cuda")
        s["counts"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
        s["coef"] = torch.empty((S, E), device="cuda")
        s["dlogits"] = torch.empty((T, E), device="cuda")
        return s
    T, d, h, E, k = case["T"], case["d"], case["h"], case["E"], case["k"]
    s = dict(op=op, T=T, d=d, h=h, E=E, x=randn(T, d).to(torch.bfloat16))
    key = randn(T, E) - case["skew"] * torch.log1p(torch.arange(E, device="cuda"))
    ids = torch.topk(key, k, 1).indices.flatten()
    order = torch.argsort(ids, stable=True)
    n = torch.bincount(ids, minlength=E)
    s["token_ids"] = (order // k).to(torch.int32)
    s["expert_ids"] = ids[order]
    s["offsets"] = torch.cat([torch.zeros(1, device="cuda"), torch.cumsum(n, 0)]).to(torch.int32)
    s["active"] = torch.nonzero(n).flatten()
    s["cap"] = int(n.max())
    # each row's place among its expert's rows, and its expert's among the active ones
    s["place"] = torch.arange(T * k, device="cuda") - s["offsets"][s["expert_ids"]].long()
    s["slot"] = (torch.cumsum((n > 0).int(), 0) - 1)[s["expert_ids"]]
    for name, N, K in (("w1", h, d), ("w3", h, d), ("w2", d, h)):
        q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty((E, -(-K // 128), N, 4), dtype=torch.uint8, device="cuda")
        for e in range(0, E, 16):
            m = min(16, E - e)
            a, b = _quantize(randn(m, N, K) * K ** -0.5)
            q[e:e + m], sc[e:e + m] = a, _scale_groups(b)
        s[name], s[name + "s"] = q, sc
    R = T * k
    f8 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    s["xq"], s["xqs"] = torch.empty((T, d), **f8), torch.empty((-(-d // 128), T, 4), **u8)
    s["act"], s["acts"] = torch.empty((R, h), **f8), torch.empty((-(-h // 128), R, 4), **u8)
    s["ye"] = torch.empty((R, d), dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _rows8(v):
    """The values that fp32 rows [n, K] stand for in 8 bits."""
    q, s = _quantize(v)
    return torch.ldexp(q.float().unflatten(-1, (-1, 32)), s.int().unsqueeze(-1) - 127).flatten(-2)


def _weights8(q, s, active):
    """The fp32 values [A, N, K] of the active experts' weights."""
    if active.numel() < q.shape[0]:
        q, s = q.view(torch.uint8)[active].view(torch.float8_e4m3fn), s[active]
    K = q.shape[-1]
    s = s.transpose(-3, -2).flatten(-2)[..., : K // 32]
    return (q.float().unflatten(-1, (-1, 32)) * torch.exp2(s.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _plain_norm(s):
    out = {}
    v = s["x"]
    if s["res"] is not None:
        v = (v.float() + s["res"].float()).to(v.dtype)
        out["sum"] = v
    f = v.float()
    y = f * (1.0 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)) * s["gamma"].float()
    if "y" in s["out"]:
        out["y"] = y.to(v.dtype)
    if "q" in s["out"]:
        out["q"] = _rows8(y).to(torch.bfloat16)
    return out


def _plain_norm_bwd(s):
    n = s["x"].float() * s["rstd"].unsqueeze(1)
    dy = s["dy"].float()
    u = dy * s["gamma"].float()
    dx = s["rstd"].unsqueeze(1) * (u - n * (u * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * n).sum(0)}


def _members(s):
    """[S, T] in fp32: 1 where a token counts for a sequence."""
    T = s["logits"].shape[0]
    at = torch.arange(T, device="cuda")
    if s["off"] is None:
        m = torch.ones((1, T), device="cuda")
    else:
        m = ((at >= s["off"][:-1, None]) & (at < s["off"][1:, None])).float()
    return m if s["mask"] is None else m * s["mask"].float()


def _plain_balance(s):
    z = s["logits"]
    T, E = z.shape
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    m = _members(s)
    n = m.sum(1, keepdim=True)
    some = (n > 0).float()
    used = torch.zeros((T, E), device="cuda").scatter_(1, s["ids"].long(), 1.0)
    c = m @ used
    n1 = n.clamp(min=1.0)
    coef = c * (E / s["k"]) / (n1 * n1 * some.sum().clamp(min=1.0)) * ALPHA
    loss = (coef * (m @ p)).sum().reshape(1)
    g = m.t() @ coef
    dz = s["dloss"] * p * (g - (p * g).sum(1, keepdim=True))
    return {"loss": loss, "counts": c.to(torch.int32), "coef": coef, "dlogits": dz}


ALPHA = 0.01


def _plain_experts(s):
    A, cap = s["active"].numel(), s["cap"]
    x = _rows8(s["x"].float())
    xe = torch.zeros((A, cap, s["d"]), device="cuda")
    xe[s["slot"], s["place"]] = x[s["token_ids"].long()]
    a = torch.matmul(xe, _weights8(s["w1"], s["w1s"], s["active"]).transpose(1, 2))
    b = torch.matmul(xe, _weights8(s["w3"], s["w3s"], s["active"]).transpose(1, 2))
    act = _rows8(a / (1.0 + torch.exp(-a)) * b)
    y = torch.matmul(act, _weights8(s["w2"], s["w2s"], s["active"]).transpose(1, 2))
    return {"ye": y[s["slot"], s["place"]].to(s["ye"].dtype)}


# --------------------------------------------------------- the framework's

def _own_norm(s):
    import padding_free_expert_amd as xm
    xm.xmoe_add_rmsnorm(s["x"], s["res"], s["gamma"], EPS, s["sum"], s["y"], q=s["q"], scale=s["qs"])
    out = {} if s["sum"] is None else {"sum": s["sum"]}
    if s["y"] is not None:
        out["y"] = s["y"]
    if s["q"] is not None:
        xm.xmoe_mx8_dequantize(s["q"], s["qs"], s["deq"])
        out["q"] = s["deq"]
    return out


def _own_norm_bwd(s):
    import padding_free_expert_amd as xm
    xm.xmoe_add_rmsnorm_bwd(s["dy"], s["dsum"], s["x"], s["gamma"], s["rstd"], s["dx"], s["dgamma"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _own_balance(s):
    import padding_free_expert_amd as xm
    xm.xmoe_balance_loss(s["logits"], s["ids"], ALPHA, s["loss"], s["counts"], s["coef"], seq_offsets=s["off"],
                         token_mask=s["mask"])
    xm.xmoe_balance_loss_bwd(s["logits"], s["coef"], s["dlogits"], seq_offsets=s["off"], token_mask=s["mask"],
                             dloss=s["dloss"])
    return {n: s[n] for n in ("loss", "counts", "coef", "dlogits")}


def _own_experts(s):
    import padding_free_expert_amd as xm
    xm.xmoe_mx8_quantize(s["x"], s["xq"], s["xqs"])
    xm.xmoe_expert_ffn_up_mx8(s["xq"], s["xqs"], s["w1"], s["w1s"], s["w3"], s["w3s"], s["offsets"], s["act"],
                              s["acts"], token_ids=s["token_ids"])
    xm.xmoe_expert_ffn_down_mx8(s["act"], s["acts"], s["w2"], s["w2s"], s["offsets"], s["ye"])
    return {"ye": s["ye"]}


def run(state):
    op = state["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "balance": _own_balance, "experts": _own_experts}[op](state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance, "experts": _plain_experts}[op](state)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n = case["T"] * case["d"]
        es = 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            b = n * es * (3 if case["res"] else 1) + ("y" in case["out"]) * n * es + ("q" in case["out"]) * n * 33 // 32
            return {"bytes": b + case["d"] * es, "flops": 6 * n}
        return {"bytes": n * es * (4 if case["res"] else 3) + 4 * case["T"] + 4 * case["d"], "flops": 10 * n}
    if op == "balance":
        T, E = case["T"], case["E"]
        # the gradient needs the counts of all tokens: the logits are read twice
        return {"bytes": 12 * T * E + 4 * T * case["k"] + case["masked"] * T + 8 * case["S"] * E, "flops": 10 * T * E}
    T, d, h, E, k = (case[n] for n in ("T", "d", "h", "E", "k"))
    R = T * k
    active = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": 2 * T * d + 2 * R * d + active * 3 * d * h * 33 / 32 + 4 * R, "flops": 6.0 * R * d * h}


# ---------------------------------------------------- the definition, 64 bits

def _e4m3_64(v):
    """float64 [..., K] rounded to 8 bits with a scale for each 32, as float64."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().max(dim=-1, keepdim=True).values
    e = torch.ceil(torch.log2(torch.where(top > 0, top / 448.0, torch.ones_like(top))))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e)  # log2's own rounding at a border
    e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
    e = torch.where(top > 0, e, torch.zeros_like(e)).clamp(-127, 127)
    r = b * torch.exp2(-e)
    _, x = torch.frexp(r)
    step = torch.exp2((x.to(torch.float64) - 1).clamp(min=-6) - 3)
    return (torch.round(r / step) * step * torch.exp2(e)).reshape(v.shape)


def _w64(q, s):
    K = q.shape[-1]
    e = s.permute(1, 0, 2).reshape(q.shape[-2], -1)[:, : K // 32].to(torch.float64) - 127
    return q.to(torch.float64) * torch.exp2(e).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm":
        v, out = s["x"].to(f64), {}
        if s["res"] is not None:
            # the norm is defined on the stored sum
            v = (s["x"].to(f64) + s["res"].to(f64)).to(s["x"].dtype).to(f64)
            out["sum"] = v
        y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["gamma"].to(f64)
        if "y" in case["out"]:
            out["y"] = y
        if "q" in case["out"]:
            out["q"] = _e4m3_64(y)
        return out
    if op == "norm_bwd":
        x, dy, r = s["x"].to(f64), s["dy"].to(f64), s["rstd"].to(f64)[:, None]
        u = dy * s["gamma"].to(f64)
        dx = r * u - x * r ** 3 * ((u * x).sum(dim=1, keepdim=True) / case["d"])
        if s["dsum"] is not None:
            dx += s["dsum"].to(f64)
        return {"dx": dx, "dgamma": torch.mv((dy * x).t(), r[:, 0])}
    if op == "balance":
        T, E, S, k = case["T"], case["E"], case["S"], case["k"]
        p = torch.softmax(s["logits"].to(f64), dim=1)
        off = [0, T] if s["off"] is None else s["off"].tolist()
        live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
        coef = torch.zeros((S, E), dtype=f64, device="cuda")
        loss = torch.zeros(1, dtype=f64, device="cuda")
        dz = torch.zeros((T, E), dtype=f64, device="cuda")
        pick = [torch.nonzero(live[a:b]).flatten() + a for a, b in zip(off, off[1:])]
        full = max(1, sum(len(i) > 0 for i in pick))
        for n, i in enumerate(pick):
            if len(i) == 0:
                continue
            c = torch.bincount(s["ids"][i].flatten().long(), minlength=E)
            counts[n] = c
            coef[n] = ALPHA * E * c.to(f64) / (k * float(len(i)) ** 2 * full)
            loss += (coef[n] * p[i].sum(dim=0)).sum()
            dz[i] = p[i] * (coef[n] - p[i] @ coef[n][:, None])
        return {"loss": loss, "counts": counts, "coef": coef, "dlogits": dz}
    x = _e4m3_64(s["x"].to(f64))
    ye = torch.zeros((case["T"] * case["k"], case["d"]), dtype=f64, device="cuda")
    off = s["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        xe = x[s["token_ids"][lo:hi].long()]
        a, b = xe @ _w64(s["w1"][e], s["w1s"][e]).t(), xe @ _w64(s["w3"][e], s["w3s"][e]).t()
        ye[lo:hi] = _e4m3_64(a * torch.sigmoid(a) * b) @ _w64(s["w2"][e], s["w2s"][e]).t()
    return {"ye": ye}
