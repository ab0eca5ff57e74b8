"""64-bit definitions of the operators around the layer (norm, balance loss,
8-bit rows), on torch float64 tensors of any device, and the bounds that the
tests hold the kernels to."""
from __future__ import annotations

import torch

F64 = torch.float64


def half_step(dt) -> float:
    """A rounding to dt moves a value by at most this, relative to it."""
    return torch.finfo(dt).eps / 2


def norm_ref(x, res, gamma, eps):
    """(sum, rstd, y): sum rounded to the dtype as stored, the rest in 64 bits."""
    s = x if res is None else (x.to(F64) + res.to(F64)).to(torch.float32).to(x.dtype)
    v = s.to(F64)
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + eps)
    return s, rstd, v * rstd[:, None] * gamma.to(F64)


def norm_bwd_ref(dy, dsum, s, gamma, rstd):
    n = s.to(F64) * rstd.to(F64)[:, None]
    u = dy.to(F64) * gamma.to(F64)
    dx = rstd.to(F64)[:, None] * (u - n * (u * n).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.to(F64)
    return dx, (dy.to(F64) * n).sum(0)


def mx8_bytes(v):
    """Scale bytes [n, K / 32] of float64 rows, by comparison with the powers of two."""
    b = v.reshape(v.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    a = torch.where(torch.isfinite(b), b, 0.0).abs().amax(-1)
    e = torch.full(a.shape, 127, dtype=torch.int64, device=v.device)
    for byte in range(255):
        lim = 448.0 * 2.0 ** (byte - 127)
        below = 448.0 * 2.0 ** (byte - 128)
        e[(a <= lim) & ((a > below) | (byte == 0)) & (a > 0)] = byte
    e[bad] = 255
    return e


def mx8_round(v, byte):
    """float64 rows rounded to nearest even in e4m3 with the given scale bytes."""
    s = torch.exp2(byte.to(F64) - 127)
    s[byte == 255] = float("nan")
    r = v.reshape(v.shape[0], -1, 32) / s[..., None]
    x = torch.frexp(r)[1].to(F64) - 1
    step = torch.exp2(torch.clamp(x, min=-6.0) - 3)
    return (torch.round(r / step) * step * s[..., None]).reshape(v.shape)


def scale_bytes(scale, K):
    """uint8 [ceil(K / 128), n, 4] -> int64 [n, K / 32], and the bytes past K."""
    s = scale.permute(1, 0, 2).reshape(scale.shape[1], -1).to(torch.int64)
    return s[:, :K // 32], s[:, K // 32:]


def mx8_values(q, scale):
    """float64 values of 8-bit rows."""
    b, _ = scale_bytes(scale, q.shape[1])
    s = torch.exp2(b.to(F64) - 127)
    s[b == 255] = float("nan")
    return (q.to(torch.float32).to(F64).reshape(q.shape[0], -1, 32) * s[..., None]).reshape(q.shape)


def sequences(T, off, mask, device):
    """Token indices that count, for each sequence."""
    live = torch.ones(T, dtype=torch.bool, device=device) if mask is None else mask.to(torch.bool)
    off = [0, T] if off is None else off.tolist()
    return [torch.nonzero(live[max(a, 0):max(b, 0)]).flatten() + max(a, 0) for a, b in zip(off, off[1:])]


def balance_ref(logits, ids, k, off, mask, alpha):
    """(loss, counts, coef, p) in 64 bits."""
    T, E = logits.shape
    p = torch.softmax(logits.to(F64), 1)
    pick = sequences(T, off, mask, logits.device)
    some = sum(len(i) > 0 for i in pick)
    counts = torch.zeros((len(pick), E), dtype=torch.int64, device=logits.device)
    coef = torch.zeros((len(pick), E), dtype=F64, device=logits.device)
    loss = 0.0
    for s, i in enumerate(pick):
        if not len(i):
            continue
        u = ids[i].flatten().long()
        counts[s] = torch.bincount(u[(u >= 0) & (u < E)], minlength=E)
        coef[s] = alpha * E * counts[s].to(F64) / (k * float(len(i)) ** 2 * some)
        loss += float((coef[s] * p[i].sum(0)).sum())
    return loss, counts, coef, p


def balance_grad_ref(p, coef, off, mask):
    """(dlogits, scale): the gradient for an upstream gradient of 1 and the
    magnitude its two terms have (they cancel in part)."""
    T = p.shape[0]
    dz, mag = torch.zeros_like(p), torch.zeros_like(p)
    for s, i in enumerate(sequences(T, off, mask, p.device)):
        if len(i):
            c = (p[i] * coef[s]).sum(1, keepdim=True)
            dz[i] = p[i] * (coef[s] - c)
            mag[i] = p[i] * (coef[s] + c)
    return dz, mag


def close(got, ref, rel, floor=0.0, name=""):
    """|got - ref| <= rel |ref| + floor, elementwise; NaN where ref is NaN."""
    got, ref = got.to(F64), ref.to(F64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaNs differ"
    err = torch.where(nan, 0.0, (got - ref).abs())
    lim = torch.where(nan, 0.0, rel * ref.abs()) + floor
    bad = err > lim
    if bad.any():
        at = torch.nonzero(bad)[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; first at {at}: {got[i].item()!r} "
                             f"for {ref[i].item()!r}")


class Guarded:
    """Output tensors with a band of known bytes on both sides."""
    BAND = 256

    def __init__(self):
        self.all = []

    def empty(self, shape, dtype, fill=None):
        n = 1
        for s in shape:
            n *= s
        size = n * torch.empty((), dtype=dtype).element_size()
        pad = -size % 256
        raw = torch.full((2 * self.BAND + size + pad,), 0xA5, dtype=torch.uint8, device="cuda")
        t = raw[self.BAND:self.BAND + size].view(dtype).view(shape)
        self.all.append((raw, size))
        if fill is not None:
            t.fill_(fill)
        return t

    def check(self):
        torch.cuda.synchronize()
        for raw, size in self.all:
            assert bool((raw[:self.BAND] == 0xA5).all()), "wrote in front of an output"
            assert bool((raw[self.BAND + size:] == 0xA5).all()), "wrote behind an output"
