"""64-bit definition of the whole layer for a few tokens, with the error that the
formats allow to each result.

Roundings: an activation is held in fp32 (2^-24 of it), for bf16 as the sum of two bf16
values (half a step of the second, which is at most half a step of the first: 2^-16 of it
at most), with 8 bits rounded to them (2^-4 of it, or half of the smallest step, 2^-10,
times the block's scale); y is rounded once.  A sum of K products in fp32 is off by at
most K 2^-24 of the sum of their magnitudes (the down-projection of bf16 has 2 h products,
two for an activation).  silu(a) moves by at most
1.1 times a's own error, exp and the division by 2^-20 of the value."""
from __future__ import annotations

import torch

from _block_ref import half_step, mx8_bytes, mx8_round, mx8_values

F64 = torch.float64


def silu(a):
    return a * torch.sigmoid(a)


def ffn(x, w1, w3, w2, act_half):
    """(values, allowed error) of one SwiGLU FFN on float64 rows; act_half None: act in
    8 bits, else the part of it that is lost."""
    K, h = w1.shape[0], w1.shape[1]
    a, b = x @ w1, x @ w3
    d1 = K * 2.0 ** -24 * (x.abs() @ w1.abs())
    d3 = K * 2.0 ** -24 * (x.abs() @ w3.abs())
    v = silu(a) * b
    dv = 1.1 * d1 * (b.abs() + d3) + silu(a).abs() * d3 + 2.0 ** -20 * v.abs()
    if act_half is None:
        act = mx8_round(v, mx8_bytes(v)) if v.shape[0] else v
        top = torch.nn.functional.pad(v.abs() + dv, (0, -h % 32)).reshape(v.shape[0], -(-h // 32), 32).amax(-1)
        # the block's scale is less than top / 224; a smallest step is 2^-9 of it.  Against
        # the rounded reference each of the two is half a step from v
        small = (2.0 ** -10 / 224 * top).repeat_interleave(32, 1)[:, :h]
        da = 2 * (2.0 ** -4 * (v.abs() + dv) + small) + dv
    else:
        act = v
        da = act_half * (v.abs() + dv) + dv
    return act @ w2, da @ w2.abs() + 2 * h * 2.0 ** -24 * ((act.abs() + da) @ w2.abs())


def gate(x, wg, tau, lbias):
    """(logits, their allowed error)"""
    z = x @ wg * tau
    dz = x.shape[1] * 2.0 ** -24 * (x.abs() @ wg.abs()) * abs(tau) + 2.0 ** -23 * z.abs()
    if lbias is not None:
        z = z + lbias.to(F64)
        dz = dz + 2.0 ** -24 * z.abs()
    return z, dz


def layer(x, xe, wg, sets, shared, ids, tau=1.0, lbias=None, act_half=None, out_half=0.0):
    """y and its allowed error for the given ids.  x: the gate's rows, xe: the experts';
    sets(e) and shared: (w1, w3, w2) in float64."""
    z, dz = gate(x, wg, tau, lbias)
    p = torch.softmax(z, 1)
    dp = p * (2 * dz.amax(1, keepdim=True) + 2.0 ** -20)
    y, dy = torch.zeros_like(xe), torch.zeros_like(xe)
    for e in torch.unique(ids).tolist():
        t = torch.nonzero((ids == e).any(1)).flatten()
        v, dv = ffn(xe[t], *sets(e), act_half)
        w, dw = p[t, e, None], dp[t, e, None]
        y[t] += w * v
        dy[t] += w * dv + dw * (v.abs() + dv)
    if shared is not None:
        v, dv = ffn(xe, *shared, act_half)
        y += v
        dy += dv
    return z, dz, p, dp, y, dy + (out_half + 2.0 ** -20) * (y.abs() + dy)


def chosen_well(z, dz, sbias, ids):
    """Whether ids are a top-k of z (+ sbias) up to the logits' allowed error, in
    descending order."""
    sel = z if sbias is None else z + sbias.to(F64)
    slack = 2 * dz.amax(1, keepdim=True) + 2.0 ** -22 * sel.abs().amax(1, keepdim=True)
    got = torch.gather(sel, 1, ids.long())
    left = sel.scatter(1, ids.long(), -float("inf"))
    return bool((got[:, :-1] + slack >= got[:, 1:]).all() and (got[:, -1:] + slack >= left.amax(1, keepdim=True)).all())


def mx8_weights(q, scale):
    """float64 [K, N] of one expert's 8-bit weights [N, K]."""
    return mx8_values(q, scale).t()


__all__ = ["ffn", "gate", "layer", "chosen_well", "mx8_weights", "half_step", "mx8_values", "silu"]
