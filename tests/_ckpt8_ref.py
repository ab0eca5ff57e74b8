"""64-bit definition of pre-activations kept in 8 bits and of the backward that reads
them, on torch float64 tensors of any device."""
from __future__ import annotations

import torch

F64 = torch.float64


def blocks(v):
    """[n, h] -> [n, ceil(h / 32), 32], zeros behind h."""
    return torch.nn.functional.pad(v, (0, -v.shape[1] % 32)).reshape(v.shape[0], -(-v.shape[1] // 32), 32)


def scale_bytes(v):
    """Scale byte of each block of float64 rows, by comparison with the powers of two."""
    b = blocks(v)
    bad = ~torch.isfinite(b).all(-1)
    a = torch.where(torch.isfinite(b), b, 0.0).abs().amax(-1)
    e = torch.full(a.shape, 127, dtype=torch.int64, device=v.device)
    for byte in range(255):
        e[(a <= 127 * 2.0 ** (byte - 127)) & ((a > 127 * 2.0 ** (byte - 128)) | (byte == 0)) & (a > 0)] = byte
    e[bad] = 255
    return e


def round8(v):
    """(int8 values, scale bytes, float64 values) of float64 rows."""
    byte = scale_bytes(v)
    q = torch.round(blocks(v) / torch.exp2(byte.to(F64) - 127)[..., None])
    q = torch.where((byte == 255)[..., None], 0.0, q)
    val = (q * scale(byte)[..., None]).flatten(1)[:, : v.shape[1]]
    return q.flatten(1)[:, : v.shape[1]].to(torch.int8), byte, val


def scale(byte):
    s = torch.exp2(byte.to(F64) - 127)
    s[byte == 255] = float("nan")
    return s


def half(hscale, h, b):
    """(bytes [rows, ceil(h / 32)] of H1 (b = 0) or H3, the bytes past them)."""
    s = hscale[b].permute(1, 0, 2).flatten(1).to(torch.int64)
    return s[:, : -(-h // 32)], s[:, -(-h // 32):]


def values(hq, hscale):
    """float64 (H1, H3) of 8-bit pre-activations."""
    h = hq.shape[1] // 2
    out = []
    for b in range(2):
        s = scale(half(hscale, h, b)[0]).repeat_interleave(32, 1)[:, :h]
        out.append(hq[:, b * h:(b + 1) * h].to(F64) * s)
    return out


def pack(h1, h3):
    """(hq, hscale) of float64 pre-activations."""
    rows, h = h1.shape
    hq = torch.empty((rows, 2 * h), dtype=torch.int8, device=h1.device)
    hs = torch.full((2, -(-h // 128), rows, 4), 127, dtype=torch.uint8, device=h1.device)
    for b, v in enumerate((h1, h3)):
        q, byte, _ = round8(v)
        hq[:, b * h:(b + 1) * h] = q
        full = torch.full((rows, 4 * hs.shape[1]), 127, dtype=torch.int64, device=h1.device)
        full[:, : byte.shape[1]] = byte
        hs[b] = full.reshape(rows, -1, 4).permute(1, 0, 2).to(torch.uint8)
    return hq, hs


def backward(dy, tok, w2, h1, h3, weights, off):
    """(dH1, dH3, act, dots, dA, sum |dy||w2|) of rows on their experts, all in 64 bits;
    rows in no segment are NaN."""
    R, h = h1.shape
    nan = lambda *s: torch.full(s, float("nan"), dtype=F64, device=h1.device)
    da, mag = nan(R, h), nan(R, h)
    rows = dy if tok is None else dy[tok.long()]
    for e in range(w2.shape[0]):
        i = slice(off[e], off[e + 1])
        w = w2[e].to(F64).t().contiguous()
        da[i] = rows[i].to(F64) @ w
        mag[i] = rows[i].to(F64).abs() @ w.abs()
    sg = torch.sigmoid(h1)
    act = h1 * sg * h3
    dots = (da * act).sum(1)
    w = 1.0 if weights is None else weights.to(F64)[:, None]
    return w * da * h3 * (sg + h1 * sg * (1 - sg)), w * da * h1 * sg, w * act, dots, da, mag
