"""Sequences of which the balance loss counts nothing, over many pieces: results
against the 64-bit definition (bounds as in test_gpu_balance.py), and a time that
does not grow with what is masked."""
import pytest
import torch

import test_gpu_balance as tb
from test_gpu_balance import xm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,S,E,k", [
    (40000, 2, 16, 2), (40000, 16, 33, 3), (40000, 17, 16, 2), (40000, 63, 8, 2), (40000, 64, 64, 6), (40000, 65, 16, 2),
    (40000, 300, 8, 1), (65536, 3, 8, 2), (65537, 3, 8, 2), (200000, 5, 16, 2),
    (5000, 200, 1024, 8), (9000, 4096, 64, 2)])
def test_masked_sequences(xm, T, S, E, k):  # noqa: F811
    """Every second sequence masked, the first one too; then all but the last
    token; sequences up to the whole batch."""
    print(f"[balance] T={T} S={S} E={E}", flush=True)
    logits, ids, g = tb._case(T, E, k, seed=T + S)
    cut = torch.sort(torch.randint(1, T - 5, (S - 1,), generator=g, device="cuda")).values
    off = torch.cat([torch.tensor([2], device="cuda"), cut, torch.tensor([T - 1], device="cuda")]).to(torch.int32)
    off = torch.sort(off).values.to(torch.int32)
    at = off.tolist()
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    for a, b in list(zip(at, at[1:]))[::2]:
        mask[a:b] = False
    tb._check(xm, logits, ids, k, off, mask)
    mask[:] = False
    mask[T - 2] = True
    tb._check(xm, logits, ids, k, off, mask)


def _us(f):
    for _ in range(3):
        f()
    r = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            f()
        b.record()
        b.synchronize()
        r.append(a.elapsed_time(b) * 100)
    return sorted(r)[3]


def test_a_masked_sequence_costs_what_a_counted_one_does(xm):  # noqa: F811
    """2^19 masked tokens are 4096 pieces: read one after another they would take
    several times what the whole call takes."""
    T, E, k = 1 << 20, 16, 2
    logits, ids, _ = tb._case(T, E, k, seed=1)
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(1, device="cuda"), torch.empty((2, E), dtype=torch.int32, device="cuda")
    coef = torch.empty((2, E), device="cuda")
    ws = torch.empty(xm.xmoe_balance_loss_workspace_size(T, E, 2), dtype=torch.uint8, device="cuda")
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    call = lambda: xm.xmoe_balance_loss(logits, ids, 0.1, loss, counts, coef, off, mask, ws)
    free = _us(call)
    mask[:T // 2] = False
    masked = _us(call)
    print(f"[balance] 2^20 tokens {free:.1f} us, half of them masked {masked:.1f} us", flush=True)
    assert masked <= 2 * free
