"""Every kernel of the 8-bit experts, each at the sizes that run it (which kernel a
case runs is checked by test_mx8_choice.py), against the 64-bit definition with
the bounds of test_gpu_mx8.py."""
import pytest
import torch

import _block_ref as br
import test_gpu_mx8 as tm
from _mx8_cases import CASES
from test_gpu_mx8 import BF, F8, U8, xm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", list(CASES))
def test_experts(xm, name):  # noqa: F811
    c = CASES[name]
    print(f"[experts8] {name}: up {c['up']}, down {c['down']}", flush=True)
    tm._check_experts(xm, c["counts"], c["d"], c["h"], c["T"], seed=len(c["counts"]) + c["d"], spare=c["spare"])


TILES = ["empty halves, K = 128", "short tiles", "heights of a second tile, not gathered"]


@pytest.mark.parametrize("name", TILES)
def test_a_nan_stays_in_its_row(xm, name):  # noqa: F811
    c = CASES[name]
    n = sum(c["counts"])
    first = c["counts"][0]
    rows = sorted({2, 5, first - 1, first, n - 1})

    def tweak(x):
        for i, r in enumerate(rows):
            x[r, (7 * i) % c["d"]] = float("nan") if i % 2 else float("inf")
    _, _, ye = tm._check_experts(xm, c["counts"], c["d"], c["h"], None, tweak=tweak)
    bad = torch.isnan(ye.float())
    assert torch.nonzero(bad.any(1)).flatten().tolist() == rows and bool(bad[rows].all())


GATHERED = ["short tiles, gathered", "empty halves, K = 96", "long and short", "one expert"]


@pytest.mark.parametrize("name", GATHERED)
def test_ids_outside_the_rows_read_zeros(xm, name):  # noqa: F811
    """At the first and last rows of tiles, whatever stands in front of and behind x."""
    c = CASES[name]
    counts, d, h = c["counts"], c["d"], c["h"]
    n, T = sum(counts), c["T"]
    w1, w1s, w3, w3s, _, _ = tm._experts(xm, len(counts), d, h, 3)
    xq, xs = tm._quantize(xm, torch.randn((T, d), generator=tm._gen(1), device="cuda").to(BF))
    ids = torch.randint(0, T, (n,), generator=tm._gen(2), device="cuda").to(torch.int32)
    off, _ = tm._rows(counts)
    act, acts = torch.empty((n, h), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(n, h), dtype=U8, device="cuda")
    xm.xmoe_expert_ffn_up_mx8(xq, xs, w1, w1s, w3, w3s, off, act, acts, token_ids=ids)
    want = br.mx8_values(act, acts)
    rows = [r for r in sorted({0, 1, counts[0] - 1, counts[0], n - 1, n // 2}) if r < n]
    for r, v in zip(rows, (-1, T, 1 << 30, -(1 << 31), (1 << 31) - 1, T + 1)):
        ids[r] = v
    xm.xmoe_expert_ffn_up_mx8(xq, xs, w1, w1s, w3, w3s, off, act, acts, token_ids=ids)
    want[rows] = 0
    assert torch.equal(br.mx8_values(act, acts), want)


@pytest.mark.parametrize("name", ["short tiles, gathered", "empty halves, K = 96", "heights of a second tile"])
def test_weights_that_are_not_finite(xm, name):  # noqa: F811
    """A NaN in a weight makes NaNs of what reads it, a row of zeros included, and of
    nothing else."""
    c = CASES[name]
    counts, d, h, T = c["counts"], c["d"], c["h"], c["T"]
    n, lo = sum(counts), counts[0]
    w1, w1s, w3, w3s, _, _ = tm._experts(xm, len(counts), d, h, 5)
    w1s[1, 0, 40, 2] = 255        # expert 1, column 40, elements 64 .. 95
    xq, xs = tm._quantize(xm, torch.randn((T, d), generator=tm._gen(1), device="cuda").to(BF))
    ids = torch.randint(0, T, (n,), generator=tm._gen(2), device="cuda").to(torch.int32)
    ids[0] = ids[lo] = ids[lo + 2] = -1
    off, _ = tm._rows(counts)
    act, acts = torch.empty((n, h), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(n, h), dtype=U8, device="cuda")
    xm.xmoe_expert_ffn_up_mx8(xq, xs, w1, w1s, w3, w3s, off, act, acts, token_ids=ids)
    v = br.mx8_values(act, acts)
    want = torch.zeros((n, h), dtype=torch.bool, device="cuda")
    want[lo: lo + counts[1], 32:64] = True  # the block of 32 that holds the column
    assert torch.equal(torch.isnan(v), want)
    assert bool((v[0] == 0).all()) and bool((v[lo][:32] == 0).all())


@pytest.mark.parametrize("name", ["short tiles, gathered", "third round split", "heights of a second tile, not gathered"])
def test_the_same_bits_again(xm, name):  # noqa: F811
    c = CASES[name]
    a, b = (tm._check_experts(xm, c["counts"], c["d"], c["h"], c["T"]) for _ in range(2))
    for x, y in zip(a, b):
        assert torch.equal(x.view(U8), y.view(U8))


def test_serving_block_of_a_long_prompt(xm):  # noqa: F811
    """Routed and shared experts on the tile kernel, the shared ones not gathered."""
    import test_gpu_block as tb
    import workloads
    from padding_free_expert_amd.layer import MoEBlock8
    wl = workloads.Workload("serve1500", "bf16", T=1500, d=1088, E=8, h=224, k=3, n_shared=1, h_shared=544, backward=True)
    inp, weights, res, _, _ = tb._inputs(wl)
    for overlap in (True, False):
        block = MoEBlock8(weights, wl.T, wl.k, wl.inv_tau, tb.EPS, overlap=overlap)
        out, s = block.forward(inp["x"], res)
        torch.cuda.synchronize()
        ref, rs = tb._serve_reference(wl, weights, inp["x"], res, block.topk_ids,
                                      [block.w1q, block.w3q, block.w2q, block.s1q, block.s3q, block.s2q])
        assert torch.equal(s, rs)
        tb._near(out, ref, 2e-2, "out")
