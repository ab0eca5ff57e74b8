"""The layers for a few tokens, as a model uses them: one call in place of the layer's
sequence, beside the layers that run the sequence."""
import pytest
import torch

import workloads
from _helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    need_gpu()
    from padding_free_expert_amd import layer
    return layer


def _weights(wl, seed=0):
    inp = {k: v.cuda() for k, v in workloads.generate(wl, backward=True).items() if v is not None}
    w = {k: inp[k] for k in ("wg", "w1", "w3", "w2", "s1", "s3", "s2", "logit_bias", "select_bias") if k in inp}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w["norm"] = (1 + 0.2 * torch.randn(wl.d, generator=g, device="cuda")).to(inp["x"].dtype)
    return inp["x"], w


def _near(a, b, rtol):
    a, b = a.double(), b.double()
    assert torch.isfinite(a).all()
    assert float((a - b).norm()) <= rtol * float(b.norm())


@pytest.mark.parametrize("name", ["tiny_f32", "dsmoe16b", "dsv3", "zipf_skew", "long_batch"])
@pytest.mark.parametrize("T", [1, 13, 64])
def test_layer(layers, name, T):
    """Against the layer's sequence on the same weights: the same choice of experts, y to
    rounding (twice the layer's tolerances, each side being within one)."""
    wl = workloads.small(name)
    x, w = _weights(wl)
    x = x[:T].contiguous()
    few = layers.PaddingFreeMoE(w, T, wl.k, wl.inv_tau, backward=False, few=True)
    full = layers.PaddingFreeMoE(w, T, wl.k, wl.inv_tau, backward=False)
    y = few.forward(x)
    assert y is few.y and few.saved_bytes() == 0
    full.forward(x)
    same = (few.topk_ids == full.topk_ids).all(1)
    assert float(same.float().mean()) > 0.9   # near ties may differ
    _near(y[same], full.y[same], 2e-4 if wl.dtype == "f32" else 4e-2)
    _near(few.topk_w[same], full.topk_w[same], 1e-4)
    _near(few.logits, full.logits, 1e-4)
    # new weights are read at the next call
    w["w2"].mul_(2.0)
    z = few.forward(x).clone()
    full.forward(x)
    _near(z[same], full.y[same], 2e-4 if wl.dtype == "f32" else 4e-2)


def test_blocks_and_a_decode_loop_in_a_graph(layers):
    """Pre-norm and layer (bf16), and with 8-bit experts, four blocks deep, captured."""
    wl = workloads.small("dsmoe16b")
    wl = workloads.Workload("w", "bf16", T=24, d=256, E=16, h=224, k=6, n_shared=2, h_shared=224, backward=True)
    x, w = _weights(wl)
    for make in (lambda few: layers.MoEBlock(w, wl.T, wl.k, backward=False, **({"few": True} if few else {})),
                 lambda few: layers.MoEBlock8(w, wl.T, wl.k, few=few)):
        few, full = [make(True) for _ in range(4)], [make(False) for _ in range(4)]

        def run(blocks, h):
            res = None
            for b in blocks:
                h, res = b.forward(h, res)
            return h, res

        want = [t.clone() for t in run(few, x)]
        one, two = few[0].forward(x)[0].clone(), full[0].forward(x)[0].clone()
        _near(one, two, 4e-2)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run(few, x)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(few, x)
        for _ in range(3):
            for t in out:
                t.zero_()
            g.replay()
            full[1].forward(x)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_block8_refreshes(layers):
    wl = workloads.Workload("w", "bf16", T=5, d=128, E=8, h=96, k=2, n_shared=1, h_shared=64, backward=True)
    x, w = _weights(wl)
    b = layers.MoEBlock8(w, wl.T, wl.k, few=True)
    y = b.forward(x)[0].clone()
    w["w2"].mul_(2.0)
    w["s2"].mul_(2.0)
    assert torch.equal(b.forward(x)[0], y)
    b.refresh_weights()
    _near(b.forward(x)[0], 2 * y.double(), 2.0 ** -7)


def test_refusals(layers):
    wl = workloads.small("dsmoe16b")
    _, w = _weights(wl)
    for kw in (dict(backward=True), dict(backward=False, merge_shared=True), dict(backward=False, balance_alpha=0.1)):
        with pytest.raises(ValueError, match="few"):
            layers.PaddingFreeMoE(w, 4, wl.k, few=True, **kw)
    with pytest.raises(ValueError, match="64 tokens"):
        layers.PaddingFreeMoE(w, 65, wl.k, backward=False, few=True)
    with pytest.raises(ValueError, match="does not take"):
        layers.MoEBlock8({**w, "w1": w["w1"][:, :, :192].contiguous(), "w3": w["w3"][:, :, :192].contiguous(),
                          "w2": w["w2"][:, :192].contiguous(), "s1": w["s1"][:, :384].contiguous(),
                          "s3": w["s3"][:, :384].contiguous(), "s2": w["s2"][:384].contiguous()}, 65, wl.k, few=True)
    m = layers.PaddingFreeMoE(w, 4, wl.k, backward=False, few=True)
    with pytest.raises(ValueError):
        m.forward(torch.empty((5, wl.d), dtype=torch.bfloat16, device="cuda"))
