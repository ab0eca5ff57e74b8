"""The layer for a few tokens where its down-projection has many strips (2048 strips of
columns of chosen experts, and more): a wave then takes strips by itself, one after the
other; and where routed activations are formed by a launch of their own."""
import pytest
import torch

from test_gpu_few import BF, F32, Case, xm  # noqa: F401  (xm is a fixture)

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f32", "mx8"]


def _case(xm, sizes, kind, **kw):  # noqa: F811
    return Case(xm, *sizes, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8", **kw)


# T, d, E, k, h, hs.  Strips of the down-projection: of 128 columns in bf16, of 64 else
MANY_STRIPS = [
    (64, 2112, 128, 8, 96, 96),       # 2176 to 4257 strips with the shared experts', the last group of four not full
    (64, 2080, 128, 8, 96, 0),        # a width that ends inside a strip
    (64, 2112, 264, 8, 64, 0),        # 8712 strips in fp32 and 8 bits: two for each wave, the last group not full
    (64, 4160, 32, 8, 544, 288),      # two row tiles, several parts, activations by a launch of their own
    (4, 4128, 96, 16, 64, 0),         # few tokens: top-k inside the up-projection, an expert a slot
    (12, 2112, 136, 9, 160, 32),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", MANY_STRIPS, ids=str)
def test_many_strips(xm, sizes, kind):  # noqa: F811
    _case(xm, sizes, kind, bias=sizes[0] != 64, seed=1).run().check(kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", [(64, 1024, 8, 2, 64, 0), (33, 1024, 16, 4, 64, 32), (64, 1024, 8, 2, 160, 0)], ids=str)
def test_activations_by_a_launch_of_their_own(xm, sizes, kind):  # noqa: F811
    """Few experts with many rows each and a d that is cut into several parts."""
    _case(xm, sizes, kind, bias=True, seed=2).run().check(kind)


@pytest.mark.parametrize("kind", KINDS)
def test_many_rows_on_a_few_of_many_experts(xm, kind):  # noqa: F811
    """Every token on the same experts: four passes of 16 rows over a wave's strips."""
    c = _case(xm, (64, 2080, 264, 8, 64, 0), kind)
    chosen = [3, 64, 65, 127, 128, 200, 262, 263]
    c.sb = torch.zeros(264, device="cuda")
    c.sb[chosen] = 100.0
    c.run().check(kind)
    assert all(sorted(r) == chosen for r in c.ids.tolist())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_infinite_weights_reach_only_their_column(xm, kind):  # noqa: F811
    c = _case(xm, (5, 2080, 136, 100, 40, 0), kind)
    clean = c.run().outs()
    e = int(c.ids[0, 0])
    for col in (5, 2079):     # the first strip, and the last column of all
        c.w[2][e, 39, col] = float("inf")
    c.run()
    other = torch.ones(2080, dtype=torch.bool, device="cuda")
    other[[5, 2079]] = False
    assert torch.equal(c.y[:, other], clean[3][:, other])
    assert not torch.isfinite(c.y[0, [5, 2079]]).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", [MANY_STRIPS[0], MANY_STRIPS[3]], ids=str)
def test_repeats_graphs_and_streams(xm, sizes, kind):  # noqa: F811
    """The same bits eager, on another stream and replayed, whatever the workspace held;
    nothing is written past its needed bytes."""
    c, other = _case(xm, sizes, kind, seed=4), _case(xm, sizes, kind, seed=5)
    n = c.need()
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    want = c.run(workspace=ws).check(kind).outs()
    assert bool((ws[n:] == 255).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (c.ids, c.p, c.z, c.y):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c.outs()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(workspace=ws)
    for i in range(3):
        for t in (c.ids, c.p, c.z, c.y):
            t.zero_()
        ws.fill_(255)
        other.run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, c.outs())), i
