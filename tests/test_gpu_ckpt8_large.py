"""8-bit pre-activations of more than 2^31 elements: the same bits as calls on parts."""
import pytest
import torch

from test_gpu_ckpt8 import BF, F32, I8, I32, U8, _gen, xm  # noqa: F401  (xm is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32])
def test_past_2_31_elements(xm, dt):  # noqa: F811
    counts, d, h = [700001, 0, 400100], 16, 1000
    E, off = 3, [0, 700001, 700001, 1100101]
    R, spare = off[-1] + 7, 7
    assert R * 2 * h > 2 ** 31
    g = _gen(4)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    x, dy, w1, w3, w2 = r(R, d), r(R, d), r(E, d, h), r(E, d, h), r(E, h, d)
    tok = torch.randperm(R, generator=g, device="cuda").to(I32)
    wt = torch.rand(R, generator=g, device="cuda")

    def run(i, e0, offsets):
        n, es = i.stop - i.start, slice(e0, e0 + len(offsets) - 1)
        o = torch.tensor(offsets, dtype=I32, device="cuda")
        t, w = tok[i].contiguous(), wt[i].contiguous()
        act = torch.full((n, h), 3.0, dtype=dt, device="cuda")
        hq = torch.full((n, 2 * h), 77, dtype=I8, device="cuda")
        hs = torch.full(xm.ckpt8_scale_shape(n, h), 99, dtype=U8, device="cuda")
        xm.xmoe_expert_ffn_up_ckpt8(x, w1[es], w3[es], o, act, hq, hs, token_ids=t)
        val = torch.full((n, 2 * h), 3.0, dtype=dt, device="cuda")
        xm.xmoe_ckpt8_dequantize(hq, hs, val)
        back = torch.full((n, h), 3.0, dtype=dt, device="cuda")
        dh, dw = torch.full((n, 2 * h), 3.0, dtype=dt, device="cuda"), torch.full((n,), 3.0, device="cuda")
        xm.xmoe_expert_ffn_bwd_dact_ckpt8(dy, w2[es], hq, hs, o, dh, back, token_ids=t, row_weights=w, dweights=dw)
        return act, hq, hs.permute(2, 0, 1, 3), val, back, dh, dw

    whole = run(slice(0, R), 0, off)
    for e in (0, 2):
        for r0 in (off[e], off[e + 1] - 3000):   # the first rows of a segment and its last ones
            i = slice(r0, r0 + 3000)
            for k, (a, b) in enumerate(zip(whole, run(i, e, [0, 3000]))):
                assert torch.equal(a[i], b), (e, r0, k)
    act, hq, hs, _, back, dh, dw = whole
    for t, v in ((act, 3), (hq, 77), (hs, 99), (back, 3), (dh, 3), (dw, 3)):
        assert bool((t[-spare:] == v).all())
