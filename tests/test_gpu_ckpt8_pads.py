"""Scale bytes of 8-bit pre-activations: those past h are 127 whatever a row of x holds,
and a row that is not finite changes no other row's."""
import pytest
import torch

from test_gpu_ckpt8 import BF, CASES, F32, _case, _up, ref, xm  # noqa: F401  (xm is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name", ["empty experts", "ragged", "narrow", "two column tiles", "wide", "large tiles, few columns"])
def test_bytes_past_h_beside_rows_that_are_not_finite(xm, name, dt):  # noqa: F811
    c = _case(name, dt)
    n, h = c["off"][-1], c["h"]
    clean = _up(xm, c, dt)
    rows = torch.arange(c["R"], device="cuda") if c["tok"] is None else c["tok"].long()
    T = c["x"].shape[0]
    bad = [0, T // 2, T - 1]
    for t, v in zip(bad, (float("inf"), float("nan"), -float("inf"))):
        c["x"][t, 3] = v
    act, hq, hs = _up(xm, c, dt)
    hit = torch.isin(rows[:n], torch.tensor(bad, device="cuda"))
    assert bool(hit.any()) and not bool(hit.all())
    for b in range(2):
        byte, pad = ref.half(hs[:, :, :n], h, b)
        assert pad.numel() > 0 and bool((byte[hit] == 255).all())
        assert bool((pad == 127).all()), f"bytes past h: {torch.unique(pad).tolist()}"
    assert torch.equal(hs[:, :, :n][:, :, ~hit], clean[2][:, :, :n][:, :, ~hit])
    assert torch.equal(hq[:n][~hit], clean[1][:n][~hit]) and torch.equal(act[:n][~hit], clean[0][:n][~hit])
    assert bool((hs[:, :, n:] == 99).all())
    val = torch.empty((c["R"], 2 * h), device="cuda")
    xm.xmoe_ckpt8_dequantize(hq, hs, val)
    assert bool(torch.isnan(val[:n][hit]).all())
