"""The norm's backward with dx in the buffer of sum, as of dy and of dsum: the bits
of a call with a buffer of its own, at every width's split over waves."""
import pytest
import torch

from test_gpu_norm import xm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (9, 512), (300, 1000), (257, 2048), (2100, 2056), (65, 4096), (40, 8192), (33, 16384)])
def test_dx_in_place_of_sum(xm, T, d, dtype):  # noqa: F811
    print(f"[norm bwd in place] T={T} d={d} {dtype}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    s, dy, dsum, gamma = r(T, d), r(T, d), r(T, d), r(d)
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-6)
    for ds in (None, dsum):
        dx, dg = torch.empty_like(s), torch.empty(d, device="cuda")
        xm.xmoe_add_rmsnorm_bwd(dy, ds, s, gamma, rstd, dx, dg)
        for at in ("sum", "dy", "dsum", "all"):
            a = dict(dy=dy.clone(), dsum=None if ds is None else ds.clone(), sum=s.clone())
            if at == "dsum" and ds is None:
                continue
            if at == "all":     # one buffer that is dy and dsum as well
                if ds is None:
                    continue
                a["dsum"] = a["dy"]
                xm.xmoe_add_rmsnorm_bwd(dy, dy, s, gamma, rstd, dx, dg)
                at = "dy"
            got, gg = a[at], torch.empty(d, device="cuda")
            xm.xmoe_add_rmsnorm_bwd(a["dy"], a["dsum"], a["sum"], gamma, rstd, got, gg)
            assert torch.equal(got, dx) and torch.equal(gg, dg), at
