"""Residual addition + RMS norm (forward, 8-bit output, backward) against the
64-bit definition.

Bounds.  The sum of squares has d positive terms: at most 32 in a lane in
sequence, then log2(64) + 16 steps, so its relative error is below 64 * 2^-24;
the square root halves it, and five more roundings follow: y carries at most
2^-18 relative before its own rounding of half a step of its type.  e4m3 adds
half a step, 2^-4 of the element, or half of its smallest step 2^-9 times the
block's scale."""
import pytest
import torch

import _block_ref as br
from _helpers import need_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6
PRE = 2.0 ** -18   # relative error of y before its rounding


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    return m


def _inputs(T, d, dt, res, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (r(T, d) * torch.exp(r(T, 1))).to(dt)
    return x, (2 * r(T, d)).to(dt) if res else None, (1 + 0.3 * r(d)).to(dt), r


def _check_q(q, scale, y, pre, name):
    """8-bit rows against float64 y whose computed value is within pre of it."""
    K = y.shape[1]
    got, pad = br.scale_bytes(scale, K)
    assert bool((pad == 127).all()), "padding bytes of the scales"
    lo, hi = br.mx8_bytes(y * (1 - pre)), br.mx8_bytes(y * (1 + pre))
    assert bool(((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all()), "scale bytes"
    s = torch.exp2(got.to(torch.float64) - 127).repeat_interleave(32, 1)
    br.close(br.mx8_values(q, scale), y, 2.0 ** -4 + pre, s * 2.0 ** -10, name)


SHAPES = [(1, 8), (1, 2048), (2, 64), (3, 32), (5, 1000), (7, 512), (9, 520), (33, 96), (1, 16384), (3, 16384),
          (130, 2048), (257, 1024), (1000, 160), (1500, 4096), (2050, 7168), (1027, 8), (4100, 2056), (66, 12288)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(xm, T, d, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for res in (False, True):
        print(f"[norm] T={T} d={d} {dtype} res={res}", flush=True)
        x, r, gamma, _ = _inputs(T, d, dt, res, seed=T + d)
        s, rstd, y = br.norm_ref(x, r, gamma, EPS)
        G = br.Guarded()
        gs, gy, gr = G.empty((T, d), dt), G.empty((T, d), dt), G.empty((T,), torch.float32)
        q8 = d % 32 == 0
        gq = G.empty((T, d), torch.float8_e4m3fn) if q8 else None
        gsc = G.empty(xm.mx8_scale_shape(T, d), torch.uint8) if q8 else None
        xm.xmoe_add_rmsnorm(x, r, gamma, EPS, gs, gy, gq, gsc, gr)
        G.check()
        assert torch.equal(gs, s)
        br.close(gr, rstd, PRE, name="rstd")
        br.close(gy, y, br.half_step(dt) + PRE, name="y")
        if q8:
            _check_q(gq, gsc, y, PRE, "q")
            # the 8-bit output alone gives the same bytes
            q2, s2 = torch.empty_like(gq), torch.empty_like(gsc)
            xm.xmoe_add_rmsnorm(x, r, gamma, EPS, q=q2, scale=s2)
            assert torch.equal(q2.view(torch.uint8), gq.view(torch.uint8)) and torch.equal(s2, gsc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(5, 16384), (700, 1024)])
def test_forward_in_place(xm, T, d, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, r, gamma, _ = _inputs(T, d, dt, True)
    s, y = torch.empty_like(x), torch.empty_like(x)
    xm.xmoe_add_rmsnorm(x, r, gamma, EPS, s, y)
    a, b = x.clone(), r.clone()
    xm.xmoe_add_rmsnorm(a, b, gamma, EPS, sum=b, y=a)
    assert torch.equal(a, y) and torch.equal(b, s)


def test_rows_of_zeros_and_non_finite_values(xm):
    T, d = 6, 256
    x = torch.ones(T, d, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3] = 1e-30
    x[4] = 3e38  # its square leaves fp32's range: the definition's value is 0
    y, q = torch.empty_like(x), torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(xm.mx8_scale_shape(T, d), dtype=torch.uint8, device="cuda")
    xm.xmoe_add_rmsnorm(x, None, gamma, EPS, y=y, q=q, scale=sc)
    b, _ = br.scale_bytes(sc, d)
    assert bool((y[0] == 0).all()) and bool((b[0] == 127).all())
    assert bool(torch.isnan(y[1]).all()) and bool((b[1] == 255).all())
    assert bool(torch.isnan(y[2, 200])) and int(b[2, 200 // 32]) == 255
    assert bool((y[2, :192] == 0).all())
    br.close(y[3], torch.full((d,), 1e-30 / EPS ** 0.5, device="cuda", dtype=torch.float64), 2.0 ** -7, name="tiny")
    assert bool((y[4] == 0).all())
    br.close(y[5], torch.ones(d, device="cuda") / (1 + EPS) ** 0.5, 2.0 ** -8, name="ones")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_backward(xm, T, d, dtype):
    """dx: u - n mean(u n) loses to cancellation, so its bound goes by the
    magnitudes of its terms; dgamma: T terms in blocks, by the sum of theirs."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for res in (False, True):
        print(f"[norm bwd] T={T} d={d} {dtype} dsum={res}", flush=True)
        s, _, gamma, r = _inputs(T, d, dt, False, seed=T + d)
        rstd = (1.0 / torch.sqrt((s.double() ** 2).mean(1) + EPS)).float()
        dy, dsum = r(T, d).to(dt), (r(T, d).to(dt) if res else None)
        dx, dg = br.norm_bwd_ref(dy, dsum, s, gamma, rstd)
        G = br.Guarded()
        gx, gg = G.empty((T, d), dt), G.empty((d,), torch.float32)
        ws = G.empty((xm.xmoe_add_rmsnorm_bwd_workspace_size(T, d, dt),), torch.uint8)
        xm.xmoe_add_rmsnorm_bwd(dy, dsum, s, gamma, rstd, gx, gg, workspace=ws)
        G.check()
        n = s.double() * rstd.double()[:, None]
        u = dy.double() * gamma.double()
        mag = rstd.double()[:, None] * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True))
        if res:
            mag = mag + dsum.double().abs()
        br.close(gx, dx, br.half_step(dt), 2.0 ** -18 * mag, "dx")
        br.close(gg, dg, 0.0, 2.0 ** -17 * (dy.double() * n).abs().sum(0), "dgamma")
        first = (gx.clone(), gg.clone())
        # in place on dy (or dsum): the same bits
        a = dy.clone()
        xm.xmoe_add_rmsnorm_bwd(a, dsum, s, gamma, rstd, a, gg)
        assert torch.equal(a, first[0]) and torch.equal(gg, first[1])
        if res:
            a = dsum.clone()
            xm.xmoe_add_rmsnorm_bwd(dy, a, s, gamma, rstd, a, gg)
            assert torch.equal(a, first[0])


def test_backward_against_differences(xm):
    """The gradient against central differences of the forward in fp32: with
    step h = 2^-7 the difference quotient carries h^2 of the third derivative
    (order 1 here: 2^-14) and 2^-22 / h of rounding."""
    T, d = 3, 64
    x, _, gamma, r = _inputs(T, d, torch.float32, False, seed=4)
    x = x / x.square().mean(1, keepdim=True).sqrt()
    dy = r(T, d)
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    xm.xmoe_add_rmsnorm(x, None, gamma, EPS, y=y, rstd=rstd)
    dx, dg = torch.empty_like(x), torch.empty(d, device="cuda")
    xm.xmoe_add_rmsnorm_bwd(dy, None, x, gamma, rstd, dx, dg)

    def f(x, gamma):
        xm.xmoe_add_rmsnorm(x, None, gamma, EPS, y=y)
        return (y.double() * dy.double()).sum(1)

    h = 2.0 ** -7
    for c in (0, 17, 63):
        e = torch.zeros(d, device="cuda")
        e[c] = h
        num = (f(x + e, gamma) - f(x - e, gamma)) / (2 * h)
        br.close(dx[:, c], num, 2.0 ** -9, 2.0 ** -9, f"dx[{c}]")
        num = (f(x, gamma + e) - f(x, gamma - e)).sum() / (2 * h)
        br.close(dg[c], num, 2.0 ** -12, 2.0 ** -10, f"dgamma[{c}]")


def test_no_rows(xm):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    xm.xmoe_add_rmsnorm(x, None, gamma, EPS, y=torch.empty_like(x))
    dg = torch.full((64,), 7.0, device="cuda")
    xm.xmoe_add_rmsnorm_bwd(x, None, x, gamma, torch.empty(0, device="cuda"), torch.empty_like(x), dg)
    assert bool((dg == 0).all())
