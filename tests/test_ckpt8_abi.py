"""Refusals of the calls for pre-activations kept in 8 bits: the C ABI's checks on the
host, before any device is touched, and the binding's checks.  No GPU needed."""
import ctypes

import pytest
import torch

BF, F32, I32, U8, I8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
REFUSED = (INVALID, UNSUPPORTED, WORKSPACE)


@pytest.fixture(scope="module")
def xm():
    import padding_free_expert_amd as m
    return m


def _at(i):
    return ctypes.c_void_p((1 + i) << 24)  # never dereferenced


ODD = ctypes.c_void_p((1 << 24) + 8)


def _caller(fn, defaults):
    def f(**kw):
        assert set(kw) <= set(defaults), kw
        return fn(*{**defaults, **kw}.values())
    return f


def test_up_rejects_on_host(xm):
    f = _caller(xm._lib_up_ck8, dict(x=_at(0), tok=None, T=10, w1=_at(1), w3=_at(2), dt=1, off=_at(3), E=4, rows=10, d=64,
                                     h=40, act=_at(4), hq=_at(5), hs=_at(6), stream=None))
    assert f() not in REFUSED and f(tok=_at(7), T=3) not in REFUSED and f(dt=0) not in REFUSED
    for n in ("x", "w1", "w3", "off", "act", "hq", "hs"):
        assert f(**{n: None}) == INVALID, n
    for n in ("x", "w1", "w3", "act", "hq", "hs"):
        assert f(**{n: ODD}) == UNSUPPORTED, n
    assert f(T=9) == INVALID and f(T=-1, tok=_at(7)) == INVALID and f(T=0, tok=_at(7)) == INVALID
    assert f(E=0) == INVALID and f(E=1025) == INVALID and f(rows=-1) == INVALID and f(rows=1 << 31, T=1 << 31) == INVALID
    assert f(d=0) == INVALID and f(d=60) == UNSUPPORTED and f(h=44) == UNSUPPORTED and f(h=(1 << 20) + 8) == UNSUPPORTED
    assert f(dt=3) == UNSUPPORTED
    assert f(tok=_at(7), T=1 << 25) == UNSUPPORTED      # 2^31 bytes to gather from
    assert f(rows=0, T=0, x=None, act=None, hq=None, hs=None) not in REFUSED


def test_dequantize_rejects_on_host(xm):
    f = _caller(xm._lib_ck8_dq, dict(hq=_at(0), hs=_at(1), dt=1, rows=10, h=40, out=_at(2), stream=None))
    assert f() not in REFUSED and f(rows=0, hq=None, hs=None, out=None) not in REFUSED
    for n in ("hq", "hs", "out"):
        assert f(**{n: None}) == INVALID and f(**{n: ODD}) == UNSUPPORTED, n
    assert f(h=36) == UNSUPPORTED and f(h=0) == INVALID and f(rows=-4) == INVALID and f(dt=5) == UNSUPPORTED
    assert f(rows=1 << 24, h=1024) == INVALID and f(rows=(1 << 24) - 2, h=1024) not in REFUSED


def test_backward_rejects_on_host(xm):
    n = 1 << 20
    f = _caller(xm._lib_dact_ck8, dict(dy=_at(0), tok=None, rw=None, T=10, w2=_at(1), hq=_at(2), hs=_at(3), dt=1, off=_at(4),
                                       E=4, rows=10, d=64, h=40, dh=_at(5), act=_at(6), s2r=None, dw=None, ws=None, n=0,
                                       stream=None))
    assert f() not in REFUSED and f(tok=_at(7), rw=_at(8), T=2) not in REFUSED
    for k in ("dy", "w2", "hq", "hs", "off", "dh", "act"):
        assert f(**{k: None}) == INVALID, k
    for k in ("dy", "w2", "hq", "hs", "dh", "act"):
        assert f(**{k: ODD}) == UNSUPPORTED, k
    assert f(s2r=_at(9)) == INVALID                       # orders nothing
    assert f(dw=_at(9)) == WORKSPACE and f(dw=_at(9), ws=ODD, n=n) == WORKSPACE and f(dw=_at(9), ws=_at(10), n=39) == WORKSPACE
    assert f(dw=_at(9), ws=_at(10), n=40) not in REFUSED and f(dw=_at(9), s2r=_at(11), ws=_at(10), n=n) not in REFUSED
    assert f(T=11) == INVALID and f(h=20) == UNSUPPORTED and f(E=0) == INVALID and f(dt=2) == UNSUPPORTED


def test_workspace_size(xm):
    f = xm.xmoe_expert_ffn_bwd_dact_ckpt8_workspace_size
    assert f(10, 40) == 40 and f(10, 72) == 80 and f(0, 40) == 0 and f(10, 36) == 0 and f(-1, 40) == 0


def test_binding_checks_its_tensors(xm):
    E, T, R, d, h = 4, 5, 10, 64, 40
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt)
    hq, hs = e(R, 2 * h, dt=I8), e(*xm.ckpt8_scale_shape(R, h), dt=U8)
    off, tok = e(E + 1, dt=I32), e(R, dt=I32)
    up = dict(x=e(T, d), w1=e(E, d, h), w3=e(E, d, h), expert_offsets=off, act=e(R, h), hq=hq, hscale=hs, token_ids=tok)
    for n, bad in (("w1", e(E, d, h, dt=F32)), ("w3", e(E, d, h + 8)), ("expert_offsets", e(E, dt=I32)), ("act", e(T, h)),
                   ("hq", e(R, 2 * h, dt=U8)), ("hq", e(R, h, dt=I8)), ("hscale", e(2, 1, R, 3, dt=U8)),
                   ("token_ids", None), ("token_ids", e(R, dt=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            xm.xmoe_expert_ffn_up_ckpt8(**{**up, n: bad})
    with pytest.raises(ValueError, match="device tensors"):
        xm.xmoe_expert_ffn_up_ckpt8(**up)
    for out in (e(R, 2 * h + 1), e(R + 1, 2 * h), e(R, 2 * h, dt=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            xm.xmoe_ckpt8_dequantize(hq, hs, out)
    back = dict(dy=e(T, d), w2=e(E, h, d), hq=hq, hscale=hs, expert_offsets=off, dh13=e(R, 2 * h), act=e(R, h),
                token_ids=tok, row_weights=e(R, dt=F32), slot_to_row=tok, dweights=e(T, 2, dt=F32))
    for n, bad in (("w2", e(E, d, h)), ("dh13", e(R, h)), ("act", e(R, h, dt=F32)), ("row_weights", e(R)),
                   ("slot_to_row", e(T, dt=I32)), ("dweights", e(R)), ("dweights", e(T, dt=F32)), ("hscale", e(R, dt=U8)),
                   ("token_ids", None)):
        with pytest.raises((ValueError, TypeError)):
            xm.xmoe_expert_ffn_bwd_dact_ckpt8(**{**back, n: bad})
