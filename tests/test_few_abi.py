"""Refusals of the whole layer for a few tokens: the C ABI's checks on the host, before
any device is touched, and the binding's checks of its tensors.  No GPU needed."""
import ctypes

import pytest
import torch

BF, F32, I32, U8, F8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
REFUSED = (INVALID, UNSUPPORTED, WORKSPACE)


@pytest.fixture(scope="module")
def xm():
    import padding_free_expert_amd as m
    return m


def _at(i):
    return ctypes.c_void_p((1 + i) << 24)  # never dereferenced


ODD = ctypes.c_void_p((1 << 24) + 8)


def _call(xm, **kw):
    a = dict(x=_at(0), wg=_at(1), w1=_at(2), w3=_at(3), w2=_at(4), s1=None, s3=None, s2=None, dt=1, T=3, d=64, E=8, k=2, h=32,
             hs=0, tau=1.0, lb=None, sb=None, ids=_at(5), w=_at(6), z=_at(7), y=_at(8), ws=_at(9), n=1 << 30, stream=None)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return xm._lib_few(*a.values())


def test_layer_few_rejects_on_host(xm):
    f = lambda **kw: _call(xm, **kw)
    assert f() not in REFUSED                                # what follows is the device check
    for n in ("x", "wg", "w1", "w3", "w2", "ids", "w", "z", "y"):
        assert f(**{n: None}) == INVALID, n
    for n in ("x", "wg", "w1", "w3", "w2", "y"):
        assert f(**{n: ODD}) == UNSUPPORTED, n
    assert f(ws=None) == WORKSPACE and f(ws=ODD) == WORKSPACE and f(n=100) == WORKSPACE
    assert f(T=-1) == INVALID and f(T=65) == UNSUPPORTED and f(T=1 << 40) == UNSUPPORTED
    assert f(d=0) == INVALID and f(h=0) == INVALID and f(hs=-8) == INVALID
    assert f(E=0) == INVALID and f(E=1032) == INVALID and f(k=0) == INVALID and f(k=9) == INVALID
    assert f(d=60) == UNSUPPORTED and f(h=36) == UNSUPPORTED and f(hs=4, s1=_at(10), s3=_at(11), s2=_at(12)) == UNSUPPORTED
    assert f(E=12) == UNSUPPORTED and f(E=12, dt=0) not in REFUSED
    assert f(d=1 << 17) == UNSUPPORTED and f(d=65536, h=65536) == UNSUPPORTED
    assert f(d=65536, h=16384) == UNSUPPORTED and f(d=65536, h=8192) not in REFUSED
    assert f(dt=2) == UNSUPPORTED
    # the shared experts: all three, when there is a width
    s = dict(s1=_at(10), s3=_at(11), s2=_at(12), hs=16)
    assert f(**s) not in REFUSED
    for n in ("s1", "s3", "s2"):
        assert f(**{**s, n: None}) == INVALID and f(**{**s, n: ODD}) == UNSUPPORTED, n
    # no tokens: outputs may be missing
    assert f(T=0, x=None, ids=None, w=None, z=None, y=None, ws=None, n=0) not in REFUSED


def test_layer_few_mx8_rejects_on_host(xm):
    def ffn(**kw):
        at = dict(w1=_at(2), w1_scale=_at(3), w3=_at(4), w3_scale=_at(5), w2=_at(6), w2_scale=_at(7))
        at.update(kw)
        return ctypes.byref(xm._CMx8Ffn(*at.values()))

    def f(**kw):
        a = dict(x=_at(0), xq=_at(20), xs=_at(21), wg=_at(1), routed=ffn(), shared=None, T=3, d=64, E=8, k=2, h=32, hs=0,
                 tau=1.0, lb=None, sb=None, ids=_at(8), w=_at(9), z=_at(10), y=_at(11), ws=_at(12), n=1 << 30, stream=None)
        assert set(kw) <= set(a), kw
        a.update(kw)
        return xm._lib_few8(*a.values())

    assert f() not in REFUSED
    for n in ("x", "xq", "xs", "wg", "routed", "ids", "w", "z", "y"):
        assert f(**{n: None}) == INVALID, n
    for n in ("w1", "w1_scale", "w3", "w3_scale", "w2", "w2_scale"):
        assert f(routed=ffn(**{n: None})) == INVALID and f(routed=ffn(**{n: ODD})) == UNSUPPORTED, n
        assert f(hs=32, shared=ffn(**{n: None})) == INVALID, n
    assert f(hs=32) == INVALID and f(hs=32, shared=ffn()) not in REFUSED
    assert f(d=40) == UNSUPPORTED and f(h=48) == UNSUPPORTED and f(hs=8, shared=ffn()) == UNSUPPORTED
    assert f(T=65) == UNSUPPORTED and f(E=12) == UNSUPPORTED and f(k=9) == INVALID
    assert f(ws=None) == WORKSPACE and f(n=64) == WORKSPACE and f(xq=ODD) == UNSUPPORTED and f(xs=ODD) == UNSUPPORTED


def test_workspace_sizes(xm):
    f = xm.xmoe_layer_few_workspace_size
    for T in (1, 7, 64):
        for dt in (BF, F32):
            assert f(T, 64, 8, 2, 32, 0, dt) >= T * 8 * 4
            assert f(T, 64, 8, 2, 32, 48, dt) > f(T, 64, 8, 2, 32, 0, dt)
    assert f(65, 64, 8, 2, 32, 0, BF) == 0 and f(1, 60, 8, 2, 32, 0, BF) == 0 and f(1, 64, 8, 9, 32, 0, BF) == 0
    g = xm.xmoe_layer_few_mx8_workspace_size
    assert g(4, 64, 8, 2, 32, 32) > 0 and g(4, 72, 8, 2, 32, 0) == 0 and g(-1, 64, 8, 2, 32, 0) == 0


def test_binding_checks_its_tensors(xm):
    T, d, E, k, h, hs = 3, 64, 8, 2, 32, 16
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt)
    good = dict(x=e(T, d), wg=e(d, E), w1=e(E, d, h), w3=e(E, d, h), w2=e(E, h, d), k=k, topk_ids=e(T, k, dt=I32),
                topk_w=e(T, k, dt=F32), logits=e(T, E, dt=F32), y=e(T, d), s1=e(d, hs), s3=e(d, hs), s2=e(hs, d))
    for n, bad in (("wg", e(d, E + 8)), ("w1", e(E, d, h, dt=F32)), ("w3", e(E, d, h + 8)), ("w2", e(E, d, h)),
                   ("topk_ids", e(T, k)), ("topk_w", e(T, k + 1, dt=F32)), ("logits", e(T, E)), ("y", e(T, d, dt=F32)),
                   ("s1", e(d, hs + 8)), ("s3", e(hs, d)), ("s2", e(hs, d, dt=F32)), ("logit_bias", e(E)),
                   ("select_bias", e(E + 1, dt=F32)), ("s3", None)):
        with pytest.raises((ValueError, TypeError)):
            xm.xmoe_layer_few(**{**good, n: bad})
    with pytest.raises(ValueError, match="device tensors"):
        xm.xmoe_layer_few(**good, workspace=e(1 << 20, dt=U8))       # host tensors
    pair = lambda n, N, K: (e(n, N, K, dt=F8), e(n, *xm.mx8_scale_shape(N, K), dt=U8))
    good8 = dict(x=e(T, d), xq=e(T, d, dt=F8), xscale=e(*xm.mx8_scale_shape(T, d), dt=U8), wg=e(d, E), w1=pair(E, h, d),
                 w3=pair(E, h, d), w2=pair(E, d, h), k=k, topk_ids=e(T, k, dt=I32), topk_w=e(T, k, dt=F32),
                 logits=e(T, E, dt=F32), y=e(T, d))
    for n, bad in (("xq", e(T, d)), ("xscale", e(T, d, dt=U8)), ("w1", pair(E, d, h)), ("w2", (good8["w2"][0], good8["w1"][1])),
                   ("w3", (e(E, h, d), good8["w3"][1])), ("x", e(T, d, dt=F32)), ("s1", pair(1, 32, d))):
        with pytest.raises((ValueError, TypeError)):
            xm.xmoe_layer_few_mx8(**{**good8, n: bad})
