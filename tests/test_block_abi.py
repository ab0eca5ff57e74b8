"""Refusals of the calls around the layer (norm, balance loss, 8-bit experts):
the C ABI's checks on the host, before any device is touched, and the
binding's checks of its tensors.  No GPU needed."""
import ctypes

import pytest
import torch

BF, F32, I32, U8, F8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
P = ctypes.c_void_p(1 << 20)       # never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
WS = 1 << 30


@pytest.fixture(scope="module")
def xm():
    import padding_free_expert_amd as m
    return m


def _at(n):
    return ctypes.c_void_p((1 << 20) + n)


def test_norm_rejects_on_host(xm):
    def f(x=P, res=None, gamma=P, dt=1, T=10, d=64, eps=1e-6, sum=None, y=_at(1 << 16), q=None, scale=None):
        return xm._lib_norm(x, res, gamma, dt, T, d, eps, sum, y, q, scale, None, None)
    assert f(x=None) == INVALID and f(gamma=None) == INVALID
    assert f(y=None) == INVALID                       # neither y nor q
    assert f(y=None, q=P) == INVALID                  # q without scale
    assert f(T=-1) == INVALID and f(d=0) == INVALID
    assert f(d=12) == UNSUPPORTED and f(d=16392) == UNSUPPORTED
    assert f(d=40, q=_at(1 << 18), scale=P) == UNSUPPORTED   # 8 bits need a multiple of 32
    assert f(T=1 << 25) == INVALID and f(T=BIG) == INVALID   # T * max(d, 512) >= 2^34
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID
    assert f(dt=2) == UNSUPPORTED
    assert f(x=ODD) == UNSUPPORTED and f(gamma=ODD) == UNSUPPORTED and f(y=ODD) == UNSUPPORTED
    assert f(y=_at(16)) == INVALID                    # overlaps x in part
    assert f(res=_at(1 << 17), sum=_at((1 << 17) + 32)) == INVALID
    assert f(sum=_at(1 << 16)) == INVALID             # sum and y
    assert f(q=P, scale=_at(1 << 18)) == INVALID      # q and x
    assert f(q=_at((1 << 16) + 64), scale=_at(1 << 18)) == INVALID   # q and y
    # in place is allowed: what follows is the device check
    assert f(y=P) not in (INVALID, UNSUPPORTED, WORKSPACE)
    assert f(res=_at(1 << 17), sum=_at(1 << 17)) not in (INVALID, UNSUPPORTED, WORKSPACE)
    assert f(x=None, y=None, T=0) not in (INVALID, UNSUPPORTED, WORKSPACE)


def test_norm_backward_rejects_on_host(xm):
    far = [_at(i << 16) for i in range(8)]

    def f(dy=far[0], dsum=None, s=far[1], gamma=far[2], rstd=far[3], dt=1, T=10, d=64, dx=far[4], dg=far[5], ws=far[6],
          n=WS):
        return xm._lib_norm_bwd(dy, dsum, s, gamma, rstd, dt, T, d, dx, dg, ws, n, None)
    for k in ("dy", "s", "gamma", "rstd", "dx", "dg"):
        assert f(**{k: None}) == INVALID, k
    assert f(d=20) == UNSUPPORTED and f(d=1 << 20) == UNSUPPORTED and f(T=-3) == INVALID and f(dt=9) == UNSUPPORTED
    assert f(dx=_at(64)) == INVALID                   # overlaps dy in part
    assert f(ws=None) == WORKSPACE and f(ws=ODD) == WORKSPACE and f(n=16) == WORKSPACE
    assert f(dg=ODD) == UNSUPPORTED
    assert xm.xmoe_add_rmsnorm_bwd_workspace_size(100, 20, BF) == 0
    assert xm.xmoe_add_rmsnorm_bwd_workspace_size(-1, 64, BF) == 0
    assert xm.xmoe_add_rmsnorm_bwd_workspace_size(0, 64, BF) >= 64 * 4


def test_balance_rejects_on_host(xm):
    def f(logits=P, ids=P, T=10, E=8, k=2, off=None, S=1, loss=P, counts=P, coef=P, ws=P, n=WS):
        return xm._lib_balance(logits, ids, T, E, k, off, S, None, 0.1, loss, counts, coef, ws, n, None)
    for k in ("logits", "ids", "loss", "counts", "coef"):
        assert f(**{k: None}) == INVALID, k
    assert f(T=-1) == INVALID and f(T=BIG) == INVALID and f(E=0) == INVALID and f(E=1025) == INVALID
    assert f(k=0) == INVALID and f(k=9) == INVALID
    assert f(S=0) == INVALID and f(S=2) == INVALID    # two sequences without offsets
    assert f(S=4097, off=P) == INVALID
    assert f(logits=ODD) == UNSUPPORTED
    assert f(ws=None) == WORKSPACE and f(ws=ODD) == WORKSPACE and f(n=64) == WORKSPACE
    assert xm.xmoe_balance_loss_workspace_size(10, 1025) == 0
    assert xm.xmoe_balance_loss_workspace_size(10, 8, 0) == 0
    assert xm.xmoe_balance_loss_workspace_size(0, 8, 1) > 0

    def b(logits=P, coef=P, T=10, E=8, off=None, S=1, dz=P):
        return xm._lib_balance_bwd(logits, coef, T, E, off, S, None, None, dz, None)
    for k in ("logits", "coef", "dz"):
        assert b(**{k: None}) == INVALID, k
    assert b(dz=ODD) == UNSUPPORTED and b(S=3) == INVALID and b(E=2000) == INVALID

    def g(x=P, wg=P, dw=P, ldw=2, coef=P, dt=1, T=10, d=64, E=8, k=2, dx=P, dwg=P, ws=P, n=WS, S=1):
        return xm._lib_rbwd_balance(x, wg, P, P, dw, ldw, coef, None, S, None, None, dt, T, d, E, k, 1.0, 1, dx, dwg,
                                    ws, n, None)
    for k in ("x", "wg", "dw", "coef", "dx", "dwg"):
        assert g(**{k: None}) == INVALID, k
    assert g(ldw=1) == INVALID and g(k=9, ldw=9) == INVALID and g(S=2) == INVALID and g(T=1 << 26, ldw=64) == INVALID
    assert g(d=12) == UNSUPPORTED and g(E=12) == UNSUPPORTED and g(x=ODD) == UNSUPPORTED
    assert g(n=16) == WORKSPACE and g(ws=None) == WORKSPACE


def test_mx8_rejects_on_host(xm):
    q = xm._lib_mx8_q
    assert q(P, 1, 10, 48, P, P, None) == UNSUPPORTED and q(P, 1, 10, 65568, P, P, None) == UNSUPPORTED
    assert q(None, 1, 10, 64, P, P, None) == INVALID and q(P, 1, -1, 64, P, P, None) == INVALID
    assert q(P, 1, 1 << 25, 64, P, P, None) == INVALID and q(P, 3, 10, 64, P, P, None) == UNSUPPORTED
    assert q(ODD, 1, 10, 64, P, P, None) == UNSUPPORTED
    assert q(_at(1 << 16), 0, 1 << 24, 544, P, P, None) == INVALID   # n * max(K, 512) >= 2^33
    assert q(P, 1, 10, 64, _at(640), P, None) == INVALID             # q and x
    dq = xm._lib_mx8_dq
    assert dq(P, None, 1, 10, 64, P, None) == INVALID and dq(P, P, 1, 10, 63, P, None) == UNSUPPORTED
    qw = xm._lib_mx8_qw
    assert qw(P, 1, 4, 64, 40, P, P, None) == UNSUPPORTED and qw(P, 1, 0, 64, 64, P, P, None) == INVALID
    assert qw(P, 1, 1024, 65536, 65536, P, P, None) == UNSUPPORTED and qw(None, 1, 4, 64, 64, P, P, None) == INVALID

    def up(x=P, xs=P, ids=None, T=10, w1=P, w1s=P, w3=P, w3s=P, off=P, E=4, rows=10, d=64, h=64, act=P, acts=P):
        return xm._lib_up8(x, xs, ids, T, w1, w1s, w3, w3s, off, E, rows, d, h, act, acts, None)
    for k in ("x", "xs", "w1", "w1s", "w3", "w3s", "off", "act", "acts"):
        assert up(**{k: None}) == INVALID, k
    assert up(T=9) == INVALID                          # not gathered: a row of x for each row
    assert up(ids=P, T=0) == INVALID and up(ids=P, T=1 << 25) == UNSUPPORTED
    assert up(d=48) == UNSUPPORTED and up(h=8) == UNSUPPORTED and up(E=0) == INVALID and up(rows=-1) == INVALID
    assert up(d=1 << 17) == UNSUPPORTED and up(act=ODD) == UNSUPPORTED
    assert up(rows=1 << 30, T=1 << 30) == INVALID      # rows * 512 >= 2^34

    def down(act=P, acts=P, w2=P, w2s=P, off=P, E=4, rows=10, d=64, h=64, ye=P):
        return xm._lib_down8(act, acts, w2, w2s, off, E, rows, d, h, ye, None)
    for k in ("act", "acts", "w2", "w2s", "off", "ye"):
        assert down(**{k: None}) == INVALID, k
    assert down(h=33) == UNSUPPORTED and down(ye=ODD) == UNSUPPORTED and down(E=5000) == INVALID
    # nothing to do passes the checks: what follows is the device check
    assert up(x=None, xs=None, act=None, acts=None, rows=0, T=0) not in (INVALID, UNSUPPORTED, WORKSPACE)
    assert down(act=None, acts=None, ye=None, rows=0) not in (INVALID, UNSUPPORTED, WORKSPACE)
    assert xm._lib_last_error() != b""


def test_binding_checks_its_tensors(xm):
    T, d, E, k, h = 6, 64, 8, 2, 96
    x, gamma = torch.zeros(T, d, dtype=BF), torch.zeros(d, dtype=BF)
    z = torch.zeros
    for kw, err in ((dict(res=z(T, d)), TypeError), (dict(res=z(T + 1, d, dtype=BF)), ValueError),
                    (dict(y=z(T, d + 8, dtype=BF)), ValueError), (dict(sum=z(T, d)), TypeError),
                    (dict(q=z(T, d, dtype=U8)), TypeError), (dict(scale=z(1, T + 1, 4, dtype=U8)), ValueError),
                    (dict(rstd=z(T, dtype=BF)), TypeError)):
        res = kw.pop("res", None)
        with pytest.raises(err):
            xm.xmoe_add_rmsnorm(x, res, gamma, 1e-6, **kw)
    with pytest.raises(ValueError, match="gamma"):
        xm.xmoe_add_rmsnorm(x, None, z(d + 8, dtype=BF), 1e-6, y=x)
    with pytest.raises(ValueError, match="dgamma"):
        xm.xmoe_add_rmsnorm_bwd(x, None, x, gamma, z(T), x, z(T))
    with pytest.raises(ValueError, match="device tensors"):
        xm.xmoe_add_rmsnorm(x, None, gamma, 1e-6, y=z(T, d, dtype=BF))
    logits, ids = z(T, E), z(T, k, dtype=I32)
    ok = dict(loss=z(1), counts=z(1, E, dtype=I32), coef=z(1, E))
    for kw, err in ((dict(counts=z(1, E)), TypeError), (dict(coef=z(2, E)), ValueError), (dict(loss=z(())), ValueError),
                    (dict(seq_offsets=z(3, dtype=I32)), ValueError), (dict(seq_offsets=z(1, dtype=I32)), ValueError),
                    (dict(token_mask=z(T)), TypeError), (dict(token_mask=z(T + 1, dtype=torch.bool)), ValueError)):
        with pytest.raises(err):
            xm.xmoe_balance_loss(logits, ids, 0.1, **{**ok, **kw})
    with pytest.raises(TypeError, match="logits"):
        xm.xmoe_balance_loss(logits.to(BF), ids, 0.1, **ok)
    with pytest.raises(TypeError, match="topk_ids"):
        xm.xmoe_balance_loss(logits, ids.long(), 0.1, **ok)
    with pytest.raises(ValueError, match="dlogits"):
        xm.xmoe_balance_loss_bwd(logits, ok["coef"], z(T, E + 1))
    with pytest.raises(ValueError, match="device tensors"):
        xm.xmoe_balance_loss(logits, ids, 0.1, **ok)
    q, s = z(T, d, dtype=F8), z(1, T, 4, dtype=U8)
    with pytest.raises(TypeError, match="q"):
        xm.xmoe_mx8_quantize(x, z(T, d, dtype=torch.float8_e5m2), s)
    with pytest.raises(ValueError, match="scale"):
        xm.xmoe_mx8_quantize(x, q, z(T, 1, 4, dtype=U8))
    with pytest.raises(TypeError, match="unsupported dtype"):
        xm._dt(x.to(torch.float16))
    w1, w1s = z(E, h, d, dtype=F8), z(E, 1, h, 4, dtype=U8)
    off = z(E + 1, dtype=I32)
    act, acts = z(T * k, h, dtype=F8), z(1, T * k, 4, dtype=U8)
    tid = z(T * k, dtype=I32)
    good = dict(w1=w1, w1_scale=w1s, w3=w1, w3_scale=w1s, expert_offsets=off, act=act, act_scale=acts, token_ids=tid)
    for kw, err in ((dict(w3=z(E, h, d + 32, dtype=F8)), ValueError), (dict(w1_scale=z(E, 1, h, 4)), TypeError),
                    (dict(expert_offsets=z(E, dtype=I32)), ValueError), (dict(token_ids=z(T, dtype=I32)), ValueError),
                    (dict(act=z(T * k, h, dtype=BF)), TypeError), (dict(act_scale=z(1, T, 4, dtype=U8)), ValueError)):
        with pytest.raises(err):
            xm.xmoe_expert_ffn_up_mx8(q, s, **{**good, **kw})
    with pytest.raises(TypeError, match="ye"):
        xm.xmoe_expert_ffn_down_mx8(act, acts, z(E, d, h, dtype=F8), z(E, 1, d, 4, dtype=U8), off, z(T * k, d))


def test_tensors_of_two_devices_are_refused(xm):
    class On:
        def __init__(self, dev):
            self.dev = dev

        def get_device(self):
            return self.dev
    with pytest.raises(ValueError, match="different devices"):
        xm._on_device(On(0), None, On(1))
    with pytest.raises(ValueError, match="different devices"):
        xm._on_device(On(0), On(-1))
    with xm._on_device(On(-1), None, On(-1)):   # host tensors: refused when their pointers are taken
        pass
