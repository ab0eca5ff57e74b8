"""Tensors of more than 2^31 elements: the rows behind that border against the
64-bit definitions, or against the same call on those rows alone (whose bits
they must have)."""
import pytest
import torch

import _block_ref as br
from _helpers import need_gpu
from test_gpu_norm import EPS, PRE

pytestmark = pytest.mark.gpu
BF, F8, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
T, D = (1 << 31) // 16384 + 3, 16384
TAIL = slice(T - 4, T)


@pytest.fixture(scope="module")
def xm():
    need_gpu()
    import padding_free_expert_amd as m
    assert m.xmoe_query_device(0)
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    yield m
    torch.cuda.empty_cache()


def _rows(n, d, seed, dt=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty((n, d), dtype=dt, device="cuda").normal_(generator=g)


def _tail_scale(s, sl):
    return s[:, sl].contiguous()


def test_norm(xm):
    print("[large] norm", flush=True)
    x, gamma = _rows(T, D, 1), _rows(1, D, 2)[0]
    y, q = torch.empty_like(x), torch.empty((T, D), dtype=F8, device="cuda")
    sc, rstd = torch.empty(xm.mx8_scale_shape(T, D), dtype=U8, device="cuda"), torch.empty(T, device="cuda")
    xm.xmoe_add_rmsnorm(x, None, gamma, EPS, y=y, q=q, scale=sc, rstd=rstd)
    for sl in (slice(0, 2), TAIL):
        want = br.norm_ref(x[sl], None, gamma, EPS)
        br.close(rstd[sl], want[1], PRE, name="rstd")
        br.close(y[sl], want[2], br.half_step(BF) + PRE, name="y")
        alone = torch.empty_like(q[sl]), torch.empty(xm.mx8_scale_shape(q[sl].shape[0], D), dtype=U8, device="cuda")
        # (few rows are spread over more waves, which sum in another order)
        xm.xmoe_mx8_quantize(want[2].float().contiguous(), *alone)
        br.close(br.mx8_values(q[sl].contiguous(), _tail_scale(sc, sl)), want[2], 2.0 ** -4 + PRE,
                 torch.exp2(br.scale_bytes(alone[1], D)[0].double() - 126).repeat_interleave(32, 1) * 2.0 ** -10, "q")
    del q, sc
    dx, dg = torch.empty_like(x), torch.empty(D, device="cuda")
    xm.xmoe_add_rmsnorm_bwd(y, None, x, gamma, rstd, dx, dg)
    n = x[TAIL].double() * rstd[TAIL].double()[:, None]
    u = y[TAIL].double() * gamma.double()
    mag = rstd[TAIL].double()[:, None] * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True))
    br.close(dx[TAIL], br.norm_bwd_ref(y[TAIL], None, x[TAIL], gamma, rstd[TAIL])[0], br.half_step(BF), 2.0 ** -18 * mag,
             "dx")


def test_rows_in_8_bits(xm):
    print("[large] rows", flush=True)
    x = _rows(T, D, 3)
    q, sc = torch.empty((T, D), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(T, D), dtype=U8, device="cuda")
    xm.xmoe_mx8_quantize(x, q, sc)
    back = torch.empty_like(x)
    xm.xmoe_mx8_dequantize(q, sc, back)
    a, s = torch.empty((4, D), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(4, D), dtype=U8, device="cuda")
    xm.xmoe_mx8_quantize(x[TAIL], a, s)
    assert torch.equal(a.view(U8), q[TAIL].view(U8)) and torch.equal(s, _tail_scale(sc, TAIL))
    assert torch.equal(back[TAIL].double(), br.mx8_values(a, s))


def test_weights_in_8_bits(xm):
    print("[large] weights", flush=True)
    E, K, N = 1024, 2048, 1056
    w = _rows(E * K, N, 4).view(E, K, N)
    q, sc = torch.empty((E, N, K), dtype=F8, device="cuda"), torch.empty((E,) + xm.mx8_scale_shape(N, K), dtype=U8, device="cuda")
    xm.xmoe_mx8_quantize_weights(w, q, sc)
    a, s = torch.empty_like(q[:1]), torch.empty_like(sc[:1])
    for e in (0, E - 1):
        xm.xmoe_mx8_quantize_weights(w[e:e + 1], a, s)
        assert torch.equal(a.view(U8), q[e:e + 1].view(U8)) and torch.equal(s, sc[e:e + 1])


@pytest.mark.parametrize("d,h,counts", [(4096, 32, [300, 525000]), (32, 4096, [300, 525000])])
def test_experts(xm, d, h, counts):
    """ye, or act, past 2^31 elements: two experts' rows gathered from a hundred."""
    print(f"[large] experts d={d} h={h}", flush=True)
    rows, E = sum(counts), 2
    off = torch.tensor([0, counts[0], rows], dtype=torch.int32, device="cuda")
    w = []
    for i, (N, K) in enumerate(((h, d), (h, d), (d, h))):
        q, s = torch.empty((E, N, K), dtype=F8, device="cuda"), torch.empty((E,) + xm.mx8_scale_shape(N, K), dtype=U8, device="cuda")
        xm.xmoe_mx8_quantize_weights(_rows(E * K, N, 5 + i).mul_(K ** -0.5).view(E, K, N), q, s)
        w += [q, s]
    x = _rows(100, d, 9)
    xq, xs = torch.empty((100, d), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(100, d), dtype=U8, device="cuda")
    xm.xmoe_mx8_quantize(x, xq, xs)
    ids = torch.arange(rows, dtype=torch.int32, device="cuda") % 97
    act, acts = torch.empty((rows, h), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(rows, h), dtype=U8, device="cuda")
    ye = torch.empty((rows, d), dtype=BF, device="cuda")
    xm.xmoe_expert_ffn_up_mx8(xq, xs, *w[:4], off, act, acts, token_ids=ids)
    xm.xmoe_expert_ffn_down_mx8(act, acts, *w[4:], off, ye)
    # rows of the second expert repeat with its tokens; a full tile's and the last tile's have the same sums
    for r in (rows - 1, rows - 97, counts[0] + 97 * 5000):
        same = counts[0] + (r - counts[0]) % 97
        assert int(ids[r]) == int(ids[same])
        assert torch.equal(act[r].view(U8), act[same].view(U8)) and torch.equal(acts[:, r], acts[:, same])
        assert torch.equal(ye[r], ye[same])
    sl = slice(rows - 3, rows)
    av = br.mx8_values(act[sl].contiguous(), _tail_scale(acts, sl))
    a2 = br.mx8_values(w[4][1], w[5][1])
    br.close(ye[sl], av @ a2.t(), br.half_step(BF), 1.01 * (2.0 ** -10 + h * 2.0 ** -24) * (av.abs() @ a2.abs().t()), "ye")
    # rows without ids: the same act from rows laid out one by one
    few = torch.empty((3, h), dtype=F8, device="cuda"), torch.empty(xm.mx8_scale_shape(3, h), dtype=U8, device="cuda")
    last = ids[sl].long()
    one = torch.tensor([0, 0, 3], dtype=torch.int32, device="cuda")
    xm.xmoe_expert_ffn_up_mx8(xq.view(U8)[last].view(F8), xs[:, last].contiguous(), *w[:4], one, *few)
    br.close(br.mx8_values(*few), av, 2.0 ** -3, torch.exp2(br.scale_bytes(few[1], h)[0].double() - 126)
             .repeat_interleave(32, 1) * 2.0 ** -9, "act")  # one step of e4m3: sums in another order


def test_balance(xm):
    print("[large] balance", flush=True)
    n, E, k = (1 << 21) + 5, 1024, 2
    logits = _rows(n, E, 11, torch.float32)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    ids = torch.randint(0, E, (n, k), generator=g, device="cuda", dtype=torch.int32)
    off = torch.tensor([0, 1 << 20, n - 1], dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(1, device="cuda"), torch.empty((2, E), dtype=torch.int32, device="cuda")
    coef, dz = torch.empty((2, E), device="cuda"), torch.empty_like(logits)
    xm.xmoe_balance_loss(logits, ids, 1.0, loss, counts, coef, off)
    xm.xmoe_balance_loss_bwd(logits, coef, dz, off)
    total = 0.0
    for s, (lo, hi) in enumerate(((0, 1 << 20), (1 << 20, n - 1))):
        c = torch.bincount(ids[lo:hi].flatten().long(), minlength=E)
        assert torch.equal(counts[s].long(), c)
        f = E * c.double() / (k * (hi - lo))
        br.close(coef[s], f / ((hi - lo) * 2), 2.0 ** -23, name="coef")
        p = torch.zeros(E, dtype=torch.float64, device="cuda")
        for i in range(lo, hi, 1 << 16):
            p += torch.softmax(logits[i:min(i + (1 << 16), hi)].double(), 1).sum(0)
        total += float((f * p).sum()) / ((hi - lo) * 2)
    br.close(loss, torch.tensor([total], device="cuda"), 2.0 ** -17, name="loss")
    p = torch.softmax(logits[n - 3:n - 1].double(), 1)
    cf = coef[1].double()
    dot = (p * cf).sum(1, keepdim=True)
    br.close(dz[n - 3:n - 1], p * (cf - dot), 0.0, 2.0 ** -17 * p * (cf.abs() + dot.abs()), "dlogits")
    assert bool((dz[n - 1] == 0).all())
