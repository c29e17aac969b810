"""Tensors of more than 2^31 values and weights of more than 2^32 bytes: rows
at their ends against the float64 oracle, within the operators' own tolerances
(u = 2^-24; see their tests)."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import moe as O
from oracle import operators as P
from tests.gpu_util import MX_ACC_REL, dev_bits, dev_bytes, dev_i32, empty_bits, empty_bytes, host_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T_, H_ = 300001, 7168                 # T_ H_ = 2^31 + 2.9e6
ROWS = [0, 1, 299592, 299593, 299594, 300000]     # (row 299593 holds value 2^31)


@pytest.fixture(scope="module")
def G():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_gemm_glu_amd as G
    G.moe_init(0)
    yield G
    torch.cuda.empty_cache()


def _normal(*shape):
    import torch
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g).view(torch.int16)


def _rows(t, rows):
    import torch
    return host_bits(t[torch.tensor(rows, device=t.device)])


f64 = F.bf16_bits_to_f64


def test_combine_and_gradients(G):
    import torch
    k, H, M = 4, H_, T_
    rng = np.random.default_rng(1)
    y = _normal(M, H)
    # few tokens, rows at the end of y
    T = 5
    dst = rng.choice(np.arange(M - 40, M), T * k, replace=False).astype(np.int32).reshape(T, k)
    dst[0, 0] = 0
    w = rng.standard_normal((T, k)).astype(np.float32)
    out = empty_bits((T, H))
    wd, dd = torch.from_numpy(w).cuda(), dev_i32(dst)
    G.moe_combine(y, M, H, dd, T, k, out, weights=wd)
    named = np.sort(dst.reshape(-1))
    small = np.searchsorted(named, dst).astype(np.int32)
    yh = _rows(y, named.tolist())
    want = P.combine(yh, small, w)
    mag = sum(np.abs(w[:, j, None] * f64(yh[small[:, j]])) for j in range(k))
    assert np.all(np.abs(f64(host_bits(out)) - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * U * mag)
    dout = _normal(T, H)
    dy, dw = torch.zeros_like(y), torch.empty(T, k, device="cuda")
    G.moe_combine_bwd(dout, y, M, H, dd, T, k, weights=wd, dy=dy, dweights=dw)
    rdy, _, rdw = P.combine_bwd(host_bits(dout), yh, small, w)
    got = f64(_rows(dy, named.tolist()))
    assert np.all(np.abs(got - rdy) <= 2.0 ** -8 * np.abs(rdy) + 1e-37)
    dmag = np.sum(np.abs(f64(host_bits(dout)))[:, None] * np.abs(f64(yh[small])), axis=2)
    assert np.all(np.abs(dw.cpu().numpy() - rdw) <= (H / 64 + 16) * U * dmag)
    assert int((dy != 0).any(1).sum()) == T * k           # no other row
    del dy
    # many tokens: the outputs themselves pass 2^31
    dst = torch.arange(M, dtype=torch.int32, device="cuda").flip(0).contiguous()
    out = torch.zeros_like(y)
    G.moe_combine(y, M, H, dst, M, 1, out)
    assert torch.equal(out, y.flip(0))
    del out


def test_norm_and_gradients(G):
    import torch
    T, H = T_, H_
    x, wt = _normal(T, H), _normal(1, H)
    h, y, rstd = torch.zeros_like(x), torch.zeros_like(x), torch.empty(T, device="cuda")
    q, s = empty_bytes((T, H)), empty_bytes((T, H // 32))
    G.moe_add_rmsnorm(x, wt, T, H, 1e-5, residual=x, h=h, y=y, rstd=rstd, mx=G.mx_out(row_q=q, row_s=s))
    hb, rs, yv = P.add_rmsnorm(_rows(x, ROWS), host_bits(wt)[0], 1e-5, _rows(x, ROWS))
    assert np.array_equal(_rows(h, ROWS), hb)
    yb = _rows(y, ROWS)
    assert np.all(np.abs(f64(yb) - yv) <= (2.0 ** -8 + (H / 64 + 32) * U) * np.abs(yv))
    rq, rsc = O.mx_quantize_rows(yb)
    assert np.array_equal(q[ROWS].cpu().numpy(), rq) and np.array_equal(s[ROWS].cpu().numpy(), rsc)
    del q, s
    dx = torch.zeros_like(x)
    G.moe_add_rmsnorm_bwd(x, h, wt, rstd, T, H, dx=dx)
    dyh = _rows(x, ROWS)
    rdx, _ = P.add_rmsnorm_bwd(dyh, hb, host_bits(wt)[0], 1e-5)
    n, g = np.abs(f64(hb)) * rs[:, None], np.abs(f64(dyh) * f64(host_bits(wt)))
    mag = rs[:, None] * (g + n * np.mean(g * n, axis=1, keepdims=True))
    err = np.abs(f64(_rows(dx, ROWS)) - rdx)
    assert np.all(err <= 2.0 ** -8 * np.abs(rdx) + 3 * (H / 64 + 32) * U * mag + 1e-38)


def test_router_and_gradient(G):
    import torch
    T, E, k = (1 << 21) + 5, 1024, 4
    x = _normal(T, E).view(torch.bfloat16)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    r = G.router("softmax", renorm=False)
    G.moe_router_topk(x, T, E, k, r, ids, w)
    rows = [0, T - 6, T - 5, T - 1]                       # (row 2^21 holds value 2^31)
    v = x[rows].double().cpu().numpy()
    rid, rw = P.router_topk(v, k, renorm=False)
    R = np.max(np.max(v, 1) - np.min(v, 1))
    assert np.array_equal(ids[rows].cpu().numpy(), rid)
    assert np.all(np.abs(w[rows].cpu().numpy() - rw) <= (2 * R + 32) * U * rw)
    d = torch.zeros_like(x)
    G.moe_router_topk_bwd(x, T, E, k, r, ids, torch.ones_like(w), d)
    want = P.router_topk_bwd(v, rid, np.ones((len(rows), k)), renorm=False)
    sc = np.exp(v - np.max(v, 1, keepdims=True))
    sc /= sc.sum(1, keepdims=True)
    sel = np.zeros_like(v)
    np.put_along_axis(sel, rid.astype(np.int64), 1.0, 1)
    mag = sc * (sel + np.sum(sc * sel, 1, keepdims=True))
    err = np.abs(d[rows].double().cpu().numpy() - want)
    assert np.all(err <= 4 * (2 * R + 32) * U * mag + 2.0 ** -8 * np.abs(want) + 1e-37)


def test_mxfp4_quantize(G):
    v = _normal(T_, H_)
    q, s = empty_bytes((T_, H_ // 2)), empty_bytes((T_, H_ // 32))
    G.moe_mxfp4_quantize(v, T_, H_, None, q, s)
    rq, rs = P.mxfp4_quantize_rows(_rows(v, ROWS))
    assert np.array_equal(q[ROWS].cpu().numpy(), rq) and np.array_equal(s[ROWS].cpu().numpy(), rs)


def _bytes(*shape):
    import torch
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda",
                         generator=torch.Generator(device="cuda").manual_seed(shape[0]))


def _tol(a, K, want, mag):
    return 2.0 ** -8 * np.abs(want) + ((K / 128 + 16) * 4 * U if a == "fp4" else MX_ACC_REL) * mag + 1e-37


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("rows", [9, 700])                # streamed; on the 256 x 256 tiles
def test_mxfp4_product_of_the_last_experts(G, a, rows):
    import torch
    E, N, K = 150, 8192, 7168                             # 4.4e9 bytes of codes
    rng = np.random.default_rng(rows)
    b, bs = _bytes(E, N, K // 2), torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    ac = rng.integers(0, 256, (rows, K // 2 if a == "fp4" else K)).astype(np.uint8)
    if a == "fp8":
        ac = np.where((ac & 0x7F) == 0x7F, ac & 0x80, ac)
    as_ = rng.integers(118, 124, (rows, K // 32)).astype(np.uint8)
    counts = np.zeros(E, np.int64)
    counts[[0, 146, 149]] = [1, rows // 2, rows - rows // 2 - 1]
    out = empty_bits((rows, N))
    A = G.operand(dev_bytes(ac), dtype=G.DT_MXFP4 if a == "fp4" else G.DT_MXFP8, scales=dev_bytes(as_))
    B = G.operand(b, dtype=G.DT_MXFP4, layout=G.B_NK, scales=bs)
    G.moe_group_gemm_quant(A, B, N, K, G.groups(dev_i32(counts), rows), out)
    got = f64(host_bits(out))
    av = P.mxfp4_dequantize_rows(ac, as_) if a == "fp4" else O.mx_dequantize_rows(ac, as_)
    cols = np.r_[0:16, N - 48:N]
    off = O.exclusive_offsets(counts)
    for e in (0, 146, 149):
        bv = P.mxfp4_dequantize_rows(b[e].cpu().numpy()[cols], bs[e].cpu().numpy()[cols])
        r = slice(int(off[e]), int(off[e + 1]))
        want, mag = av[r] @ bv.T, np.abs(av[r]) @ np.abs(bv).T
        assert np.all(np.abs(got[r][:, cols] - want) <= _tol(a, K, want, mag)), e


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_mxfp4_product_of_many_rows(G, a):
    import torch
    M, N, K = (1 << 18) + 100, 8256, 64                   # M N = 2^31 + 1.8e7
    b, bs = _bytes(2, N, K // 2), torch.full((2, N, K // 32), 126, dtype=torch.uint8, device="cuda")
    ac = _bytes(M, K // 2 if a == "fp4" else K)
    if a == "fp8":
        ac &= 0x77
    as_ = torch.full((M, K // 32), 125, dtype=torch.uint8, device="cuda")
    counts = [M - 70, 60]
    out = empty_bits((M, N))
    A = G.operand(ac, dtype=G.DT_MXFP4 if a == "fp4" else G.DT_MXFP8, scales=as_)
    G.moe_group_gemm_quant(A, G.operand(b, dtype=G.DT_MXFP4, layout=G.B_NK, scales=bs), N, K,
                           G.groups(dev_i32(counts), M), out)
    rows = [0, 260111, M - 71, M - 70, M - 11]
    deq = P.mxfp4_dequantize_rows if a == "fp4" else O.mx_dequantize_rows
    av = deq(ac[rows].cpu().numpy(), as_[rows].cpu().numpy())
    bv = P.mxfp4_dequantize_rows(b.cpu().numpy(), bs.cpu().numpy())
    got = f64(_rows(out, rows))
    for i, row in enumerate(rows):
        e = int(row >= counts[0])
        want, mag = av[i] @ bv[e].T, np.abs(av[i]) @ np.abs(bv[e]).T
        assert np.all(np.abs(got[i] - want) <= _tol(a, K, want, mag)), row
    assert np.array_equal(_rows(out, [M - 10, M - 1]), host_bits(empty_bits((2, N))))
