"""The operators around the GEMMs on a rank without tokens or rows: empty
tensors, whose addresses are NULL, are nothing to do, not an error; with tokens
but no rows the combine is the residual alone."""
import pytest

from tests.test_gpu_router import G  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _empty(*shape, dtype="bfloat16"):
    import torch
    t = torch.empty(shape, dtype=getattr(torch, dtype), device="cuda")
    assert t.numel() > 0 or t.data_ptr() == 0
    return t


def test_router_no_tokens(G):  # noqa: F811
    import torch
    for dtype in ("float32", "bfloat16"):
        x, ids, w = _empty(0, 16, dtype=dtype), _empty(0, 4, dtype="int32"), _empty(0, 4, dtype="float32")
        r = G.router("sigmoid", bias=torch.zeros(16, device="cuda"), n_groups=4, topk_groups=2)
        G.moe_router_topk(x, 0, 16, 4, r, ids, w)
        G.moe_router_topk_bwd(x, 0, 16, 4, r, ids, w, torch.empty_like(x))
    torch.cuda.synchronize()


def test_combine_no_tokens(G):  # noqa: F811
    import torch
    H, y = 64, _empty(12, 64)
    dst, w, out = _empty(0, 3, dtype="int32"), _empty(0, 3, dtype="float32"), _empty(0, H)
    G.moe_combine(y, 12, H, dst, 0, 3, out, weights=w, residual=out)
    dy = torch.full((12, H), 5.0, dtype=torch.bfloat16, device="cuda")
    G.moe_combine_bwd(out, y, 12, H, dst, 0, 3, weights=w, dy=dy, dweights=w)
    torch.cuda.synchronize()
    assert torch.all(dy == 5)
    none = _empty(0, H)
    G.moe_combine(none, 0, H, dst, 0, 3, out, weights=w)
    G.moe_combine_bwd(out, none, 0, H, dst, 0, 3, weights=w, dy=_empty(0, H), dweights=w)


def test_combine_no_rows(G):  # noqa: F811
    """Every pair dropped, or sent elsewhere."""
    import torch
    T, k, H = 5, 3, 72
    y = _empty(0, H)
    dst = torch.tensor([[-1, 0, 7]] * T, dtype=torch.int32, device="cuda")
    w, res = torch.ones(T, k, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    out = torch.full_like(res, 9.0)
    G.moe_combine(y, 0, H, dst, T, k, out, weights=w, residual=res)
    dw = torch.full((T, k), 9.0, device="cuda")
    G.moe_combine_bwd(res, y, 0, H, dst, T, k, weights=w, dy=_empty(0, H), dweights=dw)
    G.moe_combine_bwd(res, y, 0, H, dst, T, k, weights=w, dy=_empty(0, H))
    torch.cuda.synchronize()
    assert torch.equal(out, res) and torch.all(dw == 0)


def test_norm_no_tokens(G):  # noqa: F811
    import torch
    H = 96
    x, wt = _empty(0, H), torch.ones(H, dtype=torch.bfloat16, device="cuda")
    mx = G.mx_out(row_q=_empty(0, H, dtype="uint8"), row_s=_empty(0, H // 32, dtype="uint8"))
    rstd = _empty(0, dtype="float32")
    G.moe_add_rmsnorm(x, wt, 0, H, 1e-6, residual=_empty(0, H), h=_empty(0, H), y=_empty(0, H), rstd=rstd, mx=mx)
    dw = torch.full((H,), 3.0, device="cuda")
    ws = torch.empty(max(1, G.moe_add_rmsnorm_bwd_workspace_bytes(0, H)), dtype=torch.uint8, device="cuda")
    G.moe_add_rmsnorm_bwd(x, x, wt, rstd, 0, H, dh=x, dx=_empty(0, H), dweight=dw, accumulate=True, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(dw == 3)
    G.moe_add_rmsnorm_bwd(x, x, wt, rstd, 0, H, dx=_empty(0, H), dweight=dw)      # written, as ever
    G.moe_add_rmsnorm_bwd(x, x, wt, rstd, 0, H, dx=_empty(0, H))
    torch.cuda.synchronize()
    assert torch.all(dw == 0)


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_mxfp4_no_rows(G, a):  # noqa: F811
    import torch
    E, N, K = 3, 64, 96
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    offs, status = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    v, s = _empty(0, K), _empty(0, K // 32, dtype="uint8")
    q = _empty(0, K // 2 if a == "fp4" else K, dtype="uint8")
    if a == "fp4":
        G.moe_mxfp4_quantize(v, 0, K, None, q, s)
        G.moe_mxfp4_quantize(v, 0, K, G.groups(counts, 0), q, s)
    A = G.operand(q, dtype=G.DT_MXFP4 if a == "fp4" else G.DT_MXFP8, scales=s)
    B = G.operand(torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda"), dtype=G.DT_MXFP4, layout=G.B_NK,
                  scales=torch.zeros(E, N, K // 32, dtype=torch.uint8, device="cuda"))
    G.moe_group_gemm_quant(A, B, N, K, G.groups(counts, 0), _empty(0, N))
    G.moe_group_gemm_quant(A, B, N, K, G.groups(counts, 0, offsets_out=offs, status_out=status), _empty(0, N))
    torch.cuda.synchronize()
    assert offs.tolist() == [0] * (E + 1) and int(status) == 0
    counts[1] = 4                                   # more rows than the capacity
    G.moe_group_gemm_quant(A, B, N, K, G.groups(counts, 0, offsets_out=offs, status_out=status), _empty(0, N))
    torch.cuda.synchronize()
    assert offs.tolist() == [0] * (E + 1) and int(status) == 2
