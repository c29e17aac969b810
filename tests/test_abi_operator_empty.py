"""An empty batch: the arrays that have no rows may be NULL (an empty tensor's
address); those that have rows, and the sizes, are checked as ever.  Host
checks only: the calls launch nothing, or find no device."""
import ctypes

NULL_, SHAPE, DEVICE, OK = 1, 2, 6, 0
FAKE = 1 << 24


def _done(status):
    assert status in (OK, DEVICE), status


def test_no_tokens():
    import grouped_gemm_glu_amd as G
    r, B = ctypes.byref(G.router()), ctypes.byref
    _done(G.raw_call("moe_router_topk", None, G.DT_FP32, 0, 8, 2, r, None, None, None))
    _done(G.raw_call("moe_router_topk_bwd", None, G.DT_FP32, 0, 8, 2, r, None, None, None, None))
    _done(G.raw_call("moe_combine", FAKE, 8, 64, None, None, 0, 2, None, None, None))
    _done(G.raw_call("moe_combine", None, 0, 64, None, None, 0, 2, None, None, None))
    _done(G.raw_call("moe_combine_bwd", None, FAKE, 8, 64, None, None, 0, 2, 4 * FAKE, None, None))
    _done(G.raw_call("moe_combine_bwd", None, None, 0, 64, None, None, 0, 2, None, None, None))
    _done(G.raw_call("moe_add_rmsnorm", None, None, FAKE, 0, 64, 1e-6, None, None, None, None, None))
    mx = G.mx_out()
    _done(G.raw_call("moe_add_rmsnorm", None, None, FAKE, 0, 64, 1e-6, None, None, None, B(mx), None))
    _done(G.raw_call("moe_add_rmsnorm_bwd", None, None, FAKE, None, None, 0, 64, None, None, 0, None, 0, None))
    _done(G.raw_call("moe_mxfp4_quantize", None, 0, 64, None, None, None, None))
    # what is not empty is still needed, and sizes are checked
    assert G.raw_call("moe_router_topk", None, G.DT_FP32, 0, 8, 2, None, None, None, None) == NULL_
    assert G.raw_call("moe_router_topk", None, G.DT_FP32, 0, 8, 9, r, None, None, None) == SHAPE
    assert G.raw_call("moe_combine", None, 8, 64, None, None, 0, 2, None, None, None) == NULL_
    assert G.raw_call("moe_combine", None, 0, 60, None, None, 0, 2, None, None, None) == SHAPE
    assert G.raw_call("moe_add_rmsnorm", None, None, None, 0, 64, 1e-6, None, None, None, None, None) == NULL_
    assert G.raw_call("moe_add_rmsnorm_bwd", None, None, None, None, None, 0, 64, None, FAKE, 0, None, 0, None) == NULL_
    assert G.raw_call("moe_mxfp4_quantize", None, 0, 60, None, None, None, None) == SHAPE


def test_no_rows():
    """Tokens, but no expert row here: y and dy have none."""
    import grouped_gemm_glu_amd as G
    f, B = FAKE, ctypes.byref
    assert G.raw_call("moe_combine", None, 0, 64, None, None, 4, 2, None, f, None) == NULL_        # dst
    assert G.raw_call("moe_combine", None, 0, 64, f, None, 4, 2, None, None, None) == NULL_        # out
    assert G.raw_call("moe_combine", None, 5, 64, f, None, 4, 2, None, 2 * f, None) == NULL_       # y, of 5 rows
    assert G.raw_call("moe_combine_bwd", None, None, 0, 64, f, None, 4, 2, None, 2 * f, None) == NULL_   # dout
    _done(G.raw_call("moe_combine_bwd", 3 * f, None, 0, 64, f, None, 4, 2, None, None, None))      # nothing to do
    E, N, K = 2, 64, 64
    b = G.operand(3 * f, dtype=G.DT_MXFP4, layout=G.B_NK, scales=4 * f)
    for dt in (G.DT_MXFP4, G.DT_MXFP8):
        a = G.operand(None, dtype=dt)
        _done(G.raw_call("moe_group_gemm_quant", B(a), B(b), N, K, B(G.GroupsT(f, E, 0, None, None)), None, None, 0, None))
        assert G.raw_call("moe_group_gemm_quant", B(a), B(b), N, K, B(G.GroupsT(f, E, 1, None, None)), None, None, 0, None) == NULL_
    no_b = G.operand(None, dtype=G.DT_MXFP4, layout=G.B_NK)
    assert G.raw_call("moe_group_gemm_quant", B(a), B(no_b), N, K, B(G.GroupsT(f, E, 0, None, None)), None, None, 0, None) == NULL_
