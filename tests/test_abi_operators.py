"""Refusals of the router, combine, norm and MXFP4 entry points: bad arguments
return a status on the host before anything launches (no GPU is touched), also
under AddressSanitizer."""
import ctypes
import math
import os
import subprocess
import sys

import pytest

from tests.test_abi_asan import ROOT, asan_lib  # noqa: F401  (the fixture)

NULL = None
FAKE = 1 << 20          # never dereferenced: checks fail first
NULL_, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4


def test_router_refusals():
    import grouped_gemm_glu_amd as G
    f, B = FAKE, ctypes.byref

    def fwd(logits=f, dt=G.DT_FP32, T=8, E=16, k=4, r=None, ids=f, w=f):
        return G.raw_call("moe_router_topk", logits, dt, T, E, k, B(r or G.router()), ids, w, NULL)

    def bwd(logits=f, dt=G.DT_FP32, T=8, E=16, k=4, r=None, ids=f, dw=f, dl=f):
        return G.raw_call("moe_router_topk_bwd", logits, dt, T, E, k, B(r or G.router()), ids, dw, dl, NULL)

    assert G.raw_call("moe_router_topk", f, G.DT_FP32, 8, 16, 4, NULL, f, f, NULL) == NULL_
    for call in (fwd, bwd):
        assert call(logits=NULL) == NULL_ and call(ids=NULL) == NULL_
        assert call(T=-1) == SHAPE and call(T=(1 << 25) + 1) == SHAPE
        assert call(E=0) == SHAPE and call(E=1025) == SHAPE and call(k=0) == SHAPE
        assert call(E=64, k=17) == SHAPE and call(E=4, k=5) == SHAPE
        assert call(dt=G.DT_MXFP8) == UNSUP and call(dt=G.DT_MXFP4) == UNSUP
        assert call(logits=f + 4) == ALIGN and call(ids=f + 2) == ALIGN
        assert call(r=G.router(n_groups=3)) == SHAPE                      # does not divide E
        assert call(r=G.router(n_groups=0)) == SHAPE
        assert call(r=G.router(n_groups=4, topk_groups=5)) == SHAPE
        assert call(r=G.router(n_groups=4, topk_groups=0)) == SHAPE
        assert call(k=5, r=G.router(n_groups=4, topk_groups=1)) == SHAPE  # 4 experts are left
        assert call(E=128, r=G.router(n_groups=128, topk_groups=64)) == SHAPE
        assert call(r=G.router(n_groups=16, topk_groups=8, group_score="top2")) == SHAPE
        assert call(r=G.router(scale=math.inf)) == SHAPE and call(r=G.router(scale=math.nan)) == SHAPE
        assert call(r=G.router(bias=f + 2)) == ALIGN
        for field in ("score", "group_score", "renorm"):
            bad = G.router()
            setattr(bad, field, 2)
            assert call(r=bad) == UNSUP, field
    assert fwd(w=NULL) == NULL_ and fwd(w=f + 1) == ALIGN
    assert bwd(dw=NULL) == NULL_ and bwd(dl=NULL) == NULL_ and bwd(dl=f + 4) == ALIGN
    assert bwd() == UNSUP                                                 # dlogits over the logits
    with pytest.raises(TypeError):
        import torch
        G.moe_router_topk(torch.zeros(2, 4, dtype=torch.float16), 2, 4, 1, G.router(), f, f, stream=1)


def test_combine_refusals():
    import grouped_gemm_glu_amd as G
    f = FAKE

    def fwd(y=f, M=64, H=32, dst=f, w=f, T=8, k=2, res=NULL, out=f):
        return G.raw_call("moe_combine", y, M, H, dst, w, T, k, res, out, NULL)

    def bwd(dout=f, y=2 * f, M=64, H=32, dst=f, w=f, T=8, k=2, dy=3 * f, dw=f):
        return G.raw_call("moe_combine_bwd", dout, y, M, H, dst, w, T, k, dy, dw, NULL)

    for call in (fwd, bwd):
        assert call(y=NULL) == NULL_ and call(dst=NULL) == NULL_
        assert call(H=12) == SHAPE and call(H=0) == SHAPE and call(k=0) == SHAPE and call(k=17) == SHAPE
        assert call(T=-1) == SHAPE and call(M=-1) == SHAPE
        assert call(y=f + 2) == ALIGN and call(dst=f + 2) == ALIGN and call(w=f + 2) == ALIGN
    assert fwd(out=NULL) == NULL_ and fwd(out=f + 8) == ALIGN and fwd(res=f + 8) == ALIGN
    assert bwd(dout=NULL) == NULL_ and bwd(dy=NULL, dw=NULL) == NULL_ and bwd(dout=f + 8) == ALIGN
    assert bwd(dy=f) == UNSUP and bwd(dy=2 * f) == UNSUP      # over dout, over y
    assert fwd(out=f) == UNSUP                                # over y
    assert fwd(H=(1 << 26) + 8) == SHAPE and bwd(H=(1 << 31) - 8) == SHAPE
    assert bwd(dw=f + 1) == ALIGN and bwd(dy=f + 8) == ALIGN


def test_norm_refusals():
    import grouped_gemm_glu_amd as G
    f, B = FAKE, ctypes.byref

    def fwd(x=f, res=NULL, w=f, T=4, H=64, eps=1e-6, h=NULL, y=f, rstd=NULL, mx=NULL):
        return G.raw_call("moe_add_rmsnorm", x, res, w, T, H, eps, h, y, rstd, mx, NULL)

    def bwd(dy=f, h=f, w=f, rstd=f, dh=NULL, T=4, H=64, dx=f, dw=f, acc=0, ws=f, n=1 << 20):
        return G.raw_call("moe_add_rmsnorm_bwd", dy, h, w, rstd, dh, T, H, dx, dw, acc, ws, n, NULL)

    for call in (fwd, bwd):
        assert call(w=NULL) == NULL_ and call(w=f + 2) == ALIGN
        assert call(H=12) == SHAPE and call(H=16392) == SHAPE and call(H=0) == SHAPE and call(T=-1) == SHAPE
    assert fwd(x=NULL) == NULL_ and fwd(y=NULL) == NULL_ and fwd(x=f + 2) == ALIGN
    assert fwd(eps=-1.0) == SHAPE and fwd(eps=math.nan) == SHAPE and fwd(eps=math.inf) == SHAPE
    assert fwd(res=f + 2) == ALIGN and fwd(h=f + 2) == ALIGN and fwd(rstd=f + 2) == ALIGN
    assert fwd(mx=B(G.mx_out(row_q=f))) == NULL_
    assert fwd(mx=B(G.mx_out(row_q=f, row_s=f, col_q=f, col_s=f))) == UNSUP
    assert fwd(H=72, mx=B(G.mx_out(row_q=f, row_s=f))) == SHAPE
    assert bwd(dy=NULL) == NULL_ and bwd(h=NULL) == NULL_ and bwd(rstd=NULL) == NULL_
    assert bwd(dx=NULL, dw=NULL) == NULL_ and bwd(ws=NULL) == NULL_
    need = G.moe_add_rmsnorm_bwd_workspace_bytes(4, 64)
    assert need > 0 and bwd(n=need - 1) == SHAPE and bwd(ws=f + 4) == ALIGN
    assert bwd(acc=2) == UNSUP and bwd(dh=f + 2) == ALIGN and bwd(dx=f + 2) == ALIGN
    assert bwd(h=2 * f) == UNSUP and bwd(dy=2 * f) == UNSUP              # dx over dy, over h
    assert fwd(y=f) == UNSUP and fwd(x=2 * f, res=f) == UNSUP and fwd(x=2 * f, h=f) == UNSUP
    assert G.moe_add_rmsnorm_bwd_workspace_bytes(0, 64) == 0
    # the workspace stops growing with the token count
    assert (G.moe_add_rmsnorm_bwd_workspace_bytes(1 << 20, 7168)
            == G.moe_add_rmsnorm_bwd_workspace_bytes(1 << 24, 7168) <= 16 << 20)


def test_mxfp4_refusals():
    import grouped_gemm_glu_amd as G
    f, B = FAKE, ctypes.byref
    grp = G.GroupsT(f, 4, 64, None, None)

    def quant(v=f, R=64, C=64, g=NULL, q=f, s=f):
        return G.raw_call("moe_mxfp4_quantize", v, R, C, g, q, s, NULL)
    assert quant(v=NULL) == NULL_ and quant(q=NULL) == NULL_ and quant(s=NULL) == NULL_
    assert quant(C=48) == SHAPE and quant(C=0) == SHAPE and quant(R=-1) == SHAPE
    assert quant(R=63, g=B(grp)) == SHAPE and quant(v=f + 2) == ALIGN and quant(q=f + 4) == ALIGN
    assert quant(g=B(G.GroupsT(None, 4, 64, None, None))) == NULL_

    def pack(src=f, E=2, N=64, K=64, lay=G.B_KN, q=f, s=f):
        return G.raw_call("moe_pack_weight_mxfp4", src, E, N, K, lay, q, s, NULL)
    assert pack(src=NULL) == NULL_ and pack(q=NULL) == NULL_ and pack(s=NULL) == NULL_
    assert pack(N=96) == SHAPE and pack(K=48) == SHAPE and pack(E=0) == SHAPE and pack(E=65536) == SHAPE
    assert pack(E=65535, N=1 << 16) == SHAPE
    assert pack(lay=G.B_PACKED) == UNSUP and pack(q=f + 8) == ALIGN and pack(src=f + 2) == ALIGN

    a4 = G.operand(f, dtype=G.DT_MXFP4, scales=f)
    b4 = G.operand(f, dtype=G.DT_MXFP4, layout=G.B_NK, scales=f)

    def gemm(a=a4, b=b4, N=64, K=64, c=f, mx=NULL, g=grp):
        return G.raw_call("moe_group_gemm_quant", B(a), B(b), N, K, B(g), c, mx, 0, NULL)
    assert gemm(c=NULL) == NULL_ and gemm(N=96) == SHAPE and gemm(K=48) == SHAPE and gemm(K=0) == SHAPE
    assert gemm(a=G.operand(f, dtype=G.DT_MXFP4)) == NULL_
    assert gemm(b=G.operand(f, dtype=G.DT_MXFP4, layout=G.B_NK)) == NULL_
    for dt in (G.DT_BF16, G.DT_MXFP8_E5M2, G.DT_FP32):
        assert gemm(a=G.operand(f, dtype=dt, scales=f)) == UNSUP
    for lay in (G.B_KN, G.B_PACKED):
        assert gemm(b=G.operand(f, dtype=G.DT_MXFP4, layout=lay, scales=f)) == UNSUP
    # 4-bit rows need 4-bit weights
    assert gemm(b=G.operand(f, layout=G.B_NK)) == UNSUP
    assert gemm(b=G.operand(f, dtype=G.DT_MXFP8, layout=G.B_PACKED, scales=f), K=128) == UNSUP
    assert gemm(mx=B(G.mx_out(row_q=f, row_s=f))) == UNSUP
    assert gemm(a=G.operand(f + 8, dtype=G.DT_MXFP4, scales=f)) == ALIGN and gemm(c=f + 2) == ALIGN
    # 256 rows of e4m3 codes and of outputs are addressed with 32 bits
    assert gemm(K=1 << 24) == SHAPE and gemm(K=(1 << 31) - 32) == SHAPE
    assert gemm(N=1 << 23) == SHAPE and gemm(N=(1 << 31) - 64) == SHAPE
    # the other operands keep their own rule for K
    assert gemm(a=G.operand(f), b=G.operand(f, layout=G.B_KN), K=32) == SHAPE


CHILD = r"""
import ctypes, sys
sys.path.insert(0, {root!r})
import grouped_gemm_glu_amd as G
lib = ctypes.CDLL({lib!r})
for name, (args, res) in G._SIGS.items():
    f = getattr(lib, name)
    f.argtypes = args
    f.restype = res
G._lib = lib
from tests import test_abi_operators as t
t.test_router_refusals()
t.test_combine_refusals()
t.test_norm_refusals()
t.test_mxfp4_refusals()
print("asan-child-ok")
"""


def test_refusals_clean_under_asan(asan_lib):  # noqa: F811
    lib, rt = asan_lib
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt
    env["ASAN_OPTIONS"] = "detect_leaks=0:verify_asan_link_order=0:abort_on_error=0"
    env["HIP_VISIBLE_DEVICES"] = ""
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, lib=lib)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert "ERROR: AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0 and "asan-child-ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
