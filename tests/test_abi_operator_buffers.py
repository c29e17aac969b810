"""Buffers that the router, combine, norm and MXFP4 entry points refuse on the
host: an output that shares bytes with an input or another output, unless the
call allows it; also under AddressSanitizer.  No GPU is touched."""
import ctypes
import os
import subprocess
import sys

from tests.test_abi_asan import ROOT, asan_lib  # noqa: F401  (the fixture)

UNSUP = 4
STEP = 1 << 24          # buffers this far apart, never dereferenced: checks fail first


def _sweep(call, sizes, outputs, inputs, same_allowed=()):
    """Each output laid over each input's and other output's first and last 16 bytes, and over it from before: refused.
    Just behind it, and (same_allowed) exactly on it: not refused for that (the device's status, or done)."""
    at = {n: (i + 1) * STEP for i, n in enumerate(sizes)}
    assert call(**at) != UNSUP
    for o in outputs:
        for i in inputs + [x for x in outputs if x != o]:
            for where in (at[i], at[i] + (sizes[i] - 1) // 16 * 16, at[i] - (sizes[o] - 1) // 16 * 16):
                if where == at[i] and (o, i) in same_allowed:
                    assert call(**{**at, o: where}) != UNSUP, (o, i)
                    continue
                assert call(**{**at, o: where}) == UNSUP, (o, i, where - at[i])
            for where in (at[i] + (sizes[i] + 15) // 16 * 16, at[i] - (sizes[o] + 15) // 16 * 16):
                assert call(**{**at, o: where}) != UNSUP, (o, i, where - at[i])


# T = 0 and the like launch nothing, but T rows are needed for buffers to overlap: these calls would launch on a GPU
# with addresses that are none, so they are made only where there is no device
def _no_gpu():
    import pytest
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that are none")


def test_router_overlaps():
    _no_gpu()
    import grouped_gemm_glu_amd as G
    T, E, k = 33, 40, 5

    def fwd(logits, bias, ids, w):
        return G.raw_call("moe_router_topk", logits, G.DT_BF16, T, E, k, ctypes.byref(G.router(bias=bias)), ids, w, None)
    _sweep(fwd, dict(logits=T * E * 2, bias=E * 4, ids=T * k * 4, w=T * k * 4), ["ids", "w"], ["logits", "bias"])

    def bwd(logits, ids, dw, dl):
        return G.raw_call("moe_router_topk_bwd", logits, G.DT_FP32, T, E, k, ctypes.byref(G.router()), ids, dw, dl, None)
    _sweep(bwd, dict(logits=T * E * 4, ids=T * k * 4, dw=T * k * 4, dl=T * E * 4), ["dl"], ["logits", "ids", "dw"])


def test_combine_overlaps():
    _no_gpu()
    import grouped_gemm_glu_amd as G
    T, k, M, H = 9, 3, 31, 72

    def fwd(y, dst, w, res, out):
        return G.raw_call("moe_combine", y, M, H, dst, w, T, k, res, out, None)
    size = dict(y=M * H * 2, dst=T * k * 4, w=T * k * 4, res=T * H * 2, out=T * H * 2)
    _sweep(fwd, size, ["out"], ["y", "dst", "w", "res"], {("out", "res")})

    def bwd(dout, y, dst, w, dy, dw):
        return G.raw_call("moe_combine_bwd", dout, y, M, H, dst, w, T, k, dy, dw, None)
    size = dict(dout=T * H * 2, y=M * H * 2, dst=T * k * 4, w=T * k * 4, dy=M * H * 2, dw=T * k * 4)
    _sweep(bwd, size, ["dy", "dw"], ["dout", "y", "dst", "w"])


def test_norm_overlaps():
    _no_gpu()
    import grouped_gemm_glu_amd as G
    T, H = 7, 96

    def fwd(x, res, wt, h, y, rstd, q, s):
        return G.raw_call("moe_add_rmsnorm", x, res, wt, T, H, 1e-6, h, y, rstd, ctypes.byref(G.mx_out(row_q=q, row_s=s)), None)
    size = dict(x=T * H * 2, res=T * H * 2, wt=H * 2, h=T * H * 2, y=T * H * 2, rstd=T * 4, q=T * H, s=T * H // 32)
    _sweep(fwd, size, ["h", "y", "rstd", "q", "s"], ["x", "res", "wt"], {("h", "x"), ("h", "res")})

    need = G.moe_add_rmsnorm_bwd_workspace_bytes(T, H)

    def bwd(dy, h, wt, rstd, dh, dx, dwt, ws):
        return G.raw_call("moe_add_rmsnorm_bwd", dy, h, wt, rstd, dh, T, H, dx, dwt, 0, ws, need, None)
    size = dict(dy=T * H * 2, h=T * H * 2, wt=H * 2, rstd=T * 4, dh=T * H * 2, dx=T * H * 2, dwt=H * 4, ws=need)
    _sweep(bwd, size, ["dx", "dwt", "ws"], ["dy", "h", "wt", "rstd", "dh"], {("dx", "dh")})


def test_mxfp4_overlaps():
    _no_gpu()
    import grouped_gemm_glu_amd as G
    R, C, E = 40, 96, 3

    def quant(v, counts, q, s):
        return G.raw_call("moe_mxfp4_quantize", v, R, C, ctypes.byref(G.GroupsT(counts, E, R, None, None)), q, s, None)
    _sweep(quant, dict(v=R * C * 2, counts=E * 4, q=R * C // 2, s=R * C // 32), ["q", "s"], ["v", "counts"])

    def pack(src, q, s):
        return G.raw_call("moe_pack_weight_mxfp4", src, E, 64, C, G.B_KN, q, s, None)
    _sweep(pack, dict(src=E * 64 * C * 2, q=E * 64 * C // 2, s=E * 64 * C // 32), ["q", "s"], ["src"])

    for dt, bits in ((G.DT_MXFP4, 4), (G.DT_MXFP8, 8)):
        def gemm(a, sa, b, sb, counts, c, offs, status):
            A, B = G.operand(a, dtype=dt, scales=sa), G.operand(b, dtype=G.DT_MXFP4, layout=G.B_NK, scales=sb)
            return G.raw_call("moe_group_gemm_quant", ctypes.byref(A), ctypes.byref(B), 64, C,
                              ctypes.byref(G.GroupsT(counts, E, R, offs, status)), c, None, 0, None)
        size = dict(a=R * C * bits // 8, sa=R * C // 32, b=E * 64 * C // 2, sb=E * 64 * C // 32, counts=E * 4,
                    c=R * 64 * 2, offs=E * 4 + 4, status=4)
        _sweep(gemm, size, ["c", "offs", "status"], ["a", "sa", "b", "sb", "counts"])


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
from tests import test_abi_operator_buffers as t
for name in sorted(dir(t)):
    if name.startswith("test_") and "asan" not in name:
        getattr(t, name)()
print("asan-child-ok")
"""


def test_buffers_clean_under_asan(asan_lib):  # noqa: F811
    lib, rt = asan_lib
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt
    env["ASAN_OPTIONS"] = "detect_leaks=0:verify_asan_link_order=0:abort_on_error=0"
    env["HIP_VISIBLE_DEVICES"] = ""
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, lib=lib)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert "ERROR: AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0 and "asan-child-ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
