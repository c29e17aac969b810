"""Refusals of the adapter, AdamW and gradient norm entry points: bad arguments
and buffers that share bytes return a status on the host before anything
launches, also under AddressSanitizer; a plan's table is what its tensors say.
No GPU is touched."""
import ctypes
import math
import os
import subprocess
import sys

import pytest

from tests.test_abi_asan import ROOT, asan_lib  # noqa: F401  (the fixture)
from tests.test_abi_operator_buffers import _no_gpu, _sweep

NULL = None
F = 1 << 24             # addresses that are none, this far apart: checks fail first
OK, NULL_, SHAPE, ALIGN, UNSUP, DEVICE = 0, 1, 2, 3, 4, 6
BIG = 1 << 40


def _lora(G, A=F, B=2 * F, r=16, K=64, N=72, scale=NULL, x_ld=0, y_ld=0):
    return G.LoraT(A, B, scale, r, K, N, x_ld, y_ld)


def _groups(G, counts=3 * F, E=4, M=5000):
    return G.GroupsT(counts, E, M, None, None)


def test_lora_refusals():
    import grouped_gemm_glu_amd as G
    B = ctypes.byref

    def fwd(x=4 * F, T=5000, src=5 * F, g=None, lo=None, base=6 * F, y=7 * F, u=8 * F, ws=9 * F, n=BIG):
        return G.raw_call("moe_lora_fwd", x, T, src, B(g or _groups(G)), B(lo or _lora(G)), base, y, u, ws, n, NULL)

    def bwd(dy=4 * F, x=5 * F, T=5000, src=6 * F, g=None, lo=None, u=7 * F, base=8 * F, dx=9 * F, dA=10 * F, dB=11 * F,
            acc=0, ws=12 * F, n=BIG):
        return G.raw_call("moe_lora_bwd", dy, x, T, src, B(g or _groups(G)), B(lo or _lora(G)), u, base, dx, dA, dB, acc,
                          ws, n, NULL)
    for call in (fwd, bwd):
        assert call(g=_groups(G, counts=None)) == NULL_ and call(g=_groups(G, E=0)) == SHAPE
        assert call(g=_groups(G, E=1025)) == SHAPE and call(g=_groups(G, M=-1)) == SHAPE
        assert call(g=_groups(G, M=(1 << 25) + 1)) == SHAPE and call(g=_groups(G, counts=F + 2)) == ALIGN
        assert call(lo=_lora(G, A=None)) == NULL_ and call(lo=_lora(G, B=None)) == NULL_
        for bad in (dict(r=0), dict(r=4), dict(r=12), dict(r=136), dict(K=0), dict(K=12), dict(K=(1 << 17) + 8),
                    dict(N=0), dict(N=4), dict(N=(1 << 17) + 8), dict(x_ld=56), dict(x_ld=68), dict(x_ld=-64),
                    dict(y_ld=64), dict(y_ld=76), dict(x_ld=(1 << 32) + 8), dict(y_ld=(1 << 32) + 8)):
            assert call(lo=_lora(G, **bad)) == SHAPE, bad
        assert call(lo=_lora(G, A=F + 8)) == ALIGN and call(lo=_lora(G, B=F + 2)) == ALIGN
        assert call(lo=_lora(G, scale=F + 2)) == ALIGN and call(src=F + 2) == ALIGN
        assert call(T=1 << 20, lo=_lora(G, x_ld=(1 << 28) + 8)) == call(T=1 << 20, lo=_lora(G, y_ld=(1 << 28) + 8)) == SHAPE
        assert call(T=-1) == SHAPE and call(ws=NULL) == NULL_ and call(ws=9 * F + 8) == ALIGN
    assert fwd(x=NULL) == NULL_ and fwd(y=NULL) == NULL_
    assert fwd(x=4 * F + 2) == ALIGN and fwd(y=7 * F + 8) == ALIGN and fwd(base=6 * F + 8) == ALIGN and fwd(u=8 * F + 4) == ALIGN
    need = G.moe_lora_fwd_workspace_bytes(5000, 4, 16, 64, 72)
    assert need > 0 and fwd(n=need - 1) == SHAPE
    assert bwd(dy=NULL) == NULL_ and bwd(x=NULL) == NULL_ and bwd(u=NULL) == NULL_ and bwd(dx=NULL, dA=NULL, dB=NULL) == NULL_
    for name in ("dy", "x", "u", "base", "dx", "dA", "dB"):
        assert bwd(**{name: 13 * F + 8}) == ALIGN, name
    assert bwd(acc=2) == UNSUP and bwd(acc=-1) == UNSUP
    need = G.moe_lora_bwd_workspace_bytes(5000, 4, 16, 64, 72)
    assert need > 0 and bwd(n=need - 1) == SHAPE
    assert G.raw_call("moe_lora_fwd", F, 4, NULL, NULL, B(_lora(G)), NULL, 2 * F, NULL, 3 * F, BIG, NULL) == NULL_
    assert G.raw_call("moe_lora_fwd", F, 4, NULL, B(_groups(G)), NULL, NULL, 2 * F, NULL, 3 * F, BIG, NULL) == NULL_
    for f in (G.moe_lora_fwd_workspace_bytes, G.moe_lora_bwd_workspace_bytes):
        assert f(-1, 4, 16, 64, 64) == f(8, 0, 16, 64, 64) == f(8, 4, 12, 64, 64) == f(8, 4, 16, 63, 64) == 0
        assert f(8, 4, 16, 64, 1 << 18) == 0 and f((1 << 25) + 1, 4, 16, 64, 64) == 0


def test_lora_empty():
    """No rows: their arrays and the workspace may be NULL."""
    import grouped_gemm_glu_amd as G
    B = ctypes.byref
    for T, M in ((0, 0), (0, 8), (8, 0)):
        x = F if T else NULL
        st = G.raw_call("moe_lora_fwd", x, T, NULL, B(_groups(G, M=M)), B(_lora(G)), NULL, 7 * F if T else NULL, NULL, NULL, 0, NULL)
        assert st in (OK, DEVICE), (T, M, st)
        st = G.raw_call("moe_lora_bwd", x, NULL, T, NULL, B(_groups(G, M=M)), B(_lora(G)), NULL, NULL, NULL, NULL, NULL, 1, NULL, 0, NULL)
        assert st in (OK, DEVICE), (T, M, st)


def test_lora_few_rows_need_no_workspace():
    import grouped_gemm_glu_amd as G
    B = ctypes.byref
    assert G.moe_lora_fwd_workspace_bytes(100, 4, 16, 64, 72) == 0 < G.moe_lora_fwd_workspace_bytes(100, 4, 16, 8200, 72)
    for K, want in ((64, (OK, DEVICE)), (8200, (NULL_,))):
        T = 0 if K == 64 else 100      # with rows and a device it would launch with addresses that are none
        st = G.raw_call("moe_lora_fwd", F, T, NULL, B(_groups(G, M=100)), B(_lora(G, K=K)), NULL, 7 * F, NULL, NULL, 0, NULL)
        assert st in want, (K, st)


def test_lora_overlaps():
    _no_gpu()
    import grouped_gemm_glu_amd as G
    B = ctypes.byref
    E, M, T, r, K, N = 3, 4800, 4804, 16, 40, 56
    for x_ld, y_ld in ((0, 0), (48, 64)):
        xb, yb = ((T - 1) * (x_ld or K) + K) * 2, ((T - 1) * (y_ld or N) + N) * 2
        size = dict(x=xb, src=M * 4, counts=E * 4, A=E * r * K * 2, B_=E * r * N * 2, scale=E * 4, base=yb, y=yb, u=M * r * 4,
                    ws=G.moe_lora_fwd_workspace_bytes(M, E, r, K, N), offs=E * 4 + 4, status=4)

        def fwd(x, src, counts, A, B_, scale, base, y, u, ws, offs, status):
            g = G.GroupsT(counts, E, M, offs, status)
            return G.raw_call("moe_lora_fwd", x, T, src, B(g), B(G.LoraT(A, B_, scale, r, K, N, x_ld, y_ld)), base, y, u, ws,
                              size["ws"], NULL)
        _sweep(fwd, size, ["y", "u", "ws", "offs", "status"], ["x", "src", "counts", "A", "B_", "scale", "base"], {("y", "base")})

        bsize = dict(dy=yb, x=xb, src=M * 4, counts=E * 4, A=E * r * K * 2, B_=E * r * N * 2, scale=E * 4, u=M * r * 4, base=xb,
                     dx=xb, dA=E * r * K * 4, dB=E * r * N * 4, ws=G.moe_lora_bwd_workspace_bytes(M, E, r, K, N),
                     offs=E * 4 + 4, status=4)

        def bwd(dy, x, src, counts, A, B_, scale, u, base, dx, dA, dB, ws, offs, status):
            g = G.GroupsT(counts, E, M, offs, status)
            return G.raw_call("moe_lora_bwd", dy, x, T, src, B(g), B(G.LoraT(A, B_, scale, r, K, N, x_ld, y_ld)), u, base, dx, dA,
                              dB, 0, ws, bsize["ws"], NULL)
        _sweep(bwd, bsize, ["dx", "dA", "dB", "ws", "offs", "status"], ["dy", "x", "src", "counts", "A", "B_", "scale", "u", "base"],
               {("dx", "base")})


def _tensor(G, param=F, grad=2 * F, master=NULL, m=3 * F, v=4 * F, ms=NULL, vs=NULL, n=1000, lr=1.0, wd=0.0, pd=None, gd=None,
            bits=32):
    return G.AdamwTensorT(param, grad, master, m, v, ms, vs, n, lr, wd, G.DT_FP32 if pd is None else pd,
                          G.DT_FP32 if gd is None else gd, bits)


def _plan(G, tensors, table=True, n_bytes=None, out=True):
    array = (G.AdamwTensorT * max(1, len(tensors)))(*tensors)
    size = G._lib.moe_adamw_plan_bytes(array, len(tensors))
    buf = (ctypes.c_uint64 * (size // 8 + 1))()
    plan = G.AdamwPlanT()
    st = G.raw_call("moe_adamw_plan", array, len(tensors), ctypes.addressof(buf) if table else None,
                    size if n_bytes is None else n_bytes, ctypes.byref(plan) if out else None)
    return st, plan, buf, size


def test_plan_refusals():
    import grouped_gemm_glu_amd as G
    f = lambda **k: _plan(G, [_tensor(G, **k)])[0]  # noqa: E731
    assert f() == OK and f(n=0, grad=NULL, m=NULL, v=NULL) == OK and f(param=NULL, m=NULL, v=NULL, bits=7, pd=9) == OK
    assert f(grad=NULL) == NULL_ and f(m=NULL) == NULL_ and f(v=NULL) == NULL_
    assert f(bits=8) == NULL_ and f(bits=8, ms=5 * F) == NULL_ and f(bits=8, ms=5 * F, vs=6 * F) == OK
    assert f(n=-1) == SHAPE and f(n=(1 << 42) + 1) == SHAPE
    assert f(lr=math.inf) == SHAPE and f(lr=math.nan) == SHAPE and f(wd=math.inf) == SHAPE
    assert f(bits=16) == UNSUP and f(pd=G.DT_MXFP8) == UNSUP and f(gd=G.DT_MXFP8) == UNSUP
    assert f(master=5 * F) == UNSUP and f(master=5 * F, pd=G.DT_BF16) == OK
    for name in ("param", "grad", "m", "v"):
        assert f(**{name: 7 * F + 8}) == ALIGN, name
    assert f(master=5 * F + 4, pd=G.DT_BF16) == ALIGN and f(bits=8, ms=5 * F + 2, vs=6 * F) == ALIGN
    assert _plan(G, [_tensor(G)], table=False)[0] == NULL_ and _plan(G, [_tensor(G)], out=False)[0] == NULL_
    size = _plan(G, [_tensor(G)])[3]
    assert _plan(G, [_tensor(G)], n_bytes=size - 1)[0] == SHAPE
    assert G.raw_call("moe_adamw_plan", None, -1, None, 0, ctypes.byref(G.AdamwPlanT())) == SHAPE
    assert G.raw_call("moe_adamw_plan", None, (1 << 24) + 1, None, 0, ctypes.byref(G.AdamwPlanT())) == SHAPE
    assert G.raw_call("moe_adamw_plan", None, 3, F, 0, ctypes.byref(G.AdamwPlanT())) == NULL_
    st, plan, _, size = _plan(G, [])
    assert st == OK and size == 0 and plan.n_chunks == plan.n_chunks8 == 0


def test_plan_overlaps():
    import grouped_gemm_glu_amd as G
    n = 1000
    names = ["param", "master", "m", "v", "ms", "vs", "grad"]
    size = dict(param=2 * n, master=4 * n, m=n, v=n, ms=32, vs=32, grad=4 * n)
    at = {k: (i + 1) * F for i, k in enumerate(names)}

    def one(**where):
        return _tensor(G, **{**at, **where}, n=n, pd=G.DT_BF16, bits=8)
    assert _plan(G, [one()])[0] == OK
    for o in names[:-1]:
        for i in names:
            if i == o:
                continue
            # the output over the first and last bytes of the other, and from before; just behind and before: fine
            for where in (at[i], at[i] + (size[i] - 1) // 16 * 16, at[i] - (size[o] - 1) // 16 * 16):
                assert _plan(G, [one(**{o: where})])[0] == UNSUP, (o, i)
            for where in (at[i] + (size[i] + 15) // 16 * 16, at[i] - (size[o] + 15) // 16 * 16):
                assert _plan(G, [one(**{o: where})])[0] == OK, (o, i)
    # between tensors, whatever their order; a gradient may serve twice, and behind a long one too
    far = {k: v + 64 * F for k, v in at.items()}
    assert _plan(G, [one(), one(**far)])[0] == OK
    for k in names[:-1]:
        assert _plan(G, [one(), one(**{**far, k: at[k] + 16})])[0] == UNSUP
        assert _plan(G, [one(**{**far, k: at[k] + 16}), one()])[0] == UNSUP
    assert _plan(G, [one(), one(**{**far, "grad": at["grad"]})])[0] == OK
    assert _plan(G, [one(), _tensor(G, param=NULL, grad=at["m"])])[0] == UNSUP
    long_grad = _tensor(G, param=NULL, grad=200 * F, n=F)                # 4 F bytes
    assert _plan(G, [long_grad, _tensor(G, param=NULL, grad=200 * F + 64, n=4), one(m=201 * F)])[0] == UNSUP
    assert _plan(G, [long_grad, _tensor(G, param=NULL, grad=200 * F + 64, n=4), one(m=204 * F)])[0] == OK


def test_plan_table():
    """Pieces of 2048 elements (4096 from 2^22 on) in the tensors' order, those of 8-bit states last; each begins where
    its tensor's piece does (the first words of an entry are the parameter's and the gradient's address)."""
    import grouped_gemm_glu_amd as G
    ns = [1, 0, 4096, 4097, 10000]
    ts = [_tensor(G, param=(20 * i + 1) * F, grad=(20 * i + 2) * F, m=(20 * i + 3) * F, v=(20 * i + 4) * F, n=n, lr=0.5 + i,
                  wd=0.1 * i, gd=G.DT_BF16) for i, n in enumerate(ns)]
    ts[2] = _tensor(G, param=41 * F, grad=42 * F, m=43 * F, v=44 * F, ms=45 * F, vs=46 * F, n=4096, bits=8, pd=G.DT_BF16)
    st, plan, buf, size = _plan(G, ts)
    want = [((20 * i + 1) * F + 4 * at, (20 * i + 2) * F + 2 * at) for i in (0, 3, 4) for at in range(0, ns[i], 2048)]
    want += [(41 * F + 2 * at, 42 * F + 4 * at) for at in (0, 2048)]
    assert st == OK and plan.table is None and plan.n_chunks == len(want) and plan.n_chunks8 == 2 and size % len(want) == 0
    each = size // len(want)
    word = lambda i, k: int.from_bytes(bytes(buf)[i * each + 8 * k:i * each + 8 * k + 8], "little")  # noqa: E731
    assert [(word(i, 0), word(i, 1)) for i in range(len(want))] == want
    st, plan, _, size = _plan(G, [_tensor(G, grad=64 * F, m=128 * F, v=192 * F, n=(1 << 22) + 1)])
    assert st == OK and plan.n_chunks == 1025 and plan.n_chunks8 == 0 and size == each * 1025
    bad = (G.AdamwTensorT * 1)(_tensor(G, n=-5))
    # the largest sizes
    huge = (G.AdamwTensorT * 5)(*[_tensor(G, n=1 << 42)] * 5)
    assert G._lib.moe_adamw_plan_bytes(huge, 5) == 5 * each << 30
    assert G._lib.moe_adamw_plan_bytes(bad, 1) == 0 and G._lib.moe_adamw_plan_bytes(None, 3) == 0


def test_step_refusals():
    import grouped_gemm_glu_amd as G
    B = ctypes.byref

    def step(plan=None, h=None, **k):
        return G.raw_call("moe_adamw_step", B(plan or G.AdamwPlanT(F, 1)), B(h or G.adamw(**{**dict(lr=1e-3), **k})), NULL)
    assert G.raw_call("moe_adamw_step", NULL, B(G.adamw(1e-3)), NULL) == NULL_
    assert G.raw_call("moe_adamw_step", B(G.AdamwPlanT(F, 1)), NULL, NULL) == NULL_
    assert step(plan=G.AdamwPlanT(None, 1)) == NULL_ and step(plan=G.AdamwPlanT(F + 8, 1)) == ALIGN
    assert step(plan=G.AdamwPlanT(F, -1)) == SHAPE and step(plan=G.AdamwPlanT(F, 1, 2)) == SHAPE and step(plan=G.AdamwPlanT(F, 1, -1)) == SHAPE
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf),
                dict(lr=math.inf), dict(lr=math.nan), dict(step=0), dict(step=-1)):
        assert step(**bad) == SHAPE, bad
    assert step(step_dev=F + 2) == ALIGN and step(lr_dev=F + 2) == ALIGN and step(grad_scale=F + 2) == ALIGN
    assert step(plan=G.AdamwPlanT(None, 0)) in (OK, DEVICE)

    def norm(plan=None, most=1.0, out=2 * F, ws=3 * F, n=BIG):
        return G.raw_call("moe_grad_norm", B(plan or G.AdamwPlanT(F, 1)), most, out, ws, n, NULL)
    assert norm(plan=G.AdamwPlanT(None, 1)) == NULL_ and norm(out=NULL) == NULL_ and norm(ws=NULL) == NULL_
    assert norm(most=0.0) == SHAPE and norm(most=-1.0) == SHAPE and norm(most=math.nan) == SHAPE
    assert norm(out=F) == UNSUP and norm(ws=F) == UNSUP and norm(ws=2 * F, out=2 * F + 8) == UNSUP
    assert norm(n=G.moe_grad_norm_workspace_bytes() - 1) == SHAPE and norm(out=2 * F + 2) == ALIGN and norm(ws=3 * F + 8) == ALIGN
    assert norm(out=3 * F + 8) == UNSUP
    assert G.raw_call("moe_grad_norm", NULL, 1.0, F, 2 * F, BIG, NULL) == NULL_

    def unpack(m=F, ms=2 * F, v=3 * F, vs=4 * F, n=1000, mo=5 * F, vo=6 * F):
        return G.raw_call("moe_adamw_unpack", m, ms, v, vs, n, mo, vo, NULL)
    assert unpack(n=-1) == SHAPE and unpack(n=(1 << 42) + 1) == SHAPE and unpack(mo=NULL, vo=NULL) == NULL_
    assert unpack(m=NULL) == NULL_ and unpack(ms=NULL) == NULL_ and unpack(v=NULL) == NULL_ and unpack(vs=NULL) == NULL_
    for name in ("m", "v", "mo", "vo"):
        assert unpack(**{name: 9 * F + 8}) == ALIGN, name
    assert unpack(ms=F + 2) == ALIGN and unpack(vs=F + 2) == ALIGN
    assert unpack(m=NULL, ms=NULL, v=NULL, vs=NULL, n=0, mo=NULL, vo=NULL) in (OK, DEVICE)


def test_unpack_overlaps():
    _no_gpu()
    import grouped_gemm_glu_amd as G

    def unpack(m, ms, v, vs, mo, vo):
        return G.raw_call("moe_adamw_unpack", m, ms, v, vs, 1000, mo, vo, NULL)
    _sweep(unpack, dict(m=1000, ms=32, v=1000, vs=32, mo=4000, vo=4000), ["mo", "vo"], ["m", "ms", "v", "vs"])


def test_binding_checks():
    import torch
    import grouped_gemm_glu_amd as G
    t = lambda n, d=torch.float32: torch.zeros(n, dtype=d)  # noqa: E731
    G.adamw_tensor(t(5), t(5, torch.bfloat16), t(5), t(5))
    G.adamw_tensor(t(5), t(5), t(5, torch.int8), t(5, torch.uint8), m_scale=t(1), v_scale=t(1))
    for bad in (dict(m=t(4)), dict(v=t(6)), dict(master=t(4)), dict(m_scale=t(2)), dict(param=t(4))):
        with pytest.raises(ValueError):
            G.adamw_tensor(**{**dict(param=t(5), grad=t(5), m=t(5), v=t(5)), **bad})
    with pytest.raises(ValueError):
        G.adamw_tensor(t(10)[::2], t(5), t(5), t(5))
    with pytest.raises(ValueError):
        G.adamw_plan([G.adamw_tensor(t(5), t(5), t(5), t(5))])        # not on a GPU
    for bad in (dict(m=t(5, torch.int8)), dict(grad=t(5, torch.float16)), dict(param=t(5, torch.float16)),
                dict(master=t(5, torch.bfloat16), param=t(5, torch.bfloat16)),
                dict(m=t(5, torch.int8), v=t(5, torch.uint8), m_scale=t(1), v_scale=t(1, torch.float64))):
        with pytest.raises(TypeError):
            G.adamw_tensor(**{**dict(param=t(5), grad=t(5), m=t(5), v=t(5)), **bad})


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
from tests import test_abi_training as t
for name in sorted(dir(t)):
    if name.startswith("test_") and "asan" not in name:
        getattr(t, name)()
print("asan-child-ok")
"""


def test_training_clean_under_asan(asan_lib):  # noqa: F811
    lib, rt = asan_lib
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt
    env["ASAN_OPTIONS"] = "detect_leaks=0:verify_asan_link_order=0:abort_on_error=0"
    env["HIP_VISIBLE_DEVICES"] = ""
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, lib=lib)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert "ERROR: AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0 and "asan-child-ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
