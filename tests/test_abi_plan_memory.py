"""moe_adamw_plan allocates nothing: it lays out a step of 400000 tensors, and finds
their overlaps, in a process that may take no more memory.  (CPU only, in a child,
which limits itself.)"""
import subprocess
import sys

from tests.test_abi_asan import ROOT

CHILD = r"""
import ctypes, resource, sys
sys.path.insert(0, {root!r})
import numpy as np
import grouped_gemm_glu_amd as G
n = 400000
F = 1 << 12
size = ctypes.sizeof(G.AdamwTensorT)
one = np.zeros((n, size // 8), dtype=np.uint64)
struct = lambda i: G.AdamwTensorT.from_buffer(one[i])
base = G.AdamwTensorT(0, 0, 0, 0, 0, 0, 0, 1000, 1.0, 0.0, G.DT_BF16, G.DT_BF16, 8)
one[:] = np.frombuffer(bytes(base), dtype=np.uint64)
order = np.random.default_rng(1).permutation(7 * n).reshape(n, 7).astype(np.uint64)
one[:, :7] = (order + 1) * F                     # seven buffers each, all over the addresses
array = (G.AdamwTensorT * n).from_buffer(one)
need = G._lib.moe_adamw_plan_bytes(array, n)
table, plan = np.zeros(need, dtype=np.uint8), G.AdamwPlanT()
call = lambda: G.raw_call("moe_adamw_plan", array, n, table.ctypes.data, need, ctypes.byref(plan))
now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (1 << 20), now + (1 << 20)))
first = call()
chunks = plan.n_chunks, plan.n_chunks8
one[n - 1, 4] = one[3, 0] + 16                   # a v on another tensor's parameter
print("child", first, chunks, call())
"""


def test_plan_of_many_tensors_allocates_nothing():
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.split("\n")[-2:-1] == ["child 0 (400000, 400000) 4"], (r.stdout[-2000:], r.stderr[-2000:])
