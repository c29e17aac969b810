"""The binding's current stream: torch's, also after it changes, and in a forked
child torch's own refusal, as for every other GPU call there.  CPU only: torch's
functions are stood in for, in a process of its own."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import os, sys
sys.path.insert(0, {root!r})
import torch
import grouped_gemm_glu_amd as G

now = dict(device=0, stream=[111, 222], forked=False)

def init():
    if now["forked"]:
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")
torch.cuda.init = init
torch._C._cuda_getDevice = lambda: now["device"]
torch._C._cuda_getCurrentRawStream = lambda d: now["stream"][d]

assert G._stream(None) == 111 and G._stream(None) == 111
now["stream"][0] = 333
assert G._stream(None) == 333
now["device"] = 1
assert G._stream(None) == 222 and G._stream(5) == 5
pid = os.fork()
if pid == 0:
    now["forked"] = True
    try:
        G._stream(None)
    except RuntimeError as e:
        os._exit(0 if "forked" in str(e) else 3)
    os._exit(4)
assert os.waitpid(pid, 0)[1] == 0, "a forked child was given a stream"
assert G._stream(None) == 222
print("child-ok")
"""


def test_current_stream_and_fork():
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child-ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
