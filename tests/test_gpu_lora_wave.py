"""Values that a wave's lanes hand to one another through LDS without a barrier: every
element of the result says which row and column it came from, so that a read that ran
ahead of its write, or a write ahead of the last read, shows as another's value.

x and dy hold a 1 in one column of each row, A and B rows of whole numbers: u and w are
entries of the weights, y and dx their products, exact in fp32 and bf16; dA and dB name the
rows of their columns."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from tests.gpu_util import dev_bits, empty_bits, host_bits
from tests.test_gpu_lora import G, workspace  # noqa: F401  (the fixture)
from tests.test_gpu_lora_paths import FEW, MB1, MB2, ONE, takes

pytestmark = pytest.mark.gpu

# M, groups, r, K, N, the kernels of the forward pass and of the backward
SIZES = [(37, 2, 16, 1000, 520, ONE, ONE), (50, 3, 32, 2056, 776, ONE, ONE), (40, 1, 128, 1000, 264, ONE, MB1),
         (4100, 3, 16, 520, 776, MB2, MB2), (300, 4, 32, 4104, 4168, MB1, MB1), (300, 2, 32, 4104, 4168, MB2, MB2),
         (300, 4, 64, 2056, 520, MB1, MB1), (2050, 2, 64, 520, 776, MB2, MB2), (300, 4, 128, 1032, 520, MB1, MB1),
         (1100, 2, 128, 520, 264, MB2, MB2), (60, 3, 64, 2056, 520, FEW, MB1)]


def whole(rng, *shape):
    return W.to_bf16_bits(rng.integers(-15, 16, shape).astype(np.float32))


@pytest.mark.parametrize("M,L,r,K,N,fwd,bwd", SIZES)
def test_every_place(G, M, L, r, K, N, fwd, bwd):  # noqa: F811
    import torch
    assert takes(G, M, L, r, K, N)[:2] == (fwd, bwd)
    rng = np.random.default_rng(M + r)
    counts = np.array([M // L + (e < M % L) for e in range(L)])
    group = np.repeat(np.arange(L), counts)
    rows = np.arange(M)
    kx, ny = rng.integers(0, K, M), rng.integers(0, N, M)
    x, dy = np.zeros((M, K), np.uint16), np.zeros((M, N), np.uint16)
    x[rows, kx] = dy[rows, ny] = 0x3F80
    A, B = whole(rng, L, r, K), np.zeros((L, N, r), np.uint16)
    one = rng.integers(0, r, (L, N))                          # y_in = u_i[one[n]], and w_i = a unit vector
    np.put_along_axis(B, one[:, :, None], 0x3F80, axis=2)
    A64 = F.bf16_bits_to_f64(A)
    grp = G.groups(torch.from_numpy(counts.astype(np.int32)).cuda(), M)
    lo = G.lora(dev_bits(A), dev_bits(B), r, K, N)
    y, u = empty_bits((M, N)), torch.zeros(M, r, device="cuda")
    dx, dA, dB = empty_bits((M, K)), torch.empty(L, r, K, device="cuda"), torch.empty(L, N, r, device="cuda")
    ws = workspace(max(G.moe_lora_fwd_workspace_bytes(M, L, r, K, N), G.moe_lora_bwd_workspace_bytes(M, L, r, K, N)))
    G.moe_lora_fwd(dev_bits(x), M, grp, lo, y, u=u, workspace=ws)
    G.moe_lora_bwd(dev_bits(dy), dev_bits(x), M, grp, lo, u, dx=dx, dA=dA, dB=dB, workspace=ws)
    torch.cuda.synchronize()
    want_u = A64[group, :, kx]
    assert np.array_equal(u.cpu().numpy(), want_u)
    assert np.array_equal(F.bf16_bits_to_f64(host_bits(y)), np.take_along_axis(want_u, one[group], axis=1))
    rank = one[group, ny]                                     # w_i is 1 there
    assert np.array_equal(F.bf16_bits_to_f64(host_bits(dx)), A64[group, rank])
    want_a, want_b = np.zeros((L, r, K)), np.zeros((L, N, r))
    np.add.at(want_a, (group, rank, kx), 1.0)
    np.add.at(want_b, (group, ny), want_u)
    assert np.array_equal(dA.cpu().numpy(), want_a) and np.array_equal(dB.cpu().numpy(), want_b)
