"""What the second product of an adapter takes of u and w: 2^-17 of the value.

Rows are made so that nothing else hides it.  v is any fp32 value of [1, 2), the
exact sum of its bf16 parts v1 + v2 + v3 (cut from the top, 8 bits each).  u_0 = v
from three products in different places of K, u_1 = -v2, the rows of B are (1, 1,
0, ..) and base is -v1: y is v3 and what the product takes of u_0 is off by.  Up to
four terms are not 0, each added with a rounding of 2^-24 of v or less, 8 of them at
most (of u_1, a bf16 value, nothing is lost); y's own rounding is half a bf16 step,
2^-8 of it."""
import numpy as np
import pytest

from oracle import formats as F
from tests.gpu_util import dev_bits, empty_bits, host_bits
from tests.test_gpu_lora import G, workspace  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# rows, groups, r, K, N: one launch, two of 16-row tiles, two of larger tiles
SIZES = [(40, 2, 8, 136, 72), (60, 3, 32, 520, 264), (50, 4, 40, 264, 72), (30, 2, 128, 136, 72),
         (60, 3, 16, 8200, 136), (60, 3, 32, 4104, 136), (33, 2, 64, 2056, 72), (40, 2, 128, 1032, 72),
         (4100, 3, 8, 136, 72), (300, 2, 32, 4104, 136), (300, 2, 64, 2056, 72), (1100, 2, 128, 136, 72)]


def parts(v):
    """bf16 bits of the three parts of fp32 values, and their values."""
    out, rest = [], v.astype(np.float32)
    for _ in range(3):
        b = (rest.view(np.uint32) >> 16).astype(np.uint16)
        out.append(b)
        rest = (rest - (b.astype(np.uint32) << 16).view(np.float32)).astype(np.float32)
    assert not rest.any()
    return out, [F.bf16_bits_to_f64(b) for b in out]


def values(rng, n):
    """fp32 values of [1, 2): the sums that lie in the middle between two parts' steps, then any."""
    v = (1 + rng.integers(0, 1 << 23, n) * 2.0 ** -23).astype(np.float32)
    v[:4] = [1 + 2.0 ** -8 + 2.0 ** -16, 1 + 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -7 - 2.0 ** -17]
    return v


def even_groups(M, L):
    return [M // L + (i < M % L) for i in range(L)]


def check(got, v, p, what):
    err = np.abs(got - p[2][:, None])
    tol = (2.0 ** -17 + 8 * U) * v.astype(np.float64) + 2.0 ** -8 * np.abs(p[2])
    bad = ~(err <= tol[:, None])
    assert not bad.any(), (what, int(bad.any(1).sum()), float((err / v.astype(np.float64)[:, None]).max() * 2 ** 17))


@pytest.mark.parametrize("M,L,r,K,N", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
def test_forward(G, M, L, r, K, N, sign):  # noqa: F811
    import torch
    v = values(np.random.default_rng(M + r), M) * np.float32(sign)
    bits, p = parts(v)
    at = [3, K // 2, K - 2]
    x, A, B = np.zeros((M, K), np.uint16), np.zeros((L, r, K), np.uint16), np.zeros((L, N, r), np.uint16)
    for i in range(3):
        x[:, at[i]] = bits[i]
        A[:, 0, at[i]] = 0x3F80
    A[:, 1, at[1]] = 0xBF80
    B[:, :, 0] = B[:, :, 1] = 0x3F80
    base = np.broadcast_to((bits[0] ^ 0x8000)[:, None], (M, N))
    y, u = empty_bits((M, N)), torch.zeros(M, r, device="cuda")
    grp = G.groups(torch.tensor(even_groups(M, L), dtype=torch.int32, device="cuda"), M)
    G.moe_lora_fwd(dev_bits(x), M, grp, G.lora(dev_bits(A), dev_bits(B), r, K, N), y, base=dev_bits(base), u=u,
                   workspace=workspace(G.moe_lora_fwd_workspace_bytes(M, L, r, K, N)))
    torch.cuda.synchronize()
    assert np.array_equal(u[:, 0].cpu().numpy(), v)
    check(F.bf16_bits_to_f64(host_bits(y)), np.abs(v), p, "y")


@pytest.mark.parametrize("M,L,r,N,K", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
def test_backward(G, M, L, r, K, N, sign):  # noqa: F811
    """w from dy and B, dx from w and A: the same with the weights the other way round."""
    import torch
    v = values(np.random.default_rng(M + r + 1), M) * np.float32(sign)
    bits, p = parts(v)
    at = [5, N // 2, N - 3]
    dy, A, B = np.zeros((M, N), np.uint16), np.zeros((L, r, K), np.uint16), np.zeros((L, N, r), np.uint16)
    for i in range(3):
        dy[:, at[i]] = bits[i]
        B[:, at[i], 0] = 0x3F80
    B[:, at[1], 1] = 0xBF80
    A[:, 0] = A[:, 1] = 0x3F80
    base = np.broadcast_to((bits[0] ^ 0x8000)[:, None], (M, K))
    dx = empty_bits((M, K))
    grp = G.groups(torch.tensor(even_groups(M, L), dtype=torch.int32, device="cuda"), M)
    G.moe_lora_bwd(dev_bits(dy), None, M, grp, G.lora(dev_bits(A), dev_bits(B), r, K, N), None, dx=dx, dx_base=dev_bits(base),
                   workspace=workspace(G.moe_lora_bwd_workspace_bytes(M, L, r, K, N)))
    torch.cuda.synchronize()
    check(F.bf16_bits_to_f64(host_bits(dx)), np.abs(v), p, "dx")


@pytest.mark.parametrize("M,L,r,K,N", [SIZES[0], SIZES[5], SIZES[8], SIZES[10]])
def test_largest_values(G, M, L, r, K, N):  # noqa: F811
    """u up to fp32's largest value stays finite: a part that rounded up to infinity would not."""
    import torch
    top = np.float64(np.finfo(np.float32).max)
    u0 = np.array([top, 2.0 ** 128 * (1 - 2.0 ** -9), 2.0 ** 128 * (1 - 2.0 ** -9 - 2.0 ** -24), 2.0 ** 128 * (1 - 2.0 ** -8), -top, 2.0 ** 127])
    v = np.resize(u0, M).astype(np.float32)
    bits, _ = parts(v)
    at = [3, K // 2, K - 2]
    x, A, B = np.zeros((M, K), np.uint16), np.zeros((L, r, K), np.uint16), np.zeros((L, N, r), np.uint16)
    for i in range(3):
        x[:, at[i]] = bits[i]
        A[:, 0, at[i]] = 0x3F80
    B[:, :, 0] = 0x3F00                                         # a half
    y, u = empty_bits((M, N)), torch.zeros(M, r, device="cuda")
    grp = G.groups(torch.tensor(even_groups(M, L), dtype=torch.int32, device="cuda"), M)
    G.moe_lora_fwd(dev_bits(x), M, grp, G.lora(dev_bits(A), dev_bits(B), r, K, N), y, u=u,
                   workspace=workspace(G.moe_lora_fwd_workspace_bytes(M, L, r, K, N)))
    torch.cuda.synchronize()
    assert np.array_equal(u[:, 0].cpu().numpy(), v)
    want = v.astype(np.float64)[:, None] / 2
    err = np.abs(F.bf16_bits_to_f64(host_bits(y)) - want)
    assert np.all(err <= (2.0 ** -8 + 2.0 ** -17 + 8 * U) * np.abs(want))
