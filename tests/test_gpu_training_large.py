"""Adapters and the AdamW step past 2^31 elements and 2^32 bytes: sampled rows and
elements against the float64 oracle, with the tolerances of their own tests."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import training as P
from tests.gpu_util import dev_bits, host_bits
from tests.test_gpu_lora import G, TINY, U, bits  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _u16(t):
    import torch
    return host_bits(t.view(torch.int16))


def test_lora_rows_past_4_gib(G):  # noqa: F811
    """310000 rows of 7168, as given and named by src; gradients too."""
    import torch
    T, K, N, r, E = 310000, 7168, 64, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dy = torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    rng = np.random.default_rng(1)
    A, B = bits(rng, E, r, K, std=K ** -0.5), bits(rng, E, N, r, std=r ** -0.5)
    counts = torch.tensor([100000, 5, 209990], dtype=torch.int32, device="cuda")
    grp, lo = G.groups(counts, T), G.lora(dev_bits(A), dev_bits(B), r, K, N)
    src = torch.randperm(T, generator=gen, device="cuda").int()
    ws = torch.empty(max(G.moe_lora_fwd_workspace_bytes(T, E, r, K, N), G.moe_lora_bwd_workspace_bytes(T, E, r, K, N)),
                     dtype=torch.uint8, device="cuda")
    y, u = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, r, device="cuda")
    dx = torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.empty(E, r, K, device="cuda"), torch.empty(E, N, r, device="cuda")
    for s in (None, src):
        dx.fill_(7.0)
        G.moe_lora_fwd(x, T, grp, lo, y, src=s, u=u, workspace=ws)
        G.moe_lora_bwd(dy, x, T, grp, lo, u, dx=dx, dA=dA, dB=dB, src=s, workspace=ws)
        torch.cuda.synchronize()
        g = np.array([0, 1, 63, 99999, 100000, 100004, 100005, 299590, 299593, 305000, 309994])   # grouped rows
        e = np.where(g < 100000, 0, np.where(g < 100005, 1, 2))
        rows = torch.from_numpy(g).cuda() if s is None else s[torch.from_numpy(g).cuda()].long()
        xs, ds = F.bf16_bits_to_f64(_u16(x[rows])), F.bf16_bits_to_f64(_u16(dy[rows]))
        a, b = F.bf16_bits_to_f64(A)[e], F.bf16_bits_to_f64(B)[e]
        low = np.einsum("gk,grk->gr", xs, a)
        tol_u = (K + 8) * U * np.einsum("gk,grk->gr", np.abs(xs), np.abs(a))
        assert np.all(np.abs(u[torch.from_numpy(g).cuda()].cpu().numpy() - low) <= tol_u)
        want = np.einsum("gr,gnr->gn", low, b)
        tol = np.einsum("gr,gnr->gn", tol_u + 2.0 ** -16 * np.abs(low), np.abs(b)) + 2.0 ** -8 * 1.01 * np.abs(want) + TINY
        assert np.all(np.abs(F.bf16_bits_to_f64(_u16(y[rows])) - want) <= tol)
        back = np.einsum("gn,gnr->gr", ds, b)
        tol_w = (N + 8) * U * np.einsum("gn,gnr->gr", np.abs(ds), np.abs(b))
        want = np.einsum("gr,grk->gk", back, a)
        tol = np.einsum("gr,grk->gk", tol_w + 2.0 ** -16 * np.abs(back), np.abs(a)) + 2.0 ** -8 * 1.01 * np.abs(want) + TINY
        assert np.all(np.abs(F.bf16_bits_to_f64(_u16(dx[rows])) - want) <= tol)
        untouched = torch.arange(309995, T, device="cuda") if s is None else s[309995:].long()
        assert torch.all(dx[untouched] == 7)
        # the gradients of the second group's five rows, whole
        i = torch.arange(100000, 100005, device="cuda")
        at = i if s is None else s[i].long()
        xs, ds = F.bf16_bits_to_f64(_u16(x[at])), F.bf16_bits_to_f64(_u16(dy[at]))
        u5, b1 = u[i].cpu().numpy().astype(np.float64), F.bf16_bits_to_f64(B)[1]
        w = ds @ b1
        off = (N + 40) * U * (np.abs(ds) @ np.abs(b1)).T @ np.abs(xs)
        assert np.all(np.abs(dA[1].cpu().numpy() - w.T @ xs) <= off + TINY)
        assert np.all(np.abs(dB[1].cpu().numpy() - ds.T @ u5) <= 40 * U * np.abs(ds.T) @ np.abs(u5) + TINY)
        # the largest group's, by a 64-bit product on the GPU over a slice of the columns
        c = slice(7000, 7168)
        rows2 = torch.arange(100005, 309995, device="cuda")
        at = rows2 if s is None else s[rows2].long()
        w = dy[at].double() @ torch.from_numpy(F.bf16_bits_to_f64(B)[2]).cuda()
        want = w.t() @ x[at][:, c].double()
        mag = w.abs().t() @ x[at][:, c].double().abs()
        # a path adds 2048 rows of a piece in three parts and 103 pieces, and w is off by 72 U of 64 terms' sizes
        wmag = (dy[at].double().abs() @ torch.from_numpy(np.abs(F.bf16_bits_to_f64(B)[2])).cuda()).t() @ x[at][:, c].double().abs()
        assert torch.all((dA[2][:, c].double() - want).abs() <= (3 * 2048 + 128) * U * mag + (N + 8) * U * wmag)


def test_lora_row_distance_past_2_31(G):  # noqa: F811
    import torch
    K, N, r, ld = 64, 72, 8, (1 << 30) + 8
    T = 3
    rng = np.random.default_rng(2)
    x, base, A, B = bits(rng, T, K), bits(rng, T, N), bits(rng, 1, r, K), bits(rng, 1, N, r)
    xd = torch.zeros(ld * 2 + K, dtype=torch.bfloat16, device="cuda")
    yd = torch.zeros(ld * 2 + N, dtype=torch.bfloat16, device="cuda")
    for i in range(T):
        xd[i * ld:i * ld + K] = dev_bits(x[i]).view(torch.bfloat16)
        yd[i * ld:i * ld + N] = dev_bits(base[i]).view(torch.bfloat16)
    counts = torch.tensor([T], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, G.moe_lora_fwd_workspace_bytes(T, 1, r, K, N)), dtype=torch.uint8, device="cuda")
    G.moe_lora_fwd(xd, T, G.groups(counts, T), G.lora(dev_bits(A), dev_bits(B), r, K, N, x_ld=ld, y_ld=ld), yd, base=yd, workspace=ws)
    torch.cuda.synchronize()
    _, want = P.lora_fwd(x, A, B, None, [T], T, None, base)
    _, mag = P.lora_fwd(x & 0x7FFF, A & 0x7FFF, B & 0x7FFF, None, [T], T)
    got = np.stack([F.bf16_bits_to_f64(_u16(yd[i * ld:i * ld + N])) for i in range(T)])
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (2.0 ** -17 + 2 * K * U) * mag + TINY)


@pytest.mark.parametrize("bits8", [False, True])
def test_adamw_past_2_31_elements(G, bits8):  # noqa: F811
    """A tensor of 2^31 + 5000 elements behind a small one; elements at its ends and in the middle."""
    import torch
    n = (1 << 31) + 5000
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    if bits8:
        m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
        ms, vs = torch.zeros((n + 127) // 128, device="cuda"), torch.zeros((n + 127) // 128, device="cuda")
    else:
        m, v, ms, vs = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), None, None
    at = torch.tensor([0, 1, 4095, 4096, (1 << 30) + 77, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, n - 130, n - 1], device="cuda")
    g[at] = torch.arange(1, 11, device="cuda").bfloat16()
    small = [torch.ones(10, device="cuda") for _ in range(4)]
    plan = G.adamw_plan([G.adamw_tensor(*small), G.adamw_tensor(p, g, m, v, m_scale=ms, v_scale=vs)])
    out, ws = torch.empty(2, device="cuda"), torch.empty(G.moe_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda")
    G.moe_grad_norm(plan, 1e9, out, ws)
    G.moe_adamw_step(plan, G.adamw(1e-2, eps=0.0, grad_scale=out[1:]))
    torch.cuda.synchronize()
    assert abs(float(out[0]) - np.sqrt(385 + 10)) <= 1e-5 and float(out[1]) == 1
    # the first step moves an element by lr against its gradient's sign; without a gradient 0 / 0
    assert torch.all((p[at].float() + 1e-2).abs() <= 1e-2 * 2.0 ** -7)
    if bits8:
        mo, vo = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        G.moe_adamw_unpack(m, ms, v, vs, n, mo, vo)
        torch.cuda.synchronize()
        m, v = mo, vo
    i = torch.arange(1, 11, device="cuda").double()
    assert torch.all((m[at].double() - 0.1 * i).abs() <= 0.1 * i * (0.02 if bits8 else 1e-6))
    assert torch.all((v[at].double() - 1e-3 * i * i).abs() <= 1e-3 * i * i * (0.04 if bits8 else 1e-6))
    assert int(torch.count_nonzero(m)) == 10 and int(torch.count_nonzero(v)) == 10
