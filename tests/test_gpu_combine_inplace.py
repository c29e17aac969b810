"""The combine onto its residual in place: the same bits as into another
buffer, also where a workgroup takes several tokens and where a row has more
columns than one workgroup."""
import pytest

from tests.test_gpu_router import G  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,H", [((1 << 20) + 37, 2, 8), ((1 << 21) + 1, 1, 16), (3, 16, 8200), (700, 5, 2056)])
def test_combine_in_place(G, T, k, H):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    M = 1000
    y = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    dst = torch.randint(-3, M + 3, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(T, k, generator=g, device="cuda")
    res = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    out = torch.empty_like(res)
    G.moe_combine(y, M, H, dst, T, k, out, weights=w, residual=res)
    assert not torch.equal(out, res)
    G.moe_combine(y, M, H, dst, T, k, res, weights=w, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(out, res)
