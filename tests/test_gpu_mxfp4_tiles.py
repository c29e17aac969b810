"""The 256 x 256 tiles of the MXFP4 products: several tiles per workgroup, whose
K-tiles are one stream over them.  Tolerances as in test_gpu_mxfp4."""
import numpy as np
import pytest

from tests.test_gpu_mxfp4 import G, _check, _operands, _product  # noqa: F401  (G: the fixture)

pytestmark = pytest.mark.gpu

# m-tiles of up to 128 rows and of more in turn, which store different numbers of rows; groups without rows; N that
# ends inside a tile, so that some waves store nothing
STREAM = [300, 100, 5, 513, 0, 128, 129, 700, 1, 257]


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("N", [704, 832])
@pytest.mark.parametrize("K", [32, 256, 384, 544, 1056])
def test_tiles_in_a_stream_repeat_their_bits(G, a, N, K):  # noqa: F811
    """One round of K-tiles or several behind the last tile's stores; the same bits in every run, with other values
    in the outputs and other work before."""
    import torch
    rng = np.random.default_rng(N + K)
    M = sum(STREAM)
    ops = _operands(rng, M, K, len(STREAM), N, a)
    first = None
    for i in range(6):
        junk = torch.full(((1 + i) << 20,), i, device="cuda")
        got = _product(G, STREAM, M, K, N, a, ops, cu_margin=250 if i < 4 else 253, scale_shift=i % 4)
        junk += 1
        if first is None:
            first = got
            _check(got, STREAM, M, ops[4], ops[5], a)
        assert np.array_equal(got, first), i
