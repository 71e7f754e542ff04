"""The workspace of the products with 8-bit weights, whose size is computed from
the device: it holds what the kernels write, at sizes beyond 32 bits too."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(2 ** 30, 16, 16), (2 ** 30 - 1, 1, 1), (2 ** 29 + 1, 8, 64), (5, 2 ** 30, 17),
                                   (2 ** 20, 2 ** 20, 131071), (5, 3, 1)])
@pytest.mark.parametrize("aligned", [True, False])
def test_sizes(cuda_device, lib, M, N, K, aligned):
    address = 0x7F0000000000 + (0 if aligned else 1)     # never read
    ldb = (K + 15) // 16 * 16
    for size in (lib.sgemm_i8_workspace_size, lib.sgemm_linear_i8_workspace_size):
        got = int(size(M, N, K, address, ldb))
        # a scale and FP16 codes a token, and the rows of B where they are laid out
        least = 4 * M + 2 * M * K + (0 if aligned else N * K)
        assert got >= least
        # rows padded to 16, three parts to 256, and up to 16 sums for each result
        assert got <= 4 * M + 2 * M * (K + 8) + N * ldb + 3 * 256 + 16 * 4 * M * (N + 4)
