"""4-bit products whose blocks' powers of two leave FP32 when they are multiplied with each other,
though the products of the numbers that they scale do not."""

import numpy as np
import pytest

from test_fp4_gpu import check, sg  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

TOKENS = [1, 2, 40, 300]


def both(sg, x, w):
    """The product of quantised rows, and of rows that the layer quantises."""
    a, b = sg.quantize_fp4(x, 32), sg.quantize_fp4(w, 32)
    return a, b, (sg.matmul_fp4(*a, *b), sg.linear_fp4(x, *b))


@pytest.mark.parametrize("M", TOKENS)
def test_scales_that_meet_only_zeros(sg, M):
    """Scales of 2^68 in the same block of x and w, whose columns are not the same: the sum there is 0."""
    import torch
    x, w = torch.zeros(M, 256, device="cuda"), torch.zeros(256, 256, device="cuda")
    x[:, 0], w[:, 1] = 2.0 ** 70, 2.0 ** 70
    x[:, 40], w[:, 40] = 3.0, 2.0
    for got in both(sg, x, w)[2]:
        assert bool((got == 6.0).all())


@pytest.mark.parametrize("M", TOKENS)
def test_a_product_of_scales_beyond_the_largest_number(sg, M):
    """Codes of 0.5 under scales of 2^64: 0.25 times 2^128."""
    import torch
    x, w = torch.zeros(M, 64, device="cuda"), torch.zeros(130, 64, device="cuda")
    x[:, 0], x[:, 1] = 6 * 2.0 ** 64, 0.5 * 2.0 ** 64
    w[:, 2], w[:, 1] = 6 * 2.0 ** 64, 0.5 * 2.0 ** 64
    for got in both(sg, x, w)[2]:
        assert bool((got == 2.0 ** 126).all())
    w[:, 1] = 2.0 ** 65                                   # four times as much is too large
    for got in both(sg, x, w)[2]:
        assert bool((got == float("inf")).all())


@pytest.mark.parametrize("M", TOKENS)
def test_a_product_of_scales_below_the_smallest_number(sg, M):
    """2^-69 times 2^-68 is 2^-137, a number that FP32 still holds exactly."""
    import torch
    x, w = torch.zeros(M, 64, device="cuda"), torch.zeros(130, 64, device="cuda")
    x[:, 33], w[:, 33] = 2.0 ** -69, 2.0 ** -68
    for got in both(sg, x, w)[2]:
        assert bool((got == 2.0 ** -137).all())


@pytest.mark.parametrize("up,down", [(120, -110), (-120, 124), (90, 20), (-127, 127)])
@pytest.mark.parametrize("M,N,K", [(1, 300, 1130), (3, 130, 520)])
def test_large_and_small_rows(sg, M, N, K, up, down):
    import torch
    g = torch.Generator(device="cuda").manual_seed(K)
    # (numbers of magnitude up to 1, so that those times 2^up and 2^down are finite)
    x = (2 * torch.rand(M, K, generator=g, device="cuda", dtype=torch.float64) - 1) * 2.0 ** up
    w = (2 * torch.rand(N, K, generator=g, device="cuda", dtype=torch.float64) - 1) * 2.0 ** down
    a, b, got = both(sg, x.float(), w.float())
    for c in got:
        assert np.isfinite(c.cpu().numpy()).all()
        check(c, a, b, K, 32, None, "f32")
