"""One to four tokens against 8-bit weights: the sum is an exact 32-bit integer for
every K, rounded once to FP32, and no workspace is needed.  K on both sides of
what shared memory holds of four tokens', two tokens' and one token's codes."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def operands(M, N, K, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    # mostly of one sign, so that sums pass 2^24 many times over
    x = torch.randint(60, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-20, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    x[:, 0] = 127
    return x, w


@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("K", [13312, 13313, 14336, 26640, 28672, 53249, 57344, 57345, 114688, 114689, 131071])
@pytest.mark.parametrize("quantised", [True, False])
def test_sums_are_exact_for_every_k(sg, M, K, quantised):
    import torch
    N = 70
    x, w = operands(M, N, K, M + K)
    sums = x.double() @ w.double().T                 # whole numbers below 2^53: exact
    assert float(sums.abs().max()) > 2 ** 25
    lib, stream = sg.load(), torch.cuda.current_stream().cuda_stream
    out = torch.full((M, N + 1), 7.0, device="cuda")
    one = torch.ones(N, device="cuda")
    assert lib.sgemm_i8_workspace_size(M, N, K, w.data_ptr(), K) == 0
    assert lib.sgemm_linear_i8_workspace_size(M, N, K, w.data_ptr(), K) == 0
    if quantised:
        status = lib.sgemm_i8(M, N, K, x.data_ptr(), K, one.data_ptr(), w.data_ptr(), K, one.data_ptr(), 0, out.data_ptr(),
                              N + 1, 0, 0, 0, stream)
    else:
        # whole numbers up to 127 are their own codes, with a scale of 1
        v = x.to(torch.bfloat16)
        status = lib.sgemm_linear_i8(M, N, K, 1, v.data_ptr(), K, w.data_ptr(), K, one.data_ptr(), 0, out.data_ptr(),
                                     N + 1, 0, 0, 0, stream)
    assert status == sg.SGEMM_OK
    assert torch.equal(out[:, :N], sums.float())
    assert bool((out[:, N] == 7).all())


@pytest.mark.parametrize("M,K", [(4, 57360), (3, 114704), (2, 114704), (4, 131040)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_tokens_that_take_turns(sg, M, K, dtype):
    """Rows with scales of their own, strides and every output type, where not all tokens fit at once."""
    import torch
    dt = getattr(torch, dtype)
    N = 33
    g = torch.Generator(device="cuda").manual_seed(K)
    buf = torch.full((M, K + 8), float("nan"), device="cuda", dtype=dt)
    x = buf[:, :K]
    x.copy_(torch.randn(M, K, generator=g, device="cuda") * torch.tensor([1.0, 8.0, 0.25, 3.0], device="cuda")[:M, None])
    _, w = operands(1, N, K, 3)
    ws = 0.01 + torch.rand(N, generator=g, device="cuda")
    bias = torch.randn(N, generator=g, device="cuda")
    got = sg.linear_i8(x, w, ws, bias)
    assert got.dtype is dt
    q, s = sg.quantize_i8(x)
    assert torch.equal(sg.matmul_i8(q, s, w, ws, bias, out_dtype=dt), got)
    for m in range(M):                               # a token alone has the same bits
        assert torch.equal(sg.linear_i8(x[m:m + 1], w, ws, bias), got[m:m + 1])


@pytest.mark.parametrize("M", [1, 4, 40])
def test_empty_sums_whatever_the_scales(sg, M):
    import torch
    N = 9
    bias = torch.randn(N, device="cuda")
    bad = torch.tensor([float("nan"), float("inf"), 1.0] * 3, device="cuda")
    a, b = torch.empty(M, 0, dtype=torch.int8, device="cuda"), torch.empty(N, 0, dtype=torch.int8, device="cuda")
    nan = torch.full((M,), float("nan"), device="cuda")
    lib = sg.load()
    assert lib.sgemm_i8_workspace_size(M, N, 0, 0, 1) == 0 and lib.sgemm_linear_i8_workspace_size(M, N, 0, 0, 1) == 0
    assert bool((sg.matmul_i8(a, nan, b, bad, bias) == bias).all())
    assert bool((sg.matmul_i8(a, nan, b, bad) == 0).all())
    assert bool((sg.linear_i8(torch.empty(M, 0, device="cuda"), b, bad, bias) == bias).all())
    assert bool((sg.linear_i8(torch.empty(M, 0, device="cuda", dtype=torch.bfloat16), b, bad) == 0).all())
