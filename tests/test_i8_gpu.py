"""Rows quantised to 8 bits, and the product of 8-bit operands with its scales.

The codes are defined to the bit by FP32 operations (numpy repeats them).  The
integer sums are compared as whole numbers: exact while partial sums stay below
2^24, and within the library's bound 2 K u sum |a||b| beyond.  The scales and
the bias then add three roundings: 4 u (|v| + |bias|), and the output type's."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_UNIT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def codes(x):
    """The definition in numpy's FP32: scale and codes of the rows of x."""
    x = x.astype(np.float32)
    top = np.abs(x).max(1, initial=0).astype(np.float32)
    safe = np.where(top > 0, top, np.float32(1))
    inv = np.float32(127) / safe
    q = np.rint(x * inv[:, None])
    return np.where(top[:, None] > 0, np.clip(q, -127, 127), 0).astype(np.int8), top / np.float32(127)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,pad,offset", [(1, 1, 0, 0), (3, 5, 0, 1), (1, 4096, 0, 0), (130, 512, 8, 8), (9, 1111, 0, 0),
                                            (2, 16384, 0, 0), (2, 16392, 0, 0), (70, 264, 3, 1), (2000, 64, 0, 0)])
def test_codes_are_defined_to_the_bit(sg, M, K, pad, offset, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K)
    buf = torch.full((M * (K + pad) + offset,), float("nan"), dtype=td(dtype), device="cuda")
    x = buf[offset:].view(M, K + pad)[:, :K]
    x.copy_(torch.randn(M, K, generator=g, device="cuda") * torch.exp(3 * torch.randn(M, 1, generator=g, device="cuda")))
    if M > 1:
        x[1] = 0
    q, s = sg.quantize_i8(x)
    want_q, want_s = codes(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s)


def test_codes_of_extreme_rows(sg):
    import torch
    x = torch.zeros(6, 64, device="cuda")
    x[0, 3], x[0, 5] = 1e-44, -5e-45          # below the smallest normal number
    x[1, 3], x[1, 5] = 3.4e38, -1.7e38
    x[2, 3] = float("inf")
    x[3, 3] = float("nan")
    x[4, 3], x[4, 4] = float("-inf"), float("nan")
    q, s = sg.quantize_i8(x)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert q[0, 3] == 127 and q[0, 5] in (-64, -63, -73, -72, -71)   # 5e-45 is 4 steps of 2^-149, 1e-44 is 7
    assert q[1, 3] == 127 and q[1, 5] in (-64, -63)
    assert np.isinf(s[2]) and np.isnan(s[3]) and np.isnan(s[4]) and s[5] == 0
    assert not q[2:].any()


def operands(M, N, K, seed, low=-127, high=128, pad_a=0, pad_b=0, off=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def view(rows, cols, pad):
        buf = torch.randint(-128, 128, (rows * (cols + pad) + off,), generator=g, device="cuda", dtype=torch.int8)
        v = buf[off:].view(rows, cols + pad)[:, :cols]
        v.copy_(torch.randint(low, high, (rows, cols), generator=g, device="cuda", dtype=torch.int8))
        return v
    a, b = view(M, K, pad_a), view(N, K, pad_b)
    sa = 0.01 + torch.rand(M, generator=g, device="cuda")
    sb = 0.01 + torch.rand(N, generator=g, device="cuda")
    bias = torch.randn(N, generator=g, device="cuda") * 100
    return a, b, sa, sb, bias


def check(got, a, b, sa, sb, bias, out):
    A, B = a.cpu().numpy().astype(np.float64), b.cpu().numpy().astype(np.float64)
    sums = A @ B.T                                   # whole numbers below 2^53: exact
    size = np.abs(A) @ np.abs(B).T
    K = A.shape[1]
    slack = np.where(size < 2 ** 24, 0, 2 * K * U * size)
    s = np.outer(sa.double().cpu().numpy(), sb.double().cpu().numpy())
    extra = np.abs(bias.double().cpu().numpy()) if bias is not None else 0
    want = sums * s + (bias.double().cpu().numpy() if bias is not None else 0)
    tol = slack * s + 4 * U * (np.abs(sums * s) + extra) + HALF_UNIT[out] * np.abs(want) * (1 + 2.0 ** -7)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst {(err / np.maximum(tol, 1e-300)).max():.3g} of the bound"


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 4096), (2, 129, 300), (3, 4, 5), (5, 257, 1024), (8, 512, 8192), (9, 130, 77),
          (15, 96, 2048), (16, 1024, 4096), (17, 200, 1040), (24, 384, 4096), (31, 65, 129), (33, 300, 640), (64, 256, 512),
          (65, 130, 2047), (127, 257, 100), (128, 512, 1024), (129, 1025, 513), (200, 136, 8192), (256, 256, 256),
          (257, 129, 1033), (300, 4999, 64), (513, 640, 2048), (1030, 260, 530)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product(sg, M, N, K, out):
    a, b, sa, sb, bias = operands(M, N, K, seed=M + N + K)
    use_bias = bias if (M + N) % 2 else None
    got = sg.matmul_i8(a, sa, b, sb, use_bias, out_dtype=td(out))
    check(got, a, b, sa, sb, use_bias, out)


@pytest.mark.parametrize("M", [1, 4, 20, 140, 300])
@pytest.mark.parametrize("pad_a,pad_b,off", [(1, 0, 0), (0, 3, 0), (16, 16, 16), (5, 11, 1), (0, 0, 8), (4, 4, 4)])
def test_strides_and_alignment(sg, M, pad_a, pad_b, off):
    import torch
    N, K = 210, 530
    a, b, sa, sb, bias = operands(M, N, K, 3, pad_a=pad_a, pad_b=pad_b, off=off)
    buf = torch.full((M, N + 3), 5.0, device="cuda", dtype=torch.float16)
    got = sg.matmul_i8(a, sa, b, sb, bias * 0, out=buf[:, :N].zero_())
    want = sg.matmul_i8(a.contiguous(), sa, b.contiguous(), sb, bias * 0, out_dtype=torch.float16)
    assert bool((got == want).all()) and bool((buf[:, N:] == 5.0).all())


@pytest.mark.parametrize("M", [1, 7, 16, 40, 150, 600])
def test_extreme_codes_and_a_long_sum(sg, M):
    import torch
    # every product 127 * 127 or 128 * 128: the sum passes 2^24
    N, K = 70, 5000
    for va, vb in ((127, 127), (-128, -128), (-128, 127)):
        a = torch.full((M, K), va, dtype=torch.int8, device="cuda")
        b = torch.full((N, K), vb, dtype=torch.int8, device="cuda")
        one_m, one_n = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        check(sg.matmul_i8(a, one_m, b, one_n), a, b, one_m, one_n, None, "f32")


@pytest.mark.parametrize("M", [1, 5, 33, 200])
def test_a_scale_that_is_not_finite_stays_in_its_row(sg, M):
    import torch
    a, b, sa, sb, _ = operands(M, 100, 256, 8)
    sa[0] = float("nan")
    got = sg.matmul_i8(a, sa, b, sb)
    assert bool(torch.isnan(got[0]).all()) and bool(torch.isfinite(got[1:]).all())


def test_empty_sums(sg):
    import torch
    a, b = torch.empty(3, 0, dtype=torch.int8, device="cuda"), torch.empty(5, 0, dtype=torch.int8, device="cuda")
    bias = torch.randn(5, device="cuda")
    got = sg.matmul_i8(a, torch.ones(3, device="cuda"), b, torch.ones(5, device="cuda"), bias)
    assert bool((got == bias).all())
    got = sg.linear_i8(torch.empty(3, 0, device="cuda"), b, torch.ones(5, device="cuda"))
    assert bool((got == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (1, 130, 1111), (6, 200, 512), (24, 260, 1000), (130, 300, 768),
                                   (400, 512, 2048)])
def test_linear_is_quantise_and_product(sg, M, N, K, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, generator=g, device="cuda").to(td(dtype))
    w, ws = sg.quantize_i8(0.05 * torch.randn(N, K, generator=g, device="cuda"))
    bias = torch.randn(N, generator=g, device="cuda")
    got = sg.linear_i8(x, w, ws, bias)
    assert got.dtype == td(dtype)
    q, s = codes(x.float().cpu().numpy())
    check(got, torch.from_numpy(q), w, torch.from_numpy(s), ws, bias, dtype)


def test_another_stream_a_graph_and_the_same_bits(sg):
    import torch
    for M in (1, 20, 300):
        x = torch.randn(M, 1024, device="cuda").to(torch.bfloat16)
        w, ws = sg.quantize_i8(torch.randn(520, 1024, device="cuda"))
        want = sg.linear_i8(x, w, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = sg.linear_i8(x, w, ws, stream=side)
        side.synchronize()
        assert bool((got == want).all())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = sg.linear_i8(x, w, ws)
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        assert bool((out == -want).all())
    assert sg.sgemm_device_status() == sg.SGEMM_OK


def test_python_refusals(sg):
    import torch
    a, b, sa, sb, bias = operands(4, 6, 64, 1)
    with pytest.raises(TypeError):
        sg.matmul_i8(a.float(), sa, b, sb)
    with pytest.raises(ValueError):
        sg.matmul_i8(a, sa, b[:, :32].contiguous(), sb)
    with pytest.raises(ValueError):
        sg.matmul_i8(a, sa[:3], b, sb)
    with pytest.raises(TypeError):
        sg.matmul_i8(a, sa.double(), b, sb)
    with pytest.raises(ValueError):
        sg.matmul_i8(a, sa, b, sb, out=torch.empty(4, 5, device="cuda"))
    with pytest.raises(TypeError):
        sg.linear_i8(a, b, sb)
    with pytest.raises(sg.SgemmError):
        sg.linear_i8(torch.randn(40, 64, device="cuda"), b, sb, workspace=torch.empty(16, device="cuda"))


@pytest.mark.parametrize("M,N,K", [(40, 4096, 512), (40, 130, 8192), (300, 520, 4096)])
def test_a_wait_that_runs_out_is_reported(sg, M, N, K):
    import torch
    a, b, sa, sb, _ = operands(M, N, K, 12)
    want = sg.matmul_i8(a, sa, b, sb)
    out = torch.full((M, N), 3.0, device="cuda")
    sg.sgemm_test_switches(1, 50_000_000)     # no copies: every wait runs out after 50 ms
    try:
        sg.matmul_i8(a, sa, b, sb, out=out)
        assert sg.sgemm_device_status() == sg.SGEMM_ERR_TIMEOUT
    finally:
        sg.sgemm_test_switches(0)
    # nothing was stored, or (with the sums over k divided) NaN
    assert bool(((out == 3.0) | torch.isnan(out)).all())
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert bool((sg.matmul_i8(a, sa, b, sb) == want).all())


@pytest.mark.parametrize("M", [5, 24, 100, 200])
def test_many_steps_wrap_the_rings(sg, M):
    # every tile of B on one SM over a long k: each ring of stages is walked many times
    N, K = 4096, 16384
    a, b, sa, sb, bias = operands(M, N, K, M)
    got = sg.matmul_i8(a, sa, b, sb, bias)
    rows = slice(0, 3)
    check(got[rows], a[rows], b, sa[rows], sb, bias, "f32")
    again = sg.matmul_i8(a, sa, b, sb, bias)
    assert bool((got == again).all())
