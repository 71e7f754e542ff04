"""Rows quantised to 4-bit floating point, and the product of such operands.

Codes and scales are defined to the bit by FP32 operations (numpy repeats them, with
its own roundings to 4 and 8 bits).  The products of codes and block scales are exact,
their sum over K is held to the library's 2 K u sum |a||b|; the rows' scales and the
bias then add three roundings, 4 u (|v| + |bias|), and the output type's."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_UNIT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
# every value of e4m3 up to its largest, 448, by its bits
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def nearest(table, v):
    """Indexes of the nearest entries, of two the even one; values beyond the last go to it."""
    v = np.minimum(v.astype(np.float64), table[-1])
    low = np.clip(np.searchsorted(table, v, side="right") - 1, 0, len(table) - 1)
    high = np.minimum(low + 1, len(table) - 1)
    up, down = table[high] - v, v - table[low]
    return np.where((up < down) | ((up == down) & (low % 2 == 1)), high, low)


def quantized(x, block):
    """(codes, bits of the blocks' scales, rows' scales) of the definition, in FP32 steps."""
    x = x.astype(np.float32)
    M, K = x.shape
    n = -(-K // block)
    b = np.zeros((M, n * block), np.float32)
    b[:, :K] = x
    b = b.reshape(M, n, block)
    with np.errstate(all="ignore"):
        if block == 16:
            top = np.abs(b).max((1, 2))
            pre = np.where(top < 2.0 ** -100, np.float32(2.0 ** 64), np.float32(1))
            t = np.where(top > 0, np.float32(2688) / (top * pre), np.float32(0)).astype(np.float32)
            y = b * pre[:, None, None] * t[:, None, None]
            bits = nearest(E4M3, np.abs(y).max(2) * (np.float32(1) / np.float32(6)))
            s = E4M3[bits].astype(np.float32)
            inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
            v = y * inv[:, :, None]
            rows = top / np.float32(2688)
        else:
            f, e = np.frexp(np.abs(b).max(2))
            e = np.where(f == 0, -127, np.clip(np.where(f <= 0.75, e - 3, e - 2), -127, 127))
            bits, rows = e + 127, None
            v = np.ldexp(b.astype(np.float64), -e[:, :, None])
    code = nearest(LEVELS, np.abs(v)) + 8 * (np.signbit(v))
    return code.reshape(M, -1)[:, :K], bits, rows


def codes_of(q, K):
    q = q.cpu().numpy()
    return np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)[:, :K]


def tile_bytes(s):
    import torch
    return s.view(torch.uint8).cpu().numpy()


def bits_of(s, rows, blocks):
    r, j = np.arange(rows)[:, None], np.arange(blocks)[None]
    return tile_bytes(s)[r // 128, j // 4 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4]


def values_of(q, s, K, block):
    """What codes and block scales stand for, in 64 bits."""
    code = codes_of(q, K)
    bits = bits_of(s, code.shape[0], -(-K // block))
    if block == 16:
        with_nan = np.append(E4M3, np.nan)
        scale = with_nan[np.minimum(bits, 127)]
    else:
        scale = np.where(bits == 255, np.nan, np.ldexp(1.0, bits.astype(np.int64) - 127))
    return LEVELS[code % 8] * np.where(code >= 8, -1.0, 1.0) * np.repeat(scale, block, 1)[:, :K]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,K,pad,offset", [(1, 1, 0, 0), (3, 5, 0, 1), (1, 4096, 0, 0), (130, 512, 8, 8), (9, 1111, 0, 0),
                                            (2, 16384, 0, 0), (2, 16392, 0, 0), (3, 40017, 0, 0), (70, 264, 3, 1),
                                            (2000, 64, 0, 0), (33, 528, 0, 0)])
def test_codes_are_defined_to_the_bit(sg, M, K, pad, offset, block, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K)
    buf = torch.full((M * (K + pad) + offset,), float("nan"), dtype=td(dtype), device="cuda")
    x = buf[offset:].view(M, K + pad)[:, :K]
    x.copy_(torch.randn(M, K, generator=g, device="cuda") * torch.exp(2 * torch.randn(M, 1, generator=g, device="cuda")))
    x[:, :K // 3] *= 2.0 ** -9                  # blocks whose scale is small, or comes out as 0
    if M > 1:
        x[1] = 0
    q, s, rows = sg.quantize_fp4(x, block)
    code, bits, want_rows = quantized(x.float().cpu().numpy(), block)
    got = codes_of(q, K)
    n = -(-K // block)
    assert np.array_equal(bits_of(s, M, n), bits)
    # a zero may carry either sign
    assert np.array_equal(np.where(got == 8, 0, got), np.where(code == 8, 0, code))
    if block == 16:
        assert np.array_equal(rows.cpu().numpy(), want_rows)
    else:
        assert rows is None
    if K % 2:
        assert not (q[:, -1] >> 4).any()
    # nothing but zeros behind the matrix
    assert np.count_nonzero(tile_bytes(s)) == np.count_nonzero(bits)


@pytest.mark.parametrize("block", [16, 32])
def test_halves_go_to_the_even_code(sg, block):
    import torch
    x = torch.zeros(1, 64, device="cuda")
    # 6 as the largest of every block: scales of 448 (times 6 / 2688) and of 1
    x[0] = torch.tensor([6.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]).repeat(4)
    q, _, _ = sg.quantize_fp4(x, block)
    assert codes_of(q, 16)[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 10, 12, 12, 14, 14, 15]


@pytest.mark.parametrize("block", [16, 32])
def test_codes_of_extreme_rows(sg, block):
    import torch
    x = torch.zeros(6, 64, device="cuda")
    x[0, 3], x[0, 5] = 1e-44, -5e-45          # below the smallest normal number
    x[1, 3], x[1, 5] = 3.4e38, -1.7e38
    x[2, 3] = float("inf")
    x[3, 3] = float("nan")
    x[4, 3], x[4, 4] = float("-inf"), float("nan")
    q, s, rows = sg.quantize_fp4(x, block)
    code = codes_of(q, 64)
    # the largest is 6 steps of its scale in the one format; in the other it is 3.997 times 2^126
    assert not code[2:].any() and code[1, 3] == (7 if block == 16 else 6) and not code[:2, 6:].any()
    if block == 16:
        rows = rows.cpu().numpy()
        assert code[0, 3] == 7 and np.isinf(rows[2]) and np.isnan(rows[3]) and np.isnan(rows[4]) and rows[5] == 0
    else:
        # 2^127 is the largest power of two the codes can be scaled by: 1e-44 2^127 is 0
        bits = bits_of(s, 6, 2)
        assert not (code[0] % 8).any() and bits[0].tolist() == [0, 0] and (bits[2:5, 0] == 255).all() and bits[5, 0] == 0
        assert values_of(q, s, 64, 32)[1, 3] == pytest.approx(3.4e38, rel=0.25)


def operands(sg, M, N, K, seed, block, dtype="f32"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(M, 1, generator=g, device="cuda"))).to(td(dtype))
    w = torch.randn(N, K, generator=g, device="cuda")
    return x, sg.quantize_fp4(w, block), torch.randn(N, generator=g, device="cuda") * 10


def check(got, a, w, K, block, bias, out):
    A, B = values_of(a[0], a[1], K, block), values_of(w[0], w[1], K, block)
    s = 1.0
    if block == 16:
        s = np.outer(a[2].double().cpu().numpy(), w[2].double().cpu().numpy())
    extra = bias.double().cpu().numpy() if bias is not None else 0.0
    v, size = A @ B.T * s, np.abs(A) @ np.abs(B).T * s
    want = v + extra
    tol = 2 * K * U * size + 4 * U * (np.abs(v) + np.abs(extra)) + HALF_UNIT[out] * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -126
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound, {np.count_nonzero(~(err <= tol))} of {err.size}"


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 4096), (2, 129, 300), (3, 4, 5), (5, 257, 1024), (8, 512, 8192), (9, 130, 77),
          (15, 96, 2048), (16, 1024, 4096), (17, 200, 1040), (24, 384, 4096), (31, 65, 129), (33, 300, 640), (64, 256, 512),
          (65, 130, 2047), (127, 257, 100), (128, 512, 1024), (129, 1025, 513), (200, 136, 8192), (256, 256, 256),
          (257, 129, 1033), (300, 4999, 64), (513, 640, 2048), (1030, 260, 530), (2050, 4100, 300)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", [16, 32])
def test_product(sg, M, N, K, block):
    out = ["f32", "bf16", "f16"][(M + N + K) % 3]
    x, w, bias = operands(sg, M, N, K, M + N + K, block)
    use_bias = bias if (M + N) % 2 else None
    a = sg.quantize_fp4(x, block)
    got = sg.matmul_fp4(*a, *w, use_bias, out_dtype=td(out))
    check(got, a, w, K, block, use_bias, out)
    # the layer quantises the same codes itself
    assert bool((sg.linear_fp4(x, *w, bias=use_bias, out_dtype=td(out)) == got).all())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", [(1, 4200, 5000), (1, 300, 90112), (1, 128, 90120), (2, 128, 90113),
                                   (20, 512, 8192), (14, 260, 20000), (50, 1000, 3000),
                                   (100, 128, 16384), (64, 4096, 2112), (600, 520, 4096), (1100, 4200, 1000), (700, 9000, 2113),
                                   (2000, 2300, 4160), (257, 20000, 64), (4100, 4000, 40)])
def test_product_of_every_plan(sg, M, N, K, block):
    """One token; few tiles that clusters share; tiles of 64 and 128 tokens; pairs of SMs; K that ends
    inside a step, with one to four products of it."""
    x, w, bias = operands(sg, M, N, K, M + K, block, "bf16")
    a = sg.quantize_fp4(x, block)
    out = "bf16" if (M + N) % 3 else "f32"
    got = sg.matmul_fp4(*a, *w, bias, out_dtype=td(out))
    check(got, a, w, K, block, bias, out)
    assert bool((sg.linear_fp4(x, *w, bias=bias, out_dtype=td(out)) == got).all())
    assert sg.sgemm_device_status() == sg.SGEMM_OK


@pytest.mark.parametrize("M,N", [(3, 5000), (30, 700), (130, 256), (300, 4096), (1500, 4608)])
def test_many_steps_wrap_the_rings(sg, M, N):
    K = 12000
    x, w, _ = operands(sg, M, N, K, 5, 16)
    a = sg.quantize_fp4(x)
    got = sg.matmul_fp4(*a, *w)
    rows = [0, M // 2, M - 1]
    few = (a[0][rows], a[1], a[2][rows])
    A = values_of(a[0], a[1], K, 16)[rows]
    B = values_of(w[0], w[1], K, 16)
    s = np.outer(few[2].double().cpu().numpy(), w[2].double().cpu().numpy())
    err = np.abs(got[rows].double().cpu().numpy() - A @ B.T * s)
    assert (err <= (2 * K * U * (np.abs(A) @ np.abs(B).T) + 4 * U * np.abs(A @ B.T)) * s).all()
    assert bool((sg.matmul_fp4(*a, *w) == got).all())


@pytest.mark.parametrize("M", [1, 7, 60, 200, 1300])
@pytest.mark.parametrize("block", [16, 32])
def test_strides_and_what_lies_around(sg, M, block):
    """Rows of codes further apart than they are long, with anything between them and behind; scales
    of rows behind the matrix that are not numbers; an output inside a wider one."""
    import torch
    N, K = 4300, 1130
    x, w, bias = operands(sg, M, N, K, 3, block)
    a = sg.quantize_fp4(x, block)
    want = sg.matmul_fp4(*a, *w, bias)

    def apart(q, rows):
        big = torch.full((rows + 3, q.shape[1] // 16 * 16 + 80), 0x5D, dtype=torch.uint8, device="cuda")
        big[:rows, :q.shape[1]] = q
        return big[:rows, :q.shape[1]]

    def dirty(s, rows):
        t = s.view(torch.uint8).clone()
        r, j = torch.arange(128, device="cuda")[:, None], torch.arange(t.shape[1] // 128, device="cuda")[None]
        if rows % 128:
            at = (j // 4 * 512 + r % 32 * 16 + r // 32 * 4 + j % 4)[rows % 128:].reshape(-1)
            t[-1, at] = 0x7F if block == 16 else 0xFF
        return t.view(s.dtype)
    out = torch.full((M + 2, N + 7), 5.0, device="cuda")
    got = sg.matmul_fp4(apart(a[0], M), dirty(a[1], M), a[2], apart(w[0], N), dirty(w[1], N), w[2], bias, out=out[1:M + 1, 3:N + 3])
    assert torch.equal(got, want)
    out[1:M + 1, 3:N + 3] = 5.0
    assert bool((out == 5.0).all()), "wrote outside C"


@pytest.mark.parametrize("dtype,offset,pad", [("f32", 1, 0), ("f32", 3, 2), ("bf16", 1, 0), ("bf16", 5, 3), ("f16", 7, 1), ("bf16", 8, 8)])
@pytest.mark.parametrize("M,K", [(1, 1111), (1, 5000), (9, 2047), (140, 600), (2, 16400)])
def test_rows_of_any_alignment(sg, M, K, dtype, offset, pad):
    import torch
    g = torch.Generator(device="cuda").manual_seed(offset)
    buf = torch.full((M * (K + pad) + offset + 9,), float("nan"), dtype=td(dtype), device="cuda")
    x = buf[offset:offset + M * (K + pad)].view(M, K + pad)[:, :K]
    x.copy_(torch.randn(M, K, generator=g, device="cuda"))
    w = sg.quantize_fp4(torch.randn(300, K, generator=g, device="cuda"))
    for block in (16, 32):
        for p, q in zip(sg.quantize_fp4(x, block), sg.quantize_fp4(x.contiguous().clone(), block)):
            assert p is None and q is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(sg.linear_fp4(x, *w), sg.linear_fp4(x.contiguous().clone(), *w))


@pytest.mark.parametrize("M", [1, 5, 70, 1200])
@pytest.mark.parametrize("block", [16, 32])
def test_a_row_that_is_not_finite_stays_alone(sg, M, block):
    import torch
    x, w, bias = operands(sg, M, 4200, 300, 9, block)
    want = sg.linear_fp4(x, *w, bias=bias)
    for value in (float("nan"), float("inf"), float("-inf")):
        y = x.clone()
        y[M // 2, 17] = value
        got = sg.linear_fp4(y, *w, bias=bias)
        assert bool(torch.isnan(got[M // 2]).all())
        rest = [i for i in range(M) if i != M // 2]
        assert torch.equal(got[rest], want[rest])


def test_empty_sums_and_empty_matrices(sg):
    import torch
    bias = torch.randn(5, device="cuda")
    for block in (16, 32):
        a, w = (sg.quantize_fp4(torch.empty(n, 0, device="cuda"), block) for n in (3, 5))
        assert a[0].shape == (3, 0) and a[1].shape == (1, 0)
        if block == 16:
            assert bool((a[2] == 0).all())
        for scale in (a[2], None if a[2] is None else torch.full((3,), float("nan"), device="cuda")):
            assert bool((sg.matmul_fp4(a[0], a[1], scale, *w, bias=bias) == bias).all())
        assert bool((sg.linear_fp4(torch.empty(3, 0, device="cuda"), *w, out_dtype=torch.bfloat16) == 0).all())
        none, w = sg.quantize_fp4(torch.empty(0, 64, device="cuda"), block), sg.quantize_fp4(torch.randn(5, 64, device="cuda"), block)
        assert sg.matmul_fp4(*none, *w).shape == (0, 5) and sg.matmul_fp4(*w, *none).shape == (5, 0)
        assert sg.linear_fp4(torch.empty(0, 64, device="cuda"), *w).shape == (0, 5)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("rows,K", [(1, 1), (5, 100), (130, 64), (300, 1111)])
def test_scales_laid_out(sg, rows, K, block):
    import torch
    q, s, _ = sg.quantize_fp4(torch.randn(rows, K, device="cuda"), block)
    n = -(-K // block)
    plain = torch.zeros(rows, n + 3, dtype=torch.uint8, device="cuda")[:, :n]
    plain.copy_(torch.from_numpy(bits_of(s, rows, n).astype(np.uint8)))
    got = sg.lay_out_fp4_scales(plain.view(s.dtype))
    assert got.dtype is s.dtype and torch.equal(got.view(torch.uint8), s.view(torch.uint8))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 2048), (20, 4096, 2048), (200, 6000, 1024), (1300, 8000, 1024)])
def test_weights_and_tokens_that_are_written_just_before(sg, M, N, K):
    """A product whose weights the call before quantised, with other bytes in their place until then."""
    import torch
    x = torch.randn(M, K, device="cuda")
    sets = [torch.randn(N, K, device="cuda") for _ in range(2)]
    done = [sg.quantize_fp4(w) for w in sets]
    torch.cuda.synchronize()
    want = [sg.linear_fp4(x, *w) for w in done]
    a = sg.quantize_fp4(x)
    lib = sg.load()
    q, s, r = (t.clone() for t in done[0])
    stream = torch.cuda.current_stream().cuda_stream
    for turn in range(10):
        w = sets[turn % 2]
        status = lib.sgemm_quantize_fp4(N, K, 0, w.data_ptr(), K, 16, q.data_ptr(), K // 2, s.data_ptr(), r.data_ptr(), stream)
        assert status == 0
        got = sg.matmul_fp4(*a, q, s, r)
        assert torch.equal(got, want[turn % 2]), f"call {turn}"
        status = lib.sgemm_quantize_fp4(N, K, 0, sets[1 - turn % 2].data_ptr(), K, 16, q.data_ptr(), K // 2, s.data_ptr(), r.data_ptr(),
                                        stream)
        assert status == 0 and torch.equal(sg.linear_fp4(x, q, s, r), want[1 - turn % 2])


@pytest.mark.parametrize("M", [1, 20, 300, 1300])
def test_another_stream_a_graph_and_the_same_bits(sg, M):
    import torch
    x = torch.randn(M, 1024, device="cuda").to(torch.bfloat16)
    w = sg.quantize_fp4(torch.randn(4100, 1024, device="cuda"))
    want = sg.linear_fp4(x, *w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sg.linear_fp4(x, *w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        got = sg.linear_fp4(x, *w)
    side.synchronize()
    assert torch.equal(got, want)
    # two graphs of the same call, replayed one after the other
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(sg.linear_fp4(x, *w))
    x.neg_()
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, -want)
    assert sg.sgemm_device_status() == sg.SGEMM_OK


@pytest.mark.parametrize("M,N,K", [(5, 512, 8192), (40, 4096, 512), (300, 520, 4096), (1300, 8000, 1024)])
def test_a_wait_that_runs_out_is_reported(sg, M, N, K):
    import torch
    x, w, _ = operands(sg, M, N, K, 12, 16)
    a = sg.quantize_fp4(x)
    want = sg.matmul_fp4(*a, *w)
    sg.sgemm_test_switches(1, 50_000_000)     # no copies: every wait runs out after 50 ms
    try:
        sg.matmul_fp4(*a, *w)
        assert sg.sgemm_device_status() == sg.SGEMM_ERR_TIMEOUT
    finally:
        sg.sgemm_test_switches(0)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert torch.equal(sg.matmul_fp4(*a, *w), want)


def test_refusals(sg):
    import torch
    x = torch.randn(4, 64, device="cuda")
    a, w = sg.quantize_fp4(x), sg.quantize_fp4(torch.randn(6, 64, device="cuda"))
    b32 = sg.quantize_fp4(x, 32)
    tight = torch.zeros(4, 20, dtype=torch.uint8, device="cuda")
    for call, error, match in [
            (lambda: sg.quantize_fp4(x, 64), ValueError, "block"), (lambda: sg.quantize_fp4(x.int()), TypeError, "float32"),
            (lambda: sg.quantize_fp4(x.T), ValueError, "stride"), (lambda: sg.quantize_fp4(x[0]), TypeError, "2-D"),
            (lambda: sg.matmul_fp4(a[0].int(), *a[1:], *w), TypeError, "uint8"),
            (lambda: sg.matmul_fp4(*b32, *w), ValueError, "blocks of 32"),
            (lambda: sg.matmul_fp4(a[0], a[1].view(torch.uint8), a[2], *w), TypeError, "float8"),
            (lambda: sg.matmul_fp4(*a, w[0], w[1][:, :-1], w[2]), ValueError, "tiles"),
            (lambda: sg.matmul_fp4(*a, w[0], w[1], w[2][:5]), ValueError, "elements"),
            (lambda: sg.matmul_fp4(*a, w[0], w[1], w[2].double()), TypeError, "w_scale"),
            (lambda: sg.matmul_fp4(*a, w[0][:, :16], w[1], w[2]), ValueError, "w is"),
            (lambda: sg.linear_fp4(torch.randn(4, 40, device="cuda"), tight, w[1], None), ValueError, "multiple of 16"),
            (lambda: sg.linear_fp4(x, w[0][:, 1:], w[1], w[2]), ValueError, "w is"),
            (lambda: sg.matmul_fp4(*a, *w, out=torch.empty(4, 5, device="cuda")), ValueError, "out is"),
            (lambda: sg.matmul_fp4(*a, *w, out_dtype=torch.int32), TypeError, "out_dtype"),
            (lambda: sg.matmul_fp4(*a, *w, bias=torch.zeros(6, 1, device="cuda")), TypeError, "bias"),
            (lambda: sg.linear_fp4(x, *w, workspace=torch.empty(16, device="cuda")), sg.SgemmError, "linear_fp4"),
            (lambda: sg.linear_fp4(x, *w, workspace=torch.empty(1 << 16)), TypeError, "workspace"),
            (lambda: sg.linear_fp4(x, *w, workspace=torch.empty(2, 1 << 16, device="cuda").T), ValueError, "workspace"),
            (lambda: sg.linear_fp4(x, *w, out=x[:, :6]), sg.SgemmError, "linear_fp4"),
            (lambda: sg.lay_out_fp4_scales(x), TypeError, "float8"),
            (lambda: sg.linear_fp4(x, *w, None, None, None, None, None, 3), TypeError, "positional")]:
        with pytest.raises(error, match=match):
            call()
    # a view that starts inside 16 bytes
    off = torch.zeros(200, dtype=torch.uint8, device="cuda")[4:36].view(1, 32)
    with pytest.raises(ValueError, match="16 bytes"):
        sg.matmul_fp4(off, a[1], None, *w)


# ---------------------------------------------------------------- pairs of SMs
#
# Which sizes go to pairs is a matter of measured times; these do (rounds of tiles that fill them).

@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", [(4300, 4100, 40), (9000, 4100, 64), (6000, 4999, 130), (1300, 8000, 1400), (1300, 8001, 1450),
                                   (1300, 8000, 1500), (1700, 4301, 1130)])
def test_product_on_pairs(sg, M, N, K, block):
    test_product_of_every_plan(sg, M, N, K, block)


@pytest.mark.parametrize("M", [1700, 2900])
@pytest.mark.parametrize("block", [16, 32])
def test_strides_and_what_lies_around_on_pairs(sg, M, block):
    test_strides_and_what_lies_around(sg, M, block)


def test_weights_and_tokens_that_are_written_just_before_pairs(sg):
    test_weights_and_tokens_that_are_written_just_before(sg, 1300, 8000, 2048)


@pytest.mark.parametrize("M", [3000, 4100])
def test_another_stream_a_graph_and_the_same_bits_on_pairs(sg, M):
    test_another_stream_a_graph_and_the_same_bits(sg, M)


@pytest.mark.parametrize("M,N,K", [(1300, 8000, 1500), (4300, 4100, 512), (10, 6400, 4096)])
def test_a_wait_that_runs_out_on_pairs_and_halves(sg, M, N, K):
    test_a_wait_that_runs_out_is_reported(sg, M, N, K)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", [(10, 6400, 4096), (3, 5001, 3300)])
def test_product_of_halves(sg, M, N, K, block):
    """Clusters of two."""
    test_product_of_every_plan(sg, M, N, K, block)


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("N", [8000, 8001, 7937])
def test_16_bit_results_on_pairs_anywhere(sg, N, out):
    """Rows that start on four bytes are stored two columns at a time, others one by one; the same bits."""
    import torch
    M, K = 1301, 1450
    x, w, bias = operands(sg, M, N, K, N, 16)
    a = sg.quantize_fp4(x)
    want = sg.matmul_fp4(*a, *w, bias).to(td(out))   # FP32 results, rounded once
    for start, pitch in ((0, N + N % 2), (1, N + N % 2), (2, N + 9 - N % 2), (0, N + 6 + N % 2)):
        room = torch.full((M + 2, pitch + 16), 7.0, dtype=td(out), device="cuda").view(-1)
        to = room[pitch + start:pitch + start + M * pitch].view(M, pitch)[:, :N]
        got = sg.matmul_fp4(*a, *w, bias, out=to)
        assert torch.equal(got, want)
        to.fill_(7.0)
        assert bool((room == 7.0).all()), "wrote outside C"
