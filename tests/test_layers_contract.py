"""More of include/sgemm_layers.h without a GPU: what is refused on the host before
any CUDA call."""

import pytest

import dense_fp32_matrix_04_gb300 as sg
from dense_fp32_matrix_04_gb300 import build

BAD, ALIAS, OK = sg.SGEMM_ERR_INVALID_ARG, sg.SGEMM_ERR_ALIAS, sg.SGEMM_OK
F32, BF16, F16 = 0, 1, 2
#: device-looking addresses, 16-byte aligned and far apart; never dereferenced
P = [0x7F0000000000 + (i << 36) for i in range(24)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sg.load()


@pytest.mark.parametrize("change", [dict(lddg=63), dict(dgate=P[14] + 1), dict(dgate=0), dict(dw_post=0), dict(dw_pre=0)])
def test_block_norm_backward_over_no_rows_refuses(lib, change):
    a = dict(T=0, D=64, dtype=BF16, x=P[0], ldx=64, y=P[1], ldy=64, w_pre=P[2], w_post=P[3], wdtype=F32, gate=P[4],
             ldg=64, gate_rows=2, scale=1.0, rstd=P[7], dn=P[8], lddn=64, dr=P[9], lddr=64, dx=P[10], lddx=64,
             dy=P[11], lddy=64, dw_pre=P[12], dw_post=P[13], dgate=P[14], lddg=64, ws=P[15], ws_bytes=1 << 30,
             stream=None)
    a.update(change)
    assert lib.sgemm_block_norm_backward(*a.values()) == BAD


@pytest.mark.parametrize("scale,want", [(2.0 ** 127 * (1 + 2.0 ** -23), BAD), (3.4e38, BAD), (2.0 ** 127, OK), (1e-45, OK)])
def test_logprobs_scales(lib, scale, want):
    # no rows: nothing is launched for what is accepted
    assert lib.sgemm_logprobs(0, 100, F32, P[0], 100, scale, 0, 0, 0, P[2], P[3], P[4], P[5], 0, 0, 0, None) == want
    assert lib.sgemm_logprobs_backward(0, 100, F32, P[0], 100, scale, 0, 0, 0, P[2], P[3], P[4], P[5], P[6], P[7], 100,
                                       None) == want


def test_first_argument_by_name():
    """Every call takes its first tensor by the name that its signature shows."""
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 8), torch.ones(8)
    y = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: sg.block_norm(x=x, y=x, w_pre=w), lambda: sg.quantize_i8(x=x),
                 lambda: sg.block_norm_backward(x=x, y=x, w_pre=w, rstd=x, dn=x), lambda: sg.logprobs(logits=x, target=y),
                 lambda: sg.linear_i8(x=x, w=x, w_scale=w), lambda: sg.matmul_i8(a=x.to(torch.int8), a_scale=w, w=x, w_scale=w),
                 lambda: sg.logprobs_backward(logits=x, target=y, lse=w, entropy=w, g_logprob=w)):
        with pytest.raises(TypeError, match="must be a 2-D CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="missing"):
        sg.quantize_i8()


def test_binding_refuses_sizes_beyond_32_bits():
    """ctypes drops the upper half of such a number without a word; tensors without storage show it."""
    torch = pytest.importorskip("torch")
    from dense_fp32_matrix_04_gb300 import layers

    def rows(shape, stride):
        return layers._rows(torch.empty_strided(shape, stride, device="meta"), "x", *shape)

    assert rows((2, 8), (2 ** 31 - 1, 1))[1] == 2 ** 31 - 1
    assert rows((1, 8), (2 ** 40, 1))[1] == 8            # one row: its stride does not matter
    for shape, stride in (((2, 8), (2 ** 31, 1)), ((2, 8), (2 ** 32 + 8, 1)), ((2 ** 31, 1), (1, 1)), ((2 ** 32 + 3, 1), (1, 1)),
                          ((2 ** 32, 4), (8, 1)), ((1, 2 ** 31), (2 ** 31, 1)), ((1, 2 ** 32 + 5), (2 ** 32 + 5, 1))):
        with pytest.raises(ValueError, match="2\\^31"):
            rows(shape, stride)


@pytest.mark.parametrize("change", [dict(M=2 ** 30 + 1), dict(N=2 ** 30 + 1, ldc=2 ** 30 + 1), dict(M=2 ** 31 - 1),
                                    dict(N=2 ** 31 - 1, ldc=2 ** 31 - 1), dict(K=131072, lda=131072, ldb=131072)])
def test_i8_sizes_are_bounded(lib, change):
    a = dict(M=40, N=8, K=64, A=P[0], lda=64, a_scale=P[1], B=P[2], ldb=64, b_scale=P[3], bias=P[4], C=P[5], ldc=8,
             ctype=F32, ws=P[6], ws_bytes=1 << 30, stream=None)
    a.update(change)
    assert lib.sgemm_i8(*a.values()) == BAD
    assert lib.sgemm_i8_workspace_size(a["M"], a["N"], a["K"], a["B"], a["ldb"]) == 0
    del a["a_scale"]
    b = list(a.values())
    assert lib.sgemm_linear_i8(*b[:3], BF16, *b[3:]) == BAD
