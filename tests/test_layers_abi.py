"""The operators of include/sgemm_layers.h without a GPU: every bad argument is
refused on the host with a status, before any CUDA call, and empty work
succeeds without one."""

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


def norm_args(**change):
    a = dict(T=4, D=64, dtype=BF16, x=P[0], ldx=64, y=P[1], ldy=64, w_pre=P[2], w_post=P[3], wdtype=F32, gate=P[4],
             ldg=64, gate_rows=2, scale=1.0, eps=1e-6, r=P[5], ldr=64, n=P[6], ldn=64, q=0, ldq=64, q_scale=0,
             rstd=P[7], stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(D=-1), BAD), (dict(D=65537), BAD), (dict(dtype=3), BAD), (dict(dtype=-1), BAD),
    (dict(wdtype=F16), BAD),                      # weights of a third type
    (dict(ldx=63), BAD), (dict(ldy=63), BAD), (dict(ldr=63), BAD), (dict(ldn=63), BAD), (dict(ldg=63), BAD),
    (dict(x=0), BAD), (dict(y=0), BAD), (dict(w_pre=0), BAD), (dict(r=0), BAD),
    (dict(n=0), BAD),                             # neither n nor q
    (dict(x=P[0] + 1), BAD), (dict(w_pre=P[2] + 2), BAD), (dict(rstd=P[7] + 2), BAD),
    (dict(gate_rows=3), BAD),                     # does not divide T
    (dict(gate_rows=8), BAD), (dict(gate_rows=0), BAD), (dict(gate=0), BAD), (dict(gate_rows=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(q=P[8], q_scale=0), BAD), (dict(q=P[8], q_scale=P[9], ldq=63), BAD),
    (dict(r=P[1]), ALIAS), (dict(n=P[0]), ALIAS), (dict(n=P[5]), ALIAS), (dict(r=P[0], ldr=128), ALIAS),
    (dict(r=P[0] + 2), ALIAS), (dict(rstd=P[2]), ALIAS), (dict(q=P[6], q_scale=P[9]), ALIAS),
    (dict(T=0), OK), (dict(D=0, ldx=1, ldy=1), OK),
])
def test_block_norm_refuses(lib, change, want):
    assert lib.sgemm_block_norm(*norm_args(**change)) == want


def grad_args(**change):
    a = dict(T=4, D=64, dtype=BF16, x=P[0], ldx=64, y=P[1], ldy=64, w_pre=P[2], w_post=P[3], wdtype=F32, gate=P[4],
             ldg=64, gate_rows=2, scale=1.0, rstd=P[7], dn=P[8], lddn=64, dr=P[9], lddr=64, dx=P[10], lddx=64,
             dy=P[11], lddy=64, dw_pre=P[12], dw_post=P[13], dgate=P[14], lddg=64, ws=P[15], ws_bytes=1 << 30,
             stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(D=70000), dict(dtype=7), dict(dw_pre=0), dict(dw_post=0), dict(dgate=0), dict(w_post=0),
    dict(gate=0, gate_rows=0), dict(dn=0), dict(dx=0), dict(dy=0), dict(rstd=0), dict(lddx=63), dict(lddg=63),
    dict(dw_pre=P[12] + 2),
])
def test_block_norm_backward_refuses(lib, change):
    assert lib.sgemm_block_norm_backward(*grad_args(**change)) == BAD


def test_quantize_refuses(lib):
    def call(M=4, K=64, dtype=F32, x=P[0], ldx=64, q=P[1], ldq=64, s=P[2]):
        return lib.sgemm_quantize_i8(M, K, dtype, x, ldx, q, ldq, s, None)
    for change in [dict(M=-1), dict(K=-1), dict(dtype=3), dict(x=0), dict(q=0), dict(s=0), dict(ldx=63), dict(ldq=63),
                   dict(x=P[0] + 2), dict(s=P[2] + 1)]:
        assert call(**change) == BAD, change
    assert call(q=P[0]) == ALIAS and call(s=P[0]) == ALIAS and call(s=P[1]) == ALIAS
    assert call(M=0) == OK


def i8_args(**change):
    a = dict(M=4, N=8, K=64, A=P[0], lda=64, a_scale=P[1], B=P[2], ldb=64, b_scale=P[3], bias=P[4], C=P[5], ldc=8,
             ctype=F32, ws=P[6], ws_bytes=1 << 30, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(K=131072, lda=131072, ldb=131072), BAD),
    (dict(lda=63), BAD), (dict(ldb=63), BAD), (dict(ldc=7), BAD), (dict(A=0), BAD), (dict(B=0), BAD), (dict(C=0), BAD),
    (dict(a_scale=0), BAD), (dict(b_scale=0), BAD), (dict(b_scale=P[3] + 2), BAD), (dict(bias=P[4] + 1), BAD),
    (dict(C=P[5] + 2), BAD), (dict(ctype=5), BAD),
    (dict(C=P[0]), ALIAS), (dict(C=P[2]), ALIAS), (dict(C=P[3]), ALIAS), (dict(C=P[4]), ALIAS),
    (dict(M=0), OK), (dict(N=0, ldc=1), OK),
])
def test_i8_refuses(lib, change, want):
    assert lib.sgemm_i8(*i8_args(**change)) == want


def test_linear_i8_refuses(lib):
    def call(M=40, N=8, K=64, xtype=BF16, X=P[0], ldx=64, B=P[2], ldb=64, s=P[3], bias=0, C=P[5], ldc=8, ctype=BF16,
             ws=P[6], size=1 << 30):
        return lib.sgemm_linear_i8(M, N, K, xtype, X, ldx, B, ldb, s, bias, C, ldc, ctype, ws, size, None)
    for change in [dict(M=-1), dict(xtype=3), dict(X=0), dict(ldx=63), dict(X=P[0] + 1), dict(ws=0), dict(size=16),
                   dict(ws=P[6] + 4), dict(ctype=-1)]:
        assert call(**change) == BAD, change
    assert call(ws=P[0]) == ALIAS and call(C=P[6]) == ALIAS and call(C=P[0]) == ALIAS
    assert call(M=0) == OK


def logprob_args(**change):
    a = dict(T=4, V=100, dtype=F32, z=P[0], ldz=100, scale=1.0, mask=P[1], ldm=4, mask_rows=4, target=P[2],
             logprob=P[3], entropy=P[4], lse=P[5], top=5, top_logprob=P[6], top_id=P[7], stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(V=-1), BAD), (dict(dtype=3), BAD), (dict(z=0), BAD), (dict(ldz=99), BAD),
    (dict(z=P[0] + 2), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("inf")), BAD),
    (dict(scale=float("nan")), BAD), (dict(mask_rows=2), BAD), (dict(mask_rows=0), BAD), (dict(mask=0), BAD),
    (dict(ldm=3), BAD), (dict(mask=P[1] + 2), BAD), (dict(target=0), BAD), (dict(target=P[2] + 4), BAD),
    (dict(top=-1), BAD), (dict(top=33), BAD), (dict(top_id=0), BAD), (dict(top_logprob=0), BAD),
    (dict(lse=P[0]), ALIAS), (dict(entropy=P[3]), ALIAS), (dict(top_id=P[6]), ALIAS),
    (dict(T=0), OK),
])
def test_logprobs_refuses(lib, change, want):
    assert lib.sgemm_logprobs(*logprob_args(**change)) == want


@pytest.mark.parametrize("change,want", [
    (dict(dz=0), BAD), (dict(lddz=99), BAD), (dict(lse=0), BAD), (dict(g_logprob=0), BAD), (dict(entropy=0), BAD),
    (dict(target=0), BAD), (dict(scale=0.0), BAD), (dict(dz=P[10] + 2), BAD),
    (dict(dz=P[0], lddz=104), ALIAS), (dict(dz=P[0] + 4), ALIAS), (dict(dz=P[1]), ALIAS), (dict(T=0), OK),
    (dict(V=0, ldz=1, lddz=1), OK),
])
def test_logprobs_backward_refuses(lib, change, want):
    a = dict(T=4, V=100, dtype=F32, z=P[0], ldz=100, scale=1.0, mask=P[1], ldm=4, mask_rows=4, target=P[2],
             lse=P[3], entropy=P[4], g_logprob=P[5], g_entropy=P[6], dz=P[10], lddz=100, stream=None)
    a.update(change)
    assert lib.sgemm_logprobs_backward(*a.values()) == want


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    w = torch.ones(8)
    with pytest.raises(TypeError):
        sg.block_norm(x, x, w)
    with pytest.raises(TypeError):
        sg.quantize_i8(x)
    with pytest.raises(TypeError):
        sg.logprobs(x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        sg.quantize_i8(x.to(torch.int8))
