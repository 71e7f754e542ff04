"""The layer norm, the 4-bit products and the beams without a GPU: every bad argument is
refused on the host with a status, before any CUDA call, and empty work succeeds without
one."""

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


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(D=-1), BAD), (dict(D=24577), BAD), (dict(T=2 ** 30 + 1), BAD), (dict(dtype=3), BAD), (dict(wdtype=F16), BAD),
    (dict(ldx=63), BAD), (dict(lda=63), BAD), (dict(ldr=63), BAD), (dict(ldn=63), BAD), (dict(x=0), BAD), (dict(w=0), BAD), (dict(n=0), BAD),
    (dict(r=0), BAD),                             # a sum and no place for it
    (dict(add=0), BAD),                           # a place for a sum and none
    (dict(x=P[0] + 1), BAD), (dict(w=P[2] + 2), BAD), (dict(b=P[3] + 1), BAD), (dict(stats=P[6] + 2), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(r=P[0], ldr=128), ALIAS), (dict(n=P[0]), ALIAS), (dict(n=P[4]), ALIAS), (dict(n=P[1]), ALIAS), (dict(stats=P[2]), ALIAS),
    (dict(r=P[1] + 2), ALIAS),
    (dict(T=0), OK), (dict(D=0, ldx=1, lda=1), OK),
])
def test_layer_norm_refuses(lib, change, want):
    a = dict(T=4, D=64, dtype=BF16, x=P[0], ldx=64, add=P[1], lda=64, w=P[2], b=P[3], wdtype=F32, eps=1e-5, r=P[4], ldr=64, n=P[5],
             ldn=64, stats=P[6], stream=None)
    a.update(change)
    assert lib.sgemm_layer_norm(*a.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(D=30000), BAD), (dict(dtype=-1), BAD), (dict(wdtype=7), BAD), (dict(x=0), BAD), (dict(w=0), BAD),
    (dict(stats=0), BAD), (dict(stats=P[2] + 2), BAD), (dict(dn=0), BAD), (dict(lddn=63), BAD), (dict(lddr=63), BAD), (dict(dx=0), BAD),
    (dict(dw=0), BAD), (dict(dw=P[6] + 2), BAD), (dict(ws=0), BAD), (dict(ws=P[8] + 4), BAD),
    (dict(dx=P[0], lddx=128), ALIAS), (dict(dw=P[1]), ALIAS), (dict(dw=P[2]), ALIAS), (dict(db=P[6]), ALIAS), (dict(dx=P[3] + 2), ALIAS),
    (dict(T=0, dw=0), BAD), (dict(T=0, db=P[6]), ALIAS), (dict(D=0, ldx=1, lddn=1, lddr=1, lddx=1), OK),
])
def test_layer_norm_backward_refuses(lib, change, want):
    a = dict(T=4, D=64, dtype=BF16, x=P[0], ldx=64, w=P[1], wdtype=F32, stats=P[2], dn=P[3], lddn=64, dr=P[4], lddr=64, dx=P[5],
             lddx=64, dw=P[6], db=P[7], ws=P[8], ws_bytes=1 << 30, stream=None)
    a.update(change)
    assert lib.sgemm_layer_norm_backward(*a.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), BAD), (dict(K=-1), BAD), (dict(M=2 ** 30 + 1), BAD), (dict(K=2 ** 24 + 1, ldx=2 ** 24 + 1, ldq=2 ** 24), BAD), (dict(dtype=3), BAD), (dict(block=8), BAD),
    (dict(x=0), BAD), (dict(x=P[0] + 2), BAD), (dict(ldx=99), BAD), (dict(q=0), BAD), (dict(q=P[1] + 8), BAD), (dict(ldq=48), BAD),
    (dict(ldq=56), BAD), (dict(tiles=0), BAD), (dict(tiles=P[2] + 8), BAD), (dict(scale=0), BAD), (dict(scale=P[3] + 2), BAD),
    (dict(block=32), BAD),                        # blocks of 32 have no row scale
    (dict(q=P[0]), ALIAS), (dict(tiles=P[0] + 16), ALIAS), (dict(scale=P[1]), ALIAS), (dict(tiles=P[1] + 64), ALIAS),
    (dict(M=0), OK),
])
def test_quantize_fp4_refuses(lib, change, want):
    a = dict(M=4, K=100, dtype=F32, x=P[0], ldx=100, block=16, q=P[1], ldq=64, tiles=P[2], scale=P[3], stream=None)
    a.update(change)
    assert lib.sgemm_quantize_fp4(*a.values()) == want


def test_sizes_of_scales_and_workspaces(lib):
    assert lib.sgemm_fp4_scales_size(1, 1, 16) == 512 and lib.sgemm_fp4_scales_size(129, 65, 16) == 4 * 512
    assert lib.sgemm_fp4_scales_size(129, 129, 32) == 4 * 512 and lib.sgemm_fp4_scales_size(0, 64, 16) == 0
    assert lib.sgemm_fp4_scales_size(5, 0, 16) == 0 and lib.sgemm_fp4_scales_size(5, 5, 8) == 0 and lib.sgemm_fp4_scales_size(-1, 5, 16) == 0
    # beyond 32 bits: 2^30 rows of 2^12 columns have 2^38 scales
    assert lib.sgemm_fp4_scales_size(2 ** 30, 2 ** 12, 16) == 2 ** 30 * 2 ** 8
    # codes on rows of 64 bytes, scales' tiles, rows' scales
    assert lib.sgemm_linear_fp4_workspace_size(5, 100, 16) == 512 + 1024 + 256
    assert lib.sgemm_linear_fp4_workspace_size(5, 100, 32) == 512 + 512
    assert lib.sgemm_linear_fp4_workspace_size(1, 4096, 16) == 0 and lib.sgemm_linear_fp4_workspace_size(1, 90112, 32) == 0
    assert lib.sgemm_linear_fp4_workspace_size(1, 100000, 16) > 0 and lib.sgemm_linear_fp4_workspace_size(0, 64, 16) == 0
    assert lib.sgemm_beam_step_workspace_size(2, 4, 8) == 256 + 256 + 256 and lib.sgemm_beam_step_workspace_size(0, 4, 8) == 0
    assert lib.sgemm_beam_step_workspace_size(2, 33, 8) == 0 and lib.sgemm_beam_step_workspace_size(2, 4, 0) == 0


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), BAD), (dict(K=-1), BAD), (dict(block=64), BAD), (dict(s=0), BAD), (dict(lds=6), BAD), (dict(tiles=0), BAD),
    (dict(tiles=P[1] + 8), BAD), (dict(tiles=P[0] + 16), ALIAS), (dict(rows=0), OK), (dict(K=0), OK),
])
def test_lay_out_refuses(lib, change, want):
    a = dict(rows=4, K=100, block=16, s=P[0], lds=7, tiles=P[1], stream=None)
    a.update(change)
    assert lib.sgemm_fp4_lay_out_scales(*a.values()) == want


def fp4_args(**change):
    a = dict(M=4, N=8, K=100, block=16, A=P[0], lda=64, a_block=P[1], a_scale=P[2], B=P[3], ldb=64, b_block=P[4], b_scale=P[5], bias=P[6],
             C=P[7], ldc=8, ctype=F32, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(N=2 ** 30 + 1, ldc=2 ** 30 + 1), BAD), (dict(K=2 ** 24 + 1, lda=2 ** 24, ldb=2 ** 24), BAD),
    (dict(block=4), BAD),
    (dict(lda=48), BAD), (dict(ldb=48), BAD), (dict(lda=56), BAD), (dict(ldb=72), BAD), (dict(ldc=7), BAD), (dict(A=0), BAD), (dict(B=0), BAD),
    (dict(C=0), BAD), (dict(a_block=0), BAD), (dict(b_block=0), BAD), (dict(A=P[0] + 8), BAD), (dict(b_block=P[4] + 4), BAD),
    (dict(a_scale=P[2] + 2), BAD), (dict(bias=P[6] + 1), BAD), (dict(C=P[7] + 2), BAD), (dict(ctype=5), BAD),
    (dict(C=P[0]), ALIAS), (dict(C=P[1]), ALIAS), (dict(C=P[3]), ALIAS), (dict(C=P[4] + 64), ALIAS), (dict(C=P[5]), ALIAS), (dict(C=P[6]), ALIAS),
    (dict(M=0), OK), (dict(N=0, ldc=1), OK),
])
def test_fp4_refuses(lib, change, want):
    assert lib.sgemm_fp4(*fp4_args(**change)) == want


@pytest.mark.parametrize("change,want", [
    (dict(xtype=3), BAD), (dict(X=0), BAD), (dict(X=P[0] + 1), BAD), (dict(ldx=99), BAD), (dict(B=P[3] + 8), BAD), (dict(ws=0), BAD),
    (dict(ws=P[8] + 8), BAD), (dict(size=256), BAD), (dict(block=0), BAD),
    (dict(C=P[0]), ALIAS), (dict(ws=P[0]), ALIAS), (dict(ws=P[3]), ALIAS), (dict(ws=P[7]), ALIAS), (dict(M=0), OK), (dict(N=0, ldc=1), OK),
])
def test_linear_fp4_refuses(lib, change, want):
    a = dict(M=4, N=8, K=100, xtype=BF16, X=P[0], ldx=100, block=16, B=P[3], ldb=64, b_block=P[4], b_scale=0, bias=0, C=P[7], ldc=8,
             ctype=BF16, ws=P[8], size=1 << 20, stream=None)
    a.update(change)
    assert lib.sgemm_linear_fp4(*a.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), BAD), (dict(W=0), BAD), (dict(W=33), BAD), (dict(top=0), BAD), (dict(top=33), BAD), (dict(B=2 ** 30, W=2), BAD),
    (dict(V=-1), BAD), (dict(dtype=4), BAD), (dict(z=0), BAD), (dict(ldz=99), BAD), (dict(z=P[0] + 2), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(mask_rows=2), BAD), (dict(mask=0), BAD), (dict(ldm=3), BAD), (dict(score=0), BAD),
    (dict(score=P[2] + 2), BAD), (dict(end=-1), BAD), (dict(out=0), BAD), (dict(parent=0), BAD), (dict(token=0), BAD),
    (dict(parent=P[5] + 2), BAD), (dict(ws=0), BAD), (dict(ws=P[7] + 8), BAD), (dict(size=64), BAD),
    (dict(out=P[2]), ALIAS), (dict(token=P[5]), ALIAS), (dict(ws=P[0]), ALIAS), (dict(parent=P[3]), ALIAS), (dict(ws=P[1]), ALIAS),
    (dict(B=0), OK),
])
def test_beam_step_refuses(lib, change, want):
    a = dict(B=2, W=3, V=100, dtype=F32, z=P[0], ldz=100, scale=1.0, mask=P[1], ldm=4, mask_rows=6, score=P[2], finished=P[3], end=0,
             top=4, out=P[4], parent=P[5], token=P[6], ws=P[7], size=1 << 20, stream=None)
    a.update(change)
    assert lib.sgemm_beam_step(*a.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), BAD), (dict(W=0), BAD), (dict(top=33), BAD), (dict(outer=-1), BAD), (dict(inner=-1), BAD), (dict(inner=2 ** 44 + 1), BAD),
    (dict(src=0), BAD), (dict(out=0), BAD), (dict(parent=0), BAD), (dict(parent=P[1] + 2), BAD), (dict(in_row=-1), BAD), (dict(out_outer=-1), BAD),
    (dict(in_row=2 ** 62), BAD), (dict(out_row=2 ** 43), BAD), (dict(in_outer=2 ** 44), BAD),
    (dict(out_row=100), BAD), (dict(out_outer=32), BAD),   # rows, or runs, of out over each other
    (dict(out_row=0), BAD),
    (dict(out=P[0] + 64), ALIAS), (dict(out=P[0], out_row=512), ALIAS), (dict(out=P[1]), ALIAS), (dict(out=P[0], top=2), ALIAS),
    (dict(B=0), OK), (dict(outer=0), OK), (dict(inner=0), OK),
])
def test_beam_reorder_refuses(lib, change, want):
    a = dict(B=2, W=3, top=3, outer=4, inner=48, src=P[0], in_row=256, in_outer=64, parent=P[1], out=P[2], out_row=256, out_outer=64,
             stream=None)
    a.update(change)
    assert lib.sgemm_beam_reorder(*a.values()) == want


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda **k: sg.layer_norm(x, w, **k), lambda **k: sg.layer_norm(x=x, w=w, **k), lambda **k: sg.layer_norm_backward(x, w, x, x, **k),
                 lambda **k: sg.quantize_fp4(x, **k), lambda **k: sg.linear_fp4(x, x, x, **k), lambda **k: sg.matmul_fp4(x.byte(), x, None, x, x, None, **k),
                 lambda **k: sg.beam_step(x, x, **k), lambda **k: sg.beam_reorder(x, x, **k), lambda **k: sg.lay_out_fp4_scales(x.to(torch.float8_e4m3fn), **k),
                 lambda **k: sg.layer_norm(None, w, **k), lambda **k: sg.quantize_fp4([1.0], **k)):
        for stream in ({}, {"stream": 0}):
            with pytest.raises(TypeError, match="CUDA tensor"):
                call(**stream)
    with pytest.raises(TypeError):
        sg.quantize_fp4()
    with pytest.raises(TypeError):
        sg.layer_norm(x, w, epsilon=1.0)
