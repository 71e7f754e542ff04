"""Views whose numbers are not those in memory (a conjugate, the imaginary part of one) are refused
by the native binding, which reads memory, wherever they are given."""

import pytest

import dense_fp32_matrix_04_gb300 as sg
from dense_fp32_matrix_04_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_views_that_are_not_what_lies_in_memory_are_refused():
    torch = pytest.importorskip("torch")
    conj = torch.zeros(4, 8, dtype=torch.complex64).conj()
    neg = conj.imag
    assert conj.is_conj() and neg.is_neg()
    for call in (lambda **k: sg.beam_reorder(conj, neg, **k), lambda **k: sg.layer_norm(neg, neg, **k), lambda **k: sg.quantize_fp4(neg, **k),
                 lambda **k: sg.layer_norm_backward(neg, neg, neg, neg, **k), lambda **k: sg.linear_fp4(neg, neg, neg, **k),
                 lambda **k: sg.beam_step(neg, neg, **k)):
        for stream in ({}, {"stream": 0}):
            with pytest.raises(ValueError, match="conjugate or negated"):
                call(**stream)


@pytest.mark.gpu
def test_plain_forms_of_such_views_are_taken(cuda_device):
    import torch
    state = torch.randn(4, 6, dtype=torch.complex64, device="cuda").conj()
    parent = torch.tensor([[1, 0, 3, 2]], dtype=torch.int32, device="cuda")
    want = state[[1, 0, 3, 2]].resolve_conj()
    assert torch.equal(sg.beam_reorder(state.resolve_conj(), parent), want)
    out = torch.empty(4, 6, dtype=torch.complex64, device="cuda")
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for call in (lambda: sg.beam_reorder(state, parent), lambda: sg.beam_reorder(state.resolve_conj(), parent, out=out.conj()),
                 lambda: sg.layer_norm(x, torch._neg_view(w)), lambda: sg.layer_norm(x, w, w, torch._neg_view(x)),
                 lambda: sg.layer_norm(x, w, w, x, out=torch._neg_view(x.clone()))):
        with pytest.raises(ValueError, match="conjugate or negated"):
            call()
