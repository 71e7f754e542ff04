"""What the native binding returns is a tensor with a storage of its own, however small: it can be
saved beside the others, and given back alone."""

import io

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def results(sg, T, stream):
    """The new tensors of every operator, from small calls; by operator."""
    import torch
    D = 96
    x, w = torch.randn(T, D, device="cuda", dtype=torch.bfloat16), torch.ones(D, device="cuda")
    q = sg.quantize_fp4(torch.randn(300, D, device="cuda"))
    n = sg.layer_norm(x, w, w, x, stream=stream)
    score = torch.zeros(T, 1, device="cuda")
    best = sg.beam_step(x, score, top=4, stream=stream)
    return {"layer_norm": n, "layer_norm_backward": sg.layer_norm_backward(x, w, n[2], x, stream=stream),
            "quantize_fp4": sg.quantize_fp4(x, stream=stream), "quantize_fp4 32": sg.quantize_fp4(x, 32, stream=stream)[:2],
            "lay_out_fp4_scales": (sg.lay_out_fp4_scales(torch.ones(T, 6, device="cuda").to(torch.float8_e4m3fn), stream=stream),),
            "linear_fp4": (sg.linear_fp4(x, *q, stream=stream),), "matmul_fp4": (sg.matmul_fp4(*sg.quantize_fp4(x), *q, stream=stream),),
            "beam_step": best, "beam_reorder": (sg.beam_reorder(x, torch.zeros(T, 3, dtype=torch.int32, device="cuda"), stream=stream),)}


@pytest.mark.parametrize("T", [1, 4, 300])
@pytest.mark.parametrize("other", [False, True])
def test_results_are_saved_together(sg, T, other):
    import torch
    made = results(sg, T, torch.cuda.Stream() if other else None)
    torch.cuda.synchronize()
    for name, tensors in made.items():
        named = {str(i): t for i, t in enumerate(tensors)}
        buf = io.BytesIO()
        torch.save(named, buf)
        buf.seek(0)
        back = torch.load(buf, weights_only=True)
        for k, t in named.items():
            assert back[k].dtype is t.dtype and back[k].stride() == t.stride(), name
            assert torch.equal(back[k].contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)), name


def test_results_have_storages_of_their_own(sg):
    import torch
    every = [t for tensors in results(sg, 5, None).values() for t in tensors]
    assert len({t.untyped_storage().data_ptr() for t in every}) == len(every)
    for t in every:
        rows = t.stride(0) if t.dim() == 2 else 1
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.shape[0] * rows * t.element_size()
    # one that is given back leaves the others as they are
    r, n, stats = sg.layer_norm(torch.randn(3, 64, device="cuda"), torch.ones(64, device="cuda"), add=torch.ones(3, 64, device="cuda"))
    kept = n.clone(), stats.clone()
    r.untyped_storage().resize_(0)
    others = [torch.full((3, 64), 7.0, device="cuda") for _ in range(8)]
    assert torch.equal(n, kept[0]) and torch.equal(stats, kept[1]) and len(others) == 8
