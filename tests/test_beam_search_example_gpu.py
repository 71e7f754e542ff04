"""The example that runs the layer norm, the 4-bit head and the beams together.

Serving: every step of a search is followed with its own states: the sum to the bit, the
norm, the product of the codes that the norm gives, the beams chosen from the logits, and
the states after they were reordered, each against its definition.  Training: the gradients
against the same model in 64-bit torch operations; with u = 2^-24 a logit is off by at most
2 D u sum|n||w| and the products after it add 2 V u of a sum whose terms cancel sqrt(V)-fold:
at D = 256 and V = 999 below 2 * 256 * u * 22 + 2 * 999 * u * 32 < 5e-3 of a gradient's norm."""

import importlib.util
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def example(cuda_device, lib):
    folder = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    sys.path.insert(0, folder)
    try:
        spec = importlib.util.spec_from_file_location("beam_search", os.path.join(folder, "beam_search.py"))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    finally:
        sys.path.remove(folder)
    return module


@pytest.mark.parametrize("block,B,W,D,V", [(16, 2, 4, 256, 999), (32, 5, 3, 320, 4001), (16, 1, 2, 100, 77)])
def test_every_step_of_a_search(example, block, B, W, D, V):
    import torch

    import dense_fp32_matrix_04_gb300 as sg
    from test_beam_gpu import check as check_beams, oracle, reordered
    from test_fp4_gpu import values_of
    model = example.Model(D, V, seed=3)
    served = model.for_serving(block)
    stream = torch.zeros(B * W, D, dtype=torch.bfloat16, device="cuda")
    score = torch.full((B, W), float("-inf"), device="cuda")
    score[:, 0] = 0
    finished = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    token = torch.arange(1, B + 1, device="cuda").repeat_interleave(W)
    for step in range(5):
        before = stream.clone()
        (best, parent, chosen), logits = example.advance(model, served, stream, token, score, finished)
        assert torch.equal(stream, (before.float() + model.embedding[token].bfloat16().float()).bfloat16())
        x = stream.double().cpu().numpy()
        d = x - x.mean(1, keepdims=True)
        n = d / np.sqrt((d ** 2).mean(1, keepdims=True) + example.EPS) * model.w.double().cpu().numpy() + model.b.double().cpu().numpy()
        _, n_got, _ = sg.layer_norm(stream, model.w, model.b, eps=example.EPS)
        assert (np.abs(n_got.double().cpu().numpy() - n) <= 2.0 ** -8 * 1.01 * np.abs(n) + 1e-5).all()
        a = sg.quantize_fp4(n_got, block)
        A, H = values_of(a[0], a[1], D, block), values_of(served[0], served[1], D, block)
        s = np.outer(a[2].double().cpu().numpy(), served[2].double().cpu().numpy()) if block == 16 else 1.0
        z, size = A @ H.T * s, np.abs(A) @ np.abs(H).T * s
        assert (np.abs(logits.double().cpu().numpy() - z) <= (2 * D + 8) * U * size).all()
        check_beams((best, parent, chosen), oracle(logits.cpu().numpy(), score.cpu().numpy(), W, 1.0, None, finished.cpu().numpy(), example.END))
        want = reordered(stream, parent, stream.clone())
        assert torch.equal(sg.beam_reorder(stream, parent, out=stream), want)
        finished = finished.gather(1, parent.clamp(min=0).long()) | (chosen <= example.END)
        score, token = best, chosen.clamp(min=example.END).view(-1).long()
    # the same search by the example's own loop
    answers, total = example.search(model, served, torch.arange(1, B + 1, device="cuda"), W, 5)
    assert torch.equal(total, score) and torch.equal(answers[:, :, -1].reshape(-1).long(), token)
    assert bool((total[:, :-1] >= total[:, 1:]).all())
    # answers that ended stay ended
    ended = (answers == example.END).int().cummax(2).values.bool()
    assert bool((answers[ended] == example.END).all())


def test_training_step(example):
    import torch
    T, D, V = 77, 256, 999
    g = torch.Generator(device="cuda").manual_seed(3)
    model = example.Model(D, V, seed=2)
    stream = torch.randn(T, D, generator=g, device="cuda")
    token = torch.randint(0, V, (T,), generator=g, device="cuda")
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::7] = -1
    loss, grad = example.loss_and_gradients(model, stream, token, target)
    leaf = {k: getattr(model, k).double().requires_grad_() for k in ("embedding", "w", "b", "head")}
    leaf["stream"] = stream.double().requires_grad_()
    r = leaf["stream"] + leaf["embedding"][token]
    d = r - r.mean(1, keepdim=True)
    n = d / (d.square().mean(1, keepdim=True) + example.EPS).sqrt() * leaf["w"] + leaf["b"]
    log_p = torch.log_softmax(n @ leaf["head"].T, 1).gather(1, target.clamp(min=0)[:, None])[:, 0]
    scored = target >= 0
    want = -(log_p * scored).sum() / scored.sum()
    want.backward()
    assert abs(loss.item() - want.item()) < 5e-3 * abs(want.item())
    for name, p in leaf.items():
        off = ((grad[name].double() - p.grad).norm() / p.grad.norm()).item()
        assert off < 5e-3, f"{name} is {off:.3g} off"


def test_main_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["beam_search.py", "--groups", "2", "--beams", "3", "--width", "128", "--vocabulary", "500", "--steps", "4"])
    example.main()
    assert "group 1" in capsys.readouterr().out
