"""The example that runs block norms, the 8-bit head and the log probabilities
together, against the same model in 64-bit torch operations.

Tolerance of the gradients, with u = 2^-24: a logit is off by at most 2 D u
sum|n||w|, about 2 D u * 0.64 sqrt(D) for weights of size 1 / sqrt(D), so a
probability is off by that share of itself; the products after it add 2 V u of
a sum whose terms cancel sqrt(V)-fold, and the norm's backward some 10 u.  At
D = 256 and V = 999 that is below 2 * 256 * u * 11 + 2 * 999 * u * 32 < 5e-3
of a gradient's norm.

Serving: x and the head have 8 bits, each rounded by at most 1 / 254 of its
row's largest value, so a logit is off by at most (max|n| sum|w| + max|w|
sum|n| + max|n| max|w| D / 254) / 254 over the rows, and a log probability by
twice that."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(cuda_device, lib):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "last_block.py")
    spec = importlib.util.spec_from_file_location("last_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_norm(x, y, w_pre, w_post, gate):
    h = y * (y.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w_post
    r = x + gate * h
    return r * (r.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w_pre


def test_training_step(example):
    import torch
    T, D, V = 77, 256, 999
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    model = example.LastBlock(D, V, seed=2)
    x, y = (torch.randn(T, D, generator=g, device="cuda") for _ in range(2))
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::7] = -1
    loss, grad = example.loss_and_gradients(model, x, y, target)

    leaf = {k: getattr(model, k).double().requires_grad_() for k in ("head", "w_pre", "w_post", "gate")}
    leaf["x"], leaf["y"] = x.double().requires_grad_(), y.double().requires_grad_()
    n = plain_norm(leaf["x"], leaf["y"], leaf["w_pre"], leaf["w_post"], leaf["gate"])
    log_p = torch.log_softmax(n @ leaf["head"].T, 1)
    entropy = -(log_p.exp() * log_p).sum(1)
    scored = target >= 0
    got = log_p.gather(1, target.clamp(min=0)[:, None])[:, 0]
    want = -((got + 0.01 * entropy) * scored).sum() / scored.sum()
    want.backward()
    assert abs(loss.item() - want.item()) < 5e-3 * abs(want.item())
    for name, p in leaf.items():
        off = (grad[name].double() - p.grad).norm() / p.grad.norm()
        assert off < 5e-3, (name, off.item())

    for name, rate in (("head", 2.0), ("w_pre", 0.1)):
        getattr(model, name).sub_(grad[name], alpha=rate)
    assert example.loss_and_gradients(model, x, y, target)[0].item() < loss.item()


@pytest.mark.parametrize("rows", [1, 6])
def test_next_tokens(example, rows):
    import torch
    D, V, top = 256, 999, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    model = example.LastBlock(D, V, seed=5)
    x, y = (torch.randn(rows, D, generator=g, device="cuda") for _ in range(2))
    allowed = torch.rand(rows, V, generator=g, device="cuda") < 0.5
    ids, log_p, entropy = example.next_tokens(model, model.for_serving(), x, y, example.mask_words(allowed), 1.0, top,
                                              generator=g)
    n = plain_norm(*(t.double() for t in (x, y, model.w_pre, model.w_post, model.gate)))
    w = model.head.double()
    logits = (n @ w.T).masked_fill(~allowed, -float("inf"))
    want = torch.log_softmax(logits, 1)
    nm, wm = n.abs().max(), w.abs().max()
    off = (nm * w.abs().sum(1).max() + wm * n.abs().sum(1).max() + nm * wm * D / 254) / 254
    for t in range(rows):
        assert allowed[t, ids[t]]
        assert abs(log_p[t].item() - want[t, ids[t]].item()) < 2 * off
        # no allowed token that is surely more likely was passed over top times
        assert (want[t] > want[t, ids[t]] + 4 * off).sum() < top
        p = want[t].exp()
        h = -(p[p > 0] * want[t][p > 0]).sum()
        assert abs(entropy[t].item() - h.item()) < 4 * off * (1 + h)


def test_it_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["last_block.py", "--tokens", "65", "--width", "128", "--vocabulary", "700",
                                     "--steps", "3"])
    example.main()
    out = capsys.readouterr().out
    assert out.count("loss") == 3 and out.count("row") == 4
