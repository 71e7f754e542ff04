"""A small recurrent model searched with beams on one GB300, and trained: the operators
of a model's end, run together as a user would run them.

The model keeps a residual stream per beam, to which each token adds its embedding; the
norm of that goes through the vocabulary head.

* ``search`` (serving): the sum and its layer norm, a head with 4-bit weights, the best
  continuations of every group's beams, and the beams' streams and answers reordered as
  they were chosen, in place.
* ``loss_and_gradients`` (training): the same end with FP32 weights, the mean negative log
  probability of the next tokens, and the gradients of everything that is learnt.

    python examples/beam_search.py [--groups B] [--beams W] [--width D] [--vocabulary V] [--steps S]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dense_fp32_matrix_04_gb300 as sg
from last_block import product

EPS = 1e-5
END = 0


class Model:
    """What is learnt: the tokens' embeddings, the norm's weights and bias, and the head."""

    def __init__(self, D, V, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.embedding = torch.randn(V, D, generator=g, device=device)
        self.w = 1 + 0.1 * torch.randn(D, generator=g, device=device)
        self.b = 0.1 * torch.randn(D, generator=g, device=device)
        self.head = 2 * torch.randn(V, D, generator=g, device=device) / D ** 0.5

    def for_serving(self, block=16):
        """The head's weights with 4 bits, a scale for each block and one for each word."""
        return sg.quantize_fp4(self.head, block)


def advance(model, served, stream, token, score, finished):
    """One step of all beams: ``stream`` ((B W) x D) takes its tokens' embeddings; returns the
    chosen continuations ``(score, parent, token)`` and the logits they were chosen from."""
    _, n, _ = sg.layer_norm(stream, model.w, model.b, add=model.embedding[token].to(stream.dtype), eps=EPS, out=stream)
    logits = sg.linear_fp4(n, *served, out_dtype=torch.float32)
    return sg.beam_step(logits, score, finished=finished, end=END), logits


def search(model, served, first, beams, steps, dtype=torch.bfloat16):
    """``(answers, score)``: for each of the ``first`` tokens (B) the ``beams`` best continuations of at
    most ``steps`` tokens, (B x beams x steps), best first, and their log probabilities."""
    B, D = first.shape[0], model.w.shape[0]
    device = first.device
    stream = torch.zeros(B * beams, D, dtype=dtype, device=device)
    # one beam a group to begin with: the others do not exist yet
    score = torch.full((B, beams), float("-inf"), device=device)
    score[:, 0] = 0
    finished = torch.zeros(B, beams, dtype=torch.bool, device=device)
    token = first.repeat_interleave(beams)
    answers = torch.full((B * beams, steps), END, dtype=torch.int32, device=device)
    for step in range(steps):
        (score, parent, chosen), _ = advance(model, served, stream, token, score, finished)
        # where there are fewer continuations than beams, the rest go on as beams that do not exist
        for state in (stream, answers):
            sg.beam_reorder(state, parent, out=state)
        chosen = chosen.clamp(min=END)
        finished = finished.gather(1, parent.clamp(min=0).long()) | (chosen == END)
        answers[:, step] = chosen.view(-1)
        token = chosen.view(-1).long()
    return answers.view(B, beams, steps), score


def loss_and_gradients(model, stream, token, target):
    """The mean over scored tokens of -log p[target] after one step from ``stream`` (T x D), and the
    gradients by name, that of the stream among them."""
    y = model.embedding[token]
    r, n, stats = sg.layer_norm(stream, model.w, model.b, add=y, eps=EPS)
    logits = product(n, model.head, transb=True)
    logprob, entropy, lse = sg.logprobs(logits, target)
    scored = (target >= 0).float()
    share = -scored / scored.sum().clamp(min=1)
    d_logits = sg.logprobs_backward(logits, target, lse, entropy, share, out=logits)
    dr, dw, db = sg.layer_norm_backward(r, model.w, stats, product(d_logits, model.head))
    d_embedding = torch.zeros_like(model.embedding).index_add_(0, token, dr)
    return (share * logprob).sum(), {"head": product(d_logits, n, transa=True), "w": dw, "b": db, "embedding": d_embedding, "stream": dr}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--groups", type=int, default=4)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--vocabulary", type=int, default=8000)
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    model = Model(a.width, a.vocabulary)
    stream = torch.randn(256, a.width, generator=g, device="cuda")
    token = torch.randint(1, a.vocabulary, (256,), generator=g, device="cuda")
    target = torch.randint(0, a.vocabulary, (256,), generator=g, device="cuda")
    for step in range(10):
        loss, grad = loss_and_gradients(model, stream, token, target)
        if step % 3 == 0:
            print(f"step {step:3d}  loss {loss.item():.4f}")
        for name, rate in (("head", 1.0), ("w", 0.05), ("b", 0.05), ("embedding", 1.0)):
            getattr(model, name).sub_(grad[name], alpha=rate)
    answers, score = search(model, model.for_serving(), token[:a.groups], a.beams, a.steps)
    for b in range(a.groups):
        print(f"group {b}: {answers[b, 0].tolist()} with log probability {score[b, 0].item():.3f}")
    if sg.sgemm_device_status() != sg.SGEMM_OK:
        raise SystemExit("a kernel reported a bounded-wait timeout")


if __name__ == "__main__":
    main()
