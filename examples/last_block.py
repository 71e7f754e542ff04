"""The end of a language model on one GB300, run as a user would run it: from the
last block's output to the next token, and the same end trained.

* ``next_tokens`` (serving): the residual stream and the last block's output go
  through the norms, the gate and the sum, which leave 8-bit rows; the
  vocabulary head holds 8-bit weights; from its logits come the alternatives
  that a mask allows, of which one is drawn, and how sure the model was.
* ``loss_and_gradients`` (training): the same path with FP32 weights, the head's
  products on the tensor cores at FP32 accuracy, the mean negative log
  probability of the next tokens less a share of their entropy, and the
  gradients of everything that is learnt.

    python examples/last_block.py [--tokens T] [--width D] [--vocabulary V] [--steps S]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dense_fp32_matrix_04_gb300 as sg

EPS = 1e-6


def product(a, b, transa=False, transb=False):
    """op(a) op(b) in FP32 on the tensor cores."""
    M, K = a.shape[::-1] if transa else a.shape
    N = b.shape[0] if transb else b.shape[1]
    c = torch.empty((M, N), dtype=torch.float32, device=a.device)
    need = sg.sgemm_gemm_workspace_size(sg.ALGO_3XTF32, int(transa), int(transb), M, N, K)
    ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=a.device)
    sg.sgemm_gemm(sg.ALGO_3XTF32, int(transa), int(transb), M, N, K, 1.0, a, a.shape[1], b, b.shape[1], 0.0, c, N, ws,
                  need)
    return c


def mask_words(allowed):
    """The words of a mask (rows x ceil(V / 32)) from a boolean matrix (rows x V)."""
    rows, V = allowed.shape
    bits = torch.zeros((rows, (V + 31) // 32 * 32), dtype=torch.int64, device=allowed.device)
    bits[:, :V] = allowed
    words = (bits.view(rows, -1, 32) << torch.arange(32, device=allowed.device)).sum(2)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


class LastBlock:
    """What is learnt: the two norms' weights, the gate and the head."""

    def __init__(self, D, V, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.w_post = 1 + 0.1 * torch.randn(D, generator=g, device=device)
        self.w_pre = 1 + 0.1 * torch.randn(D, generator=g, device=device)
        self.gate = 0.5 + 0.1 * torch.randn(1, D, generator=g, device=device)
        self.head = torch.randn(V, D, generator=g, device=device) / D ** 0.5

    def for_serving(self):
        """The head's weights with 8 bits and a scale for each word of the vocabulary."""
        return sg.quantize_i8(self.head)


def next_tokens(model, served, x, y, mask=None, temperature=0.8, top=20, generator=None):
    """One token for each row of x, drawn among the ``top`` most likely that the mask
    allows; with its log probability and the entropy of the whole distribution."""
    w, w_scale = served
    dt = x.dtype
    r, q, q_scale, _ = sg.block_norm(x, y, model.w_pre, w_post=model.w_post, gate=model.gate.to(dt), eps=EPS,
                                     quantize=True)
    logits = sg.matmul_i8(q, q_scale, w, w_scale)
    unscored = torch.full((x.shape[0],), -1, dtype=torch.int64, device=x.device)
    _, entropy, _, log_p, ids = sg.logprobs(logits, unscored, scale=1.0 / temperature, mask=mask, top=top)
    drawn = torch.multinomial(log_p.exp(), 1, generator=generator)
    return ids.gather(1, drawn)[:, 0], log_p.gather(1, drawn)[:, 0], entropy


def loss_and_gradients(model, x, y, target, entropy_share=0.01):
    """The mean over scored tokens of -(log p[target] + entropy_share * entropy), and
    its gradients by name, those of x and y among them."""
    r, n, rstd = sg.block_norm(x, y, model.w_pre, w_post=model.w_post, gate=model.gate, eps=EPS)
    logits = product(n, model.head, transb=True)
    logprob, entropy, lse = sg.logprobs(logits, target)
    scored = (target >= 0).float()
    share = -scored / scored.sum().clamp(min=1)
    loss = (share * (logprob + entropy_share * entropy)).sum()
    d_logits = sg.logprobs_backward(logits, target, lse, entropy, share, entropy_share * share, out=logits)
    dn = product(d_logits, model.head)
    d_head = product(d_logits, n, transa=True)
    dx, dy, dw_pre, dw_post, dgate = sg.block_norm_backward(x, y, model.w_pre, rstd, dn, w_post=model.w_post,
                                                            gate=model.gate)
    return loss, {"head": d_head, "w_pre": dw_pre, "w_post": dw_post, "gate": dgate, "x": dx, "y": dy}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--vocabulary", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    model = LastBlock(a.width, a.vocabulary)
    x, y = (torch.randn(a.tokens, a.width, generator=g, device="cuda") for _ in range(2))
    target = torch.randint(0, a.vocabulary, (a.tokens,), generator=g, device="cuda")
    for step in range(a.steps):
        loss, grad = loss_and_gradients(model, x, y, target)
        if step % max(1, a.steps // 5) == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {loss.item():.4f}")
        for name, rate in (("head", 5.0), ("w_pre", 0.1), ("w_post", 0.1), ("gate", 0.1)):
            getattr(model, name).sub_(grad[name], alpha=rate)
    served = model.for_serving()
    # the first half of the vocabulary only, for rows that must answer in it
    allowed = torch.ones(4, a.vocabulary, dtype=torch.bool, device="cuda")
    allowed[2:, a.vocabulary // 2:] = False
    ids, log_p, entropy = next_tokens(model, served, x[:4].bfloat16(), y[:4].bfloat16(), mask_words(allowed),
                                      generator=g)
    for t in range(4):
        print(f"row {t}: token {ids[t].item()} (its target {target[t].item()}), log probability {log_p[t].item():.3f}, "
              f"entropy {entropy[t].item():.3f}")
    if sg.sgemm_device_status() != sg.SGEMM_OK:
        raise SystemExit("a kernel reported a bounded-wait timeout")


if __name__ == "__main__":
    main()
