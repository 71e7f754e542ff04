"""Beams that have one column to go on with: its log probability is exactly 0, so the score stays what it
is, and beams whose scores are equal go by their number, whatever their logits are."""

import pytest

from test_beam_gpu import sg, td, words  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def forced(B, W, V, dtype, seed):
    """Logits, a mask that leaves a column of each row, and those columns."""
    import numpy as np
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (7 * torch.randn(B * W, V, generator=g, device="cuda")).to(td(dtype))
    column = torch.randint(0, V, (B * W,), generator=g, device="cuda")
    bits = np.zeros((B * W, V), bool)
    bits[np.arange(B * W), column.cpu().numpy()] = True
    return z, words(bits), column


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,W,V,top", [(50, 4, 1, 4), (40, 8, 300, 8), (40, 8, 300, 1), (3, 32, 2047, 32), (1, 4, 70000, 4), (20, 16, 33, 32)])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1e7])
def test_equal_scores_stay_and_go_by_the_beam(sg, B, W, V, top, dtype, scale):
    import torch
    z, mask, column = forced(B, W, V, dtype, B + V)
    for score in (torch.zeros(B, W, device="cuda"), torch.full((B, W), -3.7, device="cuda"), torch.full((B, W), -1e-30, device="cuda")):
        s, parent, token = sg.beam_step(z, score, top=top, scale=scale, mask=mask)
        n = min(W, top)
        order = torch.arange(n, device="cuda", dtype=torch.int32).expand(B, n)
        assert torch.equal(s[:, :n], score[:, :n]) and torch.equal(parent[:, :n], order)
        assert torch.equal(token[:, :n].long(), column.view(B, W)[:, :n])
        assert bool((parent[:, n:] == -1).all())


@pytest.mark.parametrize("V", [1, 1000])
def test_beside_beams_that_have_ended(sg, V):
    """Those keep their scores as well: they and the forced ones go by their number together."""
    import torch
    B, W = 30, 8
    z, mask, column = forced(B, W, V, "f32", V)
    g = torch.Generator(device="cuda").manual_seed(1)
    score = -torch.randint(0, 3, (B, W), generator=g, device="cuda").float()
    finished = torch.rand(B, W, generator=g, device="cuda") < 0.4
    s, parent, token = sg.beam_step(z, score, mask=mask, finished=finished, end=V - 1)
    want = score.sort(dim=1, descending=True, stable=True)
    assert torch.equal(s, want.values) and torch.equal(parent.long(), want.indices)
    goes_to = torch.where(finished, V - 1, column.view(B, W))
    assert torch.equal(token.long(), goes_to.gather(1, want.indices))


def test_other_columns_that_do_not_count(sg):
    """A logit so far above the others that their terms are 0 in FP32."""
    import torch
    z = torch.randn(6, 500, device="cuda")
    z[torch.arange(6), torch.arange(6) * 7] = 90 + torch.rand(6, device="cuda")
    score = torch.full((2, 3), -2.5, device="cuda")
    s, parent, token = sg.beam_step(z, score, top=3)
    assert torch.equal(s, score) and parent.tolist() == [[0, 1, 2]] * 2 and token.view(-1).tolist() == [0, 7, 14, 21, 28, 35]
