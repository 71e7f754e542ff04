"""FP32 gradients of columns whose probability is below the smallest normal number:
its product with its logarithm, the gradient of the entropy, may be above."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def test_probabilities_below_the_smallest_normal_number(cuda_device, lib):
    import torch
    import dense_fp32_matrix_04_gb300 as sg
    # log p from -80 to -110 beside one column with nearly all of it
    z = torch.cat([torch.zeros(1), torch.linspace(-80, -110, 600)])[None].cuda()
    target = torch.tensor([-1], device="cuda")
    _, H, lse = sg.logprobs(z, target)[:3]
    gh = 1000.0
    dz = sg.logprobs_backward(z, target, lse, H, torch.zeros(1, device="cuda"), torch.full((1,), gh, device="cuda"))
    logp = z.double().cpu().numpy() - float(lse)
    p = np.exp(logp)
    want = -gh * p * (logp + float(H))
    # p: 8 u (|log p| + 2) + 2^-20 relative, and half a step of 2^-149 where numbers end
    tol = gh * (np.abs(logp) + abs(float(H))) * (p * (8 * U * (np.abs(logp) + 2) + 2.0 ** -20) + 2.0 ** -149)
    got = dz.double().cpu().numpy()
    assert (np.abs(got - want) <= tol + U * np.abs(want) + 2.0 ** -149).all()
