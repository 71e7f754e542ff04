"""Gradients of rows with nearly all of the probability in one column, whose log p
is a small difference of large numbers.

With u = 2^-24, log p is rounded once, u |log p|; p is off by 8 u (|log p| + 2) +
2^-20 relative and the sums with g and the entropy by a few u of their terms, so
each term's magnitude times 8 u (|log p| + 2) + 2^-20 bounds the error; 4 u of the
target's own term, half a unit of the result's type, and 2^-150 of p's terms where
numbers end come on top."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_UNIT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V,spread,base", [(600, 448, 8.0, 0.0), (300, 323, 4.0, 60.0), (40, 5003, 9.0, -200.0),
                                             (20, 40001, 20.0, 0.0)])
@pytest.mark.parametrize("scored", [True, False])
def test_peaked_rows(cuda_device, lib, T, V, spread, base, scored, dtype):
    import torch
    import dense_fp32_matrix_04_gb300 as sg
    rng = np.random.RandomState(T + V)
    z = (base + spread * rng.randn(T, V)).astype(np.float32)
    z[np.arange(T), rng.randint(0, V, T)] = base + spread * rng.uniform(3, 5, T)
    z = torch.from_numpy(z).to(td(dtype)).cuda()
    target = torch.from_numpy(rng.randint(0, V, T) if scored else np.full(T, -1)).cuda()
    target[::3] = z[::3].float().argmax(1) if scored else -1
    scale = 1.25
    _, H, lse = sg.logprobs(z, target, scale=scale)[:3]
    g, gh = rng.randn(T).astype(np.float32), rng.randn(T).astype(np.float32)
    dz = sg.logprobs_backward(z, target, lse, H, torch.from_numpy(g).cuda(), torch.from_numpy(gh).cuda(), scale=scale)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    logp = scale * f(z) - f(lse)[:, None]
    p = np.exp(logp)
    y = target.cpu().numpy()
    gl, e, h = np.where(y >= 0, g, 0).astype(np.float64)[:, None], gh.astype(np.float64)[:, None], f(H)[:, None]
    hit = np.zeros((T, V))
    hit[np.arange(T), np.maximum(y, 0)] = gl[:, 0]
    want = scale * (hit - gl * p - e * p * (logp + h))
    terms = np.abs(gl) + np.abs(e) * (np.abs(logp) + np.abs(h))
    tol = scale * terms * (p * (8 * U * (np.abs(logp) + 2) + 2.0 ** -20) + 2.0 ** -149) + scale * 4 * U * np.abs(hit)
    tol = tol + HALF_UNIT[dtype] * np.abs(want) * 1.01 + SMALLEST[dtype]
    bad = ~(np.abs(f(dz) - want) <= tol)
    assert not bad.any(), f"{bad.sum()} off: {f(dz)[bad][:4]} against {want[bad][:4]}, worst {(np.abs(f(dz) - want) / tol).max():.3g}"
