"""Gradients of rows whose logits hold -infinity: such a column cannot occur, so its
gradient is 0 to the bit whatever the scale, the other logits and the column's
place beside the target are.

Elsewhere, with u = 2^-24, p is off by 8 u (|scale z| + |lse| + 2) + 2^-20
relative (lse, which comes rounded to FP32, enters the formula as it is), and the
result is rounded once to its type."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_UNIT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [7, 40, 1001, 9000])
@pytest.mark.parametrize("scale", [1.0, 1e-3, 1e-5, 1e-30])
def test_columns_that_cannot_occur(sg, V, scale, dtype):
    import torch
    T = 6
    rng = np.random.RandomState(V)
    z = torch.from_numpy((3 * rng.randn(T, V)).astype(np.float32)).to(td(dtype)).cuda()
    lowest = torch.finfo(td(dtype)).min
    z[0] = lowest                       # nothing but the lowest value, and -infinity
    z[1] = lowest
    z[2, 0::3] = lowest                 # all three kinds
    z[:, 1::3] = float("-inf")
    z[4, 1:] = float("-inf")            # one column
    target = torch.tensor([0, -1, 2, 1, 0, -1], device="cuda")   # the fourth row's cannot occur
    lp, H, lse = sg.logprobs(z, target, scale=scale)[:3]
    g, gh = rng.randn(T).astype(np.float32) * 1000, rng.randn(T).astype(np.float32) * 1000
    for with_entropy in (True, False):
        dz = sg.logprobs_backward(z, target, lse, H, torch.from_numpy(g).cuda(),
                                  torch.from_numpy(gh).cuda() if with_entropy else None, scale=scale)
        dead = torch.isinf(z)
        assert bool((dz[dead] == 0).all()), f"{int((dz[dead] != 0).sum())} columns that cannot occur have a gradient"
        zz, s = z.double().cpu().numpy(), float(np.float32(scale))
        got, l64, h64 = dz.double().cpu().numpy(), lse.double().cpu().numpy(), H.double().cpu().numpy()
        for t in range(T):
            if abs(l64[t]) > 1e4:
                continue                # lse holds nothing of the differences between such logits
            a = s * zz[t]
            logp = a - l64[t]
            p = np.exp(logp)
            logp = np.where(p > 0, logp, 0)
            y, e = int(target[t]), (gh[t] if with_entropy else 0.0)
            hit = np.zeros(V)
            if y >= 0 and a[y] > -np.inf:
                hit[y] = g[t]
            gl = g[t] if y >= 0 else 0.0
            want = s * (hit - gl * p - e * p * (logp + h64[t]))
            size = p * (abs(gl) + abs(e) * (np.abs(logp) + abs(h64[t])))
            rel = 8 * U * (np.abs(np.where(p > 0, a, 0)) + abs(l64[t]) + 2) + 2.0 ** -20
            tol = s * (size * rel + 4 * U * np.abs(hit)) + HALF_UNIT[dtype] * np.abs(want) * 1.01
            tol = tol + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
            assert (np.abs(got[t] - want) <= tol).all(), t
