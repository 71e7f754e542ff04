"""Log probabilities of rows whose scaled logits are large: rows of nothing but a
mask's value, plus or minus some, and large scales.  Softmax does not change when
all logits move together, so neither may its accuracy.

With u = 2^-24 and t = log2 of a term relative to the largest: a term is off by
2^-21 and 4 u |t|, a sum is added in runs of at most V / 256 + 64, so ln s is off
by at most tol = (V / 256 + 80) u + 4 u E|t| + 4 u ln s; a logit's own log
probability adds 4 u of itself, lse 4 u of the largest scaled logit, and the
entropy, which has two such terms, the second E|t| times as large, needs
tol (2 + 4 E|t|)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


# base and spread of the logits, and the scale
CASES = [
    ("f32", 1e10, 0.0, 1.0), ("f32", -1e10, 0.0, 1.0), ("f32", -1e9, 0.0, 4.0), ("f32", 3e9, 700.0, 0.01),
    ("f32", 1.1629e7, 40.0, 1.0),      # scaled by log2 e about 2^24, on both sides of it
    ("f32", -1.1629e7, 40.0, 1.0), ("f32", -2e12, 3e5, 1e-5), ("f32", 5e36, 0.0, 100.0), ("f32", 3.0, 3.0, 1e30),
    ("f32", -3e38, 1e37, 2.0), ("f32", 1e-30, 1e-30, 1e30), ("f32", 0.0, 3.0, 1e-38),
    ("bf16", 1e10, 0.0, 1.0), ("bf16", -1e9, 0.0, 1.25), ("bf16", -1e30, 1e27, 1.0), ("bf16", 2.0, 2.0, 1e10),
    ("f16", -65504.0, 0.0, 1.0), ("f16", 60000.0, 2000.0, 1e3), ("f16", 6e4, 500.0, 200.0),
]


@pytest.mark.parametrize("dtype,base,spread,scale", CASES)
@pytest.mark.parametrize("T,V", [(2, 5), (3, 1111), (2, 40000), (500, 2100)])
def test_moved_together(sg, T, V, dtype, base, spread, scale):
    import torch
    rng = np.random.RandomState(V)
    z = np.float64(base) + spread * rng.randn(T, V)
    z = torch.from_numpy(np.clip(z, -3.4e38, 3.4e38).astype(np.float32)).to(td(dtype))
    z = z.clamp(torch.finfo(td(dtype)).min, torch.finfo(td(dtype)).max).cuda()
    target = torch.from_numpy(rng.randint(0, V, T)).cuda()
    target[1] = int(z[1].float().argmax())
    logprob, entropy, lse, top_logprob, top_id = sg.logprobs(z, target, scale=scale, top=3)
    s = float(np.float32(scale))
    zz = z.double().cpu().numpy()
    m = zz.max(1, keepdims=True)
    a = s * (zz - m)
    e = np.exp(a)
    total = e.sum(1)
    p = e / total[:, None]
    et = (p * np.where(p > 0, np.abs(a), 0)).sum(1) * 1.4427
    tol = (V / 256 + 80) * U + 4 * U * et + 4 * U * np.log(total)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731

    def near(got, want, tol, what):
        tol = np.broadcast_to(tol, want.shape)
        same = (np.abs(got - want) <= tol) | ((np.abs(want) > 3.4e38) & np.isinf(got) & (np.sign(got) == np.sign(want)))
        assert same.all(), f"{what}: {got[~same][:3]} against {want[~same][:3]}"

    with np.errstate(invalid="ignore", over="ignore"):
        want = a[np.arange(T), target.cpu().numpy()] - np.log(total)
        near(f(logprob), want, tol + 4 * U * np.abs(want), "logprob")
        want = np.log(total) - (p * np.where(p > 0, a, 0)).sum(1)
        near(f(entropy), want, tol * (2 + 4 * et), "entropy")
        want = s * m[:, 0] + np.log(total)
        near(f(lse), want, tol + 4 * U * np.abs(s * m[:, 0]), "lse")
        order = np.argsort(-zz, axis=1, kind="stable")[:, :3]
        assert np.array_equal(top_id.cpu().numpy(), order)
        want = np.take_along_axis(a, order, 1) - np.log(total)[:, None]
        near(f(top_logprob), want, tol[:, None] + 4 * U * np.abs(want), "top_logprob")


def test_a_maximum_that_rises_past_the_limit(sg):
    """Threads, and a thread's later pieces, on both sides of 2^24: their sums are joined as they are."""
    import torch
    V = 60000
    z = torch.full((2, V), 1.162e7, device="cuda")
    z[0, ::2] = torch.linspace(1.1628e7, 1.163e7, V // 2, device="cuda").round()
    z[1] = z[0].flip(0)
    target = torch.tensor([0, 5], device="cuda")
    got = sg.logprobs(z, target)
    a = z.double() - z.double().max(1, keepdim=True).values
    want = torch.logsumexp(a, 1)
    p = torch.exp(a - want[:, None])
    et = float((p * a.abs()).sum(1).max()) * 1.4427
    tol = (V / 256 + 80) * U + 4 * U * et + 4 * U * float(want.max())
    lp = a[torch.arange(2), target] - want
    assert float(((got[0].double() - lp).abs() - 4 * U * lp.abs()).max()) <= tol
    h = want - (p * a).sum(1)
    assert float((got[1].double() - h).abs().max()) <= tol * (2 + 4 * et)


@pytest.mark.parametrize("dtype,base,spread,scale", [c for c in CASES if (abs(c[1]) + 4 * c[2]) * c[3] < 3e8] + [
    ("bf16", 300.0, 3.0, 1.0), ("f16", -400.0, 2.0, 1.0), ("bf16", 1e6, 0.0, 1.0), ("f16", 6e4, 30.0, 1.0),
    ("bf16", 240.0, 1.0, 1.0), ("f16", 240.0, 1.0, 1.0)])
@pytest.mark.parametrize("T,V", [(2, 5), (3, 1111), (2, 9001)])
def test_gradients_moved_together(sg, T, V, dtype, base, spread, scale):
    """lse enters the formula as the forward pass rounded it (beyond 3e8 that rounding is all that is
    left of p, and p need not be finite).  Then p is off by 8 u (|log p| + 2) +
    2^-20 relative, and for 16 bits while |lse| < 256 by another 600 u; the result by its half unit."""
    import torch
    half = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    rng = np.random.RandomState(V)
    z = np.float64(base) + spread * rng.randn(T, V)
    z = torch.from_numpy(np.clip(z, -3.4e38, 3.4e38).astype(np.float32)).to(td(dtype))
    z = z.clamp(torch.finfo(td(dtype)).min, torch.finfo(td(dtype)).max).cuda()
    target = torch.from_numpy(rng.randint(0, V, T)).cuda()
    target[0] = -1
    _, H, lse = sg.logprobs(z, target, scale=scale)[:3]
    g, gh = rng.randn(T).astype(np.float32), rng.randn(T).astype(np.float32)
    dz = sg.logprobs_backward(z, target, lse, H, torch.from_numpy(g).cuda(), torch.from_numpy(gh).cuda(), scale=scale)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    s, got, l64, h64 = float(np.float32(scale)), f(dz), f(lse), f(H)
    logp = s * f(z) - l64[:, None]
    p = np.exp(logp)
    logp = np.where(p > 0, logp, 0)
    y = target.cpu().numpy()
    gl = np.where(y >= 0, g, 0).astype(np.float64)
    hit = np.zeros((T, V))
    hit[np.arange(T), np.maximum(y, 0)] = gl
    e = gh.astype(np.float64)[:, None]
    with np.errstate(over="ignore"):
        want = s * (hit - gl[:, None] * p - e * p * (logp + h64[:, None]))
        size = p * (np.abs(gl[:, None]) + np.abs(e) * (np.abs(logp) + np.abs(h64[:, None])))
        rel = 8 * U * (np.abs(logp) + 2) + 2.0 ** -20 + (600 * U if dtype != "f32" else 0)
        tol = s * (size * rel + 4 * U * np.abs(hit)) + half * np.abs(want) * 1.01 + (2.0 ** -25 if dtype == "f16" else 2.0 ** -126)
        top = torch.finfo(td(dtype)).max
        same = (np.abs(got - want) <= tol) | ((np.abs(want) > top) & np.isinf(got) & (np.sign(got) == np.sign(want)))
        assert same.all(), f"{got[~same][:4]} against {want[~same][:4]}"


def test_the_largest_scale(sg):
    import torch
    z = torch.tensor([[0.0, 0.0, -1e-38, 0.0], [1.0, 0.5, -1.0, 0.0]], device="cuda")
    target = torch.tensor([1, 0], device="cuda")
    scale = 2.0 ** 127
    logprob, entropy, lse = sg.logprobs(z, target, scale=scale)
    a = torch.logsumexp(z[0].double() * scale, 0)
    p = torch.exp(z[0].double() * scale - a)
    # (three columns of 1, one of 2^-2.4: sums and logarithms of numbers near 1, ten roundings and 2^-21)
    assert abs(float(lse[0]) - float(a)) < 2.0 ** -19 and abs(float(logprob[0]) + float(a)) < 2.0 ** -19
    assert abs(float(entropy[0]) + float((p * p.log()).sum())) < 2.0 ** -18
    assert float(logprob[1]) == 0 and float(entropy[1]) == 0
