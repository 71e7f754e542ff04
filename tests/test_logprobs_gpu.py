"""Log probabilities, entropy, log-sum-exp and alternatives of rows of logits,
and their gradient, against the formulas in 64 bits.

Tolerances, with u = 2^-24: a term 2^t is off by 2^-21 and 4 u |t| relative, a
sum is added in runs of at most V / 256 + 64, so ln s is off by at most
tol_s = (V / 256 + 80) u + 4 u E|t|, where E|t| is the mean of |t| under p;
lse = scale m + ln s adds 4 u (|scale m| + |ln s|), log p the same for its own
logit; the entropy has two such terms, the second E|t| times as large."""

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


def pack(allowed):
    rows, V = allowed.shape
    full = np.zeros((rows, (V + 31) // 32 * 32), np.uint32)
    full[:, :V] = allowed
    words = (full.reshape(rows, -1, 32) << np.arange(32, dtype=np.uint32)).sum(2, dtype=np.uint32)
    return words.view(np.int32)


def case(T, V, dtype, mask_rows, seed, pad=0, offset=0, spread=3.0):
    import torch
    rng = np.random.RandomState(seed)
    z = rng.randn(T, V).astype(np.float32) * spread
    buf = torch.full((T * (V + pad) + offset,), float("nan"), dtype=td(dtype), device="cuda")
    v = buf[offset:].view(T, V + pad)[:, :V]
    v.copy_(torch.from_numpy(z))
    target = rng.randint(0, V, T)
    target[rng.rand(T) < 0.2] = -1
    allowed = rng.rand(mask_rows, V) < 0.7 if mask_rows else None
    mask = torch.from_numpy(pack(allowed)).cuda() if mask_rows else None
    return v, torch.from_numpy(target).cuda(), mask, allowed


def reference(z, target, allowed, scale, top):
    """The formulas in 64 bits, row by row; z already masked to -inf."""
    z = z.double().cpu().numpy()
    if allowed is not None:
        z = np.where(np.broadcast_to(allowed, z.shape), z, -np.inf)
    T, V = z.shape
    out = {k: np.zeros(T) for k in ("logprob", "entropy", "lse", "tol", "et", "m")}
    out["top_logprob"], out["top_id"] = np.full((T, top), -np.inf), np.full((T, top), -1)
    for t in range(T):
        a = scale * z[t]
        y = int(target[t])
        m = a.max() if V else -np.inf
        out["m"][t] = m
        if m == -np.inf:
            out["lse"][t] = -np.inf
            out["logprob"][t] = -np.inf if y >= 0 else 0
            continue
        e = np.exp(a - m)
        s = e.sum()
        p = e / s
        d = np.where(p > 0, a - m, 0)
        out["lse"][t] = m + np.log(s)
        out["entropy"][t] = np.log(s) - (p * d).sum()
        out["logprob"][t] = 0 if y < 0 else a[y] - m - np.log(s)
        out["et"][t] = (p * np.abs(d)).sum() * 1.4427
        out["tol"][t] = (V / 256 + 80) * U + 4 * U * out["et"][t] + 4 * U * np.log(s)
        order = np.argsort(-z[t], kind="stable")[:top]
        order = order[z[t][order] > -np.inf]
        out["top_id"][t, :len(order)] = order
        out["top_logprob"][t, :len(order)] = a[order] - out["lse"][t]
    return out


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    same = (got == want) | (np.abs(got - want) <= tol)
    assert same.all(), f"{what}: {got[~same][:4]} against {want[~same][:4]}"


def check(sg, z, target, mask, allowed, scale, top):
    got = sg.logprobs(z, target, scale=scale, mask=mask, top=top)
    scale = float(np.float32(scale))
    want = reference(z, target.cpu().numpy(), allowed, scale, top)
    tol = want["tol"]
    with np.errstate(invalid="ignore"):
        near(got[0], want["logprob"], tol + 4 * U * np.abs(np.nan_to_num(want["logprob"], neginf=0)), "logprob")
        near(got[1], want["entropy"], tol * (2 + 4 * want["et"]), "entropy")
        near(got[2], want["lse"], tol + 4 * U * np.abs(np.nan_to_num(want["m"], neginf=0)), "lse")
        if top:
            near(got[3], want["top_logprob"], tol[:, None] + 4 * U * np.abs(np.nan_to_num(want["top_logprob"], neginf=0)),
                 "top_logprob")
            assert np.array_equal(got[4].cpu().numpy(), want["top_id"])
    return got


SHAPES = [(1, 1), (2, 3), (1, 17), (5, 31), (3, 32), (4, 33), (2, 1000), (7, 1024), (3, 4097), (2, 8192), (1, 50001),
          (3, 131072), (40, 9001), (300, 1111), (700, 260)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("top", [0, 1, 20])
def test_forward(sg, T, V, top, dtype):
    mask_rows = {0: 0, 1: T, 2: 1}[(T + V + top) % 3]
    z, target, mask, allowed = case(T, V, dtype, mask_rows, T + V)
    check(sg, z, target, mask, allowed, [1.0, 0.7, 1.3][V % 3], top)


@pytest.mark.parametrize("dtype,pad,offset", [("f32", 1, 1), ("bf16", 3, 5), ("bf16", 8, 8), ("f16", 1, 7), ("f32", 0, 3)])
def test_strides_and_alignment(sg, dtype, pad, offset):
    z, target, mask, allowed = case(9, 3001, dtype, 9, 4, pad, offset)
    check(sg, z, target, mask, allowed, 1.1, 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lowest_column(sg, dtype):
    import torch
    rng = np.random.RandomState(1)
    z = torch.from_numpy(rng.randint(0, 4, (6, 9000)).astype(np.float32)).to(td(dtype)).cuda()
    z[0] = 1.5                       # every logit the same
    z[1] = torch.arange(9000, device="cuda").float() // 100          # rising, in runs of equals
    z[2] = -z[1].float()
    z[3, 5::7] = 9.0
    target = torch.arange(6, device="cuda")
    for top in (1, 7, 32):
        check(sg, z, target, None, None, 1.0, top)


def test_rising_and_falling_rows(sg):
    import torch
    up = torch.linspace(-8, 8, 40000, device="cuda")
    z = torch.stack([up, up.flip(0)])
    check(sg, z, torch.tensor([39999, 0], device="cuda"), None, None, 1.0, 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [70, 5000, 40000])
def test_masks_that_leave_little_or_nothing(sg, V, dtype):
    import torch
    T = 8
    z, target, _, _ = case(T, V, dtype, 0, 11)
    lowest = torch.finfo(td(dtype)).min
    allowed = np.ones((T, V), bool)
    allowed[0] = False                                # nothing
    allowed[1] = False
    allowed[1, V - 1] = True                          # one column
    allowed[2] = np.arange(V) % 2 == 0
    z[2, 1::2] = float("nan")                         # NaN where it is masked
    z[3, :] = float("-inf")                           # nothing without a mask
    z[4, :] = lowest                                  # all of them the lowest value
    z[5, 1:] = lowest
    z[6, 1:] = float("-inf")                          # one column without a mask
    allowed[7] = np.arange(V) != 3
    z[7, 3] = float("inf")                            # infinity where it is masked
    target[:] = torch.tensor([0, V - 1, 1, 2, 3, 0, 5, 3])
    mask = torch.from_numpy(pack(allowed)).cuda()
    zz = z.clone()
    zz[torch.from_numpy(~allowed).cuda()] = float("-inf")
    got = sg.logprobs(z, target, mask=mask, top=5)
    want = reference(zz, target.cpu().numpy(), allowed, 1.0, 5)
    near(got[2], want["lse"], want["tol"] + 8 * U * np.abs(np.nan_to_num(want["m"], neginf=0)), "lse")
    near(got[0], want["logprob"], want["tol"] + 4 * U * np.abs(np.nan_to_num(want["logprob"], neginf=0)), "logprob")
    near(got[1], want["entropy"], want["tol"] * (2 + 4 * want["et"]), "entropy")
    assert np.array_equal(got[4].cpu().numpy(), want["top_id"])
    g = torch.ones(T, device="cuda")
    dz = sg.logprobs_backward(z, target, got[2], got[1], g, g, mask=mask)
    assert bool((dz[torch.from_numpy(~allowed).cuda()] == 0).all())
    assert bool((dz[0] == 0).all()) and bool((dz[3] == 0).all())
    assert bool(torch.isfinite(dz).all())


def test_rows_that_are_not_finite(sg):
    import torch
    z, target, _, _ = case(4, 3000, "f32", 0, 2)
    target[:] = 5
    z[0, 2999] = float("nan")
    z[1, 100] = float("inf")
    z[2, :] = float("-inf")
    z[2, 17] = float("nan")
    got = sg.logprobs(z, target, top=4)
    for v in got[:3]:
        assert bool(torch.isnan(v[:3]).all()) and bool(torch.isfinite(v[3]))
    assert bool((got[4][:3] == -1).all()) and bool((got[4][3] >= 0).all())


def test_targets_outside_the_vocabulary(sg):
    import torch
    z, target, _, _ = case(3, 100, "f32", 0, 2)
    target[:] = torch.tensor([100, 2 ** 40, -5])
    got = sg.logprobs(z, target)
    assert bool(torch.isnan(got[0][:2]).all()) and float(got[0][2]) == 0
    dz = sg.logprobs_backward(z, target, got[2], got[1], torch.ones(3, device="cuda"))
    assert bool(torch.isnan(dz[:2]).all()) and bool((dz[2] == 0).all())


def gradient64(z, target, allowed, scale, lse, H, g, gh):
    z = z.double().cpu().numpy()
    a = scale * z
    if allowed is not None:
        a = np.where(np.broadcast_to(allowed, a.shape), a, -np.inf)
    T, V = a.shape
    logp = a - lse[:, None]
    p = np.exp(logp)
    lp = np.where(p > 0, logp, 0)
    gl = np.where(target >= 0, g, 0)
    d = -gl[:, None] * p - gh[:, None] * p * (lp + H[:, None])
    size = p * (np.abs(gl)[:, None] + np.abs(gh)[:, None] * (np.abs(lp) + np.abs(H)[:, None]))
    rel = 8 * U * (np.abs(np.where(p > 0, a, 0)) + np.abs(lse)[:, None] + 2) + 2.0 ** -20
    rows = np.arange(T)
    at = np.maximum(target, 0)
    hit = np.where(a[rows, at] > -np.inf, gl, 0)
    d[rows, at] += hit
    size2 = np.zeros_like(size)
    size2[rows, at] = np.abs(hit)
    return scale * d, scale * (size * rel + 4 * U * size2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V,pad,offset", [(1, 1, 0, 0), (3, 7, 0, 0), (2, 33, 1, 3), (5, 1000, 0, 0), (4, 4097, 0, 0),
                                            (3, 9001, 8, 8), (300, 260, 0, 0), (1, 131072, 0, 0)])
@pytest.mark.parametrize("entropy", [True, False])
def test_backward(sg, T, V, pad, offset, dtype, entropy):
    import torch
    mask_rows = {0: 0, 1: T, 2: 1}[(T + V) % 3]
    z, target, mask, allowed = case(T, V, dtype, mask_rows, V, pad, offset, spread=1.5)
    scale = 0.8
    lp, H, lse = sg.logprobs(z, target, scale=scale, mask=mask)[:3]
    rng = np.random.RandomState(5)
    g, gh = rng.randn(T).astype(np.float32), rng.randn(T).astype(np.float32) * entropy
    dz = sg.logprobs_backward(z, target, lse, H, torch.from_numpy(g).cuda(),
                              torch.from_numpy(gh).cuda() if entropy else None, scale=scale, mask=mask)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    finite = np.isfinite(f(lse))
    want, tol = gradient64(z, target.cpu().numpy(), allowed, float(np.float32(scale)), np.where(finite, f(lse), np.inf),
                           f(H), g.astype(np.float64), gh.astype(np.float64))
    want = np.where(finite[:, None], want, 0)
    near(dz, want, tol + HALF_UNIT[dtype] * np.abs(want) * 1.01 + (2.0 ** -25 if dtype == "f16" else 0), "dz")
    if pad == 0 and offset == 0:
        into = z.clone()
        sg.logprobs_backward(into, target, lse, H, torch.from_numpy(g).cuda(),
                             torch.from_numpy(gh).cuda() if entropy else None, scale=scale, mask=mask, out=into)
        assert bool((into == dz).all()), "in place differs"


def test_rows_at_different_alignments(sg):
    import torch
    z, target, _, _ = case(5, 1001, "bf16", 0, 3, pad=0, offset=0)
    lp, H, lse = sg.logprobs(z, target)[:3]
    g = torch.ones(5, device="cuda")
    buf = torch.full((5, 1010), 9.0, dtype=torch.bfloat16, device="cuda")
    got = sg.logprobs_backward(z, target, lse, H, g, g, out=buf[:, 3:1004])
    assert bool((got == sg.logprobs_backward(z, target, lse, H, g, g)).all())
    assert bool((buf[:, :3] == 9).all()) and bool((buf[:, 1004:] == 9).all())


def test_gradient_against_differences():
    """The formula itself: central differences of logprob and entropy in 64 bits."""
    rng = np.random.RandomState(4)
    T, V, scale = 3, 11, 0.9
    z = rng.randn(T, V)
    target = np.array([2, -1, 10])
    g, gh = rng.randn(T), rng.randn(T)

    def value(z):
        a = scale * z
        lse = np.log(np.exp(a).sum(1))
        logp = a - lse[:, None]
        H = -(np.exp(logp) * logp).sum(1)
        lp = np.where(target >= 0, logp[np.arange(T), np.maximum(target, 0)], 0)
        return lse, H, (g * lp + gh * H).sum()

    class A(np.ndarray):
        def double(self):
            return self

        def cpu(self):
            return self

        def numpy(self):
            return np.asarray(self)

    lse, H, _ = value(z)
    want, _ = gradient64(z.view(A), target, None, scale, lse, H, g, gh)
    for i in np.ndindex(T, V):
        d = np.zeros((T, V))
        d[i] = 1e-5
        assert abs((value(z + d)[2] - value(z - d)[2]) / 2e-5 - want[i]) < 1e-8


def test_another_stream_and_a_graph(sg):
    import torch
    for T in (2, 400):
        z, target, mask, _ = case(T, 5000, "bf16", 1, 6)
        want = sg.logprobs(z, target, mask=mask, top=8)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = sg.logprobs(z, target, mask=mask, top=8, stream=side)
        side.synchronize()
        assert all(bool((a == b).all()) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = sg.logprobs(z, target, mask=mask, top=8)
        z.copy_(z.flip(0).clone())
        graph.replay()
        torch.cuda.synchronize()
        assert bool((out[2] == want[2].flip(0)).all()) and bool((out[4] == want[4].flip(0)).all())


def test_offsets_beyond_32_bits(sg):
    import torch
    # 3 rows 1.5 billion elements apart: the last starts past 2^31 elements
    V, ld = 1000, 1_500_000_000
    buf = torch.zeros(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    z = buf.as_strided((3, V), (ld, 1))
    z.copy_(torch.randn(3, V, device="cuda"))
    target = torch.tensor([1, 2, 3], device="cuda")
    got = sg.logprobs(z, target, top=3)
    want = sg.logprobs(z.contiguous(), target, top=3)
    assert all(bool((a == b).all()) for a, b in zip(got, want))


def test_python_refusals(sg):
    import torch
    z, target, mask, _ = case(4, 100, "f32", 4, 1)
    with pytest.raises(ValueError):
        sg.logprobs(z, target[:3])
    with pytest.raises(TypeError):
        sg.logprobs(z, target.int())
    with pytest.raises(ValueError):
        sg.logprobs(z, target, mask=mask[:2])
    with pytest.raises(ValueError):
        sg.logprobs(z, target, mask=mask[:, :3])
    with pytest.raises(sg.SgemmError):
        sg.logprobs(z, target, top=33)
    with pytest.raises(sg.SgemmError):
        sg.logprobs(z, target, scale=0.0)
    with pytest.raises(sg.SgemmError):
        sg.logprobs_backward(z, target, torch.zeros(4, device="cuda"), None, torch.zeros(4, device="cuda"),
                             torch.zeros(4, device="cuda"))


@pytest.mark.parametrize("dtype,masked", [("f32", False), ("bf16", True)])
def test_many_long_rows(sg, dtype, masked):
    """Thousands of rows of tens of thousands of columns, which blocks of four warps walk.  As
    above, with runs of at most V / 128 + 64; a logit's own log probability adds 4 u |scale z|."""
    import torch
    T, V, top, scale = 2600, 16411, 5, 0.75
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    z = (3 * torch.randn(T, V, generator=g, device="cuda")).to(td(dtype))
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::9] = -1
    mask = allowed = None
    if masked:
        rng = np.random.RandomState(3)
        rows = rng.rand(1, V) < 0.6
        mask, allowed = torch.from_numpy(pack(rows)).cuda(), torch.from_numpy(rows).cuda()
    got = sg.logprobs(z, target, scale=scale, mask=mask, top=top)
    for r0 in range(0, T, 650):
        rows = slice(r0, r0 + 650)
        d = z[rows].double() * scale
        if masked:
            d = d.masked_fill(~allowed, -float("inf"))
        lse = torch.logsumexp(d, 1)
        lp = d - lse[:, None]
        p = lp.exp()
        h = -torch.where(p > 0, p * lp, 0.0).sum(1)
        m = d.max(1).values
        et = torch.where(p > 0, p * (d - m[:, None]).abs(), 0.0).sum(1) / np.log(2)
        tol_s = (V / 128 + 80) * U + 4 * U * et
        tol = tol_s + 4 * U * (m.abs() + (lse - m).abs())
        assert bool(((got[2][rows].double() - lse).abs() <= tol).all())
        assert bool(((got[1][rows].double() - h).abs() <= tol + (tol_s + 8 * U) * et).all())
        y = target[rows].clamp(min=0)[:, None]
        want = torch.where(target[rows] >= 0, lp.gather(1, y)[:, 0], 0.0)
        own = tol + 4 * U * d.gather(1, y)[:, 0].abs().nan_to_num(posinf=0.0)
        same = (got[0][rows].double() == want) | ((got[0][rows].double() - want).abs() <= own)
        assert bool(same.all())
        best, ids = torch.sort(d, dim=1, descending=True, stable=True)
        assert torch.equal(got[4][rows].long(), ids[:, :top])
        own = tol[:, None] + 4 * U * best[:, :top].abs()
        assert bool(((got[3][rows].double() - (best[:, :top] - lse[:, None])).abs() <= own).all())
