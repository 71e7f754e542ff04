"""sgemm_block_norm and its gradient against the formulas in 64 bits.

Tolerances, with u = 2^-24 and e the output type's half unit (u, 2^-8, 2^-11):
a sum of squares over a row is added in runs of at most 64 and then a tree, so
rho is off by at most 48 u relative; r = x + a g h by 64 u (|x| + |a g h|); n
by that times |rho2 w_pre| and another 64 u |n|; each plus e times the result
(and, for FP16, its smallest step).  The gradient's bounds follow its terms
with every one in magnitude.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = ["f32", "bf16", "f16"]
HALF_UNIT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
STEP = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -24}


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def padded(rows, cols, pad, offset, dtype, gen):
    """A rows x cols view into a larger buffer of NaN."""
    import torch
    buf = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
    return v


def inputs(T, D, dtype, groups, post, seed, pad=0, offset=0, wdtype=None):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = td(dtype)
    s = {k: padded(T, D, pad, offset, dt, g) for k in ("x", "y", "dn", "dr")}
    s["gate"] = padded(groups, D, pad, offset, dt, g) if groups else None
    wd = wdtype or torch.float32
    s["w_pre"] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wd)
    s["w_post"] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wd) if post else None
    return s


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def forward64(s, scale, eps):
    x, y, w, p, g = (f64(s[k]) for k in ("x", "y", "w_pre", "w_post", "gate"))
    T = x.shape[0]
    rho = 1 / np.sqrt((y ** 2).mean(1) + eps) if p is not None else np.ones(T)
    h = y * rho[:, None] * (p if p is not None else 1)
    gg = np.repeat(g, T // g.shape[0], 0) if g is not None else np.ones_like(x)
    r = x + scale * gg * h
    rho2 = 1 / np.sqrt((r ** 2).mean(1) + eps)
    size = np.abs(x) + np.abs(scale * gg * h)
    return r, r * rho2[:, None] * w, rho, rho2, size, h, gg


def check(got, want, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / tol):.3g} of the bound"


SHAPES = [(1, 1, 0), (1, 64, 1), (3, 7, 3), (5, 31, 1), (2, 255, 0), (7, 256, 7), (33, 264, 3), (12, 1000, 4),
          (9, 1111, 9), (4, 4096, 2), (2, 4104, 1), (3, 8192, 3), (2, 8200, 1), (2, 12345, 0), (700, 96, 10),
          (1000, 130, 4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D,groups", SHAPES)
@pytest.mark.parametrize("post", [True, False])
def test_forward(sg, T, D, groups, dtype, post):
    s = inputs(T, D, dtype, groups, post, seed=T * 7 + D)
    scale, eps = -0.75, 1e-5
    r, n, rstd = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"], scale, eps)
    r64, n64, rho, rho2, size, _, _ = forward64(s, scale, eps)
    e, step = HALF_UNIT[dtype], STEP[dtype]
    check(r, r64, 64 * U * size + e * np.abs(r64) + step, "r")
    tol_n = np.abs(rho2[:, None] * f64(s["w_pre"])) * 64 * U * size + (e + 64 * U) * np.abs(n64) + step
    check(n, n64, tol_n * (1 + 1e-3), "n")
    check(rstd, np.stack([rho, rho2]), 64 * U * np.stack([rho, rho2]) * (1 + np.stack([rho * 0, rho2 * np.sqrt((size ** 2).mean(1))])), "rstd")


@pytest.mark.parametrize("dtype,pad,offset", [("f32", 1, 1), ("bf16", 3, 5), ("bf16", 8, 8), ("f16", 8, 0), ("f32", 4, 4)])
def test_strides_and_alignment(sg, dtype, pad, offset):
    import torch
    T, D = 13, 264
    s = inputs(T, D, dtype, 13, True, 5, pad, offset)
    buf = torch.full((T, D + pad), 7.0, dtype=td(dtype), device="cuda")
    r, n, _ = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"], 0.5, 1e-6, out=buf[:, :D])
    r64, n64, _, _, size, _, _ = forward64(s, 0.5, 1e-6)
    check(r, r64, 64 * U * size + HALF_UNIT[dtype] * np.abs(r64) + STEP[dtype], "r")
    assert bool((buf[:, D:] == 7.0).all()), "wrote between the rows"
    grads = sg.block_norm_backward(s["x"], s["y"], s["w_pre"], sg.block_norm(
        s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"], 0.5)[2], s["dn"], s["dr"], s["w_post"], s["gate"], 0.5)
    c = {k: v.contiguous() if v is not None else None for k, v in s.items()}
    dense = sg.block_norm_backward(c["x"], c["y"], c["w_pre"], sg.block_norm(
        c["x"], c["y"], c["w_pre"], c["w_post"], c["gate"], 0.5)[2], c["dn"], c["dr"], c["w_post"], c["gate"], 0.5)
    e = HALF_UNIT[dtype]
    for a, b in zip(grads, dense):
        # other pieces a thread, so other sums: a rounding of the result apart at most (and of the terms)
        assert (a.double() - b.double()).abs().max() <= 4 * e * b.double().abs().max() + 1e-5


def test_in_place_on_the_residual_stream(sg):
    s = inputs(50, 520, "bf16", 1, True, 9)
    want = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"], 0.5)
    x = s["x"].clone()
    got = sg.block_norm(x, s["y"], s["w_pre"], s["w_post"], s["gate"], 0.5, out=x)
    assert bool((x == want[0]).all()) and bool((got[1] == want[1]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D", [(1, 64), (5, 1111), (3, 4096), (2, 9000), (300, 72)])
def test_quantized_rows_are_the_norm_quantised(sg, T, D, dtype):
    s = inputs(T, D, dtype, 0, True, 77)
    s["w_pre"][:2] *= 30
    r, q, scale, _ = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], None, 0.5, quantize=True)
    _, n64, _, rho2, size, _, _ = forward64(s, 0.5, 1e-6)
    top = np.abs(n64).max(1)
    tol_n = np.abs(rho2[:, None] * f64(s["w_pre"])) * 64 * U * size + 64 * U * np.abs(n64)
    assert (np.abs(f64(scale) - top / 127) <= (tol_n.max(1) + 4 * U * top) / 127).all()
    # within half a step of the value, and the roundings before it
    err = np.abs(f64(q) * (top / 127)[:, None] - n64)
    assert (err <= (top / 127)[:, None] * (0.5 + 1e-3)).all()
    assert (np.abs(f64(q)).max(1) == 127).all()


def backward64(s, scale, rstd):
    x, y, w, p, g, dn, dr = (f64(s[k]) for k in ("x", "y", "w_pre", "w_post", "gate", "dn", "dr"))
    T, D = x.shape
    rho, rho2 = rstd[0][:, None], rstd[1][:, None]
    post = p is not None
    p = p if post else np.ones(D)
    gg = np.repeat(g, T // g.shape[0], 0) if g is not None else np.ones_like(x)
    hn = y * rho
    h = hn * p
    r = x + scale * gg * h
    size = np.abs(x) + np.abs(scale * gg * h)
    u = dn * w
    drr = dr if dr is not None else np.zeros_like(x)
    dx = drr + rho2 * (u - r * rho2 ** 2 * (u * r).mean(1, keepdims=True))
    # each term in magnitude
    mx = np.abs(drr) + rho2 * (np.abs(u) + size * rho2 ** 2 * (np.abs(u) * size).mean(1, keepdims=True))
    dh, mh = scale * dx, abs(scale) * mx
    v, mv = dh * gg * p, mh * np.abs(gg * p)
    dy = rho * (v - hn * (v * hn).mean(1, keepdims=True)) if post else v
    my = rho * (mv + np.abs(hn) * (mv * np.abs(hn)).mean(1, keepdims=True)) if post else mv
    out = {"dx": (dx, mx), "dy": (dy, my), "dw_pre": ((dn * r * rho2).sum(0), (np.abs(dn) * size * rho2).sum(0)),
           "dw_post": ((dh * gg * hn).sum(0), (mh * np.abs(gg * hn)).sum(0)) if post else None}
    if g is not None:
        G = g.shape[0]
        out["dgate"] = ((dh * h).reshape(G, T // G, D).sum(1), (mh * np.abs(h)).reshape(G, T // G, D).sum(1))
    else:
        out["dgate"] = None
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D,groups", SHAPES + [(611, 40, 13), (2000, 33, 1)])
@pytest.mark.parametrize("post", [True, False])
def test_backward(sg, T, D, groups, dtype, post):
    s = inputs(T, D, dtype, groups, post, seed=T * 3 + D)
    if (T + D) % 2:
        s["dr"] = None
    _, _, rstd = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"], 0.6, 1e-6)
    got = dict(zip(("dx", "dy", "dw_pre", "dw_post", "dgate"), sg.block_norm_backward(
        s["x"], s["y"], s["w_pre"], rstd, s["dn"], s["dr"], s["w_post"], s["gate"], 0.6)))
    e, step = HALF_UNIT[dtype], STEP[dtype]
    for k, want in backward64(s, 0.6, f64(rstd)).items():
        assert (got[k] is None) == (want is None), k
        if want is None:
            continue
        half = U if k.startswith("dw") else e
        # terms within 128 u, a sum over rows in runs of at most 64
        check(got[k], want[0], 256 * U * want[1] + half * np.abs(want[0]) + (0 if k.startswith("dw") else step), k)


def test_weights_of_the_rows_type(sg):
    import torch
    s = inputs(40, 520, "bf16", 0, True, 31, wdtype=torch.bfloat16)
    r, n, rstd = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"])
    r64, n64, _, rho2, size, _, _ = forward64(s, 1.0, 1e-6)
    check(r, r64, 64 * U * size + 2.0 ** -8 * np.abs(r64), "r")
    got = sg.block_norm_backward(s["x"], s["y"], s["w_pre"], rstd, s["dn"], s["dr"], s["w_post"])
    want = backward64(s, 1.0, f64(rstd))
    assert got[2].dtype == torch.bfloat16
    check(got[2], want["dw_pre"][0], 256 * U * want["dw_pre"][1] + 2.0 ** -8 * np.abs(want["dw_pre"][0]), "dw_pre")
    check(got[3], want["dw_post"][0], 256 * U * want["dw_post"][1] + 2.0 ** -8 * np.abs(want["dw_post"][0]), "dw_post")


def test_gradient_against_differences():
    """The formula itself: central differences of the 64-bit forward pass."""
    rng = np.random.RandomState(3)
    T, D, G, scale, eps = 4, 9, 2, 0.7, 1e-6

    class A(np.ndarray):
        def double(self):
            return self

        def cpu(self):
            return self

        def numpy(self):
            return np.asarray(self)

    s = {k: rng.randn(*sh).view(A) for k, sh in (("x", (T, D)), ("y", (T, D)), ("dn", (T, D)), ("dr", (T, D)),
                                                 ("gate", (G, D)), ("w_pre", (D,)), ("w_post", (D,)))}
    r, n, rho, rho2, *_ = forward64(s, scale, eps)
    want = backward64(s, scale, np.stack([rho, rho2]))

    def loss():
        r, n, *_ = forward64(s, scale, eps)
        return (np.asarray(s["dn"]) * n).sum() + (np.asarray(s["dr"]) * r).sum()

    for name, key in (("x", "dx"), ("y", "dy"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate")):
        for i in np.ndindex(*s[name].shape):
            old, d = s[name][i], 1e-5
            s[name][i] = old + d
            up = loss()
            s[name][i] = old - d
            down = loss()
            s[name][i] = old
            assert abs((up - down) / (2 * d) - want[key][0][i]) < 1e-7 * (1 + want[key][1][i]), (name, i)


def test_rows_that_are_zero_and_not_finite(sg):
    import torch
    s = inputs(4, 128, "f32", 0, True, 1)
    s["x"][0] = 0
    s["y"][0] = 0
    s["y"][2, 5] = float("nan")
    s["x"][3, 7] = float("inf")
    r, n, _ = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"])
    assert bool((r[0] == 0).all()) and bool((n[0] == 0).all())
    assert bool(torch.isfinite(n[1]).all())
    assert bool(torch.isnan(n[2]).all())
    assert bool(torch.isnan(n[3, 7]))
    _, q, scale, _ = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], quantize=True)
    assert float(scale[0]) == 0 and bool((q[0] == 0).all())
    assert not bool(torch.isfinite(scale[2:]).any()) and bool((q[2:] == 0).all())


def test_another_stream_and_a_graph(sg):
    import torch
    s = inputs(64, 512, "bf16", 1, True, 21)
    want = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"])
    grads = sg.block_norm_backward(s["x"], s["y"], s["w_pre"], want[2], s["dn"], s["dr"], s["w_post"], s["gate"])
    side = torch.cuda.Stream()
    got = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"], stream=side)
    side.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1 = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"])
        g2 = sg.block_norm_backward(s["x"], s["y"], s["w_pre"], g1[2], s["dn"], s["dr"], s["w_post"], s["gate"])
    s["x"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    again = sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"], s["gate"])
    assert all(bool((a == b).all()) for a, b in zip(g1, again))
    assert not bool((g2[0] == grads[0]).all())


def test_python_refusals(sg):
    import torch
    s = inputs(4, 64, "bf16", 2, True, 2)
    with pytest.raises(ValueError):
        sg.block_norm(s["x"], s["y"][:3], s["w_pre"])
    with pytest.raises(TypeError):
        sg.block_norm(s["x"], s["y"].float(), s["w_pre"])
    with pytest.raises(ValueError):
        sg.block_norm(s["x"].t(), s["y"].t(), s["w_pre"][:4])
    with pytest.raises(ValueError):
        sg.block_norm(s["x"], s["y"], s["w_pre"][:32])
    with pytest.raises(TypeError):
        sg.block_norm(s["x"], s["y"], s["w_pre"], s["w_post"].to(torch.bfloat16))
    with pytest.raises(sg.SgemmError):
        sg.block_norm(s["x"], s["y"], s["w_pre"], gate=s["x"][:3])
    with pytest.raises(ValueError):
        sg.block_norm(s["x"][:1].expand(4, 64), s["y"], s["w_pre"])
    with pytest.raises(ValueError):
        sg.block_norm_backward(s["x"], s["y"], s["w_pre"], torch.zeros(4, 2, device="cuda"), s["dn"])
