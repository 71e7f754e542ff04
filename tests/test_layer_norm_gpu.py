"""sgemm_layer_norm and its gradient against the formulas in 64 bits.

The sum r = x + add is one FP32 addition and one rounding, so it is compared to the bit,
and what follows is compared with the formula of the r that came back.  Tolerances, with
u = 2^-24 and e the output type's half unit (u, 2^-8, 2^-11):

* a sum over a row is added in runs of at most 64 and then a tree: the mean is off by
  50 u mean|r| at most;
* a difference r - mean is rounded by u (|r| + |mean|), so with R the root of the mean
  square of |r| + |mean| and s = 1 / rstd the sum of squares is off by 50 u + 2 u R / s
  relative, and rstd by no more than that;
* n then adds |w| rstd times the first and the difference's rounding, |n - b| times the
  second, and five roundings;
* the gradient's bounds follow its terms with every one in magnitude, 64 u for a sum
  over a row and (T + 64) u for one over the rows.
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


def padded(rows, cols, pad, offset, dtype, gen, mean=0.0):
    """A rows x cols view into a larger buffer of NaN."""
    import torch
    buf = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.randn(rows, cols, generator=gen, device="cuda") + mean)
    return v


def inputs(T, D, dtype, add, bias, seed, pad=0, offset=0, wdtype=None, mean=0.3):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, wd = td(dtype), wdtype or torch.float32
    s = {k: padded(T, D, pad, offset, dt, g, mean if k == "x" else 0.0) for k in ("x", "add", "dn", "dr")}
    if not add:
        s["add"] = None
    s["w"] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wd)
    s["b"] = torch.randn(D, generator=g, device="cuda").to(wd) if bias else None
    return s


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, want, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / tol):.3g} of the bound"


def check_forward(s, got, eps, dtype):
    import torch
    r, n, stats = got
    if s["add"] is not None:
        assert torch.equal(r, (s["x"].float() + s["add"].float()).to(r.dtype))
    else:
        assert r is s["x"]
    x, w, b = f64(r), f64(s["w"]), f64(s["b"]) if s["b"] is not None else 0.0
    mean = x.mean(1, keepdims=True)
    sd = np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    size = np.abs(x) + np.abs(mean)
    d_mean = 50 * U * np.abs(x).mean(1, keepdims=True)
    d_rstd = 50 * U + 2 * U * np.sqrt((size ** 2).mean(1, keepdims=True)) / sd
    core = (x - mean) / sd * w
    want = core + b
    tol = np.abs(w) / sd * (d_mean + 2 * U * size) + np.abs(core) * d_rstd + 5 * U * (np.abs(core) + np.abs(b))
    check(n, want, tol * (1 + HALF_UNIT[dtype]) + HALF_UNIT[dtype] * np.abs(want) + STEP[dtype], "n")
    check(stats[0], mean[:, 0], (d_mean + 2 * U * np.abs(mean))[:, 0], "mean")
    check(stats[1], 1 / sd[:, 0], ((d_rstd + 4 * U) / sd)[:, 0], "rstd")


SHAPES = [(1, 1), (1, 64), (3, 7), (5, 31), (2, 255), (7, 256), (33, 264), (12, 1000), (9, 1111), (4, 4096), (2, 4104),
          (3, 8192), (2, 8200), (2, 12345), (1, 24576), (700, 96), (1000, 130), (3, 5121), (11, 2049)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("add", [True, False])
def test_forward(sg, T, D, dtype, add):
    s = inputs(T, D, dtype, add, D % 2 == 0, seed=T * 7 + D)
    check_forward(s, sg.layer_norm(s["x"], s["w"], s["b"], s["add"], eps=1e-5), 1e-5, dtype)


@pytest.mark.parametrize("T,D", [(5, 96), (4, 1000), (6, 1111), (3, 4096), (2, 12345)])
@pytest.mark.parametrize("mean", [1000.0, -30000.0])
def test_a_mean_far_from_zero(sg, T, D, mean):
    """A sum of squares less the squared mean would lose all of it: 30000^2 is 2^29.7."""
    s = inputs(T, D, "f32", False, True, seed=D, mean=mean)
    check_forward(s, sg.layer_norm(s["x"], s["w"], s["b"]), 1e-5, "f32")


def test_rows_of_one_value_and_rows_that_are_not_finite(sg):
    import torch
    for D in (1, 64, 257, 4096):
        x = torch.full((5, D), 3.0, device="cuda")
        x[1] = -2.0 ** 100
        x[2, D // 2] = float("inf")
        x[3, 0] = float("nan")
        w, b = torch.full((D,), 2.0, device="cuda"), torch.full((D,), 0.5, device="cuda")
        _, n, stats = sg.layer_norm(x, w, b)
        assert bool((n[0] == 0.5).all() and (n[1] == 0.5).all() and (n[4] == 0.5).all())
        assert bool(torch.isnan(n[2]).any() and torch.isnan(n[3]).all())
        assert stats[0, 0].item() == 3.0 and stats[0, 1].item() == -2.0 ** 100


@pytest.mark.parametrize("dtype,pad,offset", [("f32", 1, 1), ("bf16", 3, 5), ("bf16", 8, 8), ("f16", 8, 0), ("f32", 4, 4)])
def test_strides_and_alignment(sg, dtype, pad, offset):
    import torch
    T, D = 13, 264
    s = inputs(T, D, dtype, True, True, 5, pad, offset)
    buf = torch.full((T, D + pad), 7.0, dtype=td(dtype), device="cuda")
    got = sg.layer_norm(s["x"], s["w"], s["b"], s["add"], out=buf[:, :D])
    check_forward(s, got, 1e-5, dtype)
    assert bool((buf[:, D:] == 7.0).all()), "wrote between the rows"
    grads = sg.layer_norm_backward(s["x"], s["w"], got[2], s["dn"], s["dr"])
    c = {k: v.contiguous() for k, v in s.items()}
    for a, b in zip(grads, sg.layer_norm_backward(c["x"], c["w"], got[2], c["dn"], c["dr"])):
        # the same terms in another order
        check(a, f64(b), (2 * HALF_UNIT[dtype] if a.dim() == 2 else 200 * U) * (np.abs(f64(b)) + (a.dim() == 1)) + 1e-5, "gradient")


@pytest.mark.parametrize("which", ["x", "add"])
@pytest.mark.parametrize("D", [264, 1111])
def test_in_place(sg, which, D):
    import torch
    s = inputs(9, D, "bf16", True, True, 3)
    want = sg.layer_norm(s["x"], s["w"], s["b"], s["add"])
    got = sg.layer_norm(s["x"], s["w"], s["b"], s["add"], out=s[which])
    assert got[0] is s[which] and all(torch.equal(a, b) for a, b in zip(got, want))


def check_backward(s, stats, got, dtype, wdtype="f32"):
    dx, dw, db = got
    x, w, dn, dr = f64(s["x"]), f64(s["w"]), f64(s["dn"]), f64(s["dr"]) if s["dr"] is not None else 0.0
    mean, rstd = f64(stats)[0][:, None], f64(stats)[1][:, None]
    T = x.shape[0]
    h, hs = (x - mean) * rstd, (np.abs(x) + np.abs(mean)) * rstd
    u = dn * w
    m1, m2 = u.mean(1, keepdims=True), (u * h).mean(1, keepdims=True)
    want = dr + rstd * (u - m1 - h * m2)
    a1, a2 = np.abs(u).mean(1, keepdims=True), (np.abs(u) * hs).mean(1, keepdims=True)
    tol = 64 * U * rstd * (np.abs(u) + a1 + hs * a2) + 4 * U * np.abs(dr)
    e = HALF_UNIT[dtype]
    check(dx, want, tol * (1 + e) + e * np.abs(want) + STEP[dtype], "dx")
    e = HALF_UNIT[wdtype]
    for what, g, term, bound in (("dw", dw, dn * h, np.abs(dn) * hs), ("db", db, dn, np.abs(dn))):
        if g is not None:
            want = term.sum(0)
            check(g, want, (T + 64) * U * bound.sum(0) * (1 + e) + e * np.abs(want) + STEP[wdtype], what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D", SHAPES + [(5000, 64), (3001, 520)])
@pytest.mark.parametrize("dr", [True, False])
def test_backward(sg, T, D, dtype, dr):
    s = inputs(T, D, dtype, False, True, seed=T + D)
    if not dr:
        s["dr"] = None
    stats = sg.layer_norm(s["x"], s["w"])[2]
    got = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"], bias=D % 3 != 0)
    assert (got[2] is None) == (D % 3 == 0)
    check_backward(s, stats, got, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_of_the_rows_type(sg, dtype):
    s = inputs(37, 520, dtype, True, True, 11, wdtype=td(dtype))
    got = sg.layer_norm(s["x"], s["w"], s["b"], s["add"])
    check_forward(s, got, 1e-5, dtype)
    s["x"] = got[0]
    back = sg.layer_norm_backward(got[0], s["w"], got[2], s["dn"], s["dr"])
    assert back[1].dtype is td(dtype) and back[2].dtype is td(dtype)
    check_backward(s, got[2], back, dtype, dtype)


@pytest.mark.parametrize("T,D", [(4, 48), (3, 257)])
def test_gradient_against_differences(sg, T, D):
    """Central differences of the formula in 64 bits along ten directions, off by the step's
    square; the gradient is FP32."""
    import torch
    s = inputs(T, D, "f32", False, True, 21)
    x, w, b, dn, dr = (f64(s[k]) for k in ("x", "w", "b", "dn", "dr"))

    def value(x, w, b):
        m = x.mean(1, keepdims=True)
        n = (x - m) / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + 1e-5) * w + b
        return (n * dn).sum() + (x * dr).sum()

    stats = sg.layer_norm(s["x"], s["w"], s["b"])[2]
    dx, dw, db = (f64(t) for t in sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"]))
    rng = np.random.default_rng(2)
    step = 1e-4
    for _ in range(10):
        vx, vw, vb = rng.standard_normal(x.shape), rng.standard_normal(w.shape), rng.standard_normal(b.shape)
        slope = (value(x + step * vx, w + step * vw, b + step * vb) - value(x - step * vx, w - step * vw, b - step * vb)) / (2 * step)
        size = np.abs(dx * vx).sum() + np.abs(dw * vw).sum() + np.abs(db * vb).sum()
        assert abs((dx * vx).sum() + (dw * vw).sum() + (db * vb).sum() - slope) <= 1e-5 * size
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,D", [(0, 64), (3, 0), (0, 0)])
def test_empty(sg, T, D):
    import torch
    x = torch.empty(T, D, device="cuda")
    w = torch.ones(D, device="cuda")
    r, n, stats = sg.layer_norm(x, w, w, x.clone())
    assert r.shape == n.shape == (T, D) and stats.shape == (2, T) and bool(torch.isnan(stats).all())
    dx, dw, db = sg.layer_norm_backward(x, w, stats, x)
    assert dx.shape == (T, D) and bool((dw == 0).all() and (db == 0).all())


def test_same_bits_on_every_run(sg):
    import torch
    s = inputs(3000, 1000, "bf16", True, True, 4)
    first = sg.layer_norm(s["x"], s["w"], s["b"], s["add"])
    grads = sg.layer_norm_backward(first[0], s["w"], first[2], s["dn"], s["dr"])
    for _ in range(3):
        again = sg.layer_norm(s["x"], s["w"], s["b"], s["add"])
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(a, b) for a, b in zip(grads, sg.layer_norm_backward(first[0], s["w"], first[2], s["dn"], s["dr"])))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [1, 3, 9, 255, 257, 513, 1111, 5121, 9001])
def test_rows_anywhere_have_the_same_bits_and_leave_what_is_between_them(sg, D, dtype):
    """Every array starts and steps on its own alignment, and the outputs' rows lie in guards.
    (Widths of no whole 16 bytes, whose rows are all read alike.)"""
    import torch
    from dense_fp32_matrix_04_gb300 import layers
    T = 5
    dt, code = td(dtype), {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    s = inputs(T, D, dtype, True, True, seed=D)
    r, n, stats = sg.layer_norm(s["x"], s["w"], bias=s["b"], add=s["add"])
    dx, dw, db = sg.layer_norm_backward(r, s["w"], stats, s["dn"], s["dr"])
    stream = torch.cuda.current_stream().cuda_stream
    size = sg.layers._lib.sgemm_layer_norm_backward_workspace_size(T, D)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def room(values, start, pad):
        buf = torch.full((start + T * (D + pad) + 8,), -77.0, dtype=dt, device="cuda")
        v = buf[start:start + T * (D + pad)].view(T, D + pad)[:, :D]
        if values is not None:
            v.copy_(values)
        return buf, v

    def untouched(buf, v):
        v.fill_(-77.0)
        return bool((buf == -77.0).all())

    for k in range(8):
        start, pad = [k, (3 * k + 1) % 8, (5 * k + 2) % 8, 7 - k], [k % 3, (k + 1) % 4, 8 * k % 5, k]
        X, A, R, N = (room(v, start[i], pad[i]) for i, v in enumerate((s["x"], s["add"], None, None)))
        S = torch.zeros(2, T, device="cuda")
        assert layers._lib.sgemm_layer_norm(
            T, D, code, X[1].data_ptr(), D + pad[0], A[1].data_ptr(), D + pad[1], s["w"].data_ptr(), s["b"].data_ptr(), 0, 1e-5,
            R[1].data_ptr(), D + pad[2], N[1].data_ptr(), D + pad[3], S.data_ptr(), stream) == 0
        assert torch.equal(R[1], r) and torch.equal(N[1], n) and torch.equal(S, stats)
        DN, DR, DX = room(s["dn"], start[1], pad[1]), room(s["dr"], start[3], pad[3]), room(None, start[2], pad[2])
        DW, DB = torch.empty_like(dw), torch.empty_like(db)
        assert layers._lib.sgemm_layer_norm_backward(
            T, D, code, R[1].data_ptr(), D + pad[2], s["w"].data_ptr(), 0, S.data_ptr(), DN[1].data_ptr(), D + pad[1],
            DR[1].data_ptr(), D + pad[3], DX[1].data_ptr(), D + pad[2], DW.data_ptr(), DB.data_ptr(), ws.data_ptr(), size,
            stream) == 0
        assert torch.equal(DX[1], dx) and torch.equal(DW, dw) and torch.equal(DB, db)
        assert all(untouched(*made) for made in (R, N, DX))


@pytest.mark.parametrize("T,D", [(7, 3841), (310, 4501), (5, 5119), (3, 7777), (2, 16001), (310, 5120)])
@pytest.mark.parametrize("dr", [False, True])
def test_backward_of_wide_fp32_rows(sg, T, D, dr):
    s = inputs(T, D, "f32", False, True, seed=T + D)
    if not dr:
        s["dr"] = None
    stats = sg.layer_norm(s["x"], s["w"])[2]
    check_backward(s, stats, sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"]), "f32")
