"""Block norm over no rows: the gradients of what the rows share are sums over
nothing, zero to the bit."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("groups", [0, 1, 3])
@pytest.mark.parametrize("D", [1, 64, 1111])
def test_gradients_over_no_rows(sg, D, groups, dtype):
    import torch
    x = torch.empty(0, D, dtype=td(dtype), device="cuda")
    w = torch.ones(D, device="cuda")
    gate = torch.ones(groups, D, dtype=td(dtype), device="cuda") if groups else None
    r, n, rstd = sg.block_norm(x, x, w, w, gate)
    assert r.shape == n.shape == (0, D) and rstd.shape == (2, 0)
    # what the call allocates has been somebody else's before
    for shape, dt in (((max(groups, 1), D), td(dtype)), ((D,), torch.float32), ((D,), torch.float32)):
        torch.full(shape, float("nan"), dtype=dt, device="cuda")
    dx, dy, dw_pre, dw_post, dgate = sg.block_norm_backward(x, x, w, rstd, x, x, w, gate)
    assert dx.shape == dy.shape == (0, D)
    assert bool((dw_pre == 0).all()) and bool((dw_post == 0).all())
    assert (dgate is None) == (gate is None)
    if gate is not None:
        assert dgate.shape == gate.shape and bool((dgate == 0).all())


def test_the_gaps_between_the_gates_rows_stay(sg):
    import torch
    D, G, ld = 24, 3, 40
    gate = torch.ones(G, D, device="cuda")
    w, dw_pre = torch.ones(D, device="cuda"), torch.full((D,), 5.0, device="cuda")
    dgate = torch.full((G, ld), 5.0, device="cuda")
    lib = sg.load()
    status = lib.sgemm_block_norm_backward(0, D, 0, 0, D, 0, D, w.data_ptr(), 0, 0, gate.data_ptr(), D, G, 1.0, 0, 0, D, 0,
                                           D, 0, D, 0, D, dw_pre.data_ptr(), 0, dgate.data_ptr(), ld, 0, 0,
                                           torch.cuda.current_stream().cuda_stream)
    assert status == sg.SGEMM_OK
    assert bool((dw_pre == 0).all()) and bool((dgate[:, :D] == 0).all()) and bool((dgate[:, D:] == 5).all())


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("side", [False, True])
def test_rows_of_no_columns(sg, post, side):
    import torch
    T = 700
    x, w = torch.empty(T, 0, device="cuda"), torch.empty(0, device="cuda")
    stream = torch.cuda.Stream() if side else None
    torch.full((2, T), 5.0, device="cuda")          # what the call allocates has been somebody else's before
    torch.full((T,), 5.0, device="cuda")
    r, n, rstd = sg.block_norm(x, x, w, w if post else None, stream=stream)
    torch.cuda.synchronize()
    assert r.shape == n.shape == (T, 0)
    want = (x.square().mean(1) + 1e-6).rsqrt()      # the mean of nothing
    assert torch.equal(torch.isnan(rstd[1]), torch.isnan(want)) and bool(torch.isnan(rstd[1]).all())
    assert bool(torch.isnan(rstd[0]).all()) if post else bool((rstd[0] == 1).all())
    r, q, scale, rstd = sg.block_norm(x, x, w, w if post else None, quantize=True, stream=stream)
    torch.cuda.synchronize()
    assert q.shape == (T, 0) and torch.equal(scale, sg.quantize_i8(x)[1]) and bool((scale == 0).all())
    assert bool(torch.isnan(rstd[1]).all())
