"""The binding of the operators around the products: how arguments may be given,
and which are refused before a kernel sees them."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def same(a, b):
    import torch
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("side", [False, True])
def test_first_argument_by_name(sg, side):
    import torch
    x, w = torch.randn(6, 64, device="cuda"), torch.ones(64, device="cuda")
    q, s = sg.quantize_i8(torch.randn(10, 64, device="cuda"))
    target = torch.arange(6, device="cuda")
    norm, lp = sg.block_norm(x, x, w), sg.logprobs(x, target)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    got = [sg.block_norm(x=x, y=x, w_pre=w, stream=stream), sg.quantize_i8(x=x, stream=stream),
           sg.block_norm_backward(x=x, y=x, w_pre=w, rstd=norm[2], dn=x, stream=stream),
           [sg.linear_i8(x=x, w=q, w_scale=s, stream=stream)],
           [sg.matmul_i8(a=q, a_scale=s, w=q, w_scale=s, stream=stream)], sg.logprobs(logits=x, target=target, stream=stream),
           [sg.logprobs_backward(logits=x, target=target, lse=lp[2], entropy=lp[1], g_logprob=w[:6], stream=stream)]]
    torch.cuda.synchronize()
    want = [norm, sg.quantize_i8(x), sg.block_norm_backward(x, x, w, norm[2], x), [sg.linear_i8(x, q, s)],
            [sg.matmul_i8(q, s, q, s)], lp, [sg.logprobs_backward(x, target, lp[2], lp[1], w[:6])]]
    for a, b in zip(got, want):
        assert same(a, b)


@pytest.mark.parametrize("by_name", [True, False])
@pytest.mark.parametrize("handle", [True, False])
def test_a_call_on_another_stream_waits_for_the_memory_it_is_given(sg, by_name, handle):
    """What a call allocates may have been freed by work that torch's stream still has queued:
    here a wait and then a fill, which must not land after the call's results."""
    import torch
    x, w = torch.randn(500, 640, device="cuda"), torch.ones(640, device="cuda")
    q, s = sg.quantize_i8(torch.randn(300, 640, device="cuda"))
    target = torch.arange(500, device="cuda")
    norm, lp = sg.block_norm(x, x, w), sg.logprobs(x, target)
    g = torch.ones(500, device="cuda")
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    named = dict(stream=stream) if by_name else {}
    calls = [
        lambda on: sg.block_norm(x, x, w, None, None, 1.0, 1e-6, False, None, *on[0], **on[1]),
        lambda on: sg.block_norm(x, x, w, None, None, 1.0, 1e-6, True, None, *on[0], **on[1]),
        lambda on: sg.block_norm_backward(x, x, w, norm[2], x, None, None, None, 1.0, *on[0], **on[1]),
        lambda on: sg.quantize_i8(x, *on[0], **on[1]),
        lambda on: [sg.linear_i8(x, q, s, None, None, None, None, *on[0], **on[1])],
        lambda on: [sg.matmul_i8(q, s, q, s, None, None, None, None, *on[0], **on[1])],
        lambda on: sg.logprobs(x, target, 1.0, None, 4, *on[0], **on[1]),
        lambda on: [sg.logprobs_backward(x, target, lp[2], lp[1], g, g, 1.0, None, None, *on[0], **on[1])],
    ]
    for call in calls:
        want = call(((), {}))
        shapes = [(t.shape, t.dtype) for t in want if t is not None]
        torch.cuda.synchronize()
        held = [torch.empty(sh, dtype=dt, device="cuda") for sh, dt in shapes for _ in range(2)]
        torch.cuda._sleep(20_000_000)                 # about 10 ms
        for t in held:
            t.fill_(77)
        del held, t
        got = call(((), named) if by_name else ((stream,), {}))
        side.synchronize()
        torch.cuda.synchronize()
        assert same(got, want)


def test_a_stream_given_twice_or_out_of_place(sg):
    import torch
    x = torch.randn(4, 64, device="cuda")
    side = torch.cuda.Stream()
    with pytest.raises(TypeError):
        sg.quantize_i8(x, side, stream=side)
    with pytest.raises(TypeError):
        sg.quantize_i8(x, side, [])


@pytest.mark.parametrize("M", [3, 40])
def test_workspaces_that_are_refused(sg, M):
    import torch
    x = torch.randn(M, 64, device="cuda")
    q, s = sg.quantize_i8(x)
    w, ws = sg.quantize_i8(torch.randn(48, 64, device="cuda"))
    need = max(int(sg.load().sgemm_linear_i8_workspace_size(M, 48, 64, w.data_ptr(), 64)), 256)
    whole = torch.full((2 * need,), 9, dtype=torch.uint8, device="cuda")
    bad = [(torch.empty(need, dtype=torch.uint8), TypeError), (torch.empty(need, dtype=torch.uint8).share_memory_(), TypeError),
           (whole[::2], ValueError), (whole[:1].expand(need), ValueError),
           (torch.empty(need, dtype=torch.uint8, device="meta"), TypeError)]
    for workspace, error in bad:
        with pytest.raises(error, match="workspace"):
            sg.linear_i8(x, w, ws, workspace=workspace)
        with pytest.raises(error, match="workspace"):
            sg.matmul_i8(q, s, w, ws, workspace=workspace)
    assert bool((whole == 9).all())
    # any type and shape that is dense
    ok = torch.empty(2, (need + 7) // 8, device="cuda")
    assert torch.equal(sg.linear_i8(x, w, ws, workspace=ok), sg.linear_i8(x, w, ws))


def test_rows_too_far_apart_are_refused(sg):
    """Rows 2^32 + 64 elements apart, whose lower 32 bits are a dense row's."""
    import torch
    buf = torch.zeros(2 ** 32 + 128, dtype=torch.int8, device="cuda")
    w = buf.as_strided((2, 64), (2 ** 32 + 64, 1))
    w[1] = 5
    one = torch.ones(2, device="cuda")
    a = torch.ones(3, 64, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        sg.matmul_i8(a, torch.ones(3, device="cuda"), w, one)
    with pytest.raises(ValueError, match="2\\^31"):
        sg.quantize_i8(torch.empty(2 ** 32 + 1, 1, dtype=torch.bfloat16, device="cuda"))
    z = torch.zeros(1, 8, device="cuda")
    for top in (2 ** 32 + 1, -2 ** 32 + 1):
        with pytest.raises(ValueError, match="top"):
            sg.logprobs(z, torch.zeros(1, dtype=torch.int64, device="cuda"), top=top)


def test_a_gate_without_rows(sg):
    """The library knows no gate by its null pointer, which a tensor without rows has."""
    import torch
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    none = torch.empty(0, 64, device="cuda")
    rstd = sg.block_norm(x, x, w)[2]
    with pytest.raises(ValueError, match="gate"):
        sg.block_norm(x, x, w, gate=none)
    with pytest.raises(ValueError, match="gate"):
        sg.block_norm_backward(x, x, w, rstd, x, gate=none)
    # no rows of x, one gate a token: none is what there is
    r, n, rstd = sg.block_norm(none, none, w, gate=none)
    assert r.shape == (0, 64)
    assert sg.block_norm_backward(none, none, w, rstd, none, gate=none)[4].shape == (0, 64)


@pytest.mark.parametrize("T", [0, 3])
@pytest.mark.parametrize("mask_rows", [None, 1, 3])
def test_a_vocabulary_of_nothing(sg, T, mask_rows):
    import torch
    z = torch.empty(T, 0, device="cuda")
    target = torch.tensor([-1, 0, 7], device="cuda")[:T]
    mask = None if mask_rows is None else torch.empty(min(mask_rows, max(T, 1)), 0, dtype=torch.int32, device="cuda")
    logprob, entropy, lse, top_logprob, top_id = sg.logprobs(z, target, mask=mask, top=2)
    assert bool((entropy == 0).all()) and bool((lse == float("-inf")).all())
    assert bool((top_id == -1).all()) and bool((top_logprob == float("-inf")).all())
    assert bool((logprob[:1] == 0).all()) and bool(torch.isnan(logprob[1:]).all())     # no column is below V
    assert sg.logprobs_backward(z, target, lse, entropy, entropy, entropy, mask=mask).shape == (T, 0)
