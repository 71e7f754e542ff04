"""The native binding of the layer norm, the 4-bit products and the beams: streams, graphs,
arguments by name, and what is refused."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def same(a, b):
    import torch
    return all((x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b, strict=True))


@pytest.fixture(scope="module")
def calls(sg):
    """Each operator as a call of (positional rest, keywords) that returns all its new tensors."""
    import torch
    x, w = torch.randn(500, 640, device="cuda"), torch.ones(640, device="cuda")
    q, s, r = sg.quantize_fp4(torch.randn(300, 640, device="cuda"))
    q32, s32, _ = sg.quantize_fp4(torch.randn(300, 640, device="cuda"), 32)
    a, sa, ra = sg.quantize_fp4(x)
    stats = sg.layer_norm(x, w)[2]
    score = torch.randn(125, 4, device="cuda")
    parent = torch.randint(0, 4, (125, 4), device="cuda", dtype=torch.int32)
    plain = torch.ones(300, 40, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return [
        lambda p, k: sg.layer_norm(x, w, w, x, 1e-5, None, *p, **k),
        lambda p, k: sg.layer_norm(x, w, None, None, 1e-5, None, *p, **k)[1:],
        lambda p, k: sg.layer_norm_backward(x, w, stats, x, x, True, *p, **k),
        lambda p, k: sg.layer_norm_backward(x, w, stats, x, None, False, *p, **k),
        lambda p, k: [t for t in sg.quantize_fp4(x, 16, *p, **k)],
        lambda p, k: [t for t in sg.quantize_fp4(x, 32, *p, **k)],
        lambda p, k: [sg.lay_out_fp4_scales(plain, *p, **k)],
        lambda p, k: [sg.linear_fp4(x, q, s, r, None, None, None, None, *p, **k)],
        lambda p, k: [sg.linear_fp4(x[:1], q32, s32, None, None, None, None, None, *p, **k)],
        lambda p, k: [sg.matmul_fp4(a, sa, ra, q, s, r, None, None, None, *p, **k)],
        lambda p, k: sg.beam_step(x, score, 8, 1.0, None, None, 0, *p, **k),
        lambda p, k: [sg.beam_reorder(x, parent, None, *p, **k)],
    ]


@pytest.mark.parametrize("by_name", [True, False])
@pytest.mark.parametrize("handle", [True, False])
def test_a_call_on_another_stream_waits_for_the_memory_it_is_given(sg, calls, by_name, handle):
    """What a call allocates may have been freed by work that torch's stream still has queued:
    here a wait and then a fill, which must not land after the call's results."""
    import torch
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    for call in calls:
        want = call((), {})
        shapes = [(t.shape, t.dtype) for t in want if t is not None]
        torch.cuda.synchronize()
        held = [torch.empty(sh, dtype=dt, device="cuda") for sh, dt in shapes for _ in range(2)]
        torch.cuda._sleep(20_000_000)                 # about 10 ms
        for t in held:
            t.view(torch.uint8).fill_(77)
        del held, t
        got = call((), {"stream": stream}) if by_name else call((stream,), {})
        side.synchronize()
        torch.cuda.synchronize()
        assert same([t.contiguous() if t is not None else None for t in got], [t.contiguous() if t is not None else None for t in want])


def test_results_on_another_stream_are_not_given_away(sg, calls):
    """Memory that a call allocated on torch's stream and used on another is not handed out again
    while that one is still writing it."""
    import torch
    side = torch.cuda.Stream()
    for call in calls:
        want = call((), {})
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call((), {"stream": side})
        del got                                       # still being written, 10 ms from now
        others = [torch.full(t.shape, 1, dtype=torch.uint8, device="cuda") for t in want if t is not None for _ in range(4)]
        torch.cuda.synchronize()
        for t in others:
            assert bool((t == 1).all())


def test_two_calls_at_once_on_two_streams(sg, calls):
    import torch
    streams = [torch.cuda.Stream() for _ in range(2)]
    for call in calls:
        want = call((), {})
        torch.cuda.synchronize()
        got = [call((), {"stream": s}) for _ in range(4) for s in streams]
        torch.cuda.synchronize()
        for g in got:
            assert same([t.contiguous() if t is not None else None for t in g], [t.contiguous() if t is not None else None for t in want])


def test_captured_and_replayed(sg, calls):
    import torch
    for call in calls:
        want = call((), {})
        torch.cuda.synchronize()
        graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
        for graph in graphs:
            with torch.cuda.graph(graph):
                outs.append(call((), {}))
        for o in outs:
            for t in o:
                if t is not None:
                    t.view(torch.uint8).fill_(3) if t.is_contiguous() else t.fill_(3)
        for graph in graphs + graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert same([t.contiguous() if t is not None else None for t in o], [t.contiguous() if t is not None else None for t in want])


def test_every_argument_by_name(sg):
    import torch
    x, w = torch.randn(6, 64, device="cuda"), torch.ones(64, device="cuda")
    q, s, r = sg.quantize_fp4(x=x, block=16)
    n = sg.layer_norm(x=x, w=w, bias=w, add=x, eps=1e-5, out=None, stream=None)
    assert same(n, sg.layer_norm(x, w, w, x))
    assert same([t for t in sg.layer_norm_backward(x=x, w=w, stats=n[2], dn=x, dr=x, bias=True)], sg.layer_norm_backward(x, w, n[2], x, x))
    got = sg.linear_fp4(x=x, w=q, w_block=s, w_scale=r, bias=None, out_dtype=None, out=None, workspace=None, stream=None)
    assert torch.equal(got, sg.matmul_fp4(a=q, a_block=s, a_scale=r, w=q, w_block=s, w_scale=r, bias=None, out_dtype=torch.float32, out=None))
    score = torch.zeros(2, 3, device="cuda")
    best = sg.beam_step(logits=x, score=score, top=3, scale=1.0, mask=None, finished=None, end=0)
    assert same(best, sg.beam_step(x, score))
    assert torch.equal(sg.beam_reorder(state=x, parent=best[1], out=None), sg.beam_reorder(x, best[1]))


def test_layer_norm_refusals(sg):
    import torch
    x, w = torch.randn(6, 64, device="cuda"), torch.ones(64, device="cuda")
    _, _, stats = sg.layer_norm(x, w)
    for call, error, match in [
            (lambda: sg.layer_norm(x.double(), w), TypeError, "float32"), (lambda: sg.layer_norm(x[0], w), TypeError, "2-D"),
            (lambda: sg.layer_norm(x, w[:63]), ValueError, "w has 63"), (lambda: sg.layer_norm(x, w.half()), TypeError, "w must"),
            (lambda: sg.layer_norm(x, w, w.half()), TypeError, "bias"), (lambda: sg.layer_norm(x, w, add=x[:5]), ValueError, "add is"),
            (lambda: sg.layer_norm(x, w, add=x.half()), TypeError, "add must"), (lambda: sg.layer_norm(x, w, out=x), ValueError, "out is for"),
            (lambda: sg.layer_norm(x, w, add=x, out=torch.empty(6, 65, device="cuda")), ValueError, "out is"),
            (lambda: sg.layer_norm(x, w, eps=-1.0), sg.SgemmError, "layer_norm"), (lambda: sg.layer_norm(x.T, w[:6]), ValueError, "stride"),
            (lambda: sg.layer_norm(x, w, add=x.cpu()), TypeError, "add must"),
            (lambda: sg.layer_norm(torch.zeros(2, 24577, device="cuda"), torch.ones(24577, device="cuda")), sg.SgemmError, "layer_norm"),
            (lambda: sg.layer_norm_backward(x, w, stats[:, :5], x), ValueError, "stats"), (lambda: sg.layer_norm_backward(x, w, stats.T, x), ValueError, "stats"),
            (lambda: sg.layer_norm_backward(x, w, stats, x[:, :63]), ValueError, "dn is"), (lambda: sg.layer_norm_backward(x, w, stats, x, x.half()), TypeError, "dr"),
            (lambda: sg.layer_norm(torch.empty(2 ** 31 + 1, 0, device="cuda"), w[:0]), ValueError, "2\\^31")]:
        with pytest.raises(error, match=match):
            call()
    # 2^32 + 64 elements from row to row, whose lower 32 bits are a dense row's
    buf = torch.zeros(2 ** 32 + 128, dtype=torch.float16, device="cuda")
    far = buf.as_strided((2, 64), (2 ** 32 + 64, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        sg.layer_norm(far, w)
    with pytest.raises(ValueError, match="2\\^31"):
        sg.quantize_fp4(far)


@pytest.mark.parametrize("T", [1, 3, 400])
def test_small_results_that_share_memory_are_tensors_of_their_own(sg, T):
    """What one result is used for does not reach the others, on whichever stream."""
    import torch
    x, w = torch.randn(T, 96, device="cuda"), torch.ones(96, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        made = list(sg.layer_norm(x, w, w, x, stream=stream)) + list(sg.layer_norm_backward(x, w, torch.ones(2, T, device="cuda"), x, stream=stream))
        torch.cuda.synchronize()
        kept = [t.clone() for t in made]
        for i, t in enumerate(made):
            assert t.is_contiguous() and not t.requires_grad and t.data_ptr() % 16 == 0
            t.zero_()
            for u, k in zip(made[i + 1:], kept[i + 1:]):
                assert torch.equal(u, k)
        first = made[0]
        del made
        others = [torch.full((T, 96), 7.0, device="cuda") for _ in range(8)]
        assert bool((first == 0).all()) and all(bool((o == 7).all()) for o in others)
    leaf = x.clone().requires_grad_()
    assert not any(t.requires_grad for t in sg.layer_norm(leaf.detach(), w, add=x))
