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
