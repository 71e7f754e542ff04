"""4-bit weights that are saved, or copied to the host and back: what keeps the distance of their rows,
and what lays dense rows out again."""

import io

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("N,K", [(1, 77), (5, 31), (130, 1111), (64, 64), (70, 1040)])
def test_weights_come_back(cuda_device, lib, N, K, block):
    import torch

    import dense_fp32_matrix_04_gb300 as sg
    x = torch.randn(6, K, device="cuda")
    q, s, r = sg.quantize_fp4(torch.randn(N, K, device="cuda"), block)
    want = sg.linear_fp4(x, q, s, r)
    buf = io.BytesIO()
    torch.save({"q": q, "s": s, "r": r}, buf)
    buf.seek(0)
    back = torch.load(buf, weights_only=True)
    assert back["q"].stride() == q.stride() and torch.equal(sg.linear_fp4(x, back["q"], back["s"], back["r"]), want)
    moved = [None if t is None else t.cpu().cuda() for t in (q, s, r)]
    dense = moved[0]
    if N > 1 and K % 32:
        assert dense.stride(0) == (K + 1) // 2
        if dense.stride(0) % 16:
            with pytest.raises(ValueError, match="multiple of 16.*torch.nn.functional.pad"):
                sg.linear_fp4(x, *moved)
    moved[0] = torch.nn.functional.pad(dense, (0, -dense.shape[1] % 16))[:, :dense.shape[1]]
    assert torch.equal(moved[0], q) and torch.equal(sg.linear_fp4(x, *moved), want)
    assert torch.equal(sg.matmul_fp4(*moved, *moved), sg.matmul_fp4(q, s, r, q, s, r))
