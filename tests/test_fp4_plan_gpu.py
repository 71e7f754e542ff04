"""4-bit products of every tile and split that the plan chooses, on the GPU that the plan is for; the same
bounds as in test_fp4_gpu.py."""

import pytest

from test_fp4_gpu import HALF_UNIT, LEVELS, U, operands, sg, td  # noqa: F401  (the fixture)
from test_fp4_plan import REACHED, SMS

pytestmark = pytest.mark.gpu


def values(q, s, K, block):
    """What codes and block scales stand for, in 64 bits."""
    import torch
    i, j = torch.arange(q.shape[0], device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    code = (q[:, j[0] // 2] >> (4 * (j % 2)).to(torch.uint8)) & 15
    blk = j // block
    byte = s.view(torch.uint8)[i // 128, blk // 4 * 512 + i % 32 * 16 + i % 128 // 32 * 4 + blk % 4]
    scale = byte.view(torch.float8_e4m3fn).double() if block == 16 else torch.exp2(byte.double() - 127)
    return torch.tensor(LEVELS, device="cuda")[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0) * scale


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("plan", REACHED, ids=lambda p: f"{p[0]}x{p[1]}")
def test_product(sg, plan, block):
    import torch
    M, N, K = REACHED[plan]
    if torch.cuda.get_device_properties(0).multi_processor_count == SMS:
        assert sg.sgemm_fp4_plan_model(M, N, K, SMS) == plan
    x, w, bias = operands(sg, M, N, K, M + N, block, "bf16")
    a = sg.quantize_fp4(x, block)
    A, B = values(a[0], a[1], K, block), values(w[0], w[1], K, block)
    s = torch.outer(a[2].double(), w[2].double()) if block == 16 else 1.0
    v, size, extra = A @ B.T * s, A.abs() @ B.abs().T * s, bias.double()
    del A, B
    for out in ("f32", "bf16"):
        got = sg.matmul_fp4(*a, *w, bias, out_dtype=td(out))
        want = v + extra
        tol = 2 * K * U * size + 4 * U * (v.abs() + extra.abs()) + HALF_UNIT[out] * want.abs() * (1 + 2.0 ** -7) + 2.0 ** -126
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"
        assert torch.equal(sg.linear_fp4(x, *w, bias=bias, out_dtype=td(out)), got)
        assert torch.equal(sg.matmul_fp4(*a, *w, bias, out_dtype=td(out)), got)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
