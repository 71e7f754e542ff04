"""Products with weights whose rows do not start on 16 bytes: these are first laid
out in the workspace, by a kernel that the product may overlap.  The workspace
holds other bytes before every call and the weights change from call to call, so
that a product which reads the rows before they are written cannot agree by
chance.

K <= 1024 keeps every partial sum below 2^24: the sums are exact, and with scales
that are powers of two and no bias so is every product in FP32, to the bit.  For
longer rows the same plan adds the same terms in the same order whether the rows
were laid out or came aligned, so those two agree to the bit."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def weights(N, K, seed):
    """Codes on rows of K bytes, and the same on 16-byte aligned ones."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    w[:, 0] = 127
    aligned = torch.zeros(N, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K]
    aligned.copy_(w)
    return w, aligned


# small weights leave SMs free for the product while they are laid out; large ones are still being
# written by a second wave of blocks when the product starts
SHAPES = [(5, 130, 77), (17, 300, 1001), (32, 513, 1023), (200, 96, 513), (5, 12288, 1023), (24, 10240, 1001),
          (300, 12000, 1021), (7, 6000, 2047), (40, 5120, 2047), (600, 5001, 2047)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("quantised", [True, False])
def test_weights_that_change_under_one_workspace(sg, M, N, K, quantised):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    x[:, 0] = 127
    one_m, one_n = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    # whole numbers up to 127 are their own codes, with a scale of 1
    call = (lambda w, **k: sg.matmul_i8(x, one_m, w, one_n, **k)) if quantised else (
        lambda w, **k: sg.linear_i8(x.float(), w, one_n, **k))
    sets = [weights(N, K, seed) for seed in (1, 2)]
    want = [call(aligned) for _, aligned in sets]
    if K <= 1024:
        for (w, _), v in zip(sets, want):
            assert torch.equal(v.double(), x.double() @ w.double().T)
    assert not torch.equal(want[0], want[1])
    lib = sg.load()
    size = (lib.sgemm_i8_workspace_size if quantised else lib.sgemm_linear_i8_workspace_size)(
        M, N, K, sets[0][0].data_ptr(), K)
    assert size >= N * K
    workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, device="cuda")
    for turn in range(12):
        workspace.fill_(0x7F)
        out.fill_(float("nan"))
        call(sets[turn % 2][0], out=out, workspace=workspace)
        assert torch.equal(out, want[turn % 2]), f"call {turn}"
    assert sg.sgemm_device_status() == sg.SGEMM_OK
