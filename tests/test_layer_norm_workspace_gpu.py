"""The workspace of the layer norm's gradient: as large as the partial sums that are written, and no byte
of what lies behind it, or was in it, matters."""

import pytest

from test_layer_norm_gpu import DTYPES, inputs, sg  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_rows_of_a_warp_need_a_partial_sum_a_block(sg):
    """Four warps, one row each, add theirs up before they are written."""
    import torch
    lib, sms = sg.load(), torch.cuda.get_device_properties(0).multi_processor_count
    for D in (1, 64, 128, 200, 256):
        assert lib.sgemm_layer_norm_backward_workspace_size(64000, D) == 4 * sms * 8 * D
        assert lib.sgemm_layer_norm_backward_workspace_size(7, D) == 2 * 8 * D
        assert lib.sgemm_layer_norm_backward_workspace_size(1, D) == 8 * D


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D", [(1, 1), (7, 128), (64000, 128), (3000, 127), (64000, 64), (5, 256), (20000, 255), (20000, 256),
                                 (20000, 257), (20000, 264), (20000, 511), (20000, 512), (9000, 513), (2000, 1111), (500, 8192), (300, 9001)])
@pytest.mark.parametrize("dr", [True, False])
def test_nothing_behind_it_is_touched_and_nothing_in_it_matters(sg, T, D, dtype, dr):
    import torch
    lib, code = sg.load(), {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    s = inputs(T, D, dtype, False, True, seed=T + D)
    x, w, dn, d = s["x"], s["w"], s["dn"], s["dr"] if dr else None
    stats = sg.layer_norm(x, w)[2]
    want = sg.layer_norm_backward(x, w, stats, dn, d)
    size = lib.sgemm_layer_norm_backward_workspace_size(T, D)
    room = torch.full((size // 4 + 4096,), float("nan"), device="cuda")
    dx, dw, db = (torch.empty_like(t) for t in want)

    def call(nbytes):
        return lib.sgemm_layer_norm_backward(T, D, code, x.data_ptr(), D, w.data_ptr(), 0, stats.data_ptr(), dn.data_ptr(), D,
                                             d.data_ptr() if dr else 0, D, dx.data_ptr(), D, dw.data_ptr(), db.data_ptr(),
                                             room.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream)
    assert call(size) == sg.SGEMM_OK
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])
    assert bool(torch.isnan(room[size // 4:]).all())
    assert call(size - 1) == sg.SGEMM_ERR_INVALID_ARG
