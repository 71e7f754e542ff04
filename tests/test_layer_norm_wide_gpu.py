"""The layer norm's gradient of FP32 rows on either side of the widths where the elements a thread
takes, or the blocks that share a row, change: with a gradient from r the ring fills sooner."""

import pytest

from test_layer_norm_gpu import check_backward, inputs, sg  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(3, 3840), (5, 3841), (4, 4096), (4, 4100), (300, 5122), (7, 6001), (2, 6145), (160, 6400), (3, 6404),
                                 (310, 7168), (3, 8192), (2, 8196), (5, 10243), (160, 11001), (2, 12289), (3, 12800), (2, 14336),
                                 (2, 15363), (3, 16384), (2, 16385), (2, 20482)])
@pytest.mark.parametrize("dr", [True, False])
def test_backward_of_wide_fp32_rows(sg, T, D, dr):
    s = inputs(T, D, "f32", False, True, seed=T + D)
    if not dr:
        s["dr"] = None
    stats = sg.layer_norm(s["x"], s["w"])[2]
    got = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"])
    check_backward(s, stats, got, "f32")
    again = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"])
    assert all(bool((a == b).all()) for a, b in zip(got, again))
