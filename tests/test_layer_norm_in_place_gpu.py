"""The gradient of the layer norm written over one of its inputs, or into a tensor that is given: the
same bits as into one of its own, in each of the kernel's forms (a row a lane's piece, a warp, a block, a
cluster; whole pieces and single elements)."""

import pytest

from test_layer_norm_gpu import inputs, sg  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def same(a, b):
    import torch
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["dn", "dr", "x"])
@pytest.mark.parametrize("T,D", [(1, 1), (700, 96), (5, 97), (40, 264), (9, 1111), (4, 4096), (320, 5119), (3, 9001), (3, 12344), (2, 24576)])
@pytest.mark.parametrize("stream", [False, True])
def test_over_an_input(sg, T, D, which, dtype, stream):
    import torch
    s = inputs(T, D, dtype, False, True, seed=T + D, pad=8 if T == 4 else 0)
    stats = sg.layer_norm(s["x"], s["w"])[2]
    want = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"])
    side = torch.cuda.Stream() if stream else None
    got = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"], stream=side, out=s[which])
    torch.cuda.synchronize()
    assert got[0] is s[which] and same(got, want)
    if which == "dn":
        return
    # without a gradient from r
    s = inputs(T, D, dtype, False, True, seed=T + D)
    want = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], bias=False)
    got = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], bias=False, out=s["x"])
    assert same(got, want)


@pytest.mark.parametrize("dtype,pad,offset", [("f32", 1, 1), ("bf16", 8, 8), ("f16", 3, 5)])
def test_into_a_tensor_that_is_given(sg, dtype, pad, offset):
    import torch
    T, D = 13, 264
    s = inputs(T, D, dtype, False, True, 5, pad, offset)
    stats = sg.layer_norm(s["x"], s["w"])[2]
    want = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"])
    buf = torch.full((T, D + pad), 7.0, dtype=want[0].dtype, device="cuda")
    got = sg.layer_norm_backward(s["x"], s["w"], stats, s["dn"], s["dr"], out=buf[:, :D])
    assert got[0].data_ptr() == buf.data_ptr() and same(got, want) and bool((buf[:, D:] == 7.0).all())


def test_refusals(sg):
    import torch
    x, w = torch.randn(6, 64, device="cuda"), torch.ones(64, device="cuda")
    stats = sg.layer_norm(x, w)[2]
    room = torch.zeros(7, 64, device="cuda")
    for out, error, match in [(x[:5], ValueError, "out is"), (x.half(), TypeError, "out must"), (x.cpu(), TypeError, "out must"),
                              (x.T, ValueError, "out is"), (torch.zeros(64, 6, device="cuda").T, ValueError, "stride"),
                              (torch.zeros(1, 64, device="cuda").expand(6, 64), ValueError, "overlap")]:
        with pytest.raises(error, match=match):
            sg.layer_norm_backward(x, w, stats, x, out=out)
    # a row further on than an input
    room[1:].copy_(x)
    with pytest.raises(sg.SgemmError, match="layer_norm_backward"):
        sg.layer_norm_backward(room[1:], w, stats, x, out=room[:6])
    with pytest.raises(TypeError):
        sg.layer_norm_backward(x, w, stats, x, None, True, None, x)
    assert sg.layer_norm_backward(x[:0], w, stats[:, :0].contiguous(), x[:0], out=x[:0])[0].shape == (0, 64)
