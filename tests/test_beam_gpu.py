"""A step of beam search, and states reordered, against numpy in 64 bits.

A candidate's score is the beam's, plus a logit relative to its row's largest (exact in
64 bits), less the logarithm of an FP32 sum.  A term of the sum at t = scale (z - max) is off by
4 u |t| (the rounding of scale log2(e) and of the product) + 2^-22 (the exponential), and
e^t |t| <= 1/e of the largest; sums of up to 200000 terms in runs of about a thousand and trees:
the sum is off by less than 300 u of itself.  The logarithm and the joined parts add 4 u; the score
is then rounded once.  Columns have to be equal where the oracle's candidates lie further apart
than twice that, and within a beam always."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NEAR = 304 * U


def td(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


@pytest.fixture(scope="module")
def sg(cuda_device, lib):
    import dense_fp32_matrix_04_gb300 as sg
    return sg


def words(bits):
    import torch
    rows, V = bits.shape
    full = np.zeros((rows, (V + 31) // 32 * 32), np.uint32)
    full[:, :V] = bits
    w = (full.reshape(rows, -1, 32) << np.arange(32, dtype=np.uint32)).sum(2, dtype=np.uint32)
    return torch.from_numpy(w.view(np.int32)).cuda()


def oracle(z, score, top, scale, bits=None, finished=None, end=0):
    """(score, parent, token) of the definition, in 64 bits; z: (B W) x V."""
    B, W = score.shape
    V = z.shape[1]
    with np.errstate(all="ignore"):
        a = z.astype(np.float64)
        if bits is not None:
            a = np.where(np.broadcast_to(bits, a.shape), a, -np.inf)
        bad = np.isnan(a).any(1) | (a == np.inf).any(1) | (a == -np.inf).all(1)
        a[bad] = 0
        a = a * scale
        m = a.max(1, keepdims=True)
        p = a - m - np.log(np.exp(a - m).sum(1, keepdims=True))
        p[bad] = -np.inf
        if finished is not None:
            p[finished.reshape(-1)] = -np.inf
        s = score.reshape(-1, 1).astype(np.float64)
        total = np.where(np.isfinite(s), s + p, -np.inf)
    out = []
    for b in range(B):
        rows = total[b * W:(b + 1) * W]
        cand = [(-v, w, j) for w in range(W) for j, v in ((j, rows[w, j]) for j in np.argsort(-rows[w], kind="stable")[:top])
                if v > -np.inf]
        if finished is not None:
            cand += [(-float(score[b, w]), w, end) for w in range(W) if finished[b, w] and np.isfinite(score[b, w])]
        cand = sorted(cand)[:top]
        out.append([(-v, w, j) for v, w, j in cand] + [(-np.inf, -1, -1)] * (top - len(cand)))
    o = np.array(out, np.float64).reshape(B, top, 3)
    return o[:, :, 0], o[:, :, 1].astype(int), o[:, :, 2].astype(int)


def check(got, want):
    s, parent, token = (t.cpu().numpy() for t in got)
    ws, wp, wt = want
    near = NEAR + U * np.abs(np.where(np.isfinite(ws), ws, 0))
    assert np.array_equal(np.isfinite(s), np.isfinite(ws))
    ok = np.isfinite(ws)
    assert (np.abs(s[ok].astype(np.float64) - ws[ok]) <= near[ok]).all(), np.abs(s[ok] - ws[ok]).max()
    same = (parent == wp) & (token == wt)
    for b, k in zip(*np.nonzero(~same)):
        # another beam's candidate, as near as the sums can tell
        others = [i for i in range(ws.shape[1]) if i != k and wp[b, i] != wp[b, k] and abs(ws[b, i] - ws[b, k]) <= 2 * near[b, k]]
        assert others or (k == ws.shape[1] - 1 and abs(s[b, k] - ws[b, k]) <= 2 * near[b, k]), (b, k, parent[b, k], token[b, k], wp[b, k], wt[b, k])
    assert same.mean() > 0.99 or same.size < 100


def case(B, W, V, dtype, seed, pad=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((B * W, V + pad), float("nan"), dtype=td(dtype), device="cuda")
    z = buf[:, :V]
    z.copy_(2.5 * torch.randn(B * W, V, generator=g, device="cuda"))
    score = -10 * torch.rand(B, W, generator=g, device="cuda")
    return z, score


SHAPES = [(1, 1, 1, 1), (1, 1, 7, 3), (2, 3, 5, 16), (1, 4, 1000, 4), (3, 5, 2047, 10), (1, 4, 131072, 8), (7, 2, 50001, 2),
          (33, 8, 1501, 16), (2, 32, 3001, 32), (5, 16, 40000, 32), (1, 32, 33, 32), (200, 3, 999, 6)]


@pytest.mark.parametrize("B,W,V,top", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_step(sg, B, W, V, top, dtype):
    z, score = case(B, W, V, dtype, B + W + V, pad=V % 3)
    got = sg.beam_step(z, score, top=top, scale=0.8)
    check(got, oracle(z.float().cpu().numpy(), score.cpu().numpy(), top, np.float32(0.8).astype(np.float64)))


@pytest.mark.parametrize("mask_rows", ["one", "all"])
@pytest.mark.parametrize("B,W,V,top", [(1, 4, 1000, 8), (3, 5, 2047, 10), (40, 8, 501, 16), (1, 3, 70000, 20)])
def test_masks_finished_beams_and_beams_that_do_not_exist(sg, B, W, V, top, mask_rows):
    import torch
    z, score = case(B, W, V, "f32", V)
    rng = np.random.default_rng(V)
    bits = rng.random((1 if mask_rows == "one" else B * W, V)) < 0.3
    finished = rng.random((B, W)) < 0.3
    finished[0, 0] = True
    if mask_rows == "all":
        bits[W - 1] = False                        # a beam that may not go on at all
    zh = z.cpu().numpy()
    zh[np.broadcast_to(~bits, zh.shape)] = rng.choice([np.nan, np.inf, -np.inf, 3e38], np.broadcast_to(~bits, zh.shape).sum())
    zh[finished.reshape(-1)] = np.nan              # logits that are not read
    z.copy_(torch.from_numpy(zh))
    sh = score.cpu().numpy()
    sh[rng.random((B, W)) < 0.2] = -np.inf
    sh[-1, -1] = np.nan
    score.copy_(torch.from_numpy(sh))
    end = V // 2
    for f in (torch.from_numpy(finished).cuda(), torch.from_numpy(finished.astype(np.uint8) * 3).cuda()):
        got = sg.beam_step(z, score, top=top, scale=1.25, mask=words(bits), finished=f, end=end)
        check(got, oracle(zh, sh, top, 1.25, bits, finished, end))


def test_equal_scores_go_by_the_lower_beam_and_column(sg):
    import torch
    z = torch.zeros(4, 300, device="cuda", dtype=torch.bfloat16)
    z[:, 7], z[:, 200], z[1, 3] = 2.0, 2.0, -1.0
    z[3] = z[0]
    score = torch.tensor([[-1.0, -5.0], [-2.0, -1.0]], device="cuda")
    _, parent, token = sg.beam_step(z, score, top=5)
    assert parent[0].tolist() == [0, 0, 0, 0, 0] and token[0].tolist() == [7, 200, 0, 1, 2]
    assert parent[1].tolist() == [1, 1, 0, 0, 1] and token[1].tolist() == [7, 200, 7, 200, 0]
    # the same logits and scores: beam after beam
    _, parent, token = sg.beam_step(z[2:3].expand(4, 300).contiguous(), torch.zeros(1, 4, device="cuda"), top=10)
    assert parent[0].tolist() == [0, 0, 1, 1, 2, 2, 3, 3, 0, 0] and token[0].tolist() == [7, 200] * 4 + [0, 1]


def test_groups_without_continuations_and_rows_that_are_not_finite(sg):
    import torch
    z, score = case(4, 2, 100, "f32", 1)
    z[0, 5], z[1, 6] = float("nan"), float("inf")      # group 0: nothing
    z[2] = float("-inf")                               # group 1: its second beam only
    score[2] = float("-inf")                           # group 2: nothing
    score[3, 0] = float("inf")
    s, parent, token = sg.beam_step(z, score, top=3)
    for b in (0, 2):
        assert bool((s[b] == float("-inf")).all() and (parent[b] == -1).all() and (token[b] == -1).all())
    assert parent[1].tolist() == [1, 1, 1] and parent[3].tolist() == [1, 1, 1] and bool(torch.isfinite(s[1]).all())


def test_fewer_columns_than_wanted(sg):
    import torch
    z, score = case(2, 2, 3, "f32", 2)
    got = sg.beam_step(z, score, top=16)
    check(got, oracle(z.cpu().numpy(), score.cpu().numpy(), 16, 1.0))
    assert bool((got[2][:, 6:] == -1).all())
    none = sg.beam_step(torch.empty(4, 0, device="cuda"), score, top=2)
    assert bool((none[1] == -1).all() and (none[0] == float("-inf")).all())
    assert sg.beam_step(torch.empty(0, 9, device="cuda"), torch.empty(0, 3, device="cuda"))[0].shape == (0, 3)


def test_large_scales_and_scores(sg):
    """Sums whose reference is not taken from the scaled maximum, and scores that FP32 rounds by more
    than the candidates' distance."""
    z, score = case(2, 3, 400, "f32", 3)
    z *= 1e7
    check(sg.beam_step(z, score, top=6, scale=3.0), oracle(z.cpu().numpy(), score.cpu().numpy(), 6, 3.0))
    z, score = case(3, 4, 4000, "bf16", 4)
    score -= 5e6
    s, parent, token = sg.beam_step(z, score, top=8)
    want = oracle(z.float().cpu().numpy(), score.cpu().numpy(), 8, 1.0)
    assert np.array_equal(parent.cpu().numpy(), want[1]) and np.array_equal(token.cpu().numpy(), want[2])


# ---------------------------------------------------------------- reordering

def reordered(state, parent, out):
    """What out becomes."""
    import torch
    B, top = parent.shape
    W = state.shape[0] // B
    p = parent.cpu().long()
    src = state.clone()
    for b in range(B):
        for k in range(top):
            if 0 <= p[b, k] < W:
                out[b * top + k] = src[b * W + int(p[b, k])]
    return out


@pytest.mark.parametrize("B,W,top", [(1, 1, 1), (1, 4, 4), (5, 3, 7), (2, 32, 32), (3, 8, 2), (70, 2, 2)])
@pytest.mark.parametrize("rest", [(1,), (129,), (3, 5, 8), (2, 1000), (64, 24, 16)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32", "uint8", "int64"])
def test_reorder(sg, B, W, top, rest, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(B * W)
    dt = getattr(torch, dtype)
    state = torch.randint(0, 200, (B * W, *rest), generator=g, device="cuda").to(dt)
    parent = torch.randint(-1, W, (B, top), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full((B * top, *rest), 201, device="cuda").to(dt)
    want = reordered(state, parent, out.clone())
    got = sg.beam_reorder(state, parent, out=out)
    assert got is out and torch.equal(out, want)
    if bool((parent >= 0).all()):
        assert torch.equal(sg.beam_reorder(state, parent), want)
    if top == W:
        want = reordered(state, parent, state.clone())
        assert sg.beam_reorder(state, parent, out=state) is state and torch.equal(state, want)


@pytest.mark.parametrize("heads,most,length,dim,off", [(3, 40, 17, 8, 0), (1, 64, 64, 16, 0), (8, 9, 1, 5, 3), (2, 300, 299, 72, 1)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32", "int8"])
def test_reorder_of_the_filled_part_of_a_cache(sg, heads, most, length, dim, off, dtype):
    import torch
    B, W = 3, 4
    n = B * W * heads * most * dim
    buf = torch.arange(n + off, device="cuda").remainder(120).to(getattr(torch, dtype))
    cache = buf[off:].view(B * W, heads, most, dim)
    used = cache[:, :, :length]
    parent = torch.tensor([[0, 0, 0, 0], [3, 2, 1, 0], [0, 1, 1, 3]], device="cuda", dtype=torch.int32)
    want = reordered(used, parent, torch.empty(used.shape, dtype=used.dtype, device="cuda"))
    assert torch.equal(sg.beam_reorder(used, parent), want)
    whole = cache.clone()
    assert sg.beam_reorder(used, parent, out=used).data_ptr() == used.data_ptr()
    whole[:, :, :length] = want
    assert torch.equal(cache, whole), "what lies behind the filled part changed"
    # rows inside a cache whose first dimension is another one
    swapped = torch.arange(heads * B * W * dim, device="cuda").remainder(120).to(used.dtype).view(heads, B * W, dim).transpose(0, 1)
    want = reordered(swapped, parent, torch.empty(swapped.shape, dtype=used.dtype, device="cuda"))
    assert torch.equal(sg.beam_reorder(swapped, parent), want)
    sg.beam_reorder(swapped, parent, out=swapped)
    assert torch.equal(swapped, want)


def test_reorder_takes_no_parent_outside_its_group(sg):
    import torch
    state = torch.arange(8, device="cuda", dtype=torch.float32).view(4, 2)
    out = torch.full((4, 2), -5.0, device="cuda")
    parent = torch.tensor([[2, -1], [2 ** 31 - 1, -2 ** 31]], device="cuda", dtype=torch.int32)
    assert bool((sg.beam_reorder(state, parent, out=out) == -5.0).all())


def test_reorder_beyond_32_bits(sg):
    """Rows of more than 2^32 bytes."""
    import torch
    n = 2 ** 32 + 4112
    state = torch.zeros(2, n, dtype=torch.uint8, device="cuda")
    state[0, -40:], state[1, -40:], state[1, :3] = 7, 9, 5
    parent = torch.tensor([[1, 0]], device="cuda", dtype=torch.int32)
    got = sg.beam_reorder(state, parent)
    assert bool((got[0] == state[1]).all() and (got[1] == state[0]).all())


def test_empty_states(sg):
    import torch
    parent = torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    assert sg.beam_reorder(torch.empty(6, 0, device="cuda"), parent).shape == (6, 0)
    assert sg.beam_reorder(torch.empty(0, 5, device="cuda"), parent[:0]).shape == (0, 5)
    one = torch.arange(6, device="cuda")
    assert sg.beam_reorder(one, parent).tolist() == [0, 0, 0, 3, 3, 3]


def test_refusals(sg):
    import torch
    z, score = case(2, 3, 50, "f32", 1)
    parent = torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    state = torch.zeros(6, 4, 8, device="cuda")
    for call, error in [
            (lambda: sg.beam_step(z, score[:1]), ValueError), (lambda: sg.beam_step(z, score.double()), TypeError),
            (lambda: sg.beam_step(z, score, top=0), ValueError), (lambda: sg.beam_step(z, score, top=33), ValueError),
            (lambda: sg.beam_step(z, score.T), ValueError), (lambda: sg.beam_step(z, score.cpu()), TypeError),
            (lambda: sg.beam_step(z, score, finished=parent), TypeError), (lambda: sg.beam_step(z, score, end=-1), ValueError),
            (lambda: sg.beam_step(z, score, scale=0.0), sg.SgemmError),
            (lambda: sg.beam_step(torch.zeros(33, 5, device="cuda"), torch.zeros(1, 33, device="cuda")), ValueError),
            (lambda: sg.beam_reorder(state[:5], parent), ValueError), (lambda: sg.beam_reorder(state, parent.long()), TypeError),
            (lambda: sg.beam_reorder(state.cpu(), parent), TypeError),
            (lambda: sg.beam_reorder(state, parent, out=state[:, :, :4]), ValueError),
            (lambda: sg.beam_reorder(state, parent, out=state.half()), TypeError),
            (lambda: sg.beam_reorder(state[:, ::2, ::2], parent), ValueError),
            (lambda: sg.beam_reorder(state, parent, out=torch.zeros(1, 4, 8, device="cuda").expand(6, 4, 8)), sg.SgemmError),
            (lambda: sg.beam_reorder(state[:, :2], parent, out=state[:, 1:3]), sg.SgemmError)]:
        with pytest.raises(error):
            call()
