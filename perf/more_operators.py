"""Cases that time more of the language-model operators beside the matrix products.

Three sets, as the end of a model uses them:

* ``layer_norm``: the sum of the residual stream and a block's output, and the
  norm of it with a mean, weights and a bias; and its backward pass;
* ``linear_fp4``: activations quantised to 4-bit floating point with a scale
  for each block of 16 or 32, multiplied with weights of the same format;
* ``beam_step`` and ``beam_reorder``: the best continuations of each group's
  beams over the vocabulary, and the states reordered as the beams were.

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits (64 where candidates are put in order); with ``own`` true it makes the
calls a user makes of this package.  ``exact`` computes the same results in 64
bits from the definitions.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: the whole call is latency
        dict(name="layer_norm decode 5x4096", op="norm", T=5, D=4096, dtype="bf16", add=True, bias=True),
        # a long prompt
        dict(name="layer_norm prompt 8192x5120", op="norm", T=8192, D=5120, dtype="bf16", add=True, bias=True),
        # training in bf16; a gradient arrives from the residual stream too
        dict(name="layer_norm grad 8192x4096", op="norm_grad", T=8192, D=4096, dtype="bf16", add=True, bias=True),
        # training in FP32 with an odd width, without a bias
        dict(name="layer_norm grad 2047x1111", op="norm_grad", T=2047, D=1111, dtype="f32", add=False, bias=False),
        # one new token: the weights are read once
        dict(name="linear_fp4 1x4096x4096", op="fp4", M=1, N=4096, K=4096, dtype="bf16", out="bf16", block=16,
             bias=False),
        # a decoding batch through a wide layer
        dict(name="linear_fp4 24x16384x4096", op="fp4", M=24, N=16384, K=4096, dtype="bf16", out="bf16", block=32,
             bias=True),
        # the ragged product of this repository's benchmark
        dict(name="linear_fp4 3001x4999x2047", op="fp4", M=3001, N=4999, K=2047, dtype="f32", out="f32", block=16,
             bias=True),
        # the benchmark's square product, as a long prompt meets it
        dict(name="linear_fp4 8192x8192x8192", op="fp4", M=8192, N=8192, K=8192, dtype="bf16", out="bf16", block=16,
             bias=False),
        # one sequence searched with four beams over a large vocabulary that a mask constrains
        dict(name="beam_step 1x4x131072", op="beam", B=1, W=4, V=131072, dtype="f32", top=8, mask="row", scale=1.0,
             finished=False),
        # a batch of searches, some beams of which have ended; an odd vocabulary
        dict(name="beam_step 48x8x50001", op="beam", B=48, W=8, V=50001, dtype="bf16", top=16, mask="none", scale=0.9,
             finished=True),
        # one layer's keys for one sequence of four beams
        dict(name="beam_reorder 1x4x8x777", op="reorder", B=1, W=4, heads=8, length=777, most=1024, dim=128,
             dtype="bf16"),
        # a batch of searches deep into their answers
        dict(name="beam_reorder 8x8x16x4001", op="reorder", B=8, W=8, heads=16, length=4001, most=4096, dim=128,
             dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "fp4", "fp4", "fp4", "beam", "beam", "reorder"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op in ("norm", "norm_grad"):
        D = _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        T = _spread(rng, 1, max(1, min(16384, 32_000_000 // D)))
        return dict(op=op, T=T, D=D, dtype=dtype, add=rng.random() < 0.6, bias=rng.random() < 0.75)
    if op == "fp4":
        N, K = _spread(rng, 64, 16384), _spread(rng, 64, 16384)
        if rng.random() < 0.7:
            N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
        M = _spread(rng, 1, 8192)
        while M * N * K > 8192 ** 3:
            M = max(1, M // 2)
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, out=rng.choice(["f32", dtype]), block=rng.choice([16, 32]),
                    bias=rng.random() < 0.5)
    W = rng.choice([2, 3, 4, 5, 8, 10, 16])
    if op == "beam":
        V = _spread(rng, 1000, 200_000)
        B = _spread(rng, 1, max(1, min(64, 30_000_000 // (V * W))))
        return dict(op=op, B=B, W=W, V=V, dtype=dtype, top=rng.choice([W, min(32, 2 * W)]),
                    mask=rng.choice(["none", "none", "shared", "row"]), scale=rng.choice([1.0, 0.7, 1.25]),
                    finished=rng.random() < 0.5)
    heads, dim = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 72, 96, 128, 256])
    length = _spread(rng, 1, 8192)
    most = length if rng.random() < 0.3 else length + _spread(rng, 1, 1024)
    B = _spread(rng, 1, max(1, min(64, 500_000_000 // (W * heads * dim * most))))
    while B * W * heads * most * dim > 536_000_000:
        heads, length, most = max(1, heads // 2), (length + 1) // 2, (most + 1) // 2
    return dict(op=op, B=B, W=W, heads=heads, length=length, most=most, dim=dim, dtype=dtype)


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "norm_grad"):
        T, D = case["T"], case["D"]
        weights = (2 if case["bias"] else 1) * D * 4
        if op == "norm":      # x (and what is added) -> the norm (and the sum), two statistics a row
            return {"bytes": (4 if case["add"] else 2) * T * D * e + weights + 8 * T, "flops": 8 * T * D}
        # r, dn (dr) -> dr's sum, and the gradients of the weights
        return {"bytes": (4 if case["add"] else 3) * T * D * e + D * 4 + weights + 8 * T, "flops": 14 * T * D}
    if op == "fp4":
        M, N, K = case["M"], case["N"], case["K"]
        blocks = -(-K // case["block"])
        n = M * K * e + N * (-(-K // 2) + blocks) + (4 * N if case["block"] == 16 else 0)
        return {"bytes": n + (4 * N if case["bias"] else 0) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    B, W = case["B"], case["W"]
    if op == "beam":
        V = case["V"]
        words = {"none": 0, "shared": 1, "row": B * W}[case["mask"]] * ((V + 31) // 32) * 4
        return {"bytes": B * W * V * e + words + 5 * B * W + 12 * B * case["top"], "flops": 5 * B * W * V}
    # each parent that is taken at all is read once
    read = W * (1 - (1 - 1 / W) ** W)
    row = case["heads"] * case["length"] * case["dim"] * e
    return {"bytes": int(B * (read + W) * row) + 4 * B * W, "flops": 0}


# ---------------------------------------------------------------- the 4-bit format

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _level(v):
    """FP32 values to the nearest of the 4-bit format's, ties to the even code, none above 6."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _quantize(x, block):
    """(levels, the scale of each block, the scale of each row) of the rows of x, by FP32
    operations that are rounded one by one; levels and scales are FP32 values."""
    x = x.float()
    M, K = x.shape
    n = -(-K // block)
    x = torch.nn.functional.pad(x, (0, n * block - K)).view(M, n, block)
    if block == 32:
        # the smallest power of two that brings the block's largest to 6 or below
        m, e = torch.frexp(x.abs().amax(2))
        s = torch.ldexp(torch.ones_like(m), torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 127))
        s = torch.where(m == 0, torch.full_like(s, 2.0 ** -127), s)
        return _level(x / s[:, :, None]).view(M, -1)[:, :K], s, None
    # a quotient of two tensors is rounded once; with a number on either side it is not
    top = x.abs().amax((1, 2))
    t = torch.where(top > 0, torch.full_like(top, 2688.0) / top, torch.zeros_like(top))
    y = x * t[:, None, None]
    s = (y.abs().amax(2) * torch.tensor(1 / 6, device=x.device)).to(torch.float8_e4m3fn).float()
    inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
    return _level(y * inv[:, :, None]).view(M, -1)[:, :K], s, top / torch.full_like(top, 2688.0)


def _pack(levels):
    """Two codes a byte, the first column in the low half; rows start on 16 bytes."""
    M, K = levels.shape
    size = torch.bucketize(levels.abs(), torch.tensor(LEVELS, device=levels.device)).to(torch.uint8)
    codes = torch.where(levels < 0, size + 8, size)
    codes = torch.nn.functional.pad(codes, (0, -K % 32))
    return (codes[:, 0::2] | (codes[:, 1::2] << 4))[:, :(K + 1) // 2]


def _unpack(q, K):
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=q.device)
    return torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], 2).view(q.shape[0], -1)[:, :K]


def _tiles(s):
    """Scales (rows x blocks) as bytes in tiles of 128 rows by 4 blocks: byte 16 (r % 32) + 4 (r / 32) + j
    of a tile is that of its row r and block j; 0 behind the matrix."""
    rows, n = s.shape
    s = torch.nn.functional.pad(s, (0, -n % 4, 0, -rows % 128))
    return s.view(-1, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(s.shape[0] // 128, -1)


def _from_tiles(t, rows, n):
    t = t.view(t.shape[0], -1, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(t.shape[0] * 128, -1)[:rows, :n]


def _scale_values(t, block):
    """The values of the scales' bytes."""
    if block == 16:
        return t.view(torch.float8_e4m3fn).float()
    return torch.ldexp(torch.ones(t.shape, device=t.device), t.to(torch.int32) - 127)


# ---------------------------------------------------------------- what a user's program has in hand

def _mask_words(bits):
    """Truth values of a row as 32-bit words, bit j % 32 of word j // 32 for column j."""
    rows, V = bits.shape
    words = (V + 31) // 32
    full = torch.zeros(rows, words * 32, dtype=torch.int64, device=bits.device)
    full[:, :V] = bits
    packed = (full.view(rows, words, 32) << torch.arange(32, device=bits.device)).sum(2)
    return torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": dict(case), "op": op}
    if op in ("norm", "norm_grad"):
        T, D = case["T"], case["D"]
        # a residual stream: every channel with a size and a mean of its own, a few of them large
        size = torch.exp(0.5 * normal(D)) * torch.where(uniform(D) < 0.01, 10.0, 1.0)
        s["x"] = (normal(T, D) * size + 0.5 * normal(D) + 0.3).to(dt)
        s["w"] = 1 + 0.2 * normal(D)
        s["b"] = 0.1 * normal(D) if case["bias"] else None
        if op == "norm":
            s["add"] = normal(T, D).mul_(0.7).to(dt) if case["add"] else None
        else:
            s["dn"] = normal(T, D).to(dt)
            s["dr"] = normal(T, D).to(dt) if case["add"] else None
            # the two statistics a row that the forward pass returned
            x = s["x"].double()
            s["stats"] = torch.stack([x.mean(1), 1 / (x.var(1, correction=0) + EPS).sqrt()]).float()
    elif op == "fp4":
        M, N, K, block = case["M"], case["N"], case["K"], case["block"]
        size = torch.where(uniform(K) < 0.01, 8.0, 1.0)
        s["x"] = (normal(M, K) * size).to(dt)
        levels, scales, s["w_scale"] = _quantize(normal(N, K).mul_(0.02), block)
        s["w"] = _pack(levels)
        if block == 16:
            s["w_block"] = _tiles(scales.to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            s["w_block"] = _tiles((torch.frexp(scales).exponent + 126).to(torch.uint8))
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        s["out"] = DTYPES[case["out"]]
    elif op == "beam":
        B, W, V = case["B"], case["W"], case["V"]
        s["logits"] = normal(B * W, V).mul_(2.5).to(dt)
        s["mask"] = None
        if case["mask"] != "none":
            s["mask"] = _mask_words(uniform(1 if case["mask"] == "shared" else B * W, V) < 0.6)
        # the beams' log probabilities so far; a beam that was never filled has none
        score = -10 * uniform(B, W)
        score[uniform(B, W) < 0.05] = -math.inf
        s["score"] = score
        s["finished"] = uniform(B, W) < 0.15 if case["finished"] else None
        s["end"], s["scale"], s["top"] = 2, case["scale"], case["top"]
    else:
        B, W = case["B"], case["W"]
        cache = normal(B * W, case["heads"], case["most"], case["dim"]).to(dt)
        s["state"] = cache[:, :, :case["length"]]      # as much of the cache as is filled
        s["parent"] = torch.randint(0, W, (B, W), generator=g, device=dev, dtype=torch.int32)
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_norm(s):
    dt = s["x"].dtype
    # what is normalised is the sum as it is handed on
    r = s["x"] if s["add"] is None else (s["x"].float() + s["add"].float()).to(dt)
    x = r.float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    n = c * rstd[:, None] * s["w"]
    if s["b"] is not None:
        n = n + s["b"]
    return r, n.to(dt), torch.stack([mean, rstd])


def _plain_norm_grad(s):
    dt = s["x"].dtype
    x, dn = s["x"].float(), s["dn"].float()
    mean, rstd = s["stats"][0][:, None], s["stats"][1][:, None]
    h = (x - mean) * rstd
    u = dn * s["w"]
    dx = rstd * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {"dx": dx.to(dt), "dw": (dn * h).sum(0), "db": dn.sum(0) if s["b"] is not None else None}


def _plain_fp4(s):
    K, block = s["case"]["K"], s["case"]["block"]
    N, n = s["w"].shape[0], -(-K // block)

    def values(levels, scales):
        return levels * scales.repeat_interleave(block, 1)[:, :K]

    levels, scales, rows = _quantize(s["x"], block)
    w = values(_unpack(s["w"], K), _scale_values(_from_tiles(s["w_block"], N, n).contiguous(), block))
    y = values(levels, scales) @ w.T
    if block == 16:
        y = y * rows[:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["out"])


def _allowed(z, mask):
    """Logits with the columns that the mask leaves out at minus infinity."""
    if mask is None:
        return z
    V = z.shape[1]
    bits = (mask[:, :, None] >> torch.arange(32, device=z.device, dtype=torch.int32)) & 1
    return torch.where(bits.reshape(mask.shape[0], -1)[:, :V] != 0, z, float("-inf"))


def _plain_beam(s):
    z = _allowed(s["logits"].float(), s["mask"])
    (B, W), V, top = s["score"].shape, z.shape[1], s["top"]
    m = z.amax(1, keepdim=True)
    # each row's best: one whole number per column that orders by the logit, then by the lowest index
    order = z.view(torch.int32).to(torch.int64)
    order = torch.where(order >= 0, order, -(2 ** 31) - order)
    key = (order << 32) + (2 ** 31 - torch.arange(V, device=z.device))
    ids = 2 ** 31 - (key.topk(top, 1).values & 0xFFFFFFFF)
    # candidates of different beams can lie next to each other: in 64 bits
    total = torch.exp((z - m) * s["scale"]).sum(1, keepdim=True, dtype=torch.float64)
    logp = (z.gather(1, ids) - m).double() * s["scale"] - torch.log(total)
    if s["finished"] is not None:
        # a beam that has ended goes on as it is
        done = s["finished"].view(-1, 1)
        only = torch.full_like(logp, float("-inf"))
        only[:, 0] = 0
        logp, ids = torch.where(done, only, logp), torch.where(done, s["end"], ids)
    both = (s["score"].double().view(-1, 1) + logp).view(B, W * top)
    best, at = torch.sort(both, dim=1, descending=True, stable=True)
    best, at = best[:, :top], at[:, :top]
    has = best > float("-inf")
    return {"score": best.float(), "parent": torch.where(has, at // top, -1).to(torch.int32),
            "token": torch.where(has, ids.view(B, -1).gather(1, at), -1).to(torch.int32)}


def _plain_reorder(s):
    B, W = s["parent"].shape
    first = W * torch.arange(B, device=s["parent"].device)
    return s["state"][(first[:, None] + s["parent"]).view(-1)]


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "fp4": _plain_fp4, "beam": _plain_beam,
                "reorder": _plain_reorder}[op](s)
    import dense_fp32_matrix_04_gb300 as sg
    if op == "norm":
        return sg.layer_norm(s["x"], s["w"], bias=s["b"], add=s["add"], eps=EPS)
    if op == "norm_grad":
        dx, dw, db = sg.layer_norm_backward(s["x"], s["w"], s["stats"], s["dn"], dr=s["dr"], bias=s["b"] is not None)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "fp4":
        scales = s["w_block"].view(torch.float8_e4m3fn if s["case"]["block"] == 16 else torch.float8_e8m0fnu)
        return sg.linear_fp4(s["x"], s["w"], scales, s["w_scale"], bias=s["bias"], out_dtype=s["out"])
    if op == "beam":
        score, parent, token = sg.beam_step(s["logits"], s["score"], top=s["top"], scale=s["scale"], mask=s["mask"],
                                            finished=s["finished"], end=s["end"])
        return {"score": score, "parent": parent, "token": token}
    return sg.beam_reorder(s["state"], s["parent"])


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_codes(x, block):
    """What stands for x: whole steps of the format are defined by FP32 operations (they
    jump at halves), so these are repeated here, and everything after them is exact."""
    x = x.float()
    M, K = x.shape
    x = torch.cat([x, x.new_zeros(M, -K % block)], 1).unflatten(1, (-1, block))
    grid = torch.tensor(LEVELS, device=x.device, dtype=torch.float64)
    if block == 32:
        # the power of two by whole numbers: the exponent, one more where the rest is above 1.5
        bits = x.abs().amax(2).view(torch.int32)
        e = (bits >> 23) - 129 + ((bits & 0x7FFFFF) > 0x400000).to(torch.int32)
        s, rows = torch.pow(2.0, e.clamp(-127, 127).double()), None
        v = x.double() / s[..., None]
    else:
        top = torch.amax(torch.abs(x), (1, 2))
        y = x * torch.div(torch.tensor(2688.0, device=x.device).expand_as(top), top)[:, None, None]
        s8 = torch.mul(torch.amax(torch.abs(y), 2), torch.tensor(1 / 6, device=x.device)).to(torch.float8_e4m3fn)
        s, rows = s8.double(), top.double() / 2688
        v = (y * torch.reciprocal(s8.float())[..., None]).double()
        v = torch.where(s[..., None] > 0, v, 0.0)
    # the nearest level, of two the one with the even code
    a = v.abs().clamp(max=6.0)
    low = (torch.searchsorted(grid, a.contiguous(), right=True) - 1).clamp(0, 7)
    high = (low + 1).clamp(max=7)
    up, down = grid[high] - a, a - grid[low]
    code = torch.where((up < down) | ((up == down) & (low % 2 == 1)), high, low)
    value = torch.copysign(grid[code], v) * s[..., None]
    return value.flatten(1)[:, :K], rows


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    op = s["op"]
    if op == "norm":
        r = s["x"].to(f)
        handed_on = s["x"]
        if s["add"] is not None:
            r = r + s["add"].to(f)
            handed_on = r.float().to(s["x"].dtype)
        x = handed_on.to(f)
        mean, var = x.mean(1), x.var(1, correction=0)
        n = torch.einsum("td,t,d->td", x - mean[:, None], 1 / torch.sqrt(var + EPS), s["w"].to(f))
        if s["b"] is not None:
            n = n + s["b"].to(f)
        return r, n, torch.stack([mean, 1 / torch.sqrt(var + EPS)])
    if op == "norm_grad":
        names = ["x", "w"] + (["b"] if s["b"] is not None else [])
        leaf = {k: s[k].to(f).requires_grad_() for k in names}
        x = leaf["x"]
        n = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, correction=0, keepdim=True) + EPS) * leaf["w"]
        if "b" in leaf:
            n = n + leaf["b"]
        outs, grads = (n,), (s["dn"].to(f),)
        if s["dr"] is not None:
            outs, grads = (n, x * 1), (s["dn"].to(f), s["dr"].to(f))
        got = dict(zip(names, torch.autograd.grad(outs, [leaf[k] for k in names], grads)))
        return {"dx": got["x"], "dw": got["w"], "db": got.get("b")}
    if op == "fp4":
        K, block = case["K"], case["block"]
        x, rows = _exact_codes(s["x"], block)
        grid = torch.tensor(LEVELS, device=x.device, dtype=f)
        codes = torch.stack([s["w"] % 16, s["w"] // 16], -1).flatten(1)[:, :K].long()
        w = grid[codes % 8] * (1.0 - 2.0 * (codes // 8))
        r, j = torch.arange(s["w"].shape[0], device=x.device)[:, None], torch.arange(K, device=x.device)[None] // block
        byte = s["w_block"][r // 128, (j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4]
        w = w * (byte.view(torch.float8_e4m3fn).to(f) if block == 16 else torch.pow(2.0, byte.to(f) - 127))
        y = torch.einsum("mk,nk->mn", x, w)
        if block == 16:
            y = y * torch.outer(rows, s["w_scale"].to(f))
        return y if s["bias"] is None else y + s["bias"].to(f)
    if op == "reorder":
        group = torch.arange(case["B"], device=s["parent"].device).repeat_interleave(case["W"])
        return s["state"].unflatten(0, (case["B"], case["W"]))[group, s["parent"].flatten().long()].to(f)
    z = s["logits"].to(f) * s["scale"]
    (B, W), V = s["score"].shape, z.shape[1]
    if s["mask"] is not None:
        col = torch.arange(V, device=z.device)
        word = s["mask"].to(torch.int64)[:, col // 32]
        z = z.masked_fill(((word >> (col % 32)) & 1) == 0, -math.inf)
    p = torch.log_softmax(z, 1)
    if s["finished"] is not None:
        ended = torch.full((V,), -math.inf, dtype=f, device=z.device)
        ended[s["end"]] = 0
        p = torch.where(s["finished"].flatten()[:, None], ended, p)
    total = (p + s["score"].to(f).flatten()[:, None]).view(B, W * V)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :s["top"]], at[:, :s["top"]]
    none = torch.isinf(best)
    return {"score": best, "parent": torch.where(none, -1, at // V).to(torch.int32),
            "token": torch.where(none, -1, at % V).to(torch.int32)}
