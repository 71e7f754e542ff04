"""Cases that time the language-model operators which sit beside the matrix products.

Three operators, as a block of a model and the head that scores its answers
use them:

* ``block_norm``: the norm after a block, its gate and residual scale, the
  residual sum and the norm before the next block; and its backward pass;
* ``linear_i8``: activations quantised per token to 8-bit integers, multiplied
  with 8-bit weights that carry a scale per output channel;
* ``logprobs``: log probability of a given token per row of logits, entropy,
  log-sum-exp and the most likely alternatives; and the gradient of the first
  two with respect to the logits.

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it makes the calls a user makes of this package.
``exact`` computes the same results in 64 bits from the definitions.
"""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: the whole call is latency
        dict(name="block_norm decode 7x4096", op="norm", T=7, D=4096, dtype="bf16", gate="channel", post=True),
        # a long prompt; the gate is one learnt vector
        dict(name="block_norm prompt 8192x5120", op="norm", T=8192, D=5120, dtype="bf16", gate="channel", post=True),
        # training in bf16: four sequences, each with its own gate (a conditioning signal)
        dict(name="block_norm grad 8192x4096", op="norm_grad", T=8192, D=4096, dtype="bf16", gate="group:2048",
             post=True),
        # training in FP32 with an odd width, the gate computed per token
        dict(name="block_norm grad 2047x1111", op="norm_grad", T=2047, D=1111, dtype="f32", gate="token", post=True),
        # one new token: the weights are read once
        dict(name="linear_i8 1x4096x4096", op="i8", M=1, N=4096, K=4096, dtype="bf16", out="bf16", bias=False),
        # a decoding batch through a wide layer
        dict(name="linear_i8 24x16384x4096", op="i8", M=24, N=16384, K=4096, dtype="bf16", out="bf16", bias=True),
        # the ragged product of this repository's benchmark
        dict(name="linear_i8 3001x4999x2047", op="i8", M=3001, N=4999, K=2047, dtype="f32", out="f32", bias=True),
        # the benchmark's square product, as a long prompt meets it
        dict(name="linear_i8 8192x8192x8192", op="i8", M=8192, N=8192, K=8192, dtype="bf16", out="bf16", bias=False),
        # sampling: a few rows over a large vocabulary, constrained by a mask, with alternatives
        dict(name="logprobs sample 3x131072", op="logprobs", T=3, V=131072, dtype="f32", top=20, mask="row", scale=1.25),
        # scoring a prompt: many rows, an odd vocabulary
        dict(name="logprobs score 4096x50001", op="logprobs", T=4096, V=50001, dtype="bf16", top=5, mask="none",
             scale=1.0),
        # policy gradients with an entropy term
        dict(name="logprobs grad 4096x32000", op="logprobs_grad", T=4096, V=32000, dtype="f32", mask="none", scale=1.0,
             entropy=True),
        dict(name="logprobs grad 511x128001", op="logprobs_grad", T=511, V=128001, dtype="bf16", mask="shared",
             scale=0.7, entropy=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "i8", "i8", "logprobs", "logprobs_grad"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op in ("norm", "norm_grad"):
        D = _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        T = _spread(rng, 1, max(1, min(16384, 32_000_000 // D)))
        gate = rng.choice(["none", "channel", "token", "group"])
        if gate == "group":
            per = _spread(rng, 1, T)
            T = max(1, T // per) * per
            gate = "group:%d" % per
        return dict(op=op, T=T, D=D, dtype=dtype, gate=gate, post=rng.random() < 0.75)
    if op == "i8":
        N, K = _spread(rng, 64, 16384), _spread(rng, 64, 16384)
        if rng.random() < 0.7:
            N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
        M = _spread(rng, 1, 8192)
        while M * N * K > 8192 ** 3:
            M = max(1, M // 2)
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, out=rng.choice(["f32", dtype]), bias=rng.random() < 0.5)
    V = _spread(rng, 1000, 200_000)
    T = _spread(rng, 1, max(1, min(8192, 100_000_000 // V)))
    case = dict(op=op, T=T, V=V, dtype=dtype, mask=rng.choice(["none", "none", "shared", "row"]),
                scale=rng.choice([1.0, 0.7, 1.25]))
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20])
    else:
        case["entropy"] = rng.random() < 0.6
    return case


def _gate_rows(case):
    kind = case["gate"]
    if kind == "none":
        return 0
    if kind == "channel":
        return 1
    return case["T"] if kind == "token" else case["T"] // int(kind.split(":")[1])


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "norm_grad"):
        T, D, G = case["T"], case["D"], _gate_rows(case)
        weights = (2 if case["post"] else 1) * D * 4
        if op == "norm":      # x, y -> r, n and two statistics a row
            return {"bytes": 4 * T * D * e + G * D * e + weights + 8 * T, "flops": 10 * T * D}
        # x, y, dn, dr -> dx, dy, and the gradients of the weights and the gate
        return {"bytes": 6 * T * D * e + 2 * G * D * e + 2 * weights + 8 * T, "flops": 25 * T * D}
    if op == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        n = M * K * e + N * K + 4 * N * (2 if case["bias"] else 1) + M * N * SIZE[case["out"]]
        return {"bytes": n, "flops": 2 * M * N * K}
    T, V = case["T"], case["V"]
    words = {"none": 0, "shared": 1, "row": T}[case["mask"]] * ((V + 31) // 32) * 4
    if op == "logprobs":
        return {"bytes": T * V * e + words + 8 * T + 12 * T + 8 * T * case["top"], "flops": 6 * T * V}
    return {"bytes": 2 * T * V * e + words + 8 * T + 16 * T, "flops": 7 * T * V}


# ---------------------------------------------------------------- what a user's program has in hand

def _pack(bits):
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
        T, D, G = case["T"], case["D"], _gate_rows(case)
        # a residual stream: every channel with a size of its own, a few of them large
        size = torch.exp(0.5 * normal(D)) * torch.where(uniform(D) < 0.01, 10.0, 1.0)
        s["x"] = (normal(T, D) * size).to(dt)
        s["y"] = normal(T, D).mul_(0.7).to(dt)
        s["w_pre"] = 1 + 0.2 * normal(D)
        s["w_post"] = 1 + 0.2 * normal(D) if case["post"] else None
        s["gate"] = (0.5 + 0.5 * normal(G, D)).to(dt) if G else None
        s["scale"] = 0.8
        if op == "norm_grad":
            s["dn"] = normal(T, D).to(dt)
            s["dr"] = normal(T, D).to(dt)
            # the two statistics a row that the forward pass returned
            x, y = s["x"].float(), s["y"].float()
            rho = (y.square().mean(1) + EPS).rsqrt()
            h = y * rho[:, None] * s["w_post"] if case["post"] else y
            if G:
                h = h * s["gate"].float().repeat_interleave(T // G, 0)
            r = x + s["scale"] * h
            s["rstd"] = torch.stack([rho if case["post"] else torch.ones_like(rho),
                                     (r.square().mean(1) + EPS).rsqrt()])
    elif op == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        size = torch.where(uniform(K) < 0.01, 8.0, 1.0)
        s["x"] = (normal(M, K) * size).to(dt)
        w = normal(N, K).mul_(0.02)
        top = w.abs().amax(1)
        s["w"] = (w * (127.0 / top)[:, None]).round_().to(torch.int8)
        s["w_scale"] = top / 127.0
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        s["out"] = DTYPES[case["out"]]
    else:
        T, V = case["T"], case["V"]
        z = normal(T, V).mul_(2.5)
        target = torch.randint(0, V, (T,), generator=g, device=dev)
        # the given token is mostly a likely one; some rows are not scored
        z[torch.arange(T, device=dev), target] += 9 * uniform(T)
        s["logits"] = z.to(dt)
        s["mask"] = None
        if case["mask"] != "none":
            bits = uniform(1 if case["mask"] == "shared" else T, V) < 0.6
            s["mask"] = _pack(bits)
        s["target"] = torch.where(uniform(T) < 0.05, torch.full_like(target, -1), target)
        s["scale"] = case["scale"]
        if op == "logprobs":
            s["top"] = case["top"]
        else:
            a = _allowed(s["logits"].float() * s["scale"], s["mask"])
            s["lse"] = torch.logsumexp(a, 1)
            p = torch.exp(a - s["lse"][:, None])
            s["entropy"] = s["lse"] - (p * torch.where(p > 0, a, torch.zeros_like(a))).sum(1)
            s["g_logprob"] = normal(T)
            s["g_entropy"] = 0.1 * normal(T) if case["entropy"] else None
    return s


# ---------------------------------------------------------------- the plain forms

def _allowed(z, mask):
    """Logits with the columns that the mask leaves out at minus infinity."""
    if mask is None:
        return z
    V = z.shape[1]
    bits = (mask[:, :, None] >> torch.arange(32, device=z.device, dtype=torch.int32)) & 1
    return torch.where(bits.reshape(mask.shape[0], -1)[:, :V] != 0, z, float("-inf"))


def _plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    T, D = x.shape
    if s["w_post"] is not None:
        rho = torch.rsqrt((y * y).mean(1) + EPS)
        h = y * rho[:, None] * s["w_post"]
    else:
        rho, h = torch.ones(T, device=x.device), y
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        h = (h.view(G, T // G, D) * s["gate"].float()[:, None, :]).view(T, D)
    r = x + s["scale"] * h
    rho2 = torch.rsqrt((r * r).mean(1) + EPS)
    n = r * rho2[:, None] * s["w_pre"]
    return r.to(s["x"].dtype), n.to(s["x"].dtype), torch.stack([rho, rho2])


def _plain_norm_grad(s):
    dt = s["x"].dtype
    x, y, dn, dr = s["x"].float(), s["y"].float(), s["dn"].float(), s["dr"].float()
    T, D = x.shape
    rho, rho2 = s["rstd"][0][:, None], s["rstd"][1][:, None]
    h = y * rho * s["w_post"] if s["w_post"] is not None else y
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        gate = s["gate"].float()[:, None, :].expand(G, T // G, D).reshape(T, D)
        r = x + s["scale"] * gate * h
    else:
        r = x + s["scale"] * h
    dw_pre = (dn * r * rho2).sum(0)
    u = dn * s["w_pre"]
    dx = dr + rho2 * u - r * (rho2 ** 3 * (u * r).mean(1, keepdim=True))
    dh = s["scale"] * dx
    dgate = None
    if s["gate"] is not None:
        dgate = (dh * h).view(G, T // G, D).sum(1).to(dt)
        dh = dh * gate
    dw_post = None
    if s["w_post"] is not None:
        dw_post = (dh * y * rho).sum(0)
        v = dh * s["w_post"]
        dy = rho * v - y * (rho ** 3 * (v * y).mean(1, keepdim=True))
    else:
        dy = dh
    return {"dx": dx.to(dt), "dy": dy.to(dt), "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


def _plain_i8(s):
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    # a quotient of two tensors is rounded once; with a number on either side it is not
    q = (x * (torch.full_like(top, 127.0) / top)).round()
    y = (q @ s["w"].float().T) * (top / torch.full_like(top, 127.0)) * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["out"])


def _plain_logprobs(s):
    z = s["logits"].float()
    a = _allowed(z * s["scale"], s["mask"])
    T, V = a.shape
    m = a.amax(1, keepdim=True)
    e = torch.exp(a - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    mean = (e * torch.where(e > 0, a - m, 0.0)).sum(1) / total[:, 0]
    entropy = torch.log(total)[:, 0] - mean
    at = a.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    out = {"logprob": torch.where(s["target"] >= 0, at - lse, 0.0), "entropy": entropy, "lse": lse}
    if s["top"]:
        # one whole number per column that orders by the logit, then by the lowest index
        order = _allowed(z, s["mask"]).view(torch.int32).to(torch.int64)
        order = torch.where(order >= 0, order, -(2 ** 31) - order)
        key = (order << 32) + (2 ** 31 - torch.arange(V, device=z.device))
        ids = (2 ** 31 - (key.topk(s["top"], 1).values & 0xFFFFFFFF))
        best = a.gather(1, ids)
        out["top_logprob"] = best - lse[:, None]
        out["top_id"] = torch.where(best > float("-inf"), ids, -1).to(torch.int32)
    return out


def _plain_logprobs_grad(s):
    z = s["logits"]
    a = _allowed(z.float() * s["scale"], s["mask"])
    T = a.shape[0]
    logp = a - s["lse"][:, None]
    p = torch.exp(logp)
    gl = torch.where(s["target"] >= 0, s["g_logprob"], 0.0)
    d = -gl[:, None] * p
    if s["g_entropy"] is not None:
        d = d - s["g_entropy"][:, None] * p * (torch.where(p > 0, logp, 0.0) + s["entropy"][:, None])
    rows = torch.arange(T, device=z.device)
    at = s["target"].clamp(min=0)
    d[rows, at] += torch.where(a[rows, at] > float("-inf"), gl, 0.0)
    return (s["scale"] * d).to(z.dtype)


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "i8": _plain_i8, "logprobs": _plain_logprobs,
                "logprobs_grad": _plain_logprobs_grad}[op](s)
    import dense_fp32_matrix_04_gb300 as sg
    if op == "norm":
        return sg.block_norm(s["x"], s["y"], s["w_pre"], w_post=s["w_post"], gate=s["gate"], scale=s["scale"], eps=EPS)
    if op == "norm_grad":
        dx, dy, dw_pre, dw_post, dgate = sg.block_norm_backward(
            s["x"], s["y"], s["w_pre"], s["rstd"], s["dn"], s["dr"], w_post=s["w_post"], gate=s["gate"],
            scale=s["scale"])
        return {"dx": dx, "dy": dy, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
    if op == "i8":
        return sg.linear_i8(s["x"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=s["out"])
    if op == "logprobs":
        got = sg.logprobs(s["logits"], s["target"], scale=s["scale"], mask=s["mask"], top=s["top"])
        return dict(zip(("logprob", "entropy", "lse", "top_logprob", "top_id"), got))
    return sg.logprobs_backward(s["logits"], s["target"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"],
                                scale=s["scale"], mask=s["mask"])


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    op = s["op"]
    if op in ("norm", "norm_grad"):
        leaf = {k: s[k].to(f).requires_grad_() for k in ("x", "y", "w_pre", "w_post", "gate") if s[k] is not None}
        x, y = leaf["x"], leaf["y"]
        T = x.shape[0]
        one = torch.ones(T, dtype=f, device=x.device)
        rho = 1 / torch.sqrt((y ** 2).mean(1) + EPS) if "w_post" in leaf else one
        h = torch.einsum("td,t->td", y, rho)
        if "w_post" in leaf:
            h = h * leaf["w_post"]
        if "gate" in leaf:
            G = leaf["gate"].shape[0]
            h = h * leaf["gate"][torch.arange(T, device=x.device) // (T // G)]
        r = x + s["scale"] * h
        rho2 = 1 / torch.sqrt((r ** 2).mean(1) + EPS)
        n = torch.einsum("td,t->td", r, rho2) * leaf["w_pre"]
        if op == "norm":
            return r.detach(), n.detach(), torch.stack([rho, rho2]).detach()
        names = list(leaf)
        got = torch.autograd.grad((n, r), [leaf[k] for k in names], (s["dn"].to(f), s["dr"].to(f)))
        d = dict(zip(names, got))
        return {"dx": d["x"], "dy": d["y"], "dw_pre": d["w_pre"], "dw_post": d.get("w_post"), "dgate": d.get("gate")}
    if op == "i8":
        # the whole numbers that stand for x are defined by FP32 operations (they jump at
        # halves); everything after them is exact: sums below 2^53 in any order
        x = s["x"].float()
        largest = torch.amax(torch.abs(x), 1)
        q = torch.round(x * torch.div(torch.tensor(127.0, device=x.device).expand_as(largest), largest)[:, None]).to(f)
        y = torch.einsum("mk,nk->mn", q, s["w"].to(f))
        y = y * torch.outer(largest.to(f) / 127, s["w_scale"].to(f))
        return y if s["bias"] is None else y + s["bias"].to(f)
    z = s["logits"].to(f) * s["scale"]
    T, V = z.shape
    if s["mask"] is not None:
        col = torch.arange(V, device=z.device)
        word = s["mask"].to(torch.int64)[:, col // 32]
        z = z.masked_fill(((word >> (col % 32)) & 1) == 0, -math.inf)
    logp = torch.log_softmax(z, 1)
    p = logp.exp()
    entropy = -torch.xlogy(p, p).sum(1)
    scored = s["target"] >= 0
    pick = torch.where(scored, s["target"], 0)
    rows = torch.arange(T, device=z.device)
    if op == "logprobs":
        out = {"logprob": torch.where(scored, logp[rows, pick], 0.0), "entropy": entropy,
               "lse": torch.logsumexp(z, 1)}
        if s["top"]:
            best, ids = torch.sort(z, dim=1, descending=True, stable=True)
            best, ids = best[:, :s["top"]], ids[:, :s["top"]]
            out["top_logprob"] = torch.gather(logp, 1, ids)
            out["top_id"] = torch.where(torch.isinf(best), -1, ids).to(torch.int32)
        return out
    gl = torch.where(scored, s["g_logprob"].to(f), 0.0)
    dz = p * -gl[:, None]
    hit = torch.where(torch.isinf(z[rows, pick]), 0.0, gl)
    dz.index_put_((rows, pick), hit, accumulate=True)
    if s["g_entropy"] is not None:
        dz -= s["g_entropy"].to(f)[:, None] * (torch.xlogy(p, p) + p * entropy[:, None])
    return dz * s["scale"]
