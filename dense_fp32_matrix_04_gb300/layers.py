"""The operators of a language model around its matrix products, on CUDA tensors.

Thin forms of the entry points of include/sgemm_layers.h, which states their
formulas and contracts: tensors are checked here, outputs and workspaces are
allocated with torch when they are not given, and every computation runs in the
library's kernels.  A call runs on ``stream`` (a ``torch.cuda.Stream``, a raw
handle, or None: torch's current stream).  Tensors that are used on a stream
other than the one they were made on are the caller's to order, as with any
torch operation; what a call allocates itself is marked as used on its stream.
"""

from __future__ import annotations

import ctypes

_I, _F, _P, _S = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t

SIGNATURES = {
    "sgemm_block_norm": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _F, _F, _P, _I, _P, _I, _P, _I, _P,
                              _P, _P]),
    "sgemm_block_norm_backward": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _F, _P, _P, _I, _P, _I,
                                       _P, _I, _P, _I, _P, _P, _P, _I, _P, _S, _P]),
    "sgemm_block_norm_backward_workspace_size": (_S, [_I, _I]),
    "sgemm_quantize_i8": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P]),
    "sgemm_i8": (_I, [_I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _P, _I, _I, _P, _S, _P]),
    "sgemm_i8_workspace_size": (_S, [_I, _I, _I, _P, _I]),
    "sgemm_linear_i8": (_I, [_I, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _I, _I, _P, _S, _P]),
    "sgemm_linear_i8_workspace_size": (_S, [_I, _I, _I, _P, _I]),
    "sgemm_logprobs": (_I, [_I, _I, _I, _P, _I, _F, _P, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P]),
    "sgemm_logprobs_backward": (_I, [_I, _I, _I, _P, _I, _F, _P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
}

_codes = None
_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load
        _lib = load()
    return _lib


def _check(status, where):
    if status:
        from . import SgemmError
        raise SgemmError(status, where)


def _dtype(t, name):
    """The library's code of a tensor's element type."""
    global _codes
    if _codes is None:
        import torch
        _codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    code = _codes.get(t if not hasattr(t, "dtype") else t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    return code


def _matrix(t, name, dtype, rows=None, cols=None, device=None):
    """(pointer, leading dimension) of a 2-D CUDA tensor with unit column stride."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a 2-D {dtype} CUDA tensor")
    if (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} is {tuple(shape)}, not ({rows}, {cols})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    s0, s1 = t.stride()
    if shape[1] > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride")
    if shape[0] > 1:
        if s0 < shape[1]:
            raise ValueError(f"{name} has rows that overlap")
        return t.data_ptr(), max(s0, 1)
    return t.data_ptr(), max(shape[1], 1)


def _vector(t, name, n, dtypes, device):
    """Pointer of a dense 1-D CUDA tensor of n elements."""
    if t.dtype not in dtypes or not t.is_cuda or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} elements, not {n}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be dense")
    return t.data_ptr()


class _Call:
    """The device and stream of a call: makes the tensors' device current, and
    marks what the call allocated as used on a stream that is not torch's."""

    def __init__(self, device, stream):
        import torch
        self.torch, self.device = torch, device
        self.other = None
        if torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)
            self.guard.__enter__()
        else:
            self.guard = None
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            self.handle = stream if isinstance(stream, int) else int(stream.cuda_stream)
            if self.handle != torch._C._cuda_getCurrentRawStream(device.index):
                self.other = (stream if not isinstance(stream, int)
                              else torch.cuda.ExternalStream(stream, device=device))

    def __enter__(self):
        return self

    def __exit__(self, *_):
        if self.guard is not None:
            self.guard.__exit__(None, None, None)

    def empty(self, shape, dtype):
        t = self.torch.empty(shape, dtype=dtype, device=self.device)
        if self.other is not None:
            # allocated on torch's current stream, used on another
            self.other.wait_stream(self.torch.cuda.current_stream(self.device))
            t.record_stream(self.other)
        return t


def block_norm(x, y, w_pre, w_post=None, gate=None, scale=1.0, eps=1e-6, quantize=False, out=None, stream=None):
    """The step from one block's output ``y`` and the residual stream ``x`` (T x D)
    to the next block's input:

        h = y * rsqrt(mean(y^2) + eps) * w_post      (h = y without ``w_post``)
        r = x + scale * gate * h                     (``gate``: G x D, G divides T; row t takes row t // (T / G))
        n = r * rsqrt(mean(r^2) + eps) * w_pre

    Returns ``(r, n, rstd)``, or with ``quantize`` ``(r, q, q_scale, rstd)``: n as
    8-bit integers with a scale per row.  ``rstd`` (2 x T) is for the backward
    pass.  ``out`` receives r; it may be x.
    """
    import torch
    dt, dev = x.dtype, x.device
    T, D = x.shape
    px, ldx = _matrix(x, "x", dt)
    py, ldy = _matrix(y, "y", dt, T, D, dev)
    code = _dtype(x, "x")
    weights = (torch.float32, dt)
    p_pre = _vector(w_pre, "w_pre", D, weights, dev)
    p_post = _vector(w_post, "w_post", D, (w_pre.dtype,), dev) if w_post is not None else 0
    pg, ldg, G = 0, 1, 0
    if gate is not None:
        pg, ldg = _matrix(gate, "gate", dt, None, D, dev)
        G = gate.shape[0]
    with _Call(dev, stream) as c:
        r = c.empty((T, D), dt) if out is None else out
        pr, ldr = _matrix(r, "out", dt, T, D, dev)
        rstd = c.empty((2, T), torch.float32)
        n = q = s = None
        if quantize:
            q, s = c.empty((T, D), torch.int8), c.empty((T,), torch.float32)
        else:
            n = c.empty((T, D), dt)
        _check(_library().sgemm_block_norm(
            T, D, code, px, ldx, py, ldy, p_pre, p_post, _dtype(w_pre, "w_pre"), pg, ldg, G, scale, eps, pr, ldr,
            n.data_ptr() if n is not None else 0, max(D, 1), q.data_ptr() if quantize else 0, max(D, 1),
            s.data_ptr() if quantize else 0, rstd.data_ptr(), c.handle), "sgemm_block_norm")
    return (r, q, s, rstd) if quantize else (r, n, rstd)


def block_norm_backward(x, y, w_pre, rstd, dn, dr=None, w_post=None, gate=None, scale=1.0, stream=None):
    """Gradients ``(dx, dy, dw_pre, dw_post, dgate)`` of ``block_norm`` from those of
    its n and r (``dr`` None: zero); ``dw_post`` and ``dgate`` are None where there is
    no such input."""
    import torch
    dt, dev = x.dtype, x.device
    T, D = x.shape
    px, ldx = _matrix(x, "x", dt)
    py, ldy = _matrix(y, "y", dt, T, D, dev)
    pn, ldn = _matrix(dn, "dn", dt, T, D, dev)
    pr, ldr = _matrix(dr, "dr", dt, T, D, dev) if dr is not None else (0, max(D, 1))
    code = _dtype(x, "x")
    p_pre = _vector(w_pre, "w_pre", D, (torch.float32, dt), dev)
    p_post = _vector(w_post, "w_post", D, (w_pre.dtype,), dev) if w_post is not None else 0
    if rstd.dtype != torch.float32 or tuple(rstd.shape) != (2, T) or not rstd.is_contiguous() or rstd.device != dev:
        raise ValueError("rstd must be the (2, T) float32 tensor that block_norm returned")
    pg, ldg, G = 0, 1, 0
    if gate is not None:
        pg, ldg = _matrix(gate, "gate", dt, None, D, dev)
        G = gate.shape[0]
    with _Call(dev, stream) as c:
        dx, dy = c.empty((T, D), dt), c.empty((T, D), dt)
        dw_pre = c.empty((D,), w_pre.dtype)
        dw_post = c.empty((D,), w_pre.dtype) if w_post is not None else None
        dgate = c.empty((G, D), dt) if gate is not None else None
        lib = _library()
        need = lib.sgemm_block_norm_backward_workspace_size(T, D)
        ws = c.empty((need,), torch.uint8)
        _check(lib.sgemm_block_norm_backward(
            T, D, code, px, ldx, py, ldy, p_pre, p_post, _dtype(w_pre, "w_pre"), pg, ldg, G, scale, rstd.data_ptr(),
            pn, ldn, pr, ldr, dx.data_ptr(), max(D, 1), dy.data_ptr(), max(D, 1), dw_pre.data_ptr(),
            dw_post.data_ptr() if dw_post is not None else 0, dgate.data_ptr() if dgate is not None else 0,
            max(D, 1), ws.data_ptr(), need, c.handle), "sgemm_block_norm_backward")
    return dx, dy, dw_pre, dw_post, dgate


def quantize_i8(x, stream=None):
    """``(q, scale)``: the rows of x (M x K) as 8-bit integers, scale = max|row| / 127
    and q = rint(row * (127 / max|row|)).  For activations a scale per token, for
    weights (N x K) one per output channel."""
    import torch
    code = _dtype(x, "x")
    px, ldx = _matrix(x, "x", x.dtype)
    M, K = x.shape
    with _Call(x.device, stream) as c:
        q, s = c.empty((M, K), torch.int8), c.empty((M,), torch.float32)
        _check(_library().sgemm_quantize_i8(M, K, code, px, ldx, q.data_ptr(), max(K, 1), s.data_ptr(), c.handle),
               "sgemm_quantize_i8")
    return q, s


def matmul_i8(a, a_scale, w, w_scale, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """``a_scale[m] * w_scale[n] * sum_k a[m, k] w[n, k] + bias[n]`` for 8-bit integers
    a (M x K) and w (N x K), in ``out_dtype`` (float32 unless said otherwise)."""
    import torch
    dev = a.device
    pa, lda = _matrix(a, "a", torch.int8)
    M, K = a.shape
    pw, ldw = _matrix(w, "w", torch.int8, None, K, dev)
    N = w.shape[0]
    f32 = (torch.float32,)
    ps, pt = _vector(a_scale, "a_scale", M, f32, dev), _vector(w_scale, "w_scale", N, f32, dev)
    pb = _vector(bias, "bias", N, f32, dev) if bias is not None else 0
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty((M, N), out_dtype or torch.float32)
        code = _dtype(out, "out")
        po, ldo = _matrix(out, "out", out_dtype or out.dtype, M, N, dev)
        lib = _library()
        need = lib.sgemm_i8_workspace_size(M, N, K, pw, ldw)
        if workspace is None and need:
            workspace = c.empty((need,), torch.uint8)
        size = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib.sgemm_i8(M, N, K, pa, lda, ps, pw, ldw, pt, pb, po, ldo, code,
                            workspace.data_ptr() if size else 0, size, c.handle), "sgemm_i8")
    return out


def linear_i8(x, w, w_scale, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """``matmul_i8`` on the rows of x (M x K, float32, bfloat16 or float16), which are
    quantised first as ``quantize_i8`` does it; ``out_dtype`` is x's unless said otherwise."""
    import torch
    dev = x.device
    xcode = _dtype(x, "x")
    px, ldx = _matrix(x, "x", x.dtype)
    M, K = x.shape
    pw, ldw = _matrix(w, "w", torch.int8, None, K, dev)
    N = w.shape[0]
    f32 = (torch.float32,)
    pt = _vector(w_scale, "w_scale", N, f32, dev)
    pb = _vector(bias, "bias", N, f32, dev) if bias is not None else 0
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty((M, N), out_dtype or x.dtype)
        code = _dtype(out, "out")
        po, ldo = _matrix(out, "out", out_dtype or out.dtype, M, N, dev)
        lib = _library()
        need = lib.sgemm_linear_i8_workspace_size(M, N, K, pw, ldw)
        if workspace is None and need:
            workspace = c.empty((need,), torch.uint8)
        size = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib.sgemm_linear_i8(M, N, K, xcode, px, ldx, pw, ldw, pt, pb, po, ldo, code,
                                   workspace.data_ptr() if size else 0, size, c.handle), "sgemm_linear_i8")
    return out


def _mask(mask, T, V, device):
    """(pointer, words between rows, rows) of a mask of ceil(V / 32) words a row."""
    import torch
    if mask is None:
        return 0, 0, 0
    pm, ldm = _matrix(mask, "mask", torch.int32, None, (V + 31) // 32, device)
    if mask.shape[0] not in (1, T):
        raise ValueError(f"mask has {mask.shape[0]} rows, not 1 or {T}")
    return pm, ldm, mask.shape[0]


def logprobs(logits, target, scale=1.0, mask=None, top=0, stream=None):
    """``(logprob, entropy, lse)`` per row of ``softmax(scale * logits)`` (T x V), and with
    ``top`` > 0 also ``(top_logprob, top_id)`` (T x top), most likely first.

    ``target``: T int64 columns; a negative one is not scored (logprob 0).
    ``mask``: int32 words, 1 or T rows of ceil(V / 32), bit j % 32 of word j // 32 set
    where column j is allowed."""
    import torch
    code = _dtype(logits, "logits")
    dev = logits.device
    pz, ldz = _matrix(logits, "logits", logits.dtype)
    T, V = logits.shape
    py = _vector(target, "target", T, (torch.int64,), dev)
    pm, ldm, rows = _mask(mask, T, V, dev)
    with _Call(dev, stream) as c:
        three = c.empty((3, T), torch.float32)
        p = three.data_ptr()
        got = three.unbind(0)
        pv = pi = 0
        if top:
            values, ids = c.empty((T, top), torch.float32), c.empty((T, top), torch.int32)
            pv, pi = values.data_ptr(), ids.data_ptr()
            got = (*got, values, ids)
        _check(_library().sgemm_logprobs(T, V, code, pz, ldz, scale, pm, ldm, rows, py, p, p + 4 * T, p + 8 * T, top,
                                         pv, pi, c.handle), "sgemm_logprobs")
    return got


def logprobs_backward(logits, target, lse, entropy, g_logprob, g_entropy=None, scale=1.0, mask=None, out=None,
                      stream=None):
    """The gradient with respect to the logits of ``logprobs``' logprob and entropy, from
    theirs (``g_entropy`` None: no gradient reaches the entropy).  ``out`` may be the
    logits themselves."""
    import torch
    code = _dtype(logits, "logits")
    dev = logits.device
    pz, ldz = _matrix(logits, "logits", logits.dtype)
    T, V = logits.shape
    py = _vector(target, "target", T, (torch.int64,), dev)
    f32 = (torch.float32,)
    pl = _vector(lse, "lse", T, f32, dev)
    ph = _vector(entropy, "entropy", T, f32, dev) if entropy is not None else 0
    pg = _vector(g_logprob, "g_logprob", T, f32, dev)
    pe = _vector(g_entropy, "g_entropy", T, f32, dev) if g_entropy is not None else 0
    pm, ldm, rows = _mask(mask, T, V, dev)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty((T, V), logits.dtype)
        po, ldo = _matrix(out, "out", logits.dtype, T, V, dev)
        _check(_library().sgemm_logprobs_backward(T, V, code, pz, ldz, scale, pm, ldm, rows, py, pl, ph, pg, pe, po,
                                                  ldo, c.handle), "sgemm_logprobs_backward")
    return out
