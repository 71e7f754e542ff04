"""The operators of a language model around its matrix products, on CUDA tensors.

Thin forms of the entry points of include/sgemm_layers.h, which states their
formulas and contracts: tensors are checked here, outputs and workspaces are
allocated with torch when they are not given, and every computation runs in the
library's kernels.  A call runs on ``stream`` (a ``torch.cuda.Stream``, a raw
handle, or None: torch's current stream).  Tensors that are used on a stream
other than the one they were made on are the caller's to order, as with any
torch operation; what a call allocates itself is marked as used on its stream.

No call is recorded by torch's autograd: what comes back does not require a
gradient, whatever the inputs do, and the gradients are calls of their own.
"""

from __future__ import annotations

import ctypes
import functools
import inspect

_I, _L, _F, _P, _S = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t

SIGNATURES = {
    "sgemm_block_norm": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _F, _F, _P, _I, _P, _I, _P, _I, _P,
                              _P, _P]),
    "sgemm_block_norm_backward": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _F, _P, _P, _I, _P, _I,
                                       _P, _I, _P, _I, _P, _P, _P, _I, _P, _S, _P]),
    "sgemm_block_norm_backward_workspace_size": (_S, [_I, _I]),
    "sgemm_layer_norm": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _F, _P, _I, _P, _I, _P, _P]),
    "sgemm_layer_norm_backward": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _P, _I, _P, _P, _P, _S, _P]),
    "sgemm_layer_norm_backward_workspace_size": (_S, [_I, _I]),
    "sgemm_quantize_i8": (_I, [_I, _I, _I, _P, _I, _P, _I, _P, _P]),
    "sgemm_i8": (_I, [_I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _P, _I, _I, _P, _S, _P]),
    "sgemm_i8_workspace_size": (_S, [_I, _I, _I, _P, _I]),
    "sgemm_linear_i8": (_I, [_I, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _I, _I, _P, _S, _P]),
    "sgemm_linear_i8_workspace_size": (_S, [_I, _I, _I, _P, _I]),
    "sgemm_quantize_fp4": (_I, [_I, _I, _I, _P, _I, _I, _P, _I, _P, _P, _P]),
    "sgemm_fp4_scales_size": (_S, [_I, _I, _I]),
    "sgemm_fp4_lay_out_scales": (_I, [_I, _I, _I, _P, _I, _P, _P]),
    "sgemm_fp4": (_I, [_I, _I, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _P]),
    "sgemm_fp4_plan_model": (_I, [_I, _I, _I, _I, _P, _P]),
    "sgemm_linear_fp4": (_I, [_I, _I, _I, _I, _P, _I, _I, _P, _I, _P, _P, _P, _P, _I, _I, _P, _S, _P]),
    "sgemm_linear_fp4_workspace_size": (_S, [_I, _I, _I]),
    "sgemm_logprobs": (_I, [_I, _I, _I, _P, _I, _F, _P, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P]),
    "sgemm_beam_step": (_I, [_I, _I, _I, _I, _P, _I, _F, _P, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _S, _P]),
    "sgemm_beam_step_workspace_size": (_S, [_I, _I, _I]),
    "sgemm_beam_reorder": (_I, [_I, _I, _I, _L, _L, _P, _L, _L, _P, _P, _L, _L, _P]),
    "sgemm_logprobs_backward": (_I, [_I, _I, _I, _P, _I, _F, _P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
}

# Set on the first call: torch, the library, the codes of the element types.
# What a call costs on the host is a few microseconds, which a decoding step
# sees, so the checks below ask a tensor as little as they can.
_torch = _lib = None
_codes = {}
_raw_stream = _current_device = None


def _start():
    global _torch, _lib, _raw_stream, _current_device
    import torch

    from . import load
    _lib = load()
    _codes.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch = torch


def _check(status, where):
    from . import SgemmError
    raise SgemmError(status, where)


def _first(t, name, dtypes=None):
    """(element type, device index, shape, pointer, leading dimension) of a call's first
    tensor, a 2-D CUDA one."""
    if _torch is None:
        _start()
    dtype = t.dtype
    if dtype not in (_codes if dtypes is None else dtypes):
        raise TypeError(f"{name} must be {'float32, bfloat16 or float16' if dtypes is None else dtypes[0]}")
    index = t.get_device()
    if index < 0 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D CUDA tensor")
    shape = t.shape
    return (dtype, index, shape, *_rows(t, name, *shape))


# What the library's sizes and leading dimensions can be: ctypes would drop the upper half of a
# larger number without a word.
_MOST = 2 ** 31 - 1


def _rows(t, name, rows, n):
    """(pointer, leading dimension) of a matrix with unit column stride."""
    if rows > _MOST or n > _MOST:
        raise ValueError(f"{name} is ({rows}, {n}): rows and columns must be below 2^31")
    if t.is_contiguous():
        return t.data_ptr(), n or 1
    s0, s1 = t.stride()
    if n > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1:
        if s0 < n:
            raise ValueError(f"{name} has rows that overlap")
        if s0 > _MOST:
            raise ValueError(f"{name} has rows {s0} elements apart: they must be below 2^31")
        return t.data_ptr(), s0 or 1
    return t.data_ptr(), n or 1


def _matrix(t, name, dtype, index, shape=None, cols=None):
    """(pointer, leading dimension) of a 2-D CUDA tensor with unit column stride, of
    this shape, or of this many columns."""
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 2:
        if t.dtype is dtype and t.dim() == 2 and t.get_device() >= 0:
            raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
        raise TypeError(f"{name} must be a 2-D {dtype} CUDA tensor")
    rows, n = t.shape
    if (shape is not None and (rows != shape[0] or n != shape[1])) or (cols is not None and n != cols):
        raise ValueError(f"{name} is ({rows}, {n}), not {tuple(shape) if shape is not None else ('any', cols)}")
    return _rows(t, name, rows, n)


def _vector(t, name, n, dtypes, index):
    """Pointer of a dense 1-D CUDA tensor of n elements."""
    on = t.get_device()
    if t.dtype not in dtypes or on < 0 or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, not {n}")
    if on != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be dense")
    return t.data_ptr()


def _on(index, stream):
    """The raw handle of the stream that a call on the current device runs on."""
    if stream is None:
        return _raw_stream(index)
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def _foreign(fn):
    """Runs a call whose tensors are on another device than the current one, or whose
    stream is not torch's: with the device made current, and with what the call
    allocates (on torch's stream) ordered before and marked as used on its stream.  The
    first tensor and the stream are seen by place or by name."""
    names = list(inspect.signature(fn).parameters)
    name, more_than = names[0], names.index("stream") - 1

    @functools.wraps(fn)
    def call(first=None, /, *args, stream=None, **more):
        if _torch is None:
            _start()
        if first is None:
            if name not in more:
                return fn(*args, **more)  # refuses it
            first = more.pop(name)
        if len(args) > more_than and stream is None:
            stream, args = args[more_than], args[:more_than] + args[more_than + 1:]
        index = first.get_device() if isinstance(first, _torch.Tensor) else -1
        if stream is None and (index < 0 or index == _current_device()):
            return fn(first, *args, **more)
        if index < 0:
            return fn(first, *args, stream=stream, **more)  # refuses it
        with _torch.cuda.device(index):
            handle = _on(index, stream)
            if handle == _raw_stream(index):
                return fn(first, *args, **more)
            other = _torch.cuda.ExternalStream(handle, device=index) if isinstance(stream, int) else stream
            # the inputs are the caller's to order; what is allocated here may have been freed by
            # work that is still queued on torch's stream
            other.wait_stream(_torch.cuda.current_stream(index))
            kept = []
            got = fn(first, *args, stream=stream, keep=kept, **more)
            for t in kept:
                t.record_stream(other)
            return got
    return call


@_foreign
def block_norm(x, y, w_pre, w_post=None, gate=None, scale=1.0, eps=1e-6, quantize=False, out=None, stream=None,
               *, keep=None):
    """The step from one block's output ``y`` and the residual stream ``x`` (T x D)
    to the next block's input:

        h = y * rsqrt(mean(y^2) + eps) * w_post      (h = y without ``w_post``)
        r = x + scale * gate * h                     (``gate``: G x D, G divides T; row t takes row t // (T / G))
        n = r * rsqrt(mean(r^2) + eps) * w_pre

    Returns ``(r, n, rstd)``, or with ``quantize`` ``(r, q, q_scale, rstd)``: n as
    8-bit integers with a scale per row.  ``rstd`` (2 x T) is for the backward
    pass.  ``out`` receives r; it may be x.  Rows of no columns (D = 0) have NaN for
    the means' roots and 0 for the scale.  Autograd does not see the call: its gradient
    is ``block_norm_backward``.
    """
    dt, dev, shape, px, ldx = _first(x, "x")
    f32, empty, where = _torch.float32, _torch.empty, x.device
    T, D = shape
    py, ldy = _matrix(y, "y", dt, dev, shape)
    wt = w_pre.dtype
    p_pre = _vector(w_pre, "w_pre", D, (f32, dt), dev)
    p_post = _vector(w_post, "w_post", D, (wt,), dev) if w_post is not None else 0
    pg, ldg, G = 0, 1, 0
    if gate is not None:
        pg, ldg = _matrix(gate, "gate", dt, dev, None, D)
        G = gate.shape[0]
        if not G and T:
            raise ValueError(f"gate has no rows for the {T} of x")
    r = empty(shape, dtype=dt, device=where) if out is None else out
    pr, ldr = _matrix(r, "out", dt, dev, shape) if out is not None else (r.data_ptr(), D or 1)
    rstd = empty((2, T), dtype=f32, device=where)
    if quantize:
        q, s = empty(shape, dtype=_torch.int8, device=where), empty((T,), dtype=f32, device=where)
        made, pn, pq, ps = (r, q, s, rstd), 0, q.data_ptr(), s.data_ptr()
    else:
        n = empty(shape, dtype=dt, device=where)
        made, pn, pq, ps = (r, n, rstd), n.data_ptr(), 0, 0
    status = _lib.sgemm_block_norm(T, D, _codes[dt], px, ldx, py, ldy, p_pre, p_post, _codes[wt], pg, ldg, G, scale, eps,
                                   pr, ldr, pn, D or 1, pq, D or 1, ps, rstd.data_ptr(), _on(dev, stream))
    if status:
        _check(status, "sgemm_block_norm")
    if not D and T:
        _no_columns(rstd, w_post is not None, s if quantize else None, dev, stream)
    if keep is not None:
        keep += made
    return made


def _stream_of(index, stream):
    """The context in which torch's own calls run on the stream of a call."""
    return _torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else
                              _torch.cuda.ExternalStream(_on(index, stream), device=index))


def _no_columns(rstd, post, q_scale, index, stream):
    """What a row of no elements has beside them, which the library does not launch a kernel
    for: the mean of nothing is NaN, the largest of nothing 0."""
    with _stream_of(index, stream):
        rstd.fill_(float("nan"))
        if not post:
            rstd[0].fill_(1.0)
        if q_scale is not None:
            q_scale.zero_()


@_foreign
def block_norm_backward(x, y, w_pre, rstd, dn, dr=None, w_post=None, gate=None, scale=1.0, stream=None, *, keep=None):
    """Gradients ``(dx, dy, dw_pre, dw_post, dgate)`` of ``block_norm`` from those of
    its n and r (``dr`` None: zero); ``dw_post`` and ``dgate`` are None where there is
    no such input."""
    dt, dev, shape, px, ldx = _first(x, "x")
    f32, empty, where = _torch.float32, _torch.empty, x.device
    T, D = shape
    py, ldy = _matrix(y, "y", dt, dev, shape)
    pn, ldn = _matrix(dn, "dn", dt, dev, shape)
    pr, ldr = _matrix(dr, "dr", dt, dev, shape) if dr is not None else (0, D or 1)
    wt = w_pre.dtype
    p_pre = _vector(w_pre, "w_pre", D, (f32, dt), dev)
    p_post = _vector(w_post, "w_post", D, (wt,), dev) if w_post is not None else 0
    if rstd.dtype is not f32 or rstd.shape != (2, T) or not rstd.is_contiguous() or rstd.get_device() != dev:
        raise ValueError("rstd must be the (2, T) float32 tensor that block_norm returned")
    pg, ldg, G = 0, 1, 0
    if gate is not None:
        pg, ldg = _matrix(gate, "gate", dt, dev, None, D)
        G = gate.shape[0]
        if not G and T:
            raise ValueError(f"gate has no rows for the {T} of x")
    dx, dy = empty(shape, dtype=dt, device=where), empty(shape, dtype=dt, device=where)
    dw_pre = empty((D,), dtype=wt, device=where)
    dw_post = empty((D,), dtype=wt, device=where) if w_post is not None else None
    dgate = empty((G, D), dtype=dt, device=where) if gate is not None else None
    need = _lib.sgemm_block_norm_backward_workspace_size(T, D)
    ws = empty((need,), dtype=_torch.uint8, device=where)
    status = _lib.sgemm_block_norm_backward(
        T, D, _codes[dt], px, ldx, py, ldy, p_pre, p_post, _codes[wt], pg, ldg, G, scale, rstd.data_ptr(), pn, ldn, pr,
        ldr, dx.data_ptr(), D or 1, dy.data_ptr(), D or 1, dw_pre.data_ptr(),
        dw_post.data_ptr() if dw_post is not None else 0, dgate.data_ptr() if dgate is not None else 0, D or 1,
        ws.data_ptr(), need, _on(dev, stream))
    if status:
        _check(status, "sgemm_block_norm_backward")
    made = (dx, dy, dw_pre, dw_post, dgate)
    if keep is not None:
        keep += [t for t in (*made, ws) if t is not None]
    return made


@_foreign
def quantize_i8(x, stream=None, *, keep=None):
    """``(q, scale)``: the rows of x (M x K) as 8-bit integers, scale = max|row| / 127
    and q = rint(row * (127 / max|row|)).  For activations a scale per token, for
    weights (N x K) one per output channel.  Has no gradient, and autograd does not see it."""
    dt, dev, shape, px, ldx = _first(x, "x")
    M, K = shape
    q = _torch.empty(shape, dtype=_torch.int8, device=x.device)
    s = _torch.empty((M,), dtype=_torch.float32, device=x.device)
    status = _lib.sgemm_quantize_i8(M, K, _codes[dt], px, ldx, q.data_ptr(), K or 1, s.data_ptr(), _on(dev, stream))
    if status:
        _check(status, "sgemm_quantize_i8")
    if keep is not None:
        keep += [q, s]
    return q, s


def _workspace(t, index):
    """(pointer, bytes) of a workspace that the caller gives, or (0, 0)."""
    if t is None:
        return 0, 0
    on = t.get_device()
    if on < 0:
        raise TypeError("workspace must be a CUDA tensor")
    if on != index:
        raise ValueError(f"workspace is on {t.device}, not on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError("workspace must be dense")
    return t.data_ptr(), t.numel() * t.element_size()


def _linear(call, where, x, head, w, w_scale, bias, out_dtype, out, workspace, stream, keep, size_of):
    """What matmul_i8 and linear_i8 share: the weights, the output and the workspace."""
    dev = x.get_device()
    M, K = x.shape
    pw, ldw = _matrix(w, "w", _torch.int8, dev, None, K)
    N = w.shape[0]
    f32 = (_torch.float32,)
    pt = _vector(w_scale, "w_scale", N, f32, dev)
    pb = _vector(bias, "bias", N, f32, dev) if bias is not None else 0
    if out is None:
        if out_dtype not in _codes:
            raise TypeError("out_dtype must be float32, bfloat16 or float16")
        out = _torch.empty((M, N), dtype=out_dtype, device=x.device)
        po, ldo = out.data_ptr(), N or 1
        if keep is not None:
            keep.append(out)
    else:
        out_dtype = out.dtype
        if out_dtype not in _codes:
            raise TypeError("out must be float32, bfloat16 or float16")
        po, ldo = _matrix(out, "out", out_dtype, dev, (M, N))
    pws, size = _workspace(workspace, dev)
    if workspace is None:
        size = size_of(M, N, K, pw, ldw)
        if size:
            workspace = _torch.empty((size,), dtype=_torch.uint8, device=x.device)
            pws = workspace.data_ptr()
            if keep is not None:
                keep.append(workspace)
    status = call(M, N, K, *head, pw, ldw, pt, pb, po, ldo, _codes[out_dtype], pws, size, _on(dev, stream))
    if status:
        _check(status, where)
    return out


@_foreign
def matmul_i8(a, a_scale, w, w_scale, bias=None, out_dtype=None, out=None, workspace=None, stream=None, *, keep=None):
    """``a_scale[m] * w_scale[n] * sum_k a[m, k] w[n, k] + bias[n]`` for 8-bit integers
    a (M x K) and w (N x K), in ``out_dtype`` (float32 unless said otherwise).  For inference:
    autograd does not see it."""
    if _torch is None:
        _start()
    _, dev, shape, pa, lda = _first(a, "a", (_torch.int8,))
    ps = _vector(a_scale, "a_scale", shape[0], (_torch.float32,), dev)
    return _linear(_lib.sgemm_i8, "sgemm_i8", a, (pa, lda, ps), w, w_scale, bias, out_dtype or _torch.float32, out,
                   workspace, stream, keep, _lib.sgemm_i8_workspace_size)


@_foreign
def linear_i8(x, w, w_scale, bias=None, out_dtype=None, out=None, workspace=None, stream=None, *, keep=None):
    """``matmul_i8`` on the rows of x (M x K, float32, bfloat16 or float16), which are
    quantised first as ``quantize_i8`` does it; ``out_dtype`` is x's unless said otherwise.
    ``workspace``, here and in ``matmul_i8``: a dense tensor of any type with the bytes that
    ``sgemm_linear_i8_workspace_size`` or ``sgemm_i8_workspace_size`` gives; allocated if None.
    For inference: autograd does not see the call."""
    dt, _, _, px, ldx = _first(x, "x")
    return _linear(_lib.sgemm_linear_i8, "sgemm_linear_i8", x, (_codes[dt], px, ldx), w, w_scale, bias, out_dtype or dt,
                   out, workspace, stream, keep, _lib.sgemm_linear_i8_workspace_size)


def _mask(mask, T, V, index):
    """(pointer, words between rows, rows) of a mask of ceil(V / 32) words a row."""
    if mask is None:
        return 0, 0, 0
    pm, ldm = _matrix(mask, "mask", _torch.int32, index, None, (V + 31) // 32)
    rows = mask.shape[0]
    if rows not in (1, T):
        raise ValueError(f"mask has {rows} rows, not 1 or {T}")
    if not V:
        return 0, 0, 0  # no words, and no pointer to them
    return pm, ldm, rows


@_foreign
def logprobs(logits, target, scale=1.0, mask=None, top=0, stream=None, *, keep=None):
    """``(logprob, entropy, lse)`` per row of ``softmax(scale * logits)`` (T x V), and with
    ``top`` > 0 also ``(top_logprob, top_id)`` (T x top), most likely first.

    ``target``: T int64 columns; a negative one is not scored (logprob 0).
    ``mask``: int32 words, 1 or T rows of ceil(V / 32), bit j % 32 of word j // 32 set
    where column j is allowed.  Autograd does not see the call: its gradient is
    ``logprobs_backward``."""
    dt, dev, (T, V), pz, ldz = _first(logits, "logits")
    py = _vector(target, "target", T, (_torch.int64,), dev)
    pm, ldm, rows = _mask(mask, T, V, dev)
    empty, f32, where = _torch.empty, _torch.float32, logits.device
    got = (empty((T,), dtype=f32, device=where), empty((T,), dtype=f32, device=where),
           empty((T,), dtype=f32, device=where))
    pv = pi = 0
    if not -_MOST <= top <= _MOST:
        raise ValueError(f"top is {top}: it must be 0 .. 32")
    if top > 0:
        got += (empty((T, top), dtype=f32, device=where), empty((T, top), dtype=_torch.int32, device=where))
        pv, pi = got[3].data_ptr(), got[4].data_ptr()
    status = _lib.sgemm_logprobs(T, V, _codes[dt], pz, ldz, scale, pm, ldm, rows, py, got[0].data_ptr(),
                                 got[1].data_ptr(), got[2].data_ptr(), top, pv, pi, _on(dev, stream))
    if status:
        _check(status, "sgemm_logprobs")
    if keep is not None:
        keep += got
    return got


@_foreign
def logprobs_backward(logits, target, lse, entropy, g_logprob, g_entropy=None, scale=1.0, mask=None, out=None,
                      stream=None, *, keep=None):
    """The gradient with respect to the logits of ``logprobs``' logprob and entropy, from
    theirs (``g_entropy`` None: no gradient reaches the entropy).  ``out`` may be the
    logits themselves."""
    dt, dev, shape, pz, ldz = _first(logits, "logits")
    T, V = shape
    py = _vector(target, "target", T, (_torch.int64,), dev)
    f32 = (_torch.float32,)
    pl = _vector(lse, "lse", T, f32, dev)
    ph = _vector(entropy, "entropy", T, f32, dev) if entropy is not None else 0
    pg = _vector(g_logprob, "g_logprob", T, f32, dev)
    pe = _vector(g_entropy, "g_entropy", T, f32, dev) if g_entropy is not None else 0
    pm, ldm, rows = _mask(mask, T, V, dev)
    if out is None:
        out = _torch.empty(shape, dtype=dt, device=logits.device)
        po, ldo = out.data_ptr(), V or 1
        if keep is not None:
            keep.append(out)
    else:
        po, ldo = _matrix(out, "out", dt, dev, shape)
    status = _lib.sgemm_logprobs_backward(T, V, _codes[dt], pz, ldz, scale, pm, ldm, rows, py, pl, ph, pg, pe, po, ldo,
                                          _on(dev, stream))
    if status:
        _check(status, "sgemm_logprobs_backward")
    return out



# ---------------------------------------------------------------- through the native binding
#
# The operators below check and allocate in C++ (csrc/native.cpp): a call with three outputs
# costs the host a quarter to a half of what the ones above do.

_native = None


def _load_native():
    global _native
    if _torch is None:
        _start()
    try:
        from . import _native as module
    except ImportError as e:
        raise RuntimeError(f"the native binding is not built ({e}): run python -m dense_fp32_matrix_04_gb300.build") from e
    _native = module
    return module


def _elsewhere(fn, stream, first, *args):
    """A call on a stream that is given: where it is not torch's own, that one is ordered
    behind torch's, which the memory that the call allocates may still be in use on."""
    index = first.get_device() if isinstance(first, _torch.Tensor) else -1
    if index < 0:
        return fn(first, *args, None)  # refuses it
    with _torch.cuda.device(index):
        handle = _on(index, stream)
        if handle != _raw_stream(index):
            other = _torch.cuda.ExternalStream(handle, device=index) if isinstance(stream, int) else stream
            other.wait_stream(_torch.cuda.current_stream(index))
        return fn(first, *args, handle)


def layer_norm(x, w, bias=None, add=None, eps=1e-5, out=None, stream=None):
    """The norm of the rows of x (T x D) about their mean, after the sum with ``add``:

        r = x + add                                  (rounded to x's type; r is x without ``add``)
        n = (r - mean) * rstd * w + bias,            rstd = rsqrt(mean((r - mean)^2) + eps)

    Returns ``(r, n, stats)``, of which ``stats`` (2 x T: mean, rstd) and r are for the backward
    pass.  ``out`` receives r; it may be x or add.  Rows of no columns (D = 0) have NaN for their
    statistics.  Autograd does not see the call: its gradient is ``layer_norm_backward``.
    """
    fn = (_native or _load_native()).layer_norm
    return fn(x, w, bias, add, eps, out, None) if stream is None else _elsewhere(fn, stream, x, w, bias, add, eps, out)


def layer_norm_backward(x, w, stats, dn, dr=None, bias=True, stream=None, *, out=None):
    """Gradients ``(dx, dw, db)`` of ``layer_norm`` from those of its n and r (``dr`` None: zero);
    ``x`` is the r that it returned, and ``dx`` the gradient of x and of ``add``.  ``bias`` False: db
    is not computed, and None.  ``out`` receives dx; it may be dn, dr or x."""
    fn = (_native or _load_native()).layer_norm_backward
    if stream is not None:
        return _elsewhere(fn, stream, x, w, stats, dn, dr, bias, out)
    return fn(x, w, stats, dn, dr, bias, out, None)


def quantize_fp4(x, block=16, stream=None):
    """``(q, block_scale, scale)``: the rows of x (M x K) as 4-bit floating point, for
    ``linear_fp4`` and ``matmul_fp4``.  With ``block`` 16, blocks of 16 columns have e4m3 scales
    and rows an FP32 scale; with 32, blocks of 32 have powers of two (e8m0) and ``scale`` is None.

    ``q`` (M x ceil(K / 2), uint8) holds two codes a byte, the even column in the low half, on
    rows a multiple of 16 bytes apart; ``block_scale`` is in tiles of 128 rows by 4 blocks (one row of
    tiles a row of the tensor), with the format's type.  Has no gradient, and autograd does not
    see it.

    ``torch.save`` keeps the distance of q's rows.  ``clone``, ``contiguous`` and ``to`` another device do
    not, where K is not a multiple of 32: rows that lie beside each other are refused by the products, and

        q = torch.nn.functional.pad(q, (0, -q.shape[1] % 16))[:, :q.shape[1]]

    puts them apart again."""
    fn = (_native or _load_native()).quantize_fp4
    return fn(x, block, None) if stream is None else _elsewhere(fn, stream, x, block)


def lay_out_fp4_scales(s, stream=None):
    """Block scales (rows x blocks, float8_e4m3fn of blocks of 16 or float8_e8m0fnu of blocks of
    32) in the tiles that ``matmul_fp4`` and ``linear_fp4`` take, for weights quantised elsewhere."""
    fn = (_native or _load_native()).lay_out_fp4_scales
    return fn(s, None) if stream is None else _elsewhere(fn, stream, s)


def matmul_fp4(a, a_block, a_scale, w, w_block, w_scale, bias=None, out_dtype=None, out=None, stream=None):
    """The product of the matrices that 4-bit codes and their scales stand for, a (M x K) times
    the transpose of w (N x K), plus ``bias``, in ``out_dtype`` (float32 unless said otherwise).
    Codes and scales are as ``quantize_fp4`` returns them, of the same block; ``a_scale`` and
    ``w_scale`` may be None (1).  For inference: autograd does not see it."""
    fn = (_native or _load_native()).matmul_fp4
    if stream is not None:
        return _elsewhere(fn, stream, a, a_block, a_scale, w, w_block, w_scale, bias, out_dtype, out)
    return fn(a, a_block, a_scale, w, w_block, w_scale, bias, out_dtype, out, None)


def linear_fp4(x, w, w_block, w_scale=None, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """``matmul_fp4`` on the rows of x (M x K, float32, bfloat16 or float16), which are quantised
    first as ``quantize_fp4`` does it, in the blocks of ``w_block``; ``out_dtype`` is x's unless said
    otherwise.  ``workspace``: a dense tensor of any type with the bytes that
    ``sgemm_linear_fp4_workspace_size`` gives; allocated if None.  For inference: autograd does
    not see the call."""
    fn = (_native or _load_native()).linear_fp4
    if stream is not None:
        return _elsewhere(fn, stream, x, w, w_block, w_scale, bias, out_dtype, out, workspace)
    return fn(x, w, w_block, w_scale, bias, out_dtype, out, workspace, None)


def beam_step(logits, score, top=None, scale=1.0, mask=None, finished=None, end=0, stream=None):
    """The best continuations of B groups of W beams: ``(score, parent, token)``, each B x top,
    best first, from ``logits`` ((B W) x V; row b W + w is beam w of group b) and the beams' scores
    so far (B x W, float32; -infinity for a beam that does not exist).

    A continuation's score is the beam's plus the log probability of its column in
    ``softmax(scale * logits)`` over the columns that ``mask`` allows (as in ``logprobs``).  Equal ones go
    by the lower beam, then the lower column.  ``top`` is W unless said otherwise.  ``finished`` (B x W,
    bool or uint8): such a beam goes on as it is, with column ``end``.  Where there are fewer than
    ``top`` continuations the rest have score -infinity, parent -1 and token -1.
    Has no gradient, and autograd does not see it."""
    fn = (_native or _load_native()).beam_step
    if stream is not None:
        return _elsewhere(fn, stream, logits, score, top, scale, mask, finished, end)
    return fn(logits, score, top, scale, mask, finished, end, None)


def beam_reorder(state, parent, out=None, stream=None):
    """Rows of ``state`` ((B W) x ..., of any type) as the beams of a step were chosen: row
    b top + k of the result is row b W + parent[b, k] of the state, for ``parent`` (B x top, int32) as
    ``beam_step`` returns it.  Rows whose parent is no beam are left as they are.

    ``out`` receives the rows; it may be the state itself (top = W), which is then reordered
    in place, where rows that stay cost nothing.  What belongs to a row may be one dense run or runs at
    one distance, as in ``cache[:, :, :length]``.  Has no gradient, and autograd does not see it."""
    fn = (_native or _load_native()).beam_reorder
    return fn(state, parent, out, None) if stream is None else _elsewhere(fn, stream, state, parent, out)
