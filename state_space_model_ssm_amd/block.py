"""Python binding of libssm_block (include/ssm_block.h): gated linear
recurrence, residual addition with RMS norm, and sliding-window attention
with sinks on MI355X.

Argument marshalling only, as for libssm: PyTorch supplies device memory and
the current HIP stream; if ``libssm_block.so`` is missing the calls raise.
The names are also available from the package itself:

    import state_space_model_ssm_amd as ssm
    y, s = ssm.rms_add_fwd(x, w, residual)
    h, h_last, states = ssm.glr_fwd(u, rec, inp, A, return_states=True)
    o, lse = ssm.swa_fwd(q, k, v, window=1024, sinks=4)
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import _BLOCK, SSM_BF16, SSM_F32, SsmError

__all__ = list(_BLOCK)

GLR_STATE_STEP = 16   # steps between two saved states of the recurrence

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssm_block.so")
_lib = None
_F32, _BF16 = torch.float32, torch.bfloat16
_CODES = {_F32: SSM_F32, _BF16: SSM_BF16}

# The calls below are single kernels of a few microseconds at decoding sizes,
# so their marshalling is kept to what costs little: no context managers, no
# stream objects, no conversions.


class GlrDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("reserved2", ctypes.c_int32), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class RmsDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("group", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class SwaDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("nkv", ctypes.c_int64), ("headdim", ctypes.c_int64), ("window", ctypes.c_int64),
                ("sinks", ctypes.c_int64), ("q_batch", ctypes.c_int64), ("q_token", ctypes.c_int64),
                ("k_batch", ctypes.c_int64), ("k_token", ctypes.c_int64), ("v_batch", ctypes.c_int64),
                ("v_token", ctypes.c_int64), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


def block_library_path() -> str:
    return _LIB_PATH


def block_lib():
    """The loaded libssm_block (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m state_space_model_ssm_amd.build` "
                "(hipcc, gfx950). There is no fallback implementation.")
        L = ctypes.CDLL(_LIB_PATH)
        vp, size = ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
        for name, pointers, dims in (
                ("ssm_glr_fwd", 9, GlrDims), ("ssm_glr_bwd", 13, GlrDims), ("ssm_glr_step", 7, GlrDims),
                ("ssm_rms_add_fwd", 5, RmsDims), ("ssm_rms_add_q8_fwd", 6, RmsDims), ("ssm_rms_add_bwd", 6, RmsDims),
                ("ssm_swa_fwd", 6, SwaDims), ("ssm_swa_bwd", 10, SwaDims), ("ssm_swa_step", 7, SwaDims),
                ("ssm_swa_fill", 5, SwaDims)):
            f = getattr(L, name)
            f.argtypes = [vp] * pointers + [ctypes.POINTER(dims), vp]
            f.restype = ctypes.c_int
        for name, dims in (("ssm_glr_workspace_size", GlrDims), ("ssm_glr_bwd_workspace_size", GlrDims),
                           ("ssm_rms_add_bwd_workspace_size", RmsDims), ("ssm_swa_bwd_workspace_size", SwaDims),
                           ("ssm_swa_step_workspace_size", SwaDims)):
            f = getattr(L, name)
            f.argtypes = [ctypes.POINTER(dims), size]
            f.restype = ctypes.c_int
        L.ssm_block_last_error.argtypes = []
        L.ssm_block_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def block_last_error() -> str:
    return block_lib().ssm_block_last_error().decode()


def _check(rc: int):
    if rc:
        raise SsmError(rc, block_last_error())


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return code


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr() or None


def _stream(stream):
    """The stream's handle: the current one's of the current device, or the given one's."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
    return stream.cuda_stream or None


def _out(t, shape, dtype, like, name, stream):
    """A caller-given output, checked against what the call writes, or a new
    one, allocated on the stream the kernels will run on (the caching
    allocator reuses a freed block only for later work of that stream)."""
    if t is None:
        if stream is not None:
            with torch.cuda.stream(stream):
                return torch.empty(shape, dtype=dtype, device=like.device)
        if dtype == like.dtype and shape == like.shape and like.is_contiguous():
            return torch.empty_like(like)
        return like.new_empty(shape, dtype=dtype)
    if t.shape != shape or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on {like.device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _size(call, dims) -> int:
    n = ctypes.c_size_t(0)
    _check(call(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def glr_workspace_size(dims: GlrDims) -> int:
    return _size(block_lib().ssm_glr_workspace_size, dims)


def glr_bwd_workspace_size(dims: GlrDims) -> int:
    return _size(block_lib().ssm_glr_bwd_workspace_size, dims)


def rms_add_bwd_workspace_size(dims: RmsDims) -> int:
    return _size(block_lib().ssm_rms_add_bwd_workspace_size, dims)


def swa_bwd_workspace_size(dims: SwaDims) -> int:
    return _size(block_lib().ssm_swa_bwd_workspace_size, dims)


def swa_step_workspace_size(dims: SwaDims) -> int:
    return _size(block_lib().ssm_swa_step_workspace_size, dims)


def _scratch(dims, need: int, workspace, like, stream):
    """Give ``dims`` a workspace of ``need`` bytes: the caller's if it is large
    enough, else a new one, which the caller of this keeps until the launch."""
    if need > 0:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = _out(None, (need,), torch.uint8, like, "workspace", stream)
        dims.workspace = _ptr(workspace)
        dims.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _same(name, t, dtype, shape):
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


# ---------------------------------------------------------------------------
# Gated linear recurrence
# ---------------------------------------------------------------------------

def _glr_inputs(x, rec, inp, A, reset, lead):
    if x.dim() != lead + 1:
        raise ValueError("x must be (batch, seqlen, dim), or (batch, dim) in a step")
    if rec.dtype != x.dtype or inp.dtype != x.dtype:
        raise TypeError(f"rec and inp must have dtype {x.dtype}")
    if rec.shape != x.shape or inp.shape != x.shape:
        raise ValueError("rec and inp must have the shape of x")
    _same("A", A, _F32, x.shape[-1:])
    if reset is not None and (reset.dtype not in (torch.uint8, torch.bool) or reset.shape != x.shape[:2]):
        raise ValueError("reset must be uint8 or bool (batch, seqlen)")


def glr_fwd(x, rec, inp, A, *, h0=None, reset=None, out_dtype=None, return_h_last: bool = True,
            return_states: bool = False, y=None, h_last=None, states=None, workspace=None, stream=None):
    """Gated linear recurrence (``ssm_glr_fwd``): with r = sigmoid(rec),
    i = sigmoid(inp), a = exp(A r),

        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,   y_t = h_t

    x, rec, inp: (batch, L, dim), one dtype (float32 or bfloat16); A: (dim,)
    float32, at most 0; h0: (batch, dim) float32 (zero when None); reset:
    (batch, L) uint8 or bool, h_{t-1} counting as zero where it is set.
    Returns ``(y, h_last)``, and with ``return_states`` also the states before
    every 16th step, (batch, ceil(L / 16), dim) float32, that ``glr_bwd``
    starts from.  h_last (float32) may be h0 itself.
    """
    _glr_inputs(x, rec, inp, A, reset, 2)
    batch, L, dim = x.shape
    _same("h0", h0, _F32, (batch, dim))
    out_dt = x.dtype if out_dtype is None else out_dtype
    dims = GlrDims(batch, L, dim, _code(x.dtype), _code(out_dt))
    y = _out(y, (batch, L, dim), out_dt, x, "y", stream)
    if h_last is not None or return_h_last:
        h_last = _out(h_last, (batch, dim), _F32, x, "h_last", stream)
    if states is not None or return_states:
        states = _out(states, (batch, -(-L // GLR_STATE_STEP), dim), _F32, x, "states", stream)
    workspace = _scratch(dims, glr_workspace_size(dims), workspace, x, stream)
    _check(block_lib().ssm_glr_fwd(_ptr(x), _ptr(rec), _ptr(inp), _ptr(A), _ptr(h0), _ptr(reset), _ptr(y),
                                   _ptr(h_last), _ptr(states), ctypes.byref(dims), _stream(stream)))
    return (y, h_last, states) if return_states else (y, h_last)


def glr_bwd(x, rec, inp, A, states, dy, *, dh_last=None, reset=None, return_dh0: bool = True, out=None,
            workspace=None, stream=None):
    """Backward of ``glr_fwd`` (``ssm_glr_bwd``) from the states it saved and
    the gradients of y (x's shape and dtype) and of h_last ((batch, dim)
    float32 or None).  Returns ``(dx, drec, dinp, dA, dh0)``: the first three
    like x, dA (dim,) and dh0 (batch, dim) float32 (None without return_dh0).
    ``out``: a dict of preallocated outputs under those names.
    """
    _glr_inputs(x, rec, inp, A, reset, 2)
    batch, L, dim = x.shape
    _same("states", states, _F32, (batch, -(-L // GLR_STATE_STEP), dim))
    _same("dy", dy, x.dtype, x.shape)
    _same("dh_last", dh_last, _F32, (batch, dim))
    code = _code(x.dtype)
    dims = GlrDims(batch, L, dim, code, code)
    o = out or {}
    dx, drec, dinp = (_out(o.get(k), x.shape, x.dtype, x, k, stream) for k in ("dx", "drec", "dinp"))
    dA = _out(o.get("dA"), (dim,), _F32, x, "dA", stream)
    dh0 = _out(o.get("dh0"), (batch, dim), _F32, x, "dh0", stream) if return_dh0 else None
    workspace = _scratch(dims, glr_bwd_workspace_size(dims), workspace, x, stream)
    _check(block_lib().ssm_glr_bwd(_ptr(x), _ptr(rec), _ptr(inp), _ptr(A), _ptr(reset), _ptr(states), _ptr(dy),
                                   _ptr(dh_last), _ptr(dx), _ptr(drec), _ptr(dinp), _ptr(dA), _ptr(dh0),
                                   ctypes.byref(dims), _stream(stream)))
    return dx, drec, dinp, dA, dh0


def glr_step(x, rec, inp, A, h, *, h_out=None, out_dtype=None, y=None, stream=None):
    """One step of the recurrence (``ssm_glr_step``): x, rec, inp (batch, dim),
    h (batch, dim) float32, updated in place unless h_out is given.  Returns
    ``(y, h_out)``."""
    _glr_inputs(x, rec, inp, A, None, 1)
    batch, dim = x.shape
    _same("h", h, _F32, x.shape)
    out_dt = x.dtype if out_dtype is None else out_dtype
    dims = GlrDims(batch, 1, dim, _code(x.dtype), _code(out_dt))
    y = _out(y, x.shape, out_dt, x, "y", stream)
    h_out = h if h_out is None else _out(h_out, x.shape, _F32, x, "h_out", stream)
    _check(block_lib().ssm_glr_step(_ptr(x), _ptr(rec), _ptr(inp), _ptr(A), _ptr(h), _ptr(y), _ptr(h_out),
                                    ctypes.byref(dims), _stream(stream)))
    return y, h_out


# ---------------------------------------------------------------------------
# Residual addition with RMS norm
# ---------------------------------------------------------------------------

def _rms_dims(x, w, residual, eps, out_dt, group=0) -> RmsDims:
    if x.dim() < 1:
        raise ValueError("x must have a last axis to normalise")
    dim = x.shape[-1]
    _same("w", w, _F32, (dim,))
    _same("residual", residual, x.dtype, x.shape)
    return RmsDims(x.numel() // dim if dim else 0, dim, group, _code(x.dtype), _code(out_dt), eps)


def rms_add_fwd(x, w, residual=None, *, eps: float = 1e-5, out_dtype=None, y=None, residual_out=None, stream=None):
    """Residual addition with RMS norm (``ssm_rms_add_fwd``) over the last
    axis: s = x + residual, y = s / sqrt(mean(s^2) + eps) * w.  x, residual:
    (..., dim), one dtype; w: (dim,) float32.  Returns ``(y, s)``; s has x's
    dtype (x itself when there is no residual, a copy of it where y takes its
    place) and residual_out may be x or residual, y may be x."""
    out_dt = x.dtype if out_dtype is None else out_dtype
    dims = _rms_dims(x, w, residual, eps, out_dt)
    over = y is not None and y.data_ptr() == x.data_ptr()
    y = _out(y, x.shape, out_dt, x, "y", stream)
    if residual is not None or residual_out is not None or over:
        residual_out = _out(residual_out, x.shape, x.dtype, x, "residual_out", stream)
    _check(block_lib().ssm_rms_add_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(residual_out),
                                       ctypes.byref(dims), _stream(stream)))
    return y, x if residual_out is None else residual_out


def rms_add_q8_fwd(x, w, residual=None, *, eps: float = 1e-5, group: int = 0, q=None, scale=None, residual_out=None,
                   stream=None):
    """``rms_add_fwd`` with y in 8 bits (``ssm_rms_add_q8_fwd``): y stands for
    q * scale, q in torch.float8_e4m3fn, one float32 scale per row (group 0)
    or per ``group`` values of it (a multiple of 32).  Returns
    ``(q, scale, s)``, scale being (..., groups of a row)."""
    dims = _rms_dims(x, w, residual, eps, x.dtype, group)
    dim = x.shape[-1]
    groups = -(-dim // group) if 0 < group < dim else 1
    q = _out(q, x.shape, torch.float8_e4m3fn, x, "q", stream)
    scale = _out(scale, (*x.shape[:-1], groups), _F32, x, "scale", stream)
    if residual is not None or residual_out is not None:
        residual_out = _out(residual_out, x.shape, x.dtype, x, "residual_out", stream)
    _check(block_lib().ssm_rms_add_q8_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(q), _ptr(scale), _ptr(residual_out),
                                          ctypes.byref(dims), _stream(stream)))
    return q, scale, x if residual_out is None else residual_out


def rms_add_bwd(dy, s, w, *, dres=None, eps: float = 1e-5, return_dw: bool = True, dx=None, dw=None, workspace=None,
                stream=None):
    """Backward of ``rms_add_fwd`` (``ssm_rms_add_bwd``): dy, s (the sum the
    forward returned) and dres (the gradient arriving through s, or None)
    are (..., dim) of one dtype.  Returns ``(dx, dw)``: dx is the gradient of
    x and of residual alike, dw (dim,) float32 (None without return_dw)."""
    _same("dy", dy, s.dtype, s.shape)
    dims = _rms_dims(s, w, dres, eps, s.dtype)
    dx = _out(dx, s.shape, s.dtype, s, "dx", stream)
    if dw is not None or return_dw:
        dw = _out(dw, w.shape, _F32, s, "dw", stream)
        workspace = _scratch(dims, rms_add_bwd_workspace_size(dims), workspace, s, stream)
    _check(block_lib().ssm_rms_add_bwd(_ptr(dy), _ptr(s), _ptr(w), _ptr(dres), _ptr(dx), _ptr(dw),
                                       ctypes.byref(dims), _stream(stream)))
    return dx, dw


# ---------------------------------------------------------------------------
# Sliding-window attention with sinks
# ---------------------------------------------------------------------------

def _heads(name, t, lead, headdim) -> tuple:
    """Batch and token stride of a (batch[, seqlen], heads, headdim) tensor whose heads are adjacent."""
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    strides = t.stride()
    if (headdim > 1 and strides[-1] != 1) or (t.shape[-2] > 1 and strides[-2] != headdim):
        raise ValueError(f"{name}: the heads of a token must be adjacent (only batch and token strides are free)")
    # An axis of one element may carry any stride: it is never stepped over.
    batch = strides[0] if t.shape[0] > 1 else 0
    return batch, strides[1] if lead == 2 and t.shape[1] > 1 else 0


def _swa_dims(q, k, v, window, sinks, scale, lead) -> SwaDims:
    if q.dtype != _BF16 or k.dtype != _BF16 or v.dtype != _BF16:
        raise TypeError("q, k and v must be bfloat16")
    if q.dim() != lead + 2 or k.dim() != lead + 2 or k.shape != v.shape:
        raise ValueError("q, k and v must be (batch, seqlen, heads, headdim), or (batch, heads, headdim) in a step")
    if k.shape[:lead] != q.shape[:lead] or k.shape[-1] != q.shape[-1]:
        raise ValueError("k and v must have q's batch, seqlen and headdim")
    d = q.shape[-1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if lead == 1 and q.is_contiguous() and k.is_contiguous() and v.is_contiguous():  # a step's usual call, in less time
        if not (q.is_cuda and k.is_cuda and v.is_cuda):
            raise ValueError("tensors must be on the GPU")
        H, KV = q.shape[1], k.shape[1]
        return SwaDims(q.shape[0], 1, H, KV, d, window, sinks, H * d, 0, KV * d, 0, KV * d, 0, scale)
    return SwaDims(q.shape[0], q.shape[1] if lead == 2 else 1, q.shape[-2], k.shape[-2], d, window, sinks,
                   *_heads("q", q, lead, d), *_heads("k", k, lead, d), *_heads("v", v, lead, d), scale)


def _at(t):
    return t.data_ptr() or None


def swa_fwd(q, k, v, *, window: int, sinks: int = 0, scale=None, lengths=None, return_lse: bool = True, y=None,
            lse=None, stream=None):
    """Sliding-window attention with sinks (``ssm_swa_fwd``): query t sees key
    j when j <= t and (t - j < window or j < sinks), both below the row's
    length.  q: (batch, L, nheads, headdim); k, v: (batch, L, nkv, headdim),
    bfloat16, nkv dividing nheads, headdim 64 or 128; views with any batch and
    token strides that are multiples of 8 (the parts of one fused projection)
    are taken as they are.  lengths: (batch,) int32 or None; rows of q, k and
    v past a length may hold anything and give zeros.  scale defaults to
    headdim ** -0.5.  Returns ``(y, lse)``, lse (batch, nheads, L) float32
    (None without return_lse)."""
    dims = _swa_dims(q, k, v, window, sinks, scale, 2)
    batch, L, H, _ = q.shape
    _same("lengths", lengths, torch.int32, (batch,))
    y = _out(y, q.shape, _BF16, q, "y", stream)
    if lse is not None or return_lse:
        lse = _out(lse, (batch, H, L), _F32, q, "lse", stream)
    _check(block_lib().ssm_swa_fwd(_at(q), _at(k), _at(v), _ptr(lengths), _ptr(y), _ptr(lse), ctypes.byref(dims),
                                   _stream(stream)))
    return y, lse


def swa_bwd(q, k, v, y, lse, dy, *, window: int, sinks: int = 0, scale=None, lengths=None, out=None, workspace=None,
            stream=None):
    """Backward of ``swa_fwd`` (``ssm_swa_bwd``) from its y and lse and the
    gradient of y.  Returns ``(dq, dk, dv)``, dense, shaped like q, k and v.
    ``out``: a dict of preallocated outputs under those names."""
    dims = _swa_dims(q, k, v, window, sinks, scale, 2)
    batch, L, H, _ = q.shape
    _same("lengths", lengths, torch.int32, (batch,))
    _same("y", y, _BF16, q.shape)
    _same("dy", dy, _BF16, q.shape)
    _same("lse", lse, _F32, (batch, H, L))
    o = out or {}
    dq, dk, dv = (_out(o.get(n), t.shape, _BF16, q, n, stream) for n, t in (("dq", q), ("dk", k), ("dv", v)))
    workspace = _scratch(dims, swa_bwd_workspace_size(dims), workspace, q, stream)
    _check(block_lib().ssm_swa_bwd(_at(q), _at(k), _at(v), _ptr(lengths), _ptr(y), _ptr(lse), _ptr(dy), _ptr(dq),
                                   _ptr(dk), _ptr(dv), ctypes.byref(dims), _stream(stream)))
    return dq, dk, dv


def _swa_caches(k_cache, v_cache, batch, nkv, headdim, sinks) -> int:
    """The window of a pair of caches (batch, nkv, sinks + window, headdim)."""
    if k_cache.dim() != 4 or k_cache.shape[:2] != (batch, nkv) or k_cache.shape[3] != headdim:
        raise ValueError("the caches must be (batch, nkv, sinks + window, headdim)")
    if k_cache.dtype != _BF16 or v_cache.dtype != _BF16 or v_cache.shape != k_cache.shape:
        raise ValueError("the caches must be bfloat16 and of one shape")
    return k_cache.shape[2] - sinks


def swa_step(q, k, v, k_cache, v_cache, pos, *, sinks: int = 0, scale=None, y=None, workspace=None, stream=None):
    """One token per batch row (``ssm_swa_step``) against caches of
    (batch, nkv, sinks + window, headdim), which take the token's k and v in
    place.  q: (batch, nheads, headdim); k, v: (batch, nkv, headdim); pos:
    (batch,) int32, the token's position, negative for a row without a token.
    Returns y."""
    dims = _swa_dims(q, k, v, 1, sinks, scale, 1)
    dims.window = _swa_caches(k_cache, v_cache, k.shape[0], k.shape[1], k.shape[2], sinks)
    _same("pos", pos, torch.int32, (q.shape[0],))
    y = _out(y, q.shape, _BF16, q, "y", stream)
    workspace = _scratch(dims, swa_step_workspace_size(dims), workspace, q, stream)
    _check(block_lib().ssm_swa_step(_at(q), _at(k), _at(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos), _ptr(y),
                                    ctypes.byref(dims), _stream(stream)))
    return y


def swa_fill(k, v, k_cache, v_cache, *, sinks: int = 0, lengths=None, stream=None):
    """Store a prompt's keys and values ((batch, L, nkv, headdim)) into the
    caches that ``swa_step`` goes on from (``ssm_swa_fill``): the first
    ``sinks`` positions and the last ``window`` others below each length."""
    dims = _swa_dims(k, k, v, 1, sinks, 1.0, 2)
    dims.window = _swa_caches(k_cache, v_cache, k.shape[0], k.shape[2], k.shape[3], sinks)
    _same("lengths", lengths, torch.int32, (k.shape[0],))
    _check(block_lib().ssm_swa_fill(_at(k), _at(v), _ptr(lengths), _ptr(k_cache), _ptr(v_cache), ctypes.byref(dims),
                                    _stream(stream)))
