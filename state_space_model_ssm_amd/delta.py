"""Python binding of libssm_delta (include/ssm_delta.h): gated delta rule, norms
of queries and keys with the rotation by position, and attention steps over a
cache held in 8 bits on MI355X.

Argument marshalling only, as for libssm_block: PyTorch supplies device memory
and the current HIP stream; if ``libssm_delta.so`` is missing the calls raise.
The names are also available from the package itself:

    import state_space_model_ssm_amd as ssm
    y, h_last = ssm.gdr_fwd(q, k, v, g, beta)
    q, k = ssm.qk_norm_fwd(q, k, wq, wk, inv_freq=inv_freq, pos=pos)
    cache = ssm.swa_q8_cache(batch, nkv, window, headdim, sinks=4, device="cuda")
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from . import _DELTA, SsmError
from .block import SwaDims, _BF16, _F32, _code, _heads, _out, _ptr, _same, _stream, _swa_dims

__all__ = list(_DELTA)

GDR_STATE_STEP = 64   # tokens that the delta rule takes at a time
SWA_Q8_BLOCK = 64     # positions that share a scale in an 8-bit cache
_E4M3 = torch.float8_e4m3fn

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssm_delta.so")
_lib = None


class GdrDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nqk", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("kdim", ctypes.c_int64), ("vdim", ctypes.c_int64),
                ("q_batch", ctypes.c_int64), ("q_token", ctypes.c_int64), ("k_batch", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("v_batch", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("scale", ctypes.c_float), ("gate_dtype", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class QkNormDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("nkv", ctypes.c_int64), ("headdim", ctypes.c_int64), ("rot", ctypes.c_int64),
                ("q_batch", ctypes.c_int64), ("q_token", ctypes.c_int64), ("k_batch", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("oq_batch", ctypes.c_int64), ("oq_token", ctypes.c_int64),
                ("ok_batch", ctypes.c_int64), ("ok_token", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("neighbours", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class SwaQ8Cache(NamedTuple):
    """An 8-bit ring cache of keys and values (see ``ssm_swa_q8_step``)."""
    k_near: torch.Tensor    # (batch, nkv, sinks + 64, headdim) bfloat16: sinks, and the block that is being filled
    v_near: torch.Tensor
    k_ring: torch.Tensor    # (batch, nkv, window, headdim) float8_e4m3fn: whole blocks
    v_ring: torch.Tensor
    k_scale: torch.Tensor   # (batch, nkv, window / 64) float32
    v_scale: torch.Tensor


def delta_library_path() -> str:
    return _LIB_PATH


def delta_lib():
    """The loaded libssm_delta (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m state_space_model_ssm_amd.build` "
                "(hipcc, gfx950). There is no fallback implementation.")
        L = ctypes.CDLL(_LIB_PATH)
        vp, size = ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
        for name, pointers, dims in (("ssm_gdr_fwd", 10, GdrDims), ("ssm_gdr_bwd", 12, GdrDims), ("ssm_gdr_step", 8, GdrDims),
                                     ("ssm_qk_norm_fwd", 8, QkNormDims), ("ssm_qk_norm_bwd", 12, QkNormDims),
                                     ("ssm_swa_q8_step", 11, SwaDims), ("ssm_swa_q8_fill", 9, SwaDims)):
            f = getattr(L, name)
            f.argtypes = [vp] * pointers + [ctypes.POINTER(dims), vp]
            f.restype = ctypes.c_int
        for name, dims in (("ssm_gdr_workspace_size", GdrDims), ("ssm_gdr_states_size", GdrDims),
                           ("ssm_gdr_bwd_workspace_size", GdrDims),
                           ("ssm_qk_norm_bwd_workspace_size", QkNormDims), ("ssm_swa_q8_step_workspace_size", SwaDims)):
            f = getattr(L, name)
            f.argtypes = [ctypes.POINTER(dims), size]
            f.restype = ctypes.c_int
        L.ssm_delta_last_error.argtypes = []
        L.ssm_delta_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def delta_last_error() -> str:
    return delta_lib().ssm_delta_last_error().decode()


def _check(rc: int):
    if rc:
        raise SsmError(rc, delta_last_error())


def _size(call, dims) -> int:
    n = ctypes.c_size_t(0)
    _check(call(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def gdr_workspace_size(dims: GdrDims) -> int:
    return _size(delta_lib().ssm_gdr_workspace_size, dims)


def gdr_states_size(dims: GdrDims) -> int:
    return _size(delta_lib().ssm_gdr_states_size, dims)


def gdr_bwd_workspace_size(dims: GdrDims) -> int:
    return _size(delta_lib().ssm_gdr_bwd_workspace_size, dims)


def qk_norm_bwd_workspace_size(dims: QkNormDims) -> int:
    return _size(delta_lib().ssm_qk_norm_bwd_workspace_size, dims)


def swa_q8_step_workspace_size(dims: SwaDims) -> int:
    return _size(delta_lib().ssm_swa_q8_step_workspace_size, dims)


def _scratch(dims, need: int, workspace, like, stream):
    """Give ``dims`` a workspace of ``need`` bytes: the caller's if it is large
    enough, else a new one, which the caller of this keeps until the launch."""
    if need > 0:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = _out(None, (need,), torch.uint8, like, "workspace", stream)
        dims.workspace = _ptr(workspace)
        dims.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _one_device(stream, first, *others):
    """All tensors on the current device, where the call launches, and the stream if one is given."""
    at = first.get_device()   # -1 on the CPU
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors must be on one device, got {t.device} and {first.device}")
    if at < 0:
        raise ValueError("tensors must be on the GPU")
    here = torch._C._cuda_getDevice()
    if at != here or (stream is not None and stream.device_index != here):
        raise ValueError(f"tensors are on cuda:{at}, the current device is cuda:{here}"
                         + ("" if stream is None else f", the stream's cuda:{stream.device_index}"))


_DENSE = torch.contiguous_format


def _like(t, like, name, stream):
    """A caller-given output, or a new dense one, of ``like``'s shape and type."""
    if t is None and stream is None:
        return torch.empty_like(like, memory_format=_DENSE)
    return _out(t, like.shape, like.dtype, like, name, stream)


def _at(t):
    return t.data_ptr() or None


# ---------------------------------------------------------------------------
# Gated delta rule
# ---------------------------------------------------------------------------

def _gdr_dims(q, k, v, g, beta, scale, lead) -> GdrDims:
    if q.dtype != _BF16 or k.dtype != _BF16 or v.dtype != _BF16:
        raise TypeError("q, k and v must be bfloat16")
    qs, vs = q.shape, v.shape
    if len(qs) != lead + 2 or qs != k.shape or len(vs) != lead + 2 or vs[:lead] != qs[:lead]:
        raise ValueError("q and k must be (batch, seqlen, nqk, kdim) and v (batch, seqlen, nheads, vdim), "
                         "without seqlen in a step")
    gates, gs = g.dtype, vs[:-1]
    _same("g", g, gates, gs)
    _same("beta", beta, gates, gs)
    kd, vd = qs[-1], vs[-1]
    return GdrDims(qs[0], qs[1] if lead == 2 else 1, qs[-2], vs[-2], kd, vd, *_heads("q", q, lead, kd),
                   *_heads("k", k, lead, kd), *_heads("v", v, lead, vd), kd ** -0.5 if scale is None else scale, _code(gates))


def gdr_fwd(q, k, v, g, beta, *, h0=None, lengths=None, scale=None, return_h_last: bool = True,
            return_states: bool = False, y=None, h_last=None, states=None, workspace=None, stream=None):
    """Gated delta rule (``ssm_gdr_fwd``): per value head, with the state S
    (vdim x kdim) and a = exp(g),

        u_t = beta_t (v_t - a_t S_{t-1} k_t),  S_t = a_t S_{t-1} + u_t k_t^T,  y_t = scale S_t q_t

    q, k: (batch, L, nqk, kdim) and v: (batch, L, nheads, vdim), bfloat16, nqk
    dividing nheads, kdim and vdim 64 or 128, as views with any batch and
    token strides that are multiples of 8; g (at most 0) and beta: (batch, L,
    nheads), float32 or bfloat16.  Keys are meant to have unit length.  h0:
    (batch, nheads, vdim, kdim) float32 (zero when None); lengths: (batch,)
    int32 or None; rows past a length may hold anything and give zeros.  scale
    defaults to kdim ** -0.5.  Returns ``(y, h_last)``, and with
    ``return_states`` also what ``gdr_bwd`` starts from, a uint8 tensor of
    ``gdr_states_size`` bytes (per value head and 64 tokens 4 vdim (kdim + 64)
    + 26624: the state before them and what is needed of v, g and beta).  h_last
    (float32, after each row's last token) may be h0 itself; without it
    (return_h_last False) the call takes less time, and y's last bits may differ.
    """
    _one_device(stream, q, k, v, g, beta, h0, lengths, workspace)
    dims = _gdr_dims(q, k, v, g, beta, scale, 2)
    batch, L, H, vd = v.shape
    state = (batch, H, vd, q.shape[-1])
    _same("h0", h0, _F32, state)
    _same("lengths", lengths, torch.int32, (batch,))
    y = _like(y, v, "y", stream)
    if h_last is not None or return_h_last:
        h_last = _out(h_last, state, _F32, q, "h_last", stream)
    if states is not None or return_states:
        states = _out(states, (gdr_states_size(dims),), torch.uint8, q, "states", stream)
    workspace = _scratch(dims, gdr_workspace_size(dims), workspace, q, stream)
    _check(delta_lib().ssm_gdr_fwd(_at(q), _at(k), _at(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(lengths), _ptr(y),
                                   _ptr(h_last), _ptr(states), ctypes.byref(dims), _stream(stream)))
    return (y, h_last, states) if return_states else (y, h_last)


def gdr_bwd(q, k, v, g, beta, states, dy, *, dh_last=None, lengths=None, scale=None, return_dh0: bool = True, out=None,
            workspace=None, stream=None):
    """Backward of ``gdr_fwd`` (``ssm_gdr_bwd``) from what it saved and
    the gradients of y (v's shape, bfloat16) and of h_last ((batch, nheads,
    vdim, kdim) float32 or None); of v, g and beta it takes the shapes and
    types, their values being in what was saved.  Returns ``(dq, dk, dv, dg, dbeta, dh0)``:
    dense, shaped and typed like q, k, v, g and beta; dh0 float32 (None without
    return_dh0).  ``out``: a dict of preallocated outputs under those names.
    """
    _one_device(stream, q, k, v, g, beta, states, dy, dh_last, lengths, workspace)
    dims = _gdr_dims(q, k, v, g, beta, scale, 2)
    batch, L, H, vd = v.shape
    state = (batch, H, vd, q.shape[-1])
    _same("states", states, torch.uint8, (gdr_states_size(dims),))
    _same("dy", dy, _BF16, v.shape)
    _same("dh_last", dh_last, _F32, state)
    _same("lengths", lengths, torch.int32, (batch,))
    o = out or {}
    dq, dk, dv, dg, dbeta = (_like(o.get(n), t, n, stream)
                             for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)))
    dh0 = _out(o.get("dh0"), state, _F32, q, "dh0", stream) if return_dh0 else None
    workspace = _scratch(dims, gdr_bwd_workspace_size(dims), workspace, q, stream)
    _check(delta_lib().ssm_gdr_bwd(_at(q), _at(k), _ptr(lengths), _ptr(states), _ptr(dy), _ptr(dh_last), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0),
                                   ctypes.byref(dims), _stream(stream)))
    return dq, dk, dv, dg, dbeta, dh0


def gdr_step(q, k, v, g, beta, h, *, scale=None, h_out=None, y=None, stream=None):
    """One token of the delta rule (``ssm_gdr_step``): q, k (batch, nqk, kdim),
    v (batch, nheads, vdim), g, beta (batch, nheads), h (batch, nheads, vdim,
    kdim) float32, updated in place unless h_out is given.  Returns
    ``(y, h_out)``."""
    _one_device(stream, q, k, v, g, beta, h)
    dims = _gdr_dims(q, k, v, g, beta, scale, 1)
    _same("h", h, _F32, (*v.shape, q.shape[-1]))
    y = _like(y, v, "y", stream)
    h_out = h if h_out is None else _out(h_out, h.shape, _F32, q, "h_out", stream)
    _check(delta_lib().ssm_gdr_step(_at(q), _at(k), _at(v), _ptr(g), _ptr(beta), _ptr(h), _ptr(y), _ptr(h_out),
                                    ctypes.byref(dims), _stream(stream)))
    return y, h_out


# ---------------------------------------------------------------------------
# Norms of queries and keys with the rotation by position
# ---------------------------------------------------------------------------

def _rows(name, t, given, lead, d) -> tuple:
    """Batch and token stride of an output, which is dense if it is new."""
    if given:
        return _heads(name, t, lead, d)
    token = t.shape[-2] * d
    return (token, 0) if lead == 1 else (max(t.shape[1], 1) * token, token)


def _qk_norm_dims(q, k, wq, wk, inv_freq, pos, eps, neighbours, out_q, out_k, given_q, given_k) -> QkNormDims:
    qs, ks = q.shape, k.shape
    lead = len(qs) - 2
    if lead not in (1, 2) or len(ks) != lead + 2 or ks[:lead] != qs[:lead] or ks[-1] != qs[-1]:
        raise ValueError("q and k must be (batch, seqlen, heads, headdim), or (batch, heads, headdim) in a step, "
                         "of one batch, seqlen and headdim")
    dtype, d = q.dtype, qs[-1]
    if k.dtype != dtype:
        raise TypeError(f"k must have dtype {dtype}")
    _same("wq", wq, _F32, (d,))
    _same("wk", wk, _F32, (d,))
    rot = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be (pairs,)")
        _same("inv_freq", inv_freq, _F32, inv_freq.shape)
        rot = 2 * inv_freq.shape[0]
        if pos is None and lead == 1:
            raise ValueError("pos is required in a step")
    _same("pos", pos, torch.int32, qs[:lead])
    return QkNormDims(qs[0], qs[1] if lead == 2 else 1, qs[-2], ks[-2], d, rot, *_heads("q", q, lead, d),
                      *_heads("k", k, lead, d), *_rows("q's output", out_q, given_q, lead, d),
                      *_rows("k's output", out_k, given_k, lead, d), _code(dtype), int(neighbours), eps)


def qk_norm_fwd(q, k, wq=None, wk=None, *, inv_freq=None, pos=None, eps: float = 1e-6, neighbours: bool = False,
                q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q and of k with the rotation by position
    (``ssm_qk_norm_fwd``): n = x / sqrt(mean(x^2) + eps) * w, whose pairs i are
    then rotated by pos * inv_freq[i].  q: (batch, L, nheads, headdim); k:
    (batch, L, nkv, headdim), or both without L in a step; float32 or bfloat16,
    headdim a multiple of 16 up to 256, views with any batch and token strides
    that are multiples of 16 bytes.  wq, wk: (headdim,) float32 (ones when
    None; filled with headdim ** -0.5 they give heads of unit length).
    inv_freq: (pairs,) float32, 2 * pairs <= headdim elements of a head being
    rotated, in pairs (i, i + pairs) or, with ``neighbours``, (2 i, 2 i + 1);
    None for no rotation.  pos: (batch, L) int32 (0, 1, .. when None), (batch,)
    in a step.  Returns ``(q_out, k_out)``, dense, or where q_out and k_out (q
    and k themselves, or other views) are given."""
    _one_device(stream, q, k, wq, wk, inv_freq, pos)
    given_q, given_k = q_out is not None, k_out is not None
    q_out, k_out = _like(q_out, q, "q_out", stream), _like(k_out, k, "k_out", stream)
    dims = _qk_norm_dims(q, k, wq, wk, inv_freq, pos, eps, neighbours, q_out, k_out, given_q, given_k)
    _check(delta_lib().ssm_qk_norm_fwd(_at(q), _at(k), _ptr(wq), _ptr(wk), _ptr(inv_freq), _ptr(pos), _at(q_out),
                                       _at(k_out), ctypes.byref(dims), _stream(stream)))
    return q_out, k_out


def qk_norm_bwd(q, k, wq, wk, dq_out, dk_out, *, inv_freq=None, pos=None, eps: float = 1e-6, neighbours: bool = False,
                return_dw: bool = True, out=None, workspace=None, stream=None):
    """Backward of ``qk_norm_fwd`` (``ssm_qk_norm_bwd``) from its inputs and
    the gradients of its outputs (dense).  Returns ``(dq, dk, dwq, dwk)``: dq
    and dk shaped like q and k, dwq and dwk (headdim,) float32 (None without
    return_dw).  ``out``: a dict of preallocated outputs under those names, dq
    and dk with any strides that q and k may have."""
    _one_device(stream, q, k, wq, wk, inv_freq, pos, dq_out, dk_out, workspace)
    _same("dq_out", dq_out, q.dtype, q.shape)
    _same("dk_out", dk_out, q.dtype, k.shape)
    o = out or {}
    dq, dk = _like(o.get("dq"), q, "dq", stream), _like(o.get("dk"), k, "dk", stream)
    dims = _qk_norm_dims(q, k, wq, wk, inv_freq, pos, eps, neighbours, dq, dk, "dq" in o, "dk" in o)
    dwq = dwk = None
    if return_dw or "dwq" in o or "dwk" in o:
        dwq, dwk = (_out(o.get(n), q.shape[-1:], _F32, q, n, stream) for n in ("dwq", "dwk"))
        workspace = _scratch(dims, qk_norm_bwd_workspace_size(dims), workspace, q, stream)
    _check(delta_lib().ssm_qk_norm_bwd(_at(q), _at(k), _ptr(wq), _ptr(wk), _ptr(inv_freq), _ptr(pos), _ptr(dq_out),
                                       _ptr(dk_out), _at(dq), _at(dk), _ptr(dwq), _ptr(dwk), ctypes.byref(dims),
                                       _stream(stream)))
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------
# Sliding-window attention over a cache in 8 bits
# ---------------------------------------------------------------------------

def swa_q8_cache(batch: int, nkv: int, window: int, headdim: int, *, sinks: int = 0, device="cuda") -> SwaQ8Cache:
    """A new, empty cache for ``swa_q8_step`` and ``swa_q8_fill``; window must be a multiple of 64."""
    if window < SWA_Q8_BLOCK or window % SWA_Q8_BLOCK:
        raise ValueError(f"window must be a multiple of {SWA_Q8_BLOCK}, got {window}")
    shapes = ((sinks + SWA_Q8_BLOCK, headdim), _BF16), ((window, headdim), _E4M3), ((window // SWA_Q8_BLOCK,), _F32)
    return SwaQ8Cache(*(torch.empty(batch, nkv, *shape, dtype=dt, device=device) for shape, dt in shapes for _ in "kv"))


def _q8_cache(cache, batch, nkv, headdim, sinks) -> int:
    """The window of a cache, whose tensors are checked."""
    near_k, near_v, ring_k, ring_v, scale_k, scale_v = cache
    window = ring_k.shape[2] if ring_k.dim() == 4 else 0
    if window % SWA_Q8_BLOCK:
        raise ValueError(f"the cache's window must be a multiple of {SWA_Q8_BLOCK}, got {window}")
    near, ring = (batch, nkv, sinks + SWA_Q8_BLOCK, headdim), (batch, nkv, window, headdim)
    scale = (batch, nkv, window // SWA_Q8_BLOCK)
    if not (near_k.shape == near == near_v.shape and ring_k.shape == ring == ring_v.shape
            and scale_k.shape == scale == scale_v.shape and near_k.dtype is _BF16 is near_v.dtype
            and ring_k.dtype is _E4M3 is ring_v.dtype and scale_k.dtype is _F32 is scale_v.dtype):
        for name, t, dtype, shape in zip(SwaQ8Cache._fields, cache, (_BF16, _BF16, _E4M3, _E4M3, _F32, _F32),
                                         (near, near, ring, ring, scale, scale)):
            _same(name, t, dtype, shape)
    return window


def swa_q8_step(q, k, v, cache: SwaQ8Cache, pos, *, sinks: int = 0, scale=None, y=None, workspace=None, stream=None):
    """One token per batch row, as ``swa_step``, against an 8-bit cache
    (``ssm_swa_q8_step``), which takes the token's k and v in place.  q:
    (batch, nheads, headdim); k, v: (batch, nkv, headdim), bfloat16; pos:
    (batch,) int32, the token's position, negative for a row without a token.
    Returns y."""
    _one_device(stream, q, k, v, *cache, pos, workspace)
    dims = _swa_dims(q, k, v, 1, sinks, scale, 1)
    dims.window = _q8_cache(cache, k.shape[0], k.shape[1], k.shape[2], sinks)
    _same("pos", pos, torch.int32, (q.shape[0],))
    y = _like(y, q, "y", stream)
    workspace = _scratch(dims, swa_q8_step_workspace_size(dims), workspace, q, stream)
    _check(delta_lib().ssm_swa_q8_step(_at(q), _at(k), _at(v), *map(_ptr, cache), _ptr(pos), _ptr(y), ctypes.byref(dims),
                                       _stream(stream)))
    return y


def swa_q8_fill(k, v, cache: SwaQ8Cache, *, sinks: int = 0, lengths=None, stream=None):
    """Store a prompt's keys and values ((batch, L, nkv, headdim)) into the
    cache that ``swa_q8_step`` goes on from (``ssm_swa_q8_fill``): what a next
    token sees of the positions below each length."""
    _one_device(stream, k, v, *cache, lengths)
    dims = _swa_dims(k, k, v, 1, sinks, 1.0, 2)
    dims.window = _q8_cache(cache, k.shape[0], k.shape[2], k.shape[3], sinks)
    _same("lengths", lengths, torch.int32, (k.shape[0],))
    _check(delta_lib().ssm_swa_q8_fill(_at(k), _at(v), _ptr(lengths), *map(_ptr, cache), ctypes.byref(dims),
                                       _stream(stream)))
