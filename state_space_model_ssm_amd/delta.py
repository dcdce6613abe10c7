"""Python binding of libssm_delta (include/ssm_delta.h): gated delta rule, norms
of queries and keys with the rotation by position, and attention steps over a
cache held in 8 bits on MI355X.

Argument marshalling only, as for libssm_block: PyTorch supplies device memory
and the current HIP stream; if ``libssm_delta.so`` is missing the calls raise.
The names are also available from the package itself:

    import state_space_model_ssm_amd as ssm
    y, h_last = ssm.gdr_fwd(q, k, v, g, beta)
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _DELTA, SsmError
from .block import _BF16, _F32, _code, _heads, _out, _ptr, _same, _stream

__all__ = list(_DELTA)

GDR_STATE_STEP = 64   # steps between two saved states of the delta rule

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssm_delta.so")
_lib = None


class GdrDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nqk", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("kdim", ctypes.c_int64), ("vdim", ctypes.c_int64),
                ("q_batch", ctypes.c_int64), ("q_token", ctypes.c_int64), ("k_batch", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("v_batch", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("scale", ctypes.c_float), ("gate_dtype", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


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
        for name, pointers, dims in (("ssm_gdr_fwd", 10, GdrDims), ("ssm_gdr_bwd", 15, GdrDims), ("ssm_gdr_step", 8, GdrDims)):
            f = getattr(L, name)
            f.argtypes = [vp] * pointers + [ctypes.POINTER(dims), vp]
            f.restype = ctypes.c_int
        for name, dims in (("ssm_gdr_workspace_size", GdrDims), ("ssm_gdr_bwd_workspace_size", GdrDims)):
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


def gdr_bwd_workspace_size(dims: GdrDims) -> int:
    return _size(delta_lib().ssm_gdr_bwd_workspace_size, dims)


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
    """All tensors on the device whose stream the call goes to."""
    at = first.device
    for t in others:
        if t is not None and t.device != at:
            raise ValueError(f"tensors must be on one device, got {t.device} and {at}")
    if at.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    here = torch._C._cuda_getDevice() if stream is None else stream.device_index
    if at.index != here:
        raise ValueError(f"tensors are on {at}, the stream on cuda:{here}")


def _at(t):
    return t.data_ptr() or None


# ---------------------------------------------------------------------------
# Gated delta rule
# ---------------------------------------------------------------------------

def _gdr_dims(q, k, v, g, beta, scale, lead) -> GdrDims:
    if q.dtype != _BF16 or k.dtype != _BF16 or v.dtype != _BF16:
        raise TypeError("q, k and v must be bfloat16")
    if q.dim() != lead + 2 or q.shape != k.shape or v.dim() != lead + 2 or v.shape[:lead] != q.shape[:lead]:
        raise ValueError("q and k must be (batch, seqlen, nqk, kdim) and v (batch, seqlen, nheads, vdim), "
                         "without seqlen in a step")
    _same("g", g, g.dtype, v.shape[:-1])
    _same("beta", beta, g.dtype, v.shape[:-1])
    kd = q.shape[-1]
    return GdrDims(q.shape[0], q.shape[1] if lead == 2 else 1, q.shape[-2], v.shape[-2], kd, v.shape[-1],
                   *_heads("q", q, lead, kd), *_heads("k", k, lead, kd), *_heads("v", v, lead, v.shape[-1]),
                   kd ** -0.5 if scale is None else scale, _code(g.dtype))


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
    ``return_states`` also the states before every 64th token, (batch, nheads,
    ceil(L / 64), vdim, kdim) float32, that ``gdr_bwd`` starts from.  h_last
    (float32, after each row's last token) may be h0 itself.
    """
    _one_device(stream, q, k, v, g, beta, h0, lengths, workspace)
    dims = _gdr_dims(q, k, v, g, beta, scale, 2)
    batch, L, H, vd = v.shape
    state = (batch, H, vd, q.shape[-1])
    _same("h0", h0, _F32, state)
    _same("lengths", lengths, torch.int32, (batch,))
    y = _out(y, v.shape, _BF16, q, "y", stream)
    if h_last is not None or return_h_last:
        h_last = _out(h_last, state, _F32, q, "h_last", stream)
    if states is not None or return_states:
        states = _out(states, (batch, H, -(-L // GDR_STATE_STEP), vd, q.shape[-1]), _F32, q, "states", stream)
    workspace = _scratch(dims, gdr_workspace_size(dims), workspace, q, stream)
    _check(delta_lib().ssm_gdr_fwd(_at(q), _at(k), _at(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(lengths), _ptr(y),
                                   _ptr(h_last), _ptr(states), ctypes.byref(dims), _stream(stream)))
    return (y, h_last, states) if return_states else (y, h_last)


def gdr_bwd(q, k, v, g, beta, states, dy, *, dh_last=None, lengths=None, scale=None, return_dh0: bool = True, out=None,
            workspace=None, stream=None):
    """Backward of ``gdr_fwd`` (``ssm_gdr_bwd``) from the states it saved and
    the gradients of y (v's shape, bfloat16) and of h_last ((batch, nheads,
    vdim, kdim) float32 or None).  Returns ``(dq, dk, dv, dg, dbeta, dh0)``:
    dense, shaped and typed like q, k, v, g and beta; dh0 float32 (None without
    return_dh0).  ``out``: a dict of preallocated outputs under those names.
    """
    _one_device(stream, q, k, v, g, beta, states, dy, dh_last, lengths, workspace)
    dims = _gdr_dims(q, k, v, g, beta, scale, 2)
    batch, L, H, vd = v.shape
    state = (batch, H, vd, q.shape[-1])
    _same("states", states, _F32, (batch, H, -(-L // GDR_STATE_STEP), vd, q.shape[-1]))
    _same("dy", dy, _BF16, v.shape)
    _same("dh_last", dh_last, _F32, state)
    _same("lengths", lengths, torch.int32, (batch,))
    o = out or {}
    dq, dk, dv, dg, dbeta = (_out(o.get(n), t.shape, t.dtype, t, n, stream)
                             for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)))
    dh0 = _out(o.get("dh0"), state, _F32, q, "dh0", stream) if return_dh0 else None
    workspace = _scratch(dims, gdr_bwd_workspace_size(dims), workspace, q, stream)
    _check(delta_lib().ssm_gdr_bwd(_at(q), _at(k), _at(v), _ptr(g), _ptr(beta), _ptr(lengths), _ptr(states), _ptr(dy),
                                   _ptr(dh_last), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0),
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
    y = _out(y, v.shape, _BF16, q, "y", stream)
    h_out = h if h_out is None else _out(h_out, h.shape, _F32, q, "h_out", stream)
    _check(delta_lib().ssm_gdr_step(_at(q), _at(k), _at(v), _ptr(g), _ptr(beta), _ptr(h), _ptr(y), _ptr(h_out),
                                    ctypes.byref(dims), _stream(stream)))
    return y, h_out
