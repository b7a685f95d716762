"""Python binding of the C ABI in ``include/mlstm.h`` (ctypes).

Argument marshalling only: tensors are torch device tensors (torch supplies
device memory and the current stream); every step of the computation runs in
the HIP library.  There is no fallback: if ``libmlstm.so`` is missing or
fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmlstm.so")

F32, BF16 = 0, 1
VARIANTS = {"auto": 0, "fused": 1, "segscan": 2}
STATUS = {0: "MLSTM_OK", 1: "MLSTM_ERR_NULL", 2: "MLSTM_ERR_SHAPE", 3: "MLSTM_ERR_UNSUPPORTED",
          4: "MLSTM_ERR_STATE_ARGS", 5: "MLSTM_ERR_WORKSPACE", 6: "MLSTM_ERR_ALIAS",
          7: "MLSTM_ERR_HIP", 8: "MLSTM_ERR_ALIGN", 9: "MLSTM_ERR_BLAS", 10: "MLSTM_ERR_SCRATCH"}
# bytes of the fixed per-device scratch of mlstm_step_noalloc (MLSTM_STEP_NOALLOC_MAX_BYTES)
STEP_NOALLOC_MAX_BYTES = 32 << 20

# exported entry points and their C signatures (kept in step with include/mlstm.h)
_vp, _fp, _sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
_i = ctypes.c_int
SIGNATURES = {
    "mlstm_status_string": (ctypes.c_char_p, [_i]),
    "mlstm_version": (ctypes.c_char_p, []),
    "mlstm_fwd_chunkwise_workspace_size": (_i, [_i] * 7 + [ctypes.POINTER(_sz)]),
    "mlstm_fwd_chunkwise_workspace_size_variant": (_i, [_i] * 8 + [ctypes.POINTER(_sz)]),
    "mlstm_fwd_chunkwise_schedule": (_i, [_i] * 8 + [ctypes.POINTER(_i)] * 2),
    "mlstm_fwd_chunkwise": (_i, [_vp] * 13 + [_i] * 7 + [_vp, _sz, _vp]),
    "mlstm_fwd_chunkwise_variant": (_i, [_vp] * 13 + [_i] * 8 + [_vp, _sz, _vp]),
    "mlstm_step_workspace_size": (_i, [_i] * 5 + [ctypes.POINTER(_sz)]),
    "mlstm_step": (_i, [_vp] * 13 + [_i] * 5 + [_vp, _sz, _vp]),
    "mlstm_step_noalloc": (_i, [_vp] * 13 + [_i] * 5 + [_vp]),
    "mlstm_bwd_chunkwise_workspace_size": (_i, [_i] * 7 + [ctypes.POINTER(_sz)]),
    "mlstm_bwd_chunkwise": (_i, [_vp] * 19 + [_i] * 7 + [_vp, _sz, _vp]),
    "mlstm_layer_fwd_workspace_size": (_i, [_i] * 8 + [ctypes.POINTER(_sz)]),
    "mlstm_layer_fwd": (_i, [_vp] * 20 + [_i] * 8 + [_vp, _sz, _vp]),
    "mlstm_slstm_fwd": (_i, [_vp] * 11 + [_i] * 5 + [_vp]),
}
# the same for include/mlstm_ops.h
_f, _szp = ctypes.c_float, ctypes.POINTER(_sz)
OPS_SIGNATURES = {
    "mlstm_linattn_fwd_workspace_size": (_i, [_i] * 6 + [_szp]),
    "mlstm_linattn_fwd": (_i, [_vp] * 9 + [_f] + [_i] * 6 + [_vp, _sz, _vp]),
    "mlstm_linattn_step": (_i, [_vp] * 8 + [_f] + [_i] * 5 + [_vp]),
    "mlstm_linattn_bwd_workspace_size": (_i, [_i] * 6 + [_szp]),
    "mlstm_linattn_bwd": (_i, [_vp] * 13 + [_f] + [_i] * 6 + [_vp, _sz, _vp]),
    "mlstm_groupnorm_workspace_size": (_i, [_i] * 7 + [_szp]),
    "mlstm_groupnorm_fwd": (_i, [_vp] * 7 + [_i] * 6 + [_f, _i, _vp, _sz, _vp]),
    "mlstm_groupnorm_bwd": (_i, [_vp] * 10 + [_i] * 7 + [_vp, _sz, _vp]),
}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
NORM_OVER = {"token": 0, "sequence": 1}


class MlstmError(RuntimeError):
    """A non-OK status returned by the library."""

    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} "
                               "(run python -m xlstm_mlstm_matrix_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in {**SIGNATURES, **OPS_SIGNATURES}.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def status_string(s: int) -> str:
    return lib().mlstm_status_string(int(s)).decode()


def _check(s: int):
    if s != 0:
        raise MlstmError(s, status_string(s))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _io(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"I/O tensors must be float32 or bfloat16, got {t.dtype}")


def _req(t, name, dtype=None, device=None):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _stream(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def workspace_size(B, H, T, d_qk, d_v, chunk, io: int, variant: str = "auto") -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mlstm_fwd_chunkwise_workspace_size_variant(
        B, H, T, d_qk, d_v, chunk, io, VARIANTS[variant], ctypes.byref(n)))
    return n.value


def schedule(B, H, T, d_qk, d_v, chunk, io: int, variant: str = "auto"):
    """(kernel chunk length, segments per sequence) of a chunkwise call."""
    kc, ns = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().mlstm_fwd_chunkwise_schedule(B, H, T, d_qk, d_v, chunk, io, VARIANTS[variant],
                                              ctypes.byref(kc), ctypes.byref(ns)))
    return kc.value, ns.value


def fwd_chunkwise(q, k, v, i_pre, f_pre, o_pre, C0=None, n0=None, m0=None, *, chunk: int = 64,
                  return_state: bool = True, variant: str = "auto", h=None, C_T=None, n_T=None,
                  m_T=None, workspace=None):
    """Chunkwise forward over whole sequences.

    q, k [B,H,T,d_qk], v, o_pre [B,H,T,d_v] (float32 or bfloat16, one dtype);
    i_pre, f_pre [B,H,T] float32; optional (C0 [B,H,d_qk,d_v], n0 [B,H,d_qk],
    m0 [B,H]) float32.  Returns h, or (h, (C_T, n_T, m_T)) with
    ``return_state``.  Output buffers may be passed in (C_T may be C0 for an
    in-place state update)."""
    import torch
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io_t = q.dtype
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("o_pre", o_pre)):
        _req(t, name, io_t, dev)
    for name, t in (("i_pre", i_pre), ("f_pre", f_pre), ("C0", C0), ("n0", n0), ("m0", m0)):
        _req(t, name, torch.float32, dev)
    if h is None:
        h = torch.empty((B, H, T, dv), dtype=io_t, device=dev)
    if return_state and C_T is None:
        C_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
        n_T = torch.empty((B, H, dk), dtype=torch.float32, device=dev)
        m_T = torch.empty((B, H), dtype=torch.float32, device=dev)
    io = _io(q)
    nbytes = workspace_size(B, H, T, dk, dv, chunk, io, variant)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().mlstm_fwd_chunkwise_variant(
        _ptr(q), _ptr(k), _ptr(v), _ptr(i_pre), _ptr(f_pre), _ptr(o_pre),
        _ptr(C0), _ptr(n0), _ptr(m0), _ptr(h), _ptr(C_T), _ptr(n_T), _ptr(m_T),
        B, H, T, dk, dv, chunk, io, VARIANTS[variant],
        _ptr(workspace), ws_len, _stream(dev)))
    if return_state:
        return h, (C_T, n_T, m_T)
    return h


def bwd_workspace_size(B, H, T, d_qk, d_v, chunk, io: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mlstm_bwd_chunkwise_workspace_size(B, H, T, d_qk, d_v, chunk, io, ctypes.byref(n)))
    return n.value


def bwd_chunkwise(q, k, v, i_pre, f_pre, o_pre, dh, C0=None, n0=None, m0=None, *, chunk: int = 32,
                  state_grad: bool = False, workspace=None):
    """Gradients of a loss L given dL/dh, for the inputs of fwd_chunkwise.

    Same inputs as fwd_chunkwise plus dh [B,H,T,d_v] (the I/O dtype).
    Returns float32 (dq, dk, dv, di, df, do), and with ``state_grad`` also
    (dC0, dn0, dm0) -- of the zero state when no initial state is given."""
    import torch
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io_t = q.dtype
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("o_pre", o_pre), ("dh", dh)):
        _req(t, name, io_t, dev)
    for name, t in (("i_pre", i_pre), ("f_pre", f_pre), ("C0", C0), ("n0", n0), ("m0", m0)):
        _req(t, name, torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    gq, gk = torch.empty((B, H, T, dk), **f32), torch.empty((B, H, T, dk), **f32)
    gv, go = torch.empty((B, H, T, dv), **f32), torch.empty((B, H, T, dv), **f32)
    gi, gf = torch.empty((B, H, T), **f32), torch.empty((B, H, T), **f32)
    gC0 = gn0 = gm0 = None
    if state_grad:
        gC0, gn0, gm0 = (torch.empty((B, H, dk, dv), **f32), torch.empty((B, H, dk), **f32),
                         torch.empty((B, H), **f32))
    io = _io(q)
    nbytes = bwd_workspace_size(B, H, T, dk, dv, chunk, io)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws_len = workspace.numel() * workspace.element_size()
    _check(lib().mlstm_bwd_chunkwise(
        _ptr(q), _ptr(k), _ptr(v), _ptr(i_pre), _ptr(f_pre), _ptr(o_pre),
        _ptr(C0), _ptr(n0), _ptr(m0), _ptr(dh), _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gi), _ptr(gf),
        _ptr(go), _ptr(gC0), _ptr(gn0), _ptr(gm0), B, H, T, dk, dv, chunk, io,
        _ptr(workspace), ws_len, _stream(dev)))
    out = (gq, gk, gv, gi, gf, go)
    if state_grad:
        return out + (gC0, gn0, gm0)
    return out


def layer_workspace_size(B, T, d_model, H, d_qk, d_v, chunk, io: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mlstm_layer_fwd_workspace_size(B, T, d_model, H, d_qk, d_v, chunk, io, ctypes.byref(n)))
    return n.value


def layer_fwd(x, W_q, W_k, W_v, W_o, W_i, W_f, b_q, b_k, b_v, b_o, b_i, b_f, C0=None, n0=None,
              m0=None, *, chunk: int = 64, return_state: bool = True, workspace=None, norm=None):
    """The mLSTM layer forward (input projections, then the chunkwise cell).

    x [B,T,d_model]; W_q, W_k [H,d_qk,d_model]; W_v, W_o [H,d_v,d_model];
    W_i, W_f [H,d_model] (all the I/O dtype); biases float32 b_q, b_k [H,d_qk],
    b_v, b_o [H,d_v], b_i, b_f [H]; optional state C0 [H,B,d_qk,d_v], n0
    [H,B,d_qk], m0 [H,B].  Cells are head-major.  Returns h [H,B,T,d_v], or
    (h, (C_T, n_T, m_T)) with ``return_state``.

    ``norm``: a dict of groupnorm_fwd's weight and bias [H,d_v], eps and act
    (each optional) adds the norm of each head's output behind the cell; the
    result's first entry is then its token-major rows [B,T,H,d_v]."""
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io_t = x.dtype
    B, T, D = x.shape
    H, dk = W_q.shape[0], W_q.shape[1]
    dv = W_v.shape[1]
    for name, t in (("x", x), ("W_q", W_q), ("W_k", W_k), ("W_v", W_v), ("W_o", W_o), ("W_i", W_i),
                    ("W_f", W_f)):
        _req(t, name, io_t, dev)
    for name, t in (("b_q", b_q), ("b_k", b_k), ("b_v", b_v), ("b_o", b_o), ("b_i", b_i), ("b_f", b_f),
                    ("C0", C0), ("n0", n0), ("m0", m0)):
        _req(t, name, torch.float32, dev)
    h = torch.empty((H, B, T, dv), dtype=io_t, device=dev)
    C_T = n_T = m_T = None
    if return_state:
        f32 = dict(dtype=torch.float32, device=dev)
        C_T, n_T, m_T = (torch.empty((H, B, dk, dv), **f32), torch.empty((H, B, dk), **f32),
                         torch.empty((H, B), **f32))
    io = _io(x)
    if norm is not None:  # refused before anything runs
        bad = set(norm) - {"weight", "bias", "eps", "act"}
        if bad:
            raise TypeError(f"norm takes weight, bias, eps and act, not {sorted(bad)}")
        _dense(norm.get("weight"), "weight", (H, dv), torch.float32, dev)
        _dense(norm.get("bias"), "bias", (H, dv), torch.float32, dev)
        _choice(ACTIVATIONS, norm.get("act", "none"), "act")
        if not norm.get("eps", 1e-5) > 0:
            raise ValueError("eps must be positive")
    if workspace is None:
        workspace = torch.empty(layer_workspace_size(B, T, D, H, dk, dv, chunk, io), dtype=torch.uint8,
                                device=dev)
    ws_len = workspace.numel() * workspace.element_size()
    _check(lib().mlstm_layer_fwd(
        _ptr(x), _ptr(W_q), _ptr(W_k), _ptr(W_v), _ptr(W_o), _ptr(W_i), _ptr(W_f),
        _ptr(b_q), _ptr(b_k), _ptr(b_v), _ptr(b_o), _ptr(b_i), _ptr(b_f),
        _ptr(C0), _ptr(n0), _ptr(m0), _ptr(h), _ptr(C_T), _ptr(n_T), _ptr(m_T),
        B, T, D, H, dk, dv, chunk, io, _ptr(workspace), ws_len, _stream(dev)))
    if norm is not None:
        h = groupnorm_fwd(h.permute(1, 2, 0, 3), over="token", return_stats=False, **norm)
    return (h, (C_T, n_T, m_T)) if return_state else h


def slstm_fwd(gx, R, c0=None, n0=None, m0=None, h0=None, *, return_state: bool = True, h=None,
              c_T=None, n_T=None, m_T=None, h_T=None):
    """The sLSTM cell forward.

    gx [B,H,T,4,d] (input part of the z, i, f, o pre-activations) and R
    [H,4,d,d] (recurrent weights) in the I/O dtype; optional state c0, n0,
    m0, h0 [B,H,d] float32.  Returns h [B,H,T,d], or (h, (c_T, n_T, m_T,
    h_T)) with ``return_state``."""
    import torch
    dev = gx.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io_t = gx.dtype
    B, H, T, four, d = gx.shape
    if four != 4:
        raise ValueError("gx must be [B, H, T, 4, d]")
    _req(gx, "gx", io_t, dev)
    _req(R, "R", io_t, dev)
    for name, t in (("c0", c0), ("n0", n0), ("m0", m0), ("h0", h0)):
        _req(t, name, torch.float32, dev)
    if h is None:
        h = torch.empty((B, H, T, d), dtype=io_t, device=dev)
    if return_state and c_T is None:
        f32 = dict(dtype=torch.float32, device=dev)
        c_T, n_T, m_T, h_T = (torch.empty((B, H, d), **f32) for _ in range(4))
    _check(lib().mlstm_slstm_fwd(
        _ptr(gx), _ptr(R), _ptr(c0), _ptr(n0), _ptr(m0), _ptr(h0), _ptr(h),
        _ptr(c_T), _ptr(n_T), _ptr(m_T), _ptr(h_T), B, H, T, d, _io(gx), _stream(dev)))
    return (h, (c_T, n_T, m_T, h_T)) if return_state else h


def step_workspace_size(B, H, d_qk, d_v, io: int) -> int:
    """Bytes of workspace mlstm_step can use for this shape (0: none)."""
    n = ctypes.c_size_t(0)
    _check(lib().mlstm_step_workspace_size(B, H, d_qk, d_v, io, ctypes.byref(n)))
    return n.value


def step_workspace(B, H, d_qk, d_v, io_dtype, device):
    """A workspace for mlstm_step (None when the shape uses none): scratch that
    any later calls on the same stream may reuse."""
    import torch
    n = step_workspace_size(B, H, d_qk, d_v, BF16 if io_dtype == torch.bfloat16 else F32)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def step(q, k, v, i_pre, f_pre, o_pre, C=None, n=None, m=None, *, h=None, C_out=None,
         n_out=None, m_out=None, inplace: bool = True, split: bool = True, workspace=None):
    """One recurrent step for B*H cells.

    q, k [B,H,d_qk], v, o_pre [B,H,d_v]; i_pre, f_pre [B,H]; state (C [B,H,d_qk,
    d_v], n [B,H,d_qk], m [B,H]) float32 or None for the zero state.  With
    ``inplace`` (default) and a state given, the state tensors are updated in
    place.  ``split`` runs the row-split kernel where the shape has one, with
    ``workspace`` (from step_workspace; a fresh one per call when None); ``split=False`` streams each cell with one workgroup.  Returns (h,
    C_out, n_out, m_out)."""
    import torch
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io_t = q.dtype
    B, H, dk = q.shape
    dv = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("o_pre", o_pre)):
        _req(t, name, io_t, dev)
    for name, t in (("i_pre", i_pre), ("f_pre", f_pre), ("C", C), ("n", n), ("m", m)):
        _req(t, name, torch.float32, dev)
    if h is None:
        h = torch.empty((B, H, dv), dtype=io_t, device=dev)
    if C_out is None:
        if inplace and C is not None:
            C_out, n_out, m_out = C, n, m
        else:
            C_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
            n_out = torch.empty((B, H, dk), dtype=torch.float32, device=dev)
            m_out = torch.empty((B, H), dtype=torch.float32, device=dev)
    if not split:
        workspace = None
    elif workspace is None:
        workspace = step_workspace(B, H, dk, dv, io_t, dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().mlstm_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(i_pre), _ptr(f_pre), _ptr(o_pre),
        _ptr(C), _ptr(n), _ptr(m), _ptr(h), _ptr(C_out), _ptr(n_out), _ptr(m_out),
        B, H, dk, dv, _io(q), _ptr(workspace), ws_bytes, _stream(dev)))
    return h, C_out, n_out, m_out


def step_noalloc(q, k, v, i_pre, f_pre, o_pre, C=None, n=None, m=None, *, h=None, C_out=None,
                 n_out=None, m_out=None, inplace: bool = True):
    """``step`` through mlstm_step_noalloc: the row split's workspace is the
    library's fixed per-device scratch (nothing is allocated by the library;
    outputs not given are allocated here, by torch, before the call).  Same
    arguments and result as ``step`` with ``split=True``."""
    import torch
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io_t = q.dtype
    B, H, dk = q.shape
    dv = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("o_pre", o_pre)):
        _req(t, name, io_t, dev)
    for name, t in (("i_pre", i_pre), ("f_pre", f_pre), ("C", C), ("n", n), ("m", m)):
        _req(t, name, torch.float32, dev)
    if h is None:
        h = torch.empty((B, H, dv), dtype=io_t, device=dev)
    if C_out is None:
        if inplace and C is not None:
            C_out, n_out, m_out = C, n, m
        else:
            C_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
            n_out = torch.empty((B, H, dk), dtype=torch.float32, device=dev)
            m_out = torch.empty((B, H), dtype=torch.float32, device=dev)
    _check(lib().mlstm_step_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(i_pre), _ptr(f_pre), _ptr(o_pre),
        _ptr(C), _ptr(n), _ptr(m), _ptr(h), _ptr(C_out), _ptr(n_out), _ptr(m_out),
        B, H, dk, dv, _io(q), _stream(dev)))
    return h, C_out, n_out, m_out


# ---- operators of include/mlstm_ops.h

_NO_GUARD = contextlib.nullcontext()
_LONGS = {n: ctypes.c_longlong * n for n in (6, 9, 12, 21)}


def _guard(device):
    """The device as the current one (torch's guard only where it is not: a few
    microseconds, as much as a small kernel runs)."""
    import torch
    if device.index == torch.cuda.current_device():
        return _NO_GUARD
    return torch.cuda.device(device)


def _raw_stream(device) -> int:
    """torch's current stream of the device, without building a Stream object."""
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(device.index) if get is not None else _stream(device)


def _view(t, name, shape, dtype, device):
    """Check a strided tensor whose last dimension is contiguous."""
    import torch
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == device \
            and (t.stride(-1) == 1 or shape[-1] == 1):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must have a contiguous last dimension")


def _dense(t, name, shape, dtype, device):
    """Check a dense tensor (None passes)."""
    import torch
    if t is None or (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
                     and t.device == device and t.is_contiguous()):
        return
    _req(t, name, dtype, device)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _strides(*ts):
    """mlstm_strides_t array of [., ., ., d] tensors (of [., ., d] ones: s2 = 0),
    None where all are dense."""
    for t in ts:
        if not t.is_contiguous():
            break
    else:
        return None
    flat = []
    for t in ts:
        flat += t.stride()[:-1] if t.dim() == 4 else (*t.stride()[:-1], 0)
    return _LONGS[len(flat)](*flat)


def _hip_device(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    return t.device


def _workspace(workspace, nbytes, device):
    """(pointer, bytes) of a call's workspace, a fresh one when none is given.
    The tensor itself comes third: it has to live until the call is enqueued."""
    import torch
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


@functools.lru_cache(maxsize=4096)
def linattn_workspace_size(B, H, T, d_qk, d_v, io: int, backward: bool = False) -> int:
    """Bytes of workspace of linattn_fwd, or of linattn_bwd."""
    n = ctypes.c_size_t(0)
    f = lib().mlstm_linattn_bwd_workspace_size if backward else lib().mlstm_linattn_fwd_workspace_size
    _check(f(B, H, T, d_qk, d_v, io, ctypes.byref(n)))
    return n.value


def linattn_fwd(q, k, v, log_decay, S0=None, *, lengths=None, scale: float = 1.0,
                return_state: bool = True, o=None, S_T=None, workspace=None):
    """Linear attention with a decay for each head, over whole sequences:
    S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale * q_t^T S_t, g = log_decay[h].

    q, k [B,H,T,d_qk], v [B,H,T,d_v] (float32 or bfloat16, one dtype; any
    strides that are multiples of 16 bytes, e.g. views of token-major rows,
    the last dimension contiguous); log_decay [H] float32, <= 0; optional S0
    [B,H,d_qk,d_v] float32; optional lengths [B] int32 of a padded batch: rows
    behind a sequence's length are not read, come out as zeros, and do not
    touch its state.  Returns o [B,H,T,d_v], or (o, S_T) with
    ``return_state`` (a bfloat16 o may differ in its last bit without).  Output buffers may be passed in (S_T may be S0; o may
    be strided)."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, d]")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    _view(q, "q", (B, H, T, dk), q.dtype, dev)
    _view(k, "k", (B, H, T, dk), q.dtype, dev)
    _view(v, "v", (B, H, T, dv), q.dtype, dev)
    _dense(log_decay, "log_decay", (H,), torch.float32, dev)
    _dense(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    _dense(lengths, "lengths", (B,), torch.int32, dev)
    with _guard(dev):
        if o is None:
            o = torch.empty((B, H, T, dv), dtype=q.dtype, device=dev)
        if return_state and S_T is None:
            S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
        _view(o, "o", (B, H, T, dv), q.dtype, dev)
        _dense(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
        wp, wn, _keep = _workspace(workspace, linattn_workspace_size(B, H, T, dk, dv, io), dev)
        _check(lib().mlstm_linattn_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(S0), _ptr(lengths), _ptr(o), _ptr(S_T),
            _strides(q, k, v, o), scale, B, H, T, dk, dv, io, wp, wn, _raw_stream(dev)))
    return (o, S_T) if return_state else o


def linattn_step(q, k, v, log_decay, S=None, *, scale: float = 1.0, o=None, S_out=None,
                 inplace: bool = True):
    """One token of linear attention for B*H heads.

    q, k [B,H,d_qk], v [B,H,d_v] (strided as in linattn_fwd), log_decay [H],
    state S [B,H,d_qk,d_v] float32 or None for the zero state.  With
    ``inplace`` (default), a state and no ``S_out``, the state tensor is
    updated in place.  Returns (o, S_out)."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [B, H, d]")
    B, H, dk = q.shape
    dv = v.shape[-1]
    _view(q, "q", (B, H, dk), q.dtype, dev)
    _view(k, "k", (B, H, dk), q.dtype, dev)
    _view(v, "v", (B, H, dv), q.dtype, dev)
    _dense(log_decay, "log_decay", (H,), torch.float32, dev)
    _dense(S, "S", (B, H, dk, dv), torch.float32, dev)
    with _guard(dev):
        if o is None:
            o = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
        if S_out is None:
            S_out = S if inplace and S is not None else \
                torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
        _view(o, "o", (B, H, dv), q.dtype, dev)
        _dense(S_out, "S_out", (B, H, dk, dv), torch.float32, dev)
        _check(lib().mlstm_linattn_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(S), _ptr(o), _ptr(S_out),
            _strides(q, k, v, o), scale, B, H, dk, dv, io, _raw_stream(dev)))
    return o, S_out


def linattn_bwd(q, k, v, log_decay, do, S0=None, dS_T=None, *, lengths=None, scale: float = 1.0,
                state_grad: bool = False, dq=None, dk=None, dv=None, workspace=None):
    """Gradients of a loss L for the inputs of linattn_fwd, given dL/do [B,H,T,d_v]
    and, where the final state was used, dL/dS_T.

    Returns (dq, dk, dv) in the I/O dtype, each rounded once from float32 (zeros
    behind a sequence's length), and with ``state_grad`` also dS0 float32 (of
    the zero state when S0 is None).  bfloat16 gradients may differ in their last
    bit with and without ``state_grad``.  log_decay is a constant and gets none.
    Buffers for dq, dk and dv may be passed in, strided like the inputs."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, d]")
    B, H, T, d_qk = q.shape
    d_v = v.shape[-1]
    nk, nv, ns = (B, H, T, d_qk), (B, H, T, d_v), (B, H, d_qk, d_v)
    for name, t, shape in (("q", q, nk), ("k", k, nk), ("v", v, nv), ("do", do, nv)):
        _view(t, name, shape, q.dtype, dev)
    _dense(log_decay, "log_decay", (H,), torch.float32, dev)
    _dense(S0, "S0", ns, torch.float32, dev)
    _dense(dS_T, "dS_T", ns, torch.float32, dev)
    _dense(lengths, "lengths", (B,), torch.int32, dev)
    with _guard(dev):
        new = lambda t, shape: torch.empty(shape, dtype=q.dtype, device=dev) if t is None else t
        dq, dk, dv = new(dq, nk), new(dk, nk), new(dv, nv)
        for name, t, shape in (("dq", dq, nk), ("dk", dk, nk), ("dv", dv, nv)):
            _view(t, name, shape, q.dtype, dev)
        dS0 = torch.empty(ns, dtype=torch.float32, device=dev) if state_grad else None
        wp, wn, _keep = _workspace(workspace, linattn_workspace_size(B, H, T, d_qk, d_v, io, True), dev)
        _check(lib().mlstm_linattn_bwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(S0), _ptr(lengths), _ptr(do), _ptr(dS_T),
            _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dS0), _strides(q, k, v, do, dq, dk, dv), scale,
            B, H, T, d_qk, d_v, io, wp, wn, _raw_stream(dev)))
    return (dq, dk, dv, dS0) if state_grad else (dq, dk, dv)


def _choice(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {key!r}")
    return table[key]


@functools.lru_cache(maxsize=4096)
def groupnorm_workspace_size(N, S, G, D, over: str, io: int, backward: bool = False) -> int:
    """Bytes of workspace of groupnorm_fwd, or of groupnorm_bwd."""
    n = ctypes.c_size_t(0)
    _check(lib().mlstm_groupnorm_workspace_size(N, S, G, D, _choice(NORM_OVER, over, "over"), io,
                                                int(backward), ctypes.byref(n)))
    return n.value


def groupnorm_fwd(x, weight=None, bias=None, *, eps: float = 1e-5, act: str = "none",
                  over: str = "token", return_stats: bool = True, y=None, workspace=None):
    """Group norm with an activation, channels last.

    x [N,S,G,D] (float32 or bfloat16; N samples of S positions, G groups of D
    channels; any strides, the last dimension contiguous: cell outputs
    [B,H,T,d] go in as ``h.transpose(1, 2)``).  Statistics are taken over a
    group's channels at each position (``over="token"``: the norm of each
    head) or over all positions too (``over="sequence"``).  weight, bias
    [G,D] float32 or None; act "none", "silu" or "gelu".  Returns y
    [N,S,G,D] (dense unless a buffer is given), or (y, mean, rstd) with
    ``return_stats``: float32 [N,S,G] over tokens, [N,G] over sequences."""
    import torch
    dev = _hip_device(x, "x")
    io = _io(x)
    if x.dim() != 4:
        raise ValueError("x must be [N, S, G, D]")
    N, S, G, D = x.shape
    _view(x, "x", x.shape, x.dtype, dev)
    _dense(weight, "weight", (G, D), torch.float32, dev)
    _dense(bias, "bias", (G, D), torch.float32, dev)
    ov, ac = _choice(NORM_OVER, over, "over"), _choice(ACTIVATIONS, act, "act")
    with _guard(dev):
        if y is None:
            y = torch.empty((N, S, G, D), dtype=x.dtype, device=dev)
        _view(y, "y", x.shape, x.dtype, dev)
        mean = rstd = None
        if return_stats:
            shape = (N, S, G) if over == "token" else (N, G)
            mean = torch.empty(shape, dtype=torch.float32, device=dev)
            rstd = torch.empty(shape, dtype=torch.float32, device=dev)
        wp, wn, _keep = _workspace(workspace, groupnorm_workspace_size(N, S, G, D, over, io), dev)
        _check(lib().mlstm_groupnorm_fwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), _strides(x, y),
            N, S, G, D, ov, ac, eps, io, wp, wn, _raw_stream(dev)))
    return (y, mean, rstd) if return_stats else y


def groupnorm_bwd(x, dy, mean, rstd, weight=None, bias=None, *, act: str = "none", over: str = "token",
                  weight_grad: bool = True, dx=None, workspace=None):
    """Gradients of groupnorm_fwd, given dy [N,S,G,D] (strided like x) and the
    forward's mean and rstd.  Returns (dx, dweight, dbias), dx in the I/O
    dtype, the other two [G,D] float32 (None without ``weight_grad``)."""
    import torch
    dev = _hip_device(x, "x")
    io = _io(x)
    if x.dim() != 4:
        raise ValueError("x must be [N, S, G, D]")
    N, S, G, D = x.shape
    _view(x, "x", x.shape, x.dtype, dev)
    _view(dy, "dy", x.shape, x.dtype, dev)
    stat = (N, S, G) if over == "token" else (N, G)
    ov, ac = _choice(NORM_OVER, over, "over"), _choice(ACTIVATIONS, act, "act")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is None:
            raise TypeError(f"{name} must be a torch tensor")
        _dense(t, name, stat, torch.float32, dev)
    _dense(weight, "weight", (G, D), torch.float32, dev)
    _dense(bias, "bias", (G, D), torch.float32, dev)
    with _guard(dev):
        if dx is None:
            dx = torch.empty((N, S, G, D), dtype=x.dtype, device=dev)
        _view(dx, "dx", x.shape, x.dtype, dev)
        dw = db = None
        if weight_grad:
            dw = torch.empty((G, D), dtype=torch.float32, device=dev)
            db = torch.empty((G, D), dtype=torch.float32, device=dev)
        wp, wn, _keep = _workspace(workspace, groupnorm_workspace_size(N, S, G, D, over, io, True), dev)
        _check(lib().mlstm_groupnorm_bwd(
            _ptr(x), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(bias), _ptr(dx), _ptr(dw), _ptr(db),
            _strides(x, dy, dx), N, S, G, D, ov, ac, io, wp, wn, _raw_stream(dev)))
    return dx, dw, db
