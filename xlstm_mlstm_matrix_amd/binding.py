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
_f, _d, _szp = ctypes.c_float, ctypes.c_double, ctypes.POINTER(_sz)
_floats = ctypes.POINTER(_f)
OPS_SIGNATURES = {
    "mlstm_linattn_fwd_workspace_size": (_i, [_i] * 6 + [_szp]),
    "mlstm_linattn_fwd": (_i, [_vp] * 9 + [_f] + [_i] * 6 + [_vp, _sz, _vp]),
    "mlstm_linattn_step": (_i, [_vp] * 8 + [_f] + [_i] * 5 + [_vp]),
    "mlstm_linattn_bwd_workspace_size": (_i, [_i] * 6 + [_szp]),
    "mlstm_linattn_bwd": (_i, [_vp] * 13 + [_f] + [_i] * 6 + [_vp, _sz, _vp]),
    "mlstm_groupnorm_workspace_size": (_i, [_i] * 7 + [_szp]),
    "mlstm_groupnorm_fwd": (_i, [_vp] * 7 + [_i] * 6 + [_f, _i, _vp, _sz, _vp]),
    "mlstm_groupnorm_bwd": (_i, [_vp] * 10 + [_i] * 7 + [_vp, _sz, _vp]),
    "mlstm_deltarule_fwd_workspace_size": (_i, [_i] * 7 + [_szp]),
    "mlstm_deltarule_fwd": (_i, [_vp] * 10 + [_f] + [_i] * 7 + [_vp, _sz, _vp]),
    "mlstm_deltarule_step": (_i, [_vp] * 9 + [_f] + [_i] * 6 + [_vp]),
    "mlstm_deltarule_bwd_workspace_size": (_i, [_i] * 7 + [_szp]),
    "mlstm_deltarule_bwd": (_i, [_vp] * 16 + [_f] + [_i] * 7 + [_vp, _sz, _vp]),
    "mlstm_qknorm_fwd": (_i, [_vp] * 9 + [_i] * 7 + [_f, _i, _f, _i, _vp]),
    "mlstm_qknorm_bwd_workspace_size": (_i, [_i] * 5 + [_szp]),
    "mlstm_qknorm_bwd": (_i, [_vp] * 13 + [_i] * 7 + [_f, _i, _f, _i, _vp, _sz, _vp]),
    "mlstm_rope_frequencies": (_i, [_i, _d, _i, _d, _i, _d, _d, _floats, _floats]),
}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
NORM_OVER = {"token": 0, "sequence": 1}
QK_NORMS = {"none": 0, "rms": 1, "l2": 2}
ROTARY_LAYOUTS = {"half": 0, "pairs": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3}


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
_LONGS = {n: ctypes.c_longlong * n for n in (6, 9, 12, 18, 21, 33)}


def _guard(device):
    """The device as the current one (torch's guard only where it is not: a few
    microseconds, as much as a small kernel runs)."""
    import torch
    current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if device.index == current():
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


def _gate_strides(gates, *ts):
    """The same where the tensors at the places ``gates`` have a single value for each
    (b, h, t) or (b, h): all their strides count."""
    for t in ts:
        if not t.is_contiguous():
            break
    else:
        return None
    flat = []
    for i, t in enumerate(ts):
        st = t.stride() if i in gates else t.stride()[:-1]
        flat += st if len(st) == 3 else (*st, 0)
    return _LONGS[len(flat)](*flat)


def _strided(t, name, shape, dtype, device):
    """Check a tensor of any strides."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _hip_device(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError("tensors must be on a HIP device")
    return t.device


def _good(dtype, index, *pairs):
    """Whether all (tensor, shape) pass _view's and _strided's checks; the fast way
    through them, which says nothing about what is wrong."""
    try:
        for t, shape in pairs:
            if t.shape != shape or t.dtype is not dtype or t.get_device() != index or t.stride(-1) != 1:
                return False
    except AttributeError:
        return False
    return True


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


@functools.lru_cache(maxsize=4096)
def deltarule_workspace_size(B, Hk, H, T, d_qk, d_v, io: int, backward: bool = False) -> int:
    """Bytes of workspace of deltarule_fwd, or of deltarule_bwd."""
    n = ctypes.c_size_t(0)
    f = lib().mlstm_deltarule_bwd_workspace_size if backward else lib().mlstm_deltarule_fwd_workspace_size
    _check(f(B, Hk, H, T, d_qk, d_v, io, ctypes.byref(n)))
    return n.value


def deltarule_fwd(q, k, v, log_decay, beta, S0=None, *, lengths=None, scale: float = 1.0,
                  return_state: bool = True, o=None, S_T=None, workspace=None):
    """The gated delta rule over whole sequences:
    S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T, o_t = scale * q_t^T S_t.

    q, k [B,Hk,T,d_qk], v [B,H,T,d_v] (float32 or bfloat16, one dtype; strided as
    in linattn_fwd); H is a multiple of Hk, and H / Hk heads of v in a row share
    one of q and k.  log_decay (g <= 0, -inf allowed) and beta [B,H,T] float32,
    any strides; optional S0 [B,H,d_qk,d_v] float32; optional lengths [B] int32 of
    a padded batch, as in linattn_fwd.  The recurrence is stable for 0 <= beta |k|^2
    <= 2 (keys of unit length: qknorm_fwd).  Returns o [B,H,T,d_v], or (o, S_T)
    with ``return_state`` (a bfloat16 o may differ in its last bit without).
    Output buffers may be passed in (S_T may be S0; o may be strided)."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, d]")
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[-1]
    dt, nk, nv, ng, ns = q.dtype, (B, Hk, T, dk), (B, H, T, dv), (B, H, T), (B, H, dk, dv)
    if not _good(dt, dev.index, (q, nk), (k, nk), (v, nv)):
        _view(q, "q", nk, dt, dev)
        _view(k, "k", nk, dt, dev)
        _view(v, "v", nv, dt, dev)
    if not _good(torch.float32, dev.index, (log_decay, ng), (beta, ng)):
        _strided(log_decay, "log_decay", ng, torch.float32, dev)
        _strided(beta, "beta", ng, torch.float32, dev)
    _dense(S0, "S0", ns, torch.float32, dev)
    _dense(lengths, "lengths", (B,), torch.int32, dev)
    with _guard(dev):
        if o is None:
            o = torch.empty(nv, dtype=dt, device=dev)
        else:
            _view(o, "o", nv, dt, dev)
        if S_T is not None:
            _dense(S_T, "S_T", ns, torch.float32, dev)
        elif return_state:
            S_T = torch.empty(ns, dtype=torch.float32, device=dev)
        wp, wn, _keep = _workspace(workspace, deltarule_workspace_size(B, Hk, H, T, dk, dv, io), dev)
        _check(lib().mlstm_deltarule_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(beta), _ptr(S0), _ptr(lengths), _ptr(o),
            _ptr(S_T), _gate_strides((3, 4), q, k, v, log_decay, beta, o), scale, B, Hk, H, T, dk, dv, io,
            wp, wn, _raw_stream(dev)))
    return (o, S_T) if return_state else o


def deltarule_step(q, k, v, log_decay, beta, S=None, *, scale: float = 1.0, o=None, S_out=None,
                   inplace: bool = True):
    """One token of the gated delta rule for B*H heads.

    q, k [B,Hk,d_qk], v [B,H,d_v], log_decay, beta [B,H] (strided as in
    deltarule_fwd), state S [B,H,d_qk,d_v] float32 or None for the zero state.
    With ``inplace`` (default), a state and no ``S_out``, the state tensor is
    updated in place.  Returns (o, S_out)."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [B, H, d]")
    B, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[-1]
    dt, nk, nv, ng, ns = q.dtype, (B, Hk, dk), (B, H, dv), (B, H), (B, H, dk, dv)
    if not _good(dt, dev.index, (q, nk), (k, nk), (v, nv)):
        _view(q, "q", nk, dt, dev)
        _view(k, "k", nk, dt, dev)
        _view(v, "v", nv, dt, dev)
    if not _good(torch.float32, dev.index, (log_decay, ng), (beta, ng)):
        _strided(log_decay, "log_decay", ng, torch.float32, dev)
        _strided(beta, "beta", ng, torch.float32, dev)
    _dense(S, "S", ns, torch.float32, dev)
    with _guard(dev):
        if o is None:
            o = torch.empty(nv, dtype=dt, device=dev)
        else:
            _view(o, "o", nv, dt, dev)
        if S_out is not None:
            _dense(S_out, "S_out", ns, torch.float32, dev)
        elif inplace and S is not None:
            S_out = S
        else:
            S_out = torch.empty(ns, dtype=torch.float32, device=dev)
        _check(lib().mlstm_deltarule_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(beta), _ptr(S), _ptr(o), _ptr(S_out),
            _gate_strides((3, 4), q, k, v, log_decay, beta, o), scale, B, Hk, H, dk, dv, io, _raw_stream(dev)))
    return o, S_out


def deltarule_bwd(q, k, v, log_decay, beta, do, S0=None, dS_T=None, *, lengths=None, scale: float = 1.0,
                  state_grad: bool = False, dq=None, dk=None, dv=None, dlog_decay=None, dbeta=None,
                  workspace=None):
    """Gradients of a loss L for the inputs of deltarule_fwd, given dL/do [B,H,T,d_v]
    and, where the final state was used, dL/dS_T.

    Returns (dq, dk, dv, dlog_decay, dbeta): the first three in the I/O dtype, each
    rounded once (dq and dk [B,Hk,T,d_qk], summed over the heads that share them),
    the other two float32 [B,H,T]; zeros behind a sequence's length.  With
    ``state_grad`` also dS0 float32 (of the zero state when S0 is None).  Buffers
    for the first five may be passed in, strided like the inputs."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, d]")
    B, Hk, T, d_qk = q.shape
    H, d_v = v.shape[1], v.shape[-1]
    nk, nv, ng, ns = (B, Hk, T, d_qk), (B, H, T, d_v), (B, H, T), (B, H, d_qk, d_v)
    for name, t, shape in (("q", q, nk), ("k", k, nk), ("v", v, nv), ("do", do, nv)):
        _view(t, name, shape, q.dtype, dev)
    _strided(log_decay, "log_decay", ng, torch.float32, dev)
    _strided(beta, "beta", ng, torch.float32, dev)
    _dense(S0, "S0", ns, torch.float32, dev)
    _dense(dS_T, "dS_T", ns, torch.float32, dev)
    _dense(lengths, "lengths", (B,), torch.int32, dev)
    with _guard(dev):
        new = lambda t, shape, dt: torch.empty(shape, dtype=dt, device=dev) if t is None else t
        dq, dk, dv = new(dq, nk, q.dtype), new(dk, nk, q.dtype), new(dv, nv, q.dtype)
        dlog_decay, dbeta = new(dlog_decay, ng, torch.float32), new(dbeta, ng, torch.float32)
        for name, t, shape in (("dq", dq, nk), ("dk", dk, nk), ("dv", dv, nv)):
            _view(t, name, shape, q.dtype, dev)
        _strided(dlog_decay, "dlog_decay", ng, torch.float32, dev)
        _strided(dbeta, "dbeta", ng, torch.float32, dev)
        dS0 = torch.empty(ns, dtype=torch.float32, device=dev) if state_grad else None
        wp, wn, _keep = _workspace(workspace, deltarule_workspace_size(B, Hk, H, T, d_qk, d_v, io, True), dev)
        _check(lib().mlstm_deltarule_bwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(beta), _ptr(S0), _ptr(lengths), _ptr(do),
            _ptr(dS_T), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_decay), _ptr(dbeta), _ptr(dS0),
            _gate_strides((3, 4, 9, 10), q, k, v, log_decay, beta, do, dq, dk, dv, dlog_decay, dbeta), scale,
            B, Hk, H, T, d_qk, d_v, io, wp, wn, _raw_stream(dev)))
    out = (dq, dk, dv, dlog_decay, dbeta)
    return out + (dS0,) if state_grad else out


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


def rope_frequencies(n_freq: int, base: float = 10000.0, *, scaling: str = "plain", factor: float = 1.0,
                     context: int = 4096, fast: float = 32.0, slow: float = 1.0, device=None):
    """The table of rotations a position (radians, float32 [n_freq]) that qknorm_fwd
    takes as inv_freq, and the amplitude that goes with it: base^(-i / n_freq),
    scaled for contexts ``factor`` times the trained one.

    scaling "plain"; "linear" (every frequency divided by the factor); "base" (a
    larger base: the slowest divided by the factor, the fastest kept); "ramp" (those
    of ``fast`` turns or more over the trained ``context`` kept, those of ``slow`` turns or
    fewer divided, a ramp between; amplitude 0.1 ln(factor) + 1)."""
    import torch
    table, amp = (_f * max(int(n_freq), 1))(), _f()
    _check(lib().mlstm_rope_frequencies(n_freq, base, _choice(ROPE_SCALINGS, scaling, "scaling"), factor, context,
                                        fast, slow, table, ctypes.byref(amp)))
    return torch.tensor(list(table), dtype=torch.float32, device=device), amp.value


def _qk_checks(q, k, others, inv_freq, positions, weights, dev):
    """Shapes of a qknorm call: (B, H, Hk, T, d, n_freq)."""
    import torch
    B, H, T, d = q.shape
    Hk = 0 if k is None else k.shape[1]
    nq, nk = (B, H, T, d), (B, Hk, T, d)
    if k is None or not _good(q.dtype, dev.index, (q, nq), (k, nk), *((t, nq if h == H else nk) for _, t, h in others)):
        for name, t, h in (("q", q, H), ("k", k, Hk)) + others:
            if k is not None or h != Hk:
                _view(t, name, (B, h, T, d), q.dtype, dev)
            elif t is not None:
                raise ValueError(f"{name} without k")
    for name, w in weights:
        if w is not None:
            _dense(w, name, (d,), torch.float32, dev)
    n = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be a torch tensor of one dimension")
        n = inv_freq.shape[0]
        _dense(inv_freq, "inv_freq", (n,), torch.float32, dev)
    if positions is not None:
        _dense(positions, "positions", (B, T), torch.int32, dev)
    return B, H, Hk, T, d, n


def qknorm_fwd(q, k=None, q_weight=None, k_weight=None, *, norm: str = "rms", eps: float = 1e-6, inv_freq=None,
               positions=None, layout: str = "half", amplitude: float = 1.0, yq=None, yk=None):
    """Norm of each head's queries and keys, and their rotation by the token's
    position, in one pass.

    q [B,H,T,d], k [B,Hk,T,d] or None (float32 or bfloat16; any strides, the last
    dimension contiguous, d <= 512).  Each row is divided by its root mean square
    (``norm="rms"``), its length ("l2") or nothing ("none"), and scaled by q_weight, k_weight
    [d] float32 or None.  With inv_freq [n] float32 (rope_frequencies) the first 2 n
    channels are then rotated by positions[b,t] * inv_freq (int32 [B,T]; 0 ... T-1 when
    None) in n pairs: channels i and i + n (``layout="half"``) or 2 i and 2 i + 1
    ("pairs"), times ``amplitude``.  Returns (yq, yk), yq alone without k; buffers may be
    passed in, strided, and yq may be q itself and yk k."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    nm, ly = _choice(QK_NORMS, norm, "norm"), _choice(ROTARY_LAYOUTS, layout, "layout")
    if q.dim() != 4 or (k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 4)):
        raise ValueError("q and k must be [B, H, T, d]")
    with _guard(dev):
        if yq is None:
            yq = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if yk is None and k is not None:
            yk = torch.empty(k.shape, dtype=q.dtype, device=dev)
        B, H, Hk, T, d, n = _qk_checks(q, k, (("yq", yq, q.shape[1]), ("yk", yk, 0 if k is None else k.shape[1])),
                                       inv_freq, positions, (("q_weight", q_weight), ("k_weight", k_weight)), dev)
        kk, yy = (q, yq) if k is None else (k, yk)
        _check(lib().mlstm_qknorm_fwd(
            _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq), _ptr(positions), _ptr(yq), _ptr(yk),
            _strides(q, kk, yq, yy), B, H, Hk, T, d, n, ly, amplitude, nm, eps, io, _raw_stream(dev)))
    return yq if k is None else (yq, yk)


@functools.lru_cache(maxsize=4096)
def qknorm_bwd_workspace_size(B, H, Hk, T, d) -> int:
    """Bytes of workspace of qknorm_bwd with weight gradients (Hk = 0: queries alone)."""
    n = ctypes.c_size_t(0)
    _check(lib().mlstm_qknorm_bwd_workspace_size(B, H, Hk, T, d, ctypes.byref(n)))
    return n.value


def qknorm_bwd(q, k, dyq, dyk, q_weight=None, k_weight=None, *, norm: str = "rms", eps: float = 1e-6,
               inv_freq=None, positions=None, layout: str = "half", amplitude: float = 1.0,
               weight_grad: bool = True, dq=None, dk=None, workspace=None):
    """Gradients of qknorm_fwd, given its q and k (before the norm) and dyq and dyk.

    Returns (dq, dk, dq_weight, dk_weight), the first two in the I/O dtype, the others
    [d] float32 (None without ``weight_grad``; k, dyk None: dk and dk_weight are None).
    Buffers dq and dk may be passed in, strided; they may be dyq and dyk themselves."""
    import torch
    dev = _hip_device(q, "q")
    io = _io(q)
    nm, ly = _choice(QK_NORMS, norm, "norm"), _choice(ROTARY_LAYOUTS, layout, "layout")
    if q.dim() != 4 or (k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 4)):
        raise ValueError("q and k must be [B, H, T, d]")
    with _guard(dev):
        if dq is None:
            dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if dk is None and k is not None:
            dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
        h = 0 if k is None else k.shape[1]
        B, H, Hk, T, d, n = _qk_checks(q, k, (("dyq", dyq, q.shape[1]), ("dyk", dyk, h), ("dq", dq, q.shape[1]),
                                              ("dk", dk, h)), inv_freq, positions,
                                       (("q_weight", q_weight), ("k_weight", k_weight)), dev)
        dwq = torch.empty(d, dtype=torch.float32, device=dev) if weight_grad else None
        dwk = torch.empty(d, dtype=torch.float32, device=dev) if weight_grad and k is not None else None
        wp, wn, _keep = _workspace(workspace, qknorm_bwd_workspace_size(B, H, Hk, T, d) if weight_grad else 0, dev)
        other = (q, dyq, dq) if k is None else (k, dyk, dk)
        _check(lib().mlstm_qknorm_bwd(
            _ptr(q), _ptr(k), _ptr(dyq), _ptr(dyk), _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq),
            _ptr(positions), _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk),
            _strides(q, other[0], dyq, other[1], dq, other[2]), B, H, Hk, T, d, n, ly, amplitude, nm, eps, io,
            wp, wn, _raw_stream(dev)))
    return dq, dk, dwq, dwk
