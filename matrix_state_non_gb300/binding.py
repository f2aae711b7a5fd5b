"""Thin ctypes binding of libm2rnn.so (include/m2rnn.h).

The ``m2rnn_*`` functions mirror the C ABI one to one (raw device pointers and
sizes).  ``forward`` / ``backward`` are torch conveniences on top: they take
contiguous CUDA tensors, allocate outputs and the workspace with torch (device
memory and streams are all torch is used for) and call the C ABI on the
current stream.  Every step of both scans runs in the library's CUDA kernels;
there is no CPU path.  Loading fails loudly when the library is missing.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libm2rnn.so")

M2RNN_OK = 0
M2RNN_ERR_INVALID_ARG = -1
M2RNN_ERR_UNSUPPORTED = -2
M2RNN_ERR_WORKSPACE = -3
M2RNN_ERR_CUDA = -4
M2RNN_ERR_TIMEOUT = -5
M2RNN_ERR_DEVICE = -6
M2RNN_F32 = 0
M2RNN_BF16 = 1
M2RNN_OPT_KERNEL_FAMILY = 0
M2RNN_OPT_TEST_STALL_TILE = 1
# Kernel family codes (as m2rnn_path returns them); -1 = automatic choice.
FAMILIES = {"auto": -1, "simt": 0, "tcgen05": 1, "mma": 2}

EXPORTS = (
    "m2rnn_version", "m2rnn_status_string", "m2rnn_checkpoint_count", "m2rnn_path",
    "m2rnn_forward_workspace_size", "m2rnn_backward_workspace_size", "m2rnn_forward",
    "m2rnn_backward", "m2rnn_sync_status", "m2rnn_forward_state", "m2rnn_backward_state",
    "m2rnn_decode_step", "m2rnn_backward_state_workspace_size", "m2rnn_forward_gated",
    "m2rnn_backward_gated", "m2rnn_output_norm", "m2rnn_output_norm_backward_workspace_size",
    "m2rnn_output_norm_backward", "m2rnn_z_stash_size", "m2rnn_set_option",
    "m2rnn_backward_noalloc", "m2rnn_backward_noalloc_status",
    "m2rnn_causal_conv", "m2rnn_causal_conv_backward_workspace_size", "m2rnn_causal_conv_backward",
    "m2rnn_causal_conv_step", "m2rnn_ssm_workspace_size", "m2rnn_ssm_scan",
    "m2rnn_ssm_backward_workspace_size", "m2rnn_ssm_scan_backward", "m2rnn_ssm_step",
    "m2rnn_grad_plan_size", "m2rnn_grad_plan_build", "m2rnn_grad_workspace_size", "m2rnn_grad_norm",
    "m2rnn_grad_clip",
)

_lib = None


class M2RNNError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def load() -> ctypes.CDLL:
    """Load libm2rnn.so (built in-tree); raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m matrix_state_non_gb300.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.m2rnn_version.restype = ci
    lib.m2rnn_version.argtypes = []
    lib.m2rnn_status_string.restype = ctypes.c_char_p
    lib.m2rnn_status_string.argtypes = [ci]
    lib.m2rnn_checkpoint_count.restype = i64
    lib.m2rnn_checkpoint_count.argtypes = [i64, ci]
    lib.m2rnn_path.restype = ci
    lib.m2rnn_path.argtypes = [i64, i64, ci]
    lib.m2rnn_set_option.restype = ci
    lib.m2rnn_set_option.argtypes = [ci, ci, ctypes.POINTER(ci)]
    lib.m2rnn_forward_workspace_size.restype = sz
    lib.m2rnn_forward_workspace_size.argtypes = [i64, i64, i64, i64, i64, ci]
    lib.m2rnn_backward_workspace_size.restype = sz
    lib.m2rnn_backward_workspace_size.argtypes = [i64, i64, i64, i64, i64, ci, ci, ci]
    lib.m2rnn_forward.restype = ci
    lib.m2rnn_forward.argtypes = [vp] * 9 + [ci] + [i64] * 5 + [ci, vp, sz, vp]
    lib.m2rnn_backward.restype = ci
    lib.m2rnn_backward.argtypes = [vp] * 9 + [ci] + [vp] * 6 + [i64] * 5 + [ci, vp, sz, vp]
    lib.m2rnn_sync_status.restype = ci
    lib.m2rnn_sync_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.m2rnn_forward_state.restype = ci
    lib.m2rnn_forward_state.argtypes = [vp] * 10 + [ci, vp] + [i64] * 6 + [ci, vp, sz, vp]
    lib.m2rnn_backward_state.restype = ci
    lib.m2rnn_backward_state.argtypes = [vp] * 10 + [ci, vp] + [vp] * 7 + [ctypes.c_float] + [i64] * 6 + [ci, vp, sz, vp]
    lib.m2rnn_backward_state_workspace_size.restype = sz
    lib.m2rnn_backward_state_workspace_size.argtypes = [i64] * 6 + [ci, ci, ci]
    lib.m2rnn_decode_step.restype = ci
    lib.m2rnn_decode_step.argtypes = [vp] * 8 + [i64] * 5 + [ci, vp, sz, vp]
    fl = ctypes.c_float
    lib.m2rnn_forward_gated.restype = ci
    lib.m2rnn_forward_gated.argtypes = [vp] * 12 + [ci, vp] + [i64] * 6 + [ci, vp, sz, vp]
    lib.m2rnn_backward_gated.restype = ci
    lib.m2rnn_backward_gated.argtypes = [vp] * 12 + [ci, vp] + [vp] * 9 + [fl] + [i64] * 6 + [ci, vp, sz, vp]
    lib.m2rnn_z_stash_size.restype = sz
    lib.m2rnn_z_stash_size.argtypes = [i64] * 5 + [ci]
    lib.m2rnn_output_norm.restype = ci
    lib.m2rnn_output_norm.argtypes = [vp] * 3 + [fl] + [vp] * 2 + [i64] * 4 + [ci, vp]
    lib.m2rnn_output_norm_backward_workspace_size.restype = sz
    lib.m2rnn_output_norm_backward_workspace_size.argtypes = [i64] * 4
    lib.m2rnn_output_norm_backward.restype = ci
    lib.m2rnn_output_norm_backward.argtypes = [vp] * 4 + [fl] + [vp] * 3 + [i64] * 4 + [ci, vp, sz, vp]
    lib.m2rnn_causal_conv.restype = ci
    lib.m2rnn_causal_conv.argtypes = [vp, i64] + [vp] * 6 + [i64] * 4 + [ci, ci, vp]
    lib.m2rnn_causal_conv_backward_workspace_size.restype = sz
    lib.m2rnn_causal_conv_backward_workspace_size.argtypes = [i64] * 4
    lib.m2rnn_causal_conv_backward.restype = ci
    lib.m2rnn_causal_conv_backward.argtypes = [vp, i64] + [vp] * 10 + [i64] * 4 + [ci, ci, vp, sz, vp]
    lib.m2rnn_causal_conv_step.restype = ci
    lib.m2rnn_causal_conv_step.argtypes = [vp, vp, i64] + [vp] * 3 + [i64] * 3 + [ci, ci, vp]
    rows = [vp, i64] * 4
    lib.m2rnn_ssm_workspace_size.restype = sz
    lib.m2rnn_ssm_workspace_size.argtypes = [i64] * 6 + [ci]
    lib.m2rnn_ssm_scan.restype = ci
    lib.m2rnn_ssm_scan.argtypes = rows + [vp] * 7 + [i64] * 6 + [ci, vp, sz, vp]
    lib.m2rnn_ssm_backward_workspace_size.restype = sz
    lib.m2rnn_ssm_backward_workspace_size.argtypes = [i64] * 6 + [ci]
    lib.m2rnn_ssm_scan_backward.restype = ci
    lib.m2rnn_ssm_scan_backward.argtypes = rows + [vp] * 15 + [i64] * 6 + [ci, vp, sz, vp]
    lib.m2rnn_ssm_step.restype = ci
    lib.m2rnn_ssm_step.argtypes = [vp] + rows + [vp] * 4 + [i64] * 5 + [ci, vp]
    lib.m2rnn_grad_plan_size.restype = sz
    lib.m2rnn_grad_plan_size.argtypes = [i64, vp]
    lib.m2rnn_grad_plan_build.restype = ci
    lib.m2rnn_grad_plan_build.argtypes = [i64] + [vp] * 5 + [sz]
    lib.m2rnn_grad_workspace_size.restype = sz
    lib.m2rnn_grad_workspace_size.argtypes = []
    lib.m2rnn_grad_norm.restype = ci
    lib.m2rnn_grad_norm.argtypes = [vp, sz, vp, vp, sz, vp]
    lib.m2rnn_grad_clip.restype = ci
    lib.m2rnn_grad_clip.argtypes = [vp, sz, fl, vp, vp, sz, vp]
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# One-to-one wrappers of the C ABI (integers are device addresses).
# ---------------------------------------------------------------------------
def m2rnn_version() -> int:
    return load().m2rnn_version()


def status_string(status: int) -> str:
    return load().m2rnn_status_string(status).decode()


m2rnn_status_string = status_string


def m2rnn_checkpoint_count(T: int, ckpt_every: int) -> int:
    return load().m2rnn_checkpoint_count(T, ckpt_every)


def m2rnn_path(K: int, V: int, dtype: int) -> int:
    return load().m2rnn_path(K, V, dtype)


def m2rnn_set_option(option: int, value: int):
    """Returns (status, previous value)."""
    prev = ctypes.c_int(0)
    st = load().m2rnn_set_option(option, value, ctypes.byref(prev))
    return st, prev.value


@contextlib.contextmanager
def kernel_family(name: str):
    """Run the enclosed calls on one kernel family ("auto", "tcgen05", "mma",
    "simt"); the previous choice is restored on exit."""
    st, prev = m2rnn_set_option(M2RNN_OPT_KERNEL_FAMILY, FAMILIES[name])
    _check(st, "m2rnn_set_option")
    try:
        yield
    finally:
        m2rnn_set_option(M2RNN_OPT_KERNEL_FAMILY, prev)


@contextlib.contextmanager
def stall_tile_hook(tile: int):
    """Failure-detection test hook (see include/m2rnn.h): the warp-MMA forward
    withholds input tile `tile` of single-CTA chains inside the block."""
    st, prev = m2rnn_set_option(M2RNN_OPT_TEST_STALL_TILE, tile)
    _check(st, "m2rnn_set_option")
    try:
        yield
    finally:
        m2rnn_set_option(M2RNN_OPT_TEST_STALL_TILE, prev)


def m2rnn_forward_workspace_size(B, T, N, K, V, dtype) -> int:
    return load().m2rnn_forward_workspace_size(B, T, N, K, V, dtype)


def m2rnn_backward_workspace_size(B, T, N, K, V, dtype, ckpt_every, have_ckpt) -> int:
    return load().m2rnn_backward_workspace_size(B, T, N, K, V, dtype, ckpt_every, int(bool(have_ckpt)))


def m2rnn_forward(q, k, v, f, W, w_r, y, H_T, ckpt, ckpt_every, B, T, N, K, V, dtype,
                  workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_forward(q, k, v, f, W, w_r, y, H_T, ckpt, ckpt_every, B, T, N, K, V,
                                dtype, workspace, workspace_bytes, stream)


def m2rnn_backward(q, k, v, f, W, w_r, dy, dH_T, ckpt, ckpt_every, dq, dk, dv, df, dW, dw_r,
                   B, T, N, K, V, dtype, workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_backward(q, k, v, f, W, w_r, dy, dH_T, ckpt, ckpt_every, dq, dk, dv,
                                 df, dW, dw_r, B, T, N, K, V, dtype, workspace,
                                 workspace_bytes, stream)


def m2rnn_forward_state(q, k, v, f, W, w_r, H_0, y, H_T, ckpt, ckpt_every, z_stash, B, T, N, qk_heads, K, V,
                        dtype, workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_forward_state(q, k, v, f, W, w_r, H_0, y, H_T, ckpt, ckpt_every, z_stash, B, T, N,
                                      qk_heads, K, V, dtype, workspace, workspace_bytes, stream)


def m2rnn_z_stash_size(B, T, N, K, V, dtype) -> int:
    return load().m2rnn_z_stash_size(B, T, N, K, V, dtype)


def m2rnn_backward_state_workspace_size(B, T, N, qk_heads, K, V, dtype, ckpt_every, have_ckpt) -> int:
    return load().m2rnn_backward_state_workspace_size(B, T, N, qk_heads, K, V, dtype, ckpt_every,
                                                      int(bool(have_ckpt)))


def m2rnn_backward_state(q, k, v, f, W, w_r, H_0, dy, dH_T, ckpt, ckpt_every, z_stash, dq, dk, dv, df, dW,
                         dw_r, dH_0, state_grad_clip, B, T, N, qk_heads, K, V, dtype, workspace,
                         workspace_bytes, stream) -> int:
    return load().m2rnn_backward_state(q, k, v, f, W, w_r, H_0, dy, dH_T, ckpt, ckpt_every, z_stash, dq, dk,
                                       dv, df, dW, dw_r, dH_0, state_grad_clip, B, T, N, qk_heads, K,
                                       V, dtype, workspace, workspace_bytes, stream)


def m2rnn_decode_step(H, q, k, v, f, W, w_r, y, B, N, qk_heads, K, V, dtype, workspace,
                      workspace_bytes, stream) -> int:
    return load().m2rnn_decode_step(H, q, k, v, f, W, w_r, y, B, N, qk_heads, K, V, dtype, workspace,
                                    workspace_bytes, stream)


def m2rnn_forward_gated(q, k, v, a, alpha, beta, W, w_r, H_0, y, H_T, ckpt, ckpt_every, z_stash, B, T, N,
                        qk_heads, K, V, dtype, workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_forward_gated(q, k, v, a, alpha, beta, W, w_r, H_0, y, H_T, ckpt, ckpt_every, z_stash, B, T,
                                      N, qk_heads, K, V, dtype, workspace, workspace_bytes, stream)


def m2rnn_backward_gated(q, k, v, a, alpha, beta, W, w_r, H_0, dy, dH_T, ckpt, ckpt_every, z_stash, dq, dk, dv,
                         da, dalpha, dbeta, dW, dw_r, dH_0, state_grad_clip, B, T, N, qk_heads, K, V, dtype,
                         workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_backward_gated(q, k, v, a, alpha, beta, W, w_r, H_0, dy, dH_T, ckpt, ckpt_every, z_stash,
                                       dq, dk, dv, da, dalpha, dbeta, dW, dw_r, dH_0, state_grad_clip, B, T, N,
                                       qk_heads, K, V, dtype, workspace, workspace_bytes, stream)


def m2rnn_output_norm(y, g, w, eps, out, rstd, B, T, N, V, dtype, stream) -> int:
    return load().m2rnn_output_norm(y, g, w, eps, out, rstd, B, T, N, V, dtype, stream)


def m2rnn_output_norm_backward_workspace_size(B, T, N, V) -> int:
    return load().m2rnn_output_norm_backward_workspace_size(B, T, N, V)


def m2rnn_output_norm_backward(y, g, w, dout, eps, dy, dg, dw, B, T, N, V, dtype, workspace,
                               workspace_bytes, stream) -> int:
    return load().m2rnn_output_norm_backward(y, g, w, dout, eps, dy, dg, dw, B, T, N, V, dtype, workspace,
                                             workspace_bytes, stream)


def m2rnn_sync_status(workspace, stream):
    """Returns (status, detail)."""
    d = ctypes.c_uint32(0)
    st = load().m2rnn_sync_status(workspace, stream, ctypes.byref(d))
    return st, d.value


# ---------------------------------------------------------------------------
# torch conveniences
# ---------------------------------------------------------------------------
def _ptr(t) -> Optional[int]:
    """Address of a dense tensor (the library takes no strides here)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"expected a contiguous tensor, got strides {t.stride()} for {tuple(t.shape)}")
    return t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return M2RNN_BF16
    if t.dtype == torch.float32:
        return M2RNN_F32
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _check(st: int, what: str):
    if st != M2RNN_OK:
        raise M2RNNError(st, what)


def _stream_handle(stream) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _shapes(q, v):
    """(B, T, N, K, V, qk_heads): N from v; q, k carry 1 head when shared."""
    B, T, _, K = q.shape
    N, V = v.shape[2], v.shape[-1]
    return B, T, N, K, V, q.shape[2]


def forward(q, k, v, f, W, w_r, *, H_0=None, want_state: bool = True, ckpt_every: int = 0,
            gate=None, stash: bool = False, out=None, workspace=None, stream=None):
    """Forward scan on the GPU from ``H_0`` (fp32 [B,N,K,V]; None = zero).
    Returns dict(y, H_T[, ckpt]).

    ``ckpt_every`` > 0 also writes the checkpoints the backward can reuse.
    ``gate`` = (a, alpha, beta) with ``f`` None computes the forget gate in
    the kernels (m2rnn_forward_gated).  ``stash`` also returns "z_stash", the
    fp16 Z_t of every step for ``backward`` (bf16, V = 64 only).  ``out`` may
    hold preallocated y / H_T / ckpt / z_stash tensors.
    """
    import torch
    B, T, N, K, V, NQ = _shapes(q, v)
    dt = _dtype_code(q)
    dev = q.device
    out = dict(out or {})
    y = out.get("y")
    if y is None:
        y = torch.empty((B, T, N, V), device=dev, dtype=torch.float32)
    H_T = out.get("H_T")
    if H_T is None and want_state:
        H_T = torch.empty((B, N, K, V), device=dev, dtype=torch.float32)
    ckpt = out.get("ckpt")
    if ckpt is None and ckpt_every > 0:
        nck = m2rnn_checkpoint_count(T, ckpt_every)
        ckpt = torch.empty((B, N, max(nck, 0), K, V), device=dev, dtype=torch.float32)
    ws_bytes = m2rnn_forward_workspace_size(B, T, N, K, V, dt)
    if ws_bytes == 0:
        raise M2RNNError(M2RNN_ERR_INVALID_ARG, "m2rnn_forward_workspace_size")
    if workspace is None:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    z_stash = out.get("z_stash")
    if z_stash is None and stash:
        zb = m2rnn_z_stash_size(B, T, N, K, V, dt)
        if zb == 0:
            raise M2RNNError(M2RNN_ERR_UNSUPPORTED, "m2rnn_z_stash_size")
        z_stash = torch.empty(zb, device=dev, dtype=torch.uint8)
    ce = ckpt_every if ckpt is not None else 0
    if gate is not None:
        if f is not None:
            raise ValueError("give either f or gate=(a, alpha, beta), not both")
        a, alpha, beta = gate
        st = m2rnn_forward_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(alpha), _ptr(beta), _ptr(W),
                                 _ptr(w_r), _ptr(H_0), _ptr(y), _ptr(H_T), _ptr(ckpt), ce, _ptr(z_stash), B, T,
                                 N, NQ, K, V, dt, _ptr(workspace), workspace.numel(), _stream_handle(stream))
        _check(st, "m2rnn_forward_gated")
    else:
        st = m2rnn_forward_state(_ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W), _ptr(w_r), _ptr(H_0),
                                 _ptr(y), _ptr(H_T), _ptr(ckpt), ce, _ptr(z_stash), B, T, N, NQ, K, V, dt,
                                 _ptr(workspace), workspace.numel(), _stream_handle(stream))
        _check(st, "m2rnn_forward_state")
    res = dict(y=y, H_T=H_T, workspace=workspace)
    if ckpt is not None:
        res["ckpt"] = ckpt
    if z_stash is not None:
        res["z_stash"] = z_stash
    return res


def backward(q, k, v, f, W, w_r, dy, *, dH_T=None, H_0=None, want_dH0: bool = False, ckpt=None,
             ckpt_every: int = 14, state_grad_clip: float = 0.0, gate=None, z_stash=None, out=None,
             workspace=None, stream=None):
    """Backward scan on the GPU.  Returns dict(dq, dk, dv, df, dW, dw_r[, dH_0]);
    with ``gate`` = (a, alpha, beta) (and ``f`` None) da, dalpha, dbeta
    replace df.

    ``H_0`` is the forward's initial state (None = zero); ``ckpt``, if given,
    must come from a forward with the same ``H_0`` (and gate); ``z_stash``, with
    that forward's ``ckpt``, replaces the rerun of the transform and tanh;
    ``state_grad_clip`` > 0 clamps every new state gradient C_{t-1} to [-c, c]."""
    import torch
    B, T, N, K, V, NQ = _shapes(q, v)
    dt = _dtype_code(q)
    dev = q.device
    out = dict(out or {})

    def _get(name, shape):
        t = out.get(name)
        return t if t is not None else torch.empty(shape, device=dev, dtype=torch.float32)

    dq = _get("dq", (B, T, NQ, K))
    dk = _get("dk", (B, T, NQ, K))
    dv = _get("dv", (B, T, N, V))
    df = _get("df", (B, T, N)) if gate is None else None
    dW = _get("dW", (N, V, V))
    dw_r = _get("dw_r", (N, V))
    dH_0 = _get("dH_0", (B, N, K, V)) if want_dH0 else None
    ws_bytes = m2rnn_backward_state_workspace_size(B, T, N, NQ, K, V, dt, ckpt_every, ckpt is not None)
    if ws_bytes == 0:
        raise M2RNNError(M2RNN_ERR_INVALID_ARG, "m2rnn_backward_state_workspace_size")
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    if gate is not None:
        if f is not None:
            raise ValueError("give either f or gate=(a, alpha, beta), not both")
        a, alpha, beta = gate
        da = _get("da", (B, T, N))
        dalpha = _get("dalpha", (N,))
        dbeta = _get("dbeta", (N,))
        st = m2rnn_backward_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(alpha), _ptr(beta), _ptr(W),
                                  _ptr(w_r), _ptr(H_0), _ptr(dy), _ptr(dH_T), _ptr(ckpt), ckpt_every,
                                  _ptr(z_stash), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(da), _ptr(dalpha), _ptr(dbeta), _ptr(dW),
                                  _ptr(dw_r), _ptr(dH_0), float(state_grad_clip), B, T, N, NQ, K, V, dt,
                                  _ptr(workspace), workspace.numel(), _stream_handle(stream))
        _check(st, "m2rnn_backward_gated")
        res = dict(dq=dq, dk=dk, dv=dv, da=da, dalpha=dalpha, dbeta=dbeta, dW=dW, dw_r=dw_r,
                   workspace=workspace)
    else:
        st = m2rnn_backward_state(_ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W), _ptr(w_r), _ptr(H_0),
                                  _ptr(dy), _ptr(dH_T), _ptr(ckpt), ckpt_every, _ptr(z_stash), _ptr(dq),
                                  _ptr(dk), _ptr(dv), _ptr(df), _ptr(dW), _ptr(dw_r), _ptr(dH_0),
                                  float(state_grad_clip), B, T, N, NQ, K, V, dt, _ptr(workspace),
                                  workspace.numel(), _stream_handle(stream))
        _check(st, "m2rnn_backward_state")
        res = dict(dq=dq, dk=dk, dv=dv, df=df, dW=dW, dw_r=dw_r, workspace=workspace)
    if dH_0 is not None:
        res["dH_0"] = dH_0
    return res


def decode_step(H, q, k, v, f, W, w_r, *, y=None, workspace=None, stream=None):
    """One decoding step on the GPU: ``H`` (fp32 [B,N,K,V], contiguous) is
    updated in place; q, k [B,N,K] (or [B,1,K], shared by the heads),
    v [B,N,V], f [B,N].  Returns y [B,N,V]."""
    import torch
    B, NQ, K = q.shape
    N, V = v.shape[1], v.shape[-1]
    dt = _dtype_code(q)
    if y is None:
        y = torch.empty((B, N, V), device=q.device, dtype=torch.float32)
    ws_bytes = m2rnn_forward_workspace_size(B, 1, N, K, V, dt)
    if ws_bytes == 0:
        raise M2RNNError(M2RNN_ERR_INVALID_ARG, "m2rnn_forward_workspace_size")
    if workspace is None:
        workspace = torch.empty(ws_bytes, device=q.device, dtype=torch.uint8)
    st = m2rnn_decode_step(_ptr(H), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W), _ptr(w_r), _ptr(y),
                           B, N, NQ, K, V, dt, _ptr(workspace), workspace.numel(),
                           _stream_handle(stream))
    _check(st, "m2rnn_decode_step")
    return y


def output_norm(y, g, w, *, eps: float = 1e-6, want_rstd: bool = False, out=None, stream=None):
    """out = w * (y*g) * rms^-1 over each token's N*V elements; y fp32
    [B,T,N,V], g [B,T,N,V] (bf16 or fp32), w fp32 [N,V].  Returns out, or
    (out, rstd [B,T]) with ``want_rstd``."""
    import torch
    B, T, N, V = y.shape
    if out is None:
        out = torch.empty((B, T, N, V), device=y.device, dtype=torch.float32)
    rstd = torch.empty((B, T), device=y.device, dtype=torch.float32) if want_rstd else None
    st = m2rnn_output_norm(_ptr(y), _ptr(g), _ptr(w), float(eps), _ptr(out), _ptr(rstd), B, T, N, V,
                           _dtype_code(g), _stream_handle(stream))
    _check(st, "m2rnn_output_norm")
    return (out, rstd) if want_rstd else out


def output_norm_backward(y, g, w, dout, *, eps: float = 1e-6, out=None, workspace=None, stream=None):
    """Returns dict(dy, dg [B,T,N,V], dw [N,V]) of ``output_norm``; ``out``
    may hold preallocated dy / dg / dw."""
    import torch
    B, T, N, V = y.shape
    dev = y.device
    out = dict(out or {})

    def _get(name, shape):
        t = out.get(name)
        return t if t is not None else torch.empty(shape, device=dev, dtype=torch.float32)

    dy = _get("dy", (B, T, N, V))
    dg = _get("dg", (B, T, N, V))
    dw = _get("dw", (N, V))
    ws_bytes = m2rnn_output_norm_backward_workspace_size(B, T, N, V)
    if ws_bytes == 0:
        raise M2RNNError(M2RNN_ERR_UNSUPPORTED, "m2rnn_output_norm_backward_workspace_size")
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    st = m2rnn_output_norm_backward(_ptr(y), _ptr(g), _ptr(w), _ptr(dout), float(eps), _ptr(dy), _ptr(dg),
                                    _ptr(dw), B, T, N, V, _dtype_code(g), _ptr(workspace), workspace.numel(),
                                    _stream_handle(stream))
    _check(st, "m2rnn_output_norm_backward")
    return dict(dy=dy, dg=dg, dw=dw)


def sync_status(workspace, stream=None):
    st, detail = m2rnn_sync_status(workspace.data_ptr(), _stream_handle(stream))
    return st, detail


def to_device(inp, device="cuda"):
    """Upload an ``inputs.M2RNNInputs`` batch: bf16 bit patterns become
    torch.bfloat16 tensors, float32 stays float32."""
    import numpy as np
    import torch
    res = {}
    for name, arr in inp.store.items():
        if arr.dtype == np.uint16:
            t = torch.from_numpy(arr.view(np.int16).copy()).view(torch.bfloat16)
        else:
            t = torch.from_numpy(np.ascontiguousarray(arr))
        res[name] = t.to(device).contiguous()
    return res


def m2rnn_backward_noalloc(q, k, v, f, W, w_r, dy, dH_T, ckpt, ckpt_every, dq, dk, dv, df, dW,
                           dw_r, B, T, N, K, V, dtype, sync, stream) -> int:
    """The backward for callers that cannot allocate device memory: scratch
    comes from an array built into the library (see include/m2rnn.h for the
    limits).  Integers are device addresses, as for m2rnn_backward."""
    lib = load()
    fn = lib.m2rnn_backward_noalloc
    if fn.argtypes is None:
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        fn.restype = ci
        fn.argtypes = [vp] * 9 + [ci] + [vp] * 6 + [i64] * 5 + [ci, ci, vp]
    return fn(q, k, v, f, W, w_r, dy, dH_T, ckpt, ckpt_every, dq, dk, dv, df, dW, dw_r, B, T, N,
              K, V, dtype, sync, stream)


def m2rnn_backward_noalloc_status(stream):
    """Device-side status of the last allocation-free backward on the current
    device: returns (status, detail); synchronises `stream` first."""
    lib = load()
    fn = lib.m2rnn_backward_noalloc_status
    if fn.argtypes is None:
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    detail = ctypes.c_uint32(0)
    st = fn(stream, ctypes.byref(detail))
    return st, detail.value


# ---------------------------------------------------------------------------
# The hybrid layer: short causal convolution, selective state space scan,
# gradient clipping (raw wrappers, then torch conveniences)
# ---------------------------------------------------------------------------
def m2rnn_causal_conv(*args) -> int:
    return load().m2rnn_causal_conv(*args)


def m2rnn_causal_conv_backward_workspace_size(B, T, C, W) -> int:
    return load().m2rnn_causal_conv_backward_workspace_size(B, T, C, W)


def m2rnn_causal_conv_backward(*args) -> int:
    return load().m2rnn_causal_conv_backward(*args)


def m2rnn_causal_conv_step(*args) -> int:
    return load().m2rnn_causal_conv_step(*args)


def m2rnn_ssm_workspace_size(B, T, N, G, K, V, dtype) -> int:
    return load().m2rnn_ssm_workspace_size(B, T, N, G, K, V, dtype)


def m2rnn_ssm_scan(*args) -> int:
    return load().m2rnn_ssm_scan(*args)


def m2rnn_ssm_backward_workspace_size(B, T, N, G, K, V, dtype) -> int:
    return load().m2rnn_ssm_backward_workspace_size(B, T, N, G, K, V, dtype)


def m2rnn_ssm_scan_backward(*args) -> int:
    return load().m2rnn_ssm_scan_backward(*args)


def m2rnn_ssm_step(*args) -> int:
    return load().m2rnn_ssm_step(*args)


def m2rnn_grad_plan_size(n, counts) -> int:
    return load().m2rnn_grad_plan_size(n, counts)


def m2rnn_grad_plan_build(n, grads, outs, counts, dtypes, plan, plan_bytes) -> int:
    return load().m2rnn_grad_plan_build(n, grads, outs, counts, dtypes, plan, plan_bytes)


def m2rnn_grad_workspace_size() -> int:
    return load().m2rnn_grad_workspace_size()


def m2rnn_grad_norm(plan, plan_bytes, norm, workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_grad_norm(plan, plan_bytes, norm, workspace, workspace_bytes, stream)


def m2rnn_grad_clip(plan, plan_bytes, max_norm, norm, workspace, workspace_bytes, stream) -> int:
    return load().m2rnn_grad_clip(plan, plan_bytes, max_norm, norm, workspace, workspace_bytes, stream)


def _need(t, name: str, shape, dtype, gpu: int):
    """Address of an optional dense operand (None for None), checked."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == gpu and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, shape, dtype, gpu)
    raise ValueError(f"{name} must be contiguous")


def _refuse(t, name: str, shape, dtype, gpu: int):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != gpu:
        raise ValueError(f"{name} must be on cuda:{gpu}, is on {t.device}")


def _rows(t, name: str, shape, inner: int, width: int, dtype, gpu: int):
    """Address and row stride of an input that may be a column slice of a
    wider tensor: its last ``inner`` dimensions (the ``width`` values of one
    token) dense, the tokens of [B,T,...] evenly spaced through all sequences."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != gpu:
        _refuse(t, name, shape, dtype, gpu)
    if t.is_contiguous():
        return t.data_ptr(), width
    dense, stride, n = 1, t.stride(), len(shape) - inner
    for i in range(len(shape) - 1, n - 1, -1):
        if shape[i] != 1 and stride[i] != dense:
            raise ValueError(f"{name}: the values of one token must be dense")
        dense *= shape[i]
    if n == 2 and shape[1] > 1:
        if shape[0] > 1 and stride[0] != shape[1] * stride[1]:
            raise ValueError(f"{name}: sequences must lie T rows apart")
        return t.data_ptr(), stride[1]
    return t.data_ptr(), stride[0] if shape[0] > 1 else width


def _gpu(t) -> int:
    """The tensor's GPU, which has to be the current one: the library's launches
    go there."""
    gpu = t.get_device()
    if gpu < 0:
        raise ValueError(f"expected CUDA tensors, got one on {t.device}")
    return _current(gpu)


def _current(gpu: int) -> int:
    import torch
    if gpu != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{gpu}, the current device is cuda:{torch.cuda.current_device()}: "
                         f"call under torch.cuda.device({gpu})")
    return gpu


def _on(gpu: int, stream) -> int:
    """Handle of the given stream, else of the GPU's current one."""
    if stream is not None:
        return stream.cuda_stream
    from torch._C import _cuda_getCurrentRawStream
    return _cuda_getCurrentRawStream(gpu)


def _alloc(like, shape, dtype, stream):
    """A new tensor that belongs to the stream it is used on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _out(out, name, like, shape, dtype, stream):
    t = out.get(name) if out else None
    if t is None:
        return _alloc(like, shape, dtype, stream)
    _need(t, name, shape, dtype, like.get_device())
    return t


def _scratch(workspace, nbytes: int, like, stream, what: str):
    import torch
    if nbytes == 0:
        raise M2RNNError(M2RNN_ERR_UNSUPPORTED, what)
    if workspace is None:
        return _alloc(like, (nbytes,), torch.uint8, stream)
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{like.get_device()}, is on {workspace.device}")
    return workspace if workspace.numel() >= nbytes else _alloc(like, (nbytes,), torch.uint8, stream)


def causal_conv(x, w, bias=None, *, x0=None, lengths=None, silu: bool = True, want_state: bool = False,
                out=None, stream=None):
    """Short causal depthwise convolution, with SiLU.  ``x`` [B,T,C] (may be a
    column slice of a wider projection), ``w`` [C,W], ``bias`` [C], ``x0``
    [B,W-1,C] the inputs before the sequence (None = zero), ``lengths`` [B]
    int32.  Returns dict(y[, x_T]); x_T [B,W-1,C] continues the sequence, as
    ``x0`` of the next piece or as the state of ``causal_conv_step``.  ``out``
    may hold preallocated y / x_T."""
    import torch
    B, T, C = x.shape
    W, gpu, dt = w.shape[1], _gpu(x), x.dtype
    code = _dtype_code(x)
    xp, xs = _rows(x, "x", (B, T, C), 1, C, dt, gpu)
    y = _out(out, "y", x, (B, T, C), dt, stream)
    x_T = _out(out, "x_T", x, (B, W - 1, C), dt, stream) if want_state or (out and "x_T" in out) else None
    st = load().m2rnn_causal_conv(xp, xs, _need(w, "w", (C, W), dt, gpu), _need(bias, "bias", (C,), dt, gpu),
                                  _need(x0, "x0", (B, W - 1, C), dt, gpu),
                                  _need(lengths, "lengths", (B,), torch.int32, gpu), y.data_ptr(), _ptr(x_T), B, T, C,
                                  W, int(silu), code, _on(gpu, stream))
    _check(st, "m2rnn_causal_conv")
    return dict(y=y) if x_T is None else dict(y=y, x_T=x_T)


def causal_conv_backward(x, w, bias, dy, *, x0=None, dx_T=None, lengths=None, silu: bool = True,
                         want_dx0: bool = False, out=None, workspace=None, stream=None):
    """Backward of ``causal_conv``: ``dy`` [B,T,C] and ``dx_T`` [B,W-1,C] fp32.
    Returns dict(dx, dw[, db][, dx0]), fp32 (db when there is a bias)."""
    import torch
    B, T, C = x.shape
    W, gpu, dt, f32 = w.shape[1], _gpu(x), x.dtype, torch.float32
    code = _dtype_code(x)
    xp, xs = _rows(x, "x", (B, T, C), 1, C, dt, gpu)
    res = dict(dx=_out(out, "dx", x, (B, T, C), f32, stream), dw=_out(out, "dw", x, (C, W), f32, stream))
    if bias is not None:
        res["db"] = _out(out, "db", x, (C,), f32, stream)
    if want_dx0:
        res["dx0"] = _out(out, "dx0", x, (B, W - 1, C), f32, stream)
    ws = _scratch(workspace, m2rnn_causal_conv_backward_workspace_size(B, T, C, W), x, stream,
                  "m2rnn_causal_conv_backward_workspace_size")
    st = load().m2rnn_causal_conv_backward(
        xp, xs, _need(w, "w", (C, W), dt, gpu), _need(bias, "bias", (C,), dt, gpu),
        _need(x0, "x0", (B, W - 1, C), dt, gpu), _need(lengths, "lengths", (B,), torch.int32, gpu),
        _need(dy, "dy", (B, T, C), f32, gpu), _need(dx_T, "dx_T", (B, W - 1, C), f32, gpu), res["dx"].data_ptr(),
        res["dw"].data_ptr(), _ptr(res.get("db")), _ptr(res.get("dx0")), B, T, C, W, int(silu), code, ws.data_ptr(),
        ws.numel(), _on(gpu, stream))
    _check(st, "m2rnn_causal_conv_backward")
    return res


def causal_conv_step(state, x, w, bias=None, *, silu: bool = True, y=None, stream=None):
    """One token: ``state`` [B,W-1,C] is shifted in place and takes ``x`` [B,C]
    in.  Returns y [B,C]."""
    B, C = x.shape
    W, gpu, dt = w.shape[1], _gpu(x), x.dtype
    code = _dtype_code(x)
    xp, xs = _rows(x, "x", (B, C), 1, C, dt, gpu)
    if y is None:
        y = _alloc(x, (B, C), dt, stream)
    st = load().m2rnn_causal_conv_step(_need(state, "state", (B, W - 1, C), dt, gpu), xp, xs,
                                       _need(w, "w", (C, W), dt, gpu), _need(bias, "bias", (C,), dt, gpu),
                                       _need(y, "y", (B, C), dt, gpu), B, C, W, int(silu), code,
                                       _on(gpu, stream))
    _check(st, "m2rnn_causal_conv_step")
    return y


def ssm_scan(q, k, v, dt, A, *, dt_bias=None, w_r=None, H_0=None, lengths=None, want_state: bool = True, out=None,
             workspace=None, stream=None):
    """Selective state space scan (see m2rnn_ssm_scan): q, k [B,T,G,K], v
    [B,T,N,V], dt [B,T,N] (column slices of wider tensors are fine), A [N]
    fp32, dt_bias [N] fp32, w_r [N,V], H_0 [B,N,K,V] fp32, lengths [B] int32.
    Returns dict(y, H_T, workspace): y in the inputs' type, H_T fp32."""
    import torch
    B, T, G, K = q.shape
    N, V = v.shape[2:]
    gpu, ty, f32 = _gpu(v), v.dtype, torch.float32
    code = _dtype_code(v)
    qp, qs = _rows(q, "q", (B, T, G, K), 2, G * K, ty, gpu)
    kp, ks = _rows(k, "k", (B, T, G, K), 2, G * K, ty, gpu)
    vp, vs = _rows(v, "v", (B, T, N, V), 2, N * V, ty, gpu)
    dp, ds = _rows(dt, "dt", (B, T, N), 1, N, ty, gpu)
    y = _out(out, "y", v, (B, T, N, V), ty, stream)
    H_T = _out(out, "H_T", v, (B, N, K, V), f32, stream) if want_state else None
    ws = _scratch(workspace, m2rnn_ssm_workspace_size(B, T, N, G, K, V, code), v, stream,
                  "m2rnn_ssm_workspace_size")
    st = load().m2rnn_ssm_scan(qp, qs, kp, ks, vp, vs, dp, ds, _need(A, "A", (N,), f32, gpu),
                               _need(dt_bias, "dt_bias", (N,), f32, gpu), _need(w_r, "w_r", (N, V), ty, gpu),
                               _need(H_0, "H_0", (B, N, K, V), f32, gpu),
                               _need(lengths, "lengths", (B,), torch.int32, gpu), y.data_ptr(), _ptr(H_T), B, T, N, G,
                               K, V, code, ws.data_ptr(), ws.numel(), _on(gpu, stream))
    _check(st, "m2rnn_ssm_scan")
    return dict(y=y, H_T=H_T, workspace=ws)


def ssm_scan_backward(q, k, v, dt, A, dy, *, dt_bias=None, w_r=None, H_0=None, dH_T=None, lengths=None,
                      want_dH0: bool = False, out=None, workspace=None, stream=None):
    """Backward of ``ssm_scan``: ``dy`` [B,T,N,V] in the inputs' type, ``dH_T``
    [B,N,K,V] fp32.  Returns dict(dq, dk, dv, ddt, dA[, ddt_bias][, dw_r]
    [, dH_0], workspace), all fp32."""
    import torch
    B, T, G, K = q.shape
    N, V = v.shape[2:]
    gpu, ty, f32 = _gpu(v), v.dtype, torch.float32
    code = _dtype_code(v)
    qp, qs = _rows(q, "q", (B, T, G, K), 2, G * K, ty, gpu)
    kp, ks = _rows(k, "k", (B, T, G, K), 2, G * K, ty, gpu)
    vp, vs = _rows(v, "v", (B, T, N, V), 2, N * V, ty, gpu)
    dp, ds = _rows(dt, "dt", (B, T, N), 1, N, ty, gpu)
    shapes = dict(dq=(B, T, G, K), dk=(B, T, G, K), dv=(B, T, N, V), ddt=(B, T, N), dA=(N,))
    if dt_bias is not None:
        shapes["ddt_bias"] = (N,)
    if w_r is not None:
        shapes["dw_r"] = (N, V)
    if want_dH0:
        shapes["dH_0"] = (B, N, K, V)
    res = {n: _out(out, n, v, sh, f32, stream) for n, sh in shapes.items()}
    ws = _scratch(workspace, m2rnn_ssm_backward_workspace_size(B, T, N, G, K, V, code), v, stream,
                  "m2rnn_ssm_backward_workspace_size")
    st = load().m2rnn_ssm_scan_backward(
        qp, qs, kp, ks, vp, vs, dp, ds, _need(A, "A", (N,), f32, gpu), _need(dt_bias, "dt_bias", (N,), f32, gpu),
        _need(w_r, "w_r", (N, V), ty, gpu), _need(H_0, "H_0", (B, N, K, V), f32, gpu),
        _need(lengths, "lengths", (B,), torch.int32, gpu), _need(dy, "dy", (B, T, N, V), ty, gpu),
        _need(dH_T, "dH_T", (B, N, K, V), f32, gpu),
        *(_ptr(res.get(n)) for n in ("dq", "dk", "dv", "ddt", "dA", "ddt_bias", "dw_r", "dH_0")), B, T, N, G, K, V,
        code, ws.data_ptr(), ws.numel(), _on(gpu, stream))
    _check(st, "m2rnn_ssm_scan_backward")
    res["workspace"] = ws
    return res


def ssm_step(H, q, k, v, dt, A, *, dt_bias=None, w_r=None, y=None, stream=None):
    """One token of ``ssm_scan``: ``H`` [B,N,K,V] fp32 advances in place; q, k
    [B,G,K], v [B,N,V], dt [B,N].  Returns y [B,N,V]."""
    import torch
    B, G, K = q.shape
    N, V = v.shape[1:]
    gpu, ty, f32 = _gpu(v), v.dtype, torch.float32
    code = _dtype_code(v)
    qp, qs = _rows(q, "q", (B, G, K), 2, G * K, ty, gpu)
    kp, ks = _rows(k, "k", (B, G, K), 2, G * K, ty, gpu)
    vp, vs = _rows(v, "v", (B, N, V), 2, N * V, ty, gpu)
    dp, ds = _rows(dt, "dt", (B, N), 1, N, ty, gpu)
    if y is None:
        y = _alloc(v, (B, N, V), ty, stream)
    st = load().m2rnn_ssm_step(_need(H, "H", (B, N, K, V), f32, gpu), qp, qs, kp, ks, vp, vs, dp, ds,
                               _need(A, "A", (N,), f32, gpu), _need(dt_bias, "dt_bias", (N,), f32, gpu),
                               _need(w_r, "w_r", (N, V), ty, gpu), _need(y, "y", (B, N, V), ty, gpu), B, N, G, K, V,
                               code, _on(gpu, stream))
    _check(st, "m2rnn_ssm_step")
    return y


class GradPlan:
    """The gradient tensors of a program, listed once for ``grad_norm`` and
    ``grad_clip``.  It holds their addresses (and keeps them alive): build a new
    one when a tensor is replaced.  Calls that share a plan must not overlap."""

    def __init__(self, grads, out=None):
        import torch
        grads = list(grads)
        outs = grads if out is None else list(out)
        if len(outs) != len(grads):
            raise ValueError(f"{len(grads)} gradients, {len(outs)} outputs")
        if not grads:
            raise ValueError("no gradients")
        self.gpu = _gpu(grads[0])
        for i, (g, o) in enumerate(zip(grads, outs)):
            for t, name in ((g, f"grads[{i}]"), (o, f"out[{i}]")):
                _need(t, name, g.shape, g.dtype, self.gpu)
        n = len(grads)
        counts = (ctypes.c_int64 * n)(*(g.numel() for g in grads))
        codes = (ctypes.c_int32 * n)(*(_dtype_code(g) for g in grads))
        ptrs = (ctypes.c_void_p * n)(*(g.data_ptr() for g in grads))
        optrs = (ctypes.c_void_p * n)(*(o.data_ptr() for o in outs))
        size = m2rnn_grad_plan_size(n, counts)
        host = torch.empty(size, dtype=torch.uint8)
        _check(m2rnn_grad_plan_build(n, ptrs, optrs, counts, codes, host.data_ptr(), size), "m2rnn_grad_plan_build")
        self.stream = _on(self.gpu, None)
        self.table = host.to(grads[0].device)
        self.workspace = self.table.new_empty(m2rnn_grad_workspace_size())
        self.grads, self.outs = grads, outs


def grad_plan(grads, out=None) -> GradPlan:
    """Lists gradient tensors (contiguous, bf16 or fp32) for ``grad_clip``;
    ``out``: where the clipped ones go (None = in place)."""
    return GradPlan(grads, out)


def _keep(plan, stream, handle):
    """Tells the allocator that another stream than the plan's own uses its
    buffers, which the caller does not see."""
    import torch
    if handle != plan.stream:
        used = stream if stream is not None else torch.cuda.current_stream(plan.gpu)
        plan.table.record_stream(used)
        plan.workspace.record_stream(used)


def _norm(plan, norm, stream):
    """The one fp32 number that the calls write."""
    import torch
    if norm is None:
        return _alloc(plan.table, (), torch.float32, stream)
    if norm.dtype is not torch.float32 or norm.numel() != 1 or norm.get_device() != plan.gpu:
        raise ValueError(f"norm: expected one torch.float32 on cuda:{plan.gpu}, got {norm.numel()} {norm.dtype} on "
                         f"{norm.device}")
    return norm


def grad_norm(plan: GradPlan, *, norm=None, stream=None):
    """Global norm of the plan's tensors: a 0-dim fp32 tensor on the device."""
    _current(plan.gpu)
    norm = _norm(plan, norm, stream)
    handle = _on(plan.gpu, stream)
    st = load().m2rnn_grad_norm(plan.table.data_ptr(), plan.table.numel(), norm.data_ptr(), plan.workspace.data_ptr(),
                                plan.workspace.numel(), handle)
    _check(st, "m2rnn_grad_norm")
    _keep(plan, stream, handle)
    return norm


def grad_clip(plan: GradPlan, max_norm: float, *, norm=None, stream=None):
    """Scales the plan's tensors by min(1, max_norm / (norm + 1e-6)) into its
    outputs.  Returns the norm before clipping, a 0-dim fp32 tensor."""
    _current(plan.gpu)
    norm = _norm(plan, norm, stream)
    handle = _on(plan.gpu, stream)
    st = load().m2rnn_grad_clip(plan.table.data_ptr(), plan.table.numel(), float(max_norm), norm.data_ptr(),
                                plan.workspace.data_ptr(), plan.workspace.numel(), handle)
    _check(st, "m2rnn_grad_clip")
    _keep(plan, stream, handle)
    return norm
