"""ctypes binding of libpararnn_b200 -- argument marshalling only.

The ``pararnn_*`` functions here have the names and argument order of the C
ABI in ``include/pararnn_b200.h``; pointer arguments accept a torch tensor
(its ``data_ptr()``), an int address, or None (NULL).  ``stream`` accepts a
``torch.cuda.Stream``, an int handle or None (the legacy default stream).

Above them, :func:`newton_forward` and :func:`newton_backward` allocate the
outputs and the workspace with torch (device memory is torch's job here) and
raise :class:`PararnnError` on a non-OK status.  Every step of the
computation runs in the library's CUDA kernels; nothing here computes.  If
the library cannot be loaded, this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

LINEAR, DIAG_GRU, DIAG_LSTM = 0, 1, 2
F32, BF16 = 0, 1
CELLS = {"linear": LINEAR, "diag_gru": DIAG_GRU, "diag_lstm": DIAG_LSTM}
STATUS = {0: "PARARNN_OK", 1: "PARARNN_EINVAL", 2: "PARARNN_ENONFINITE", 3: "PARARNN_ETIMEOUT", 4: "PARARNN_ECUDA"}
OK, EINVAL, ENONFINITE, ETIMEOUT, ECUDA = 0, 1, 2, 3, 4

# every exported symbol of include/pararnn_b200.h, with its C signature
_P, _I64, _I, _SZ, _U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
_F = ctypes.c_float
SIGNATURES = {
    "pararnn_num_gates": (_I, [_I]),
    "pararnn_state_width": (_I, [_I]),
    "pararnn_workspace_bytes": (_SZ, [_I, _I64, _I64, _I64, _I]),
    "pararnn_kstar": (_I, [_I, _I64]),
    "pararnn_newton_forward": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P, _SZ, _P, _P]),
    "pararnn_newton_forward_picard": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _I, _I, _P, _P, _SZ, _P, _P]),
    "pararnn_unroll": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_newton_backward": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_status_sync": (_I, [_P, _P]),
    "pararnn_status_string": (ctypes.c_char_p, [_I]),
    "pararnn_last_error": (ctypes.c_char_p, []),
    "pararnn_probe_wait_timeout": (_I, [_P, _SZ, _U64, _P]),
    "pararnn_debug_hooks": (_I, [_U64, _I]),
    "pararnn_newton_forward_noalloc": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P, _I, _P]),
    "pararnn_newton_forward_host_workspace_bytes": (_SZ, [_I, _I64, _I64, _I64, _I, _I, _I64, _I64]),
    "pararnn_newton_forward_host": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P, _SZ, _I64, _I64, _P]),
    "pararnn_newton_step_host_workspace_bytes": (_SZ, [_I, _I64, _I64, _I64, _I, _I, _I64]),
    "pararnn_newton_step_host": (_I, [_I, _I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _SZ, _I64, _P]),
    "pararnn_head_gru_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "pararnn_head_gru_forward": (_I, [_I64, _I64, _I64, _I, _I, _P, _P, _P, _I, _P, _P, _SZ, _P, _P]),
    "pararnn_head_gru_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "pararnn_head_gru_backward": (_I, [_I64, _I64, _I64, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_head_gru_unroll": (_I, [_I64, _I64, _I64, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_gated_scan_checkpoint_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "pararnn_gated_scan_forward": (_I, [_I64, _I64, _I64, _I, _P, _P, _F, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_gated_scan_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "pararnn_gated_scan_backward": (_I, [_I64, _I64, _I64, _I, _P, _P, _F, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_gated_scan_step": (_I, [_I64, _I64, _I, _P, _P, _F, _I64, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_layer_norm_forward": (_I, [_I64, _I64, _I64, _I, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P]),
    "pararnn_layer_norm_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "pararnn_layer_norm_backward": (_I, [_I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
}

_lib = None


class PararnnError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = "%s returned %s" % (where, STATUS.get(status, status))
        if detail:
            msg += ": " + detail
        super().__init__(msg)


def load(path: str | None = None):
    """Load (building first if missing or stale) the in-tree library."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    so = path or _build.build()
    if not os.path.exists(so):
        raise RuntimeError("libpararnn_b200.so not found at %s" % so)
    lib = ctypes.CDLL(so)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ---- the C ABI, one to one -------------------------------------------------

def pararnn_num_gates(cell):
    return load().pararnn_num_gates(cell)


def pararnn_state_width(cell):
    return load().pararnn_state_width(cell)


def pararnn_workspace_bytes(cell, B, T, D, K):
    return load().pararnn_workspace_bytes(cell, B, T, D, K)


def pararnn_newton_forward(cell, B, T, D, px_dtype, preacts, diag_w, h0, K, H_out, workspace, ws_bytes,
                           resid_hist, stream):
    return load().pararnn_newton_forward(cell, B, T, D, px_dtype, _ptr(preacts), _ptr(diag_w), _ptr(h0), K,
                                         _ptr(H_out), _ptr(workspace), ws_bytes, _ptr(resid_hist), _stream(stream))


def pararnn_kstar(cell, T):
    return load().pararnn_kstar(cell, T)


def pararnn_newton_forward_picard(cell, B, T, D, px_dtype, preacts, diag_w, h0, picard_iters, K, H_out, workspace,
                                  ws_bytes, resid_hist, stream):
    return load().pararnn_newton_forward_picard(cell, B, T, D, px_dtype, _ptr(preacts), _ptr(diag_w), _ptr(h0),
                                                picard_iters, K, _ptr(H_out), _ptr(workspace), ws_bytes,
                                                _ptr(resid_hist), _stream(stream))


def pararnn_unroll(cell, B, T, D, px_dtype, preacts, diag_w, h0, H_out, workspace, ws_bytes, stream):
    return load().pararnn_unroll(cell, B, T, D, px_dtype, _ptr(preacts), _ptr(diag_w), _ptr(h0), _ptr(H_out),
                                 _ptr(workspace), ws_bytes, _stream(stream))


def pararnn_newton_backward(cell, B, T, D, px_dtype, preacts, diag_w, h0, H, dL_dH, dL_dpx, dL_da, dL_dh0,
                            workspace, ws_bytes, stream):
    return load().pararnn_newton_backward(cell, B, T, D, px_dtype, _ptr(preacts), _ptr(diag_w), _ptr(h0), _ptr(H),
                                          _ptr(dL_dH), _ptr(dL_dpx), _ptr(dL_da), _ptr(dL_dh0), _ptr(workspace),
                                          ws_bytes, _stream(stream))


def pararnn_status_sync(workspace, stream):
    return load().pararnn_status_sync(_ptr(workspace), _stream(stream))


def pararnn_status_string(status):
    return load().pararnn_status_string(status).decode()


def pararnn_last_error():
    return load().pararnn_last_error().decode()


def pararnn_probe_wait_timeout(workspace, ws_bytes, timeout_ns, stream):
    return load().pararnn_probe_wait_timeout(_ptr(workspace), ws_bytes, timeout_ns, _stream(stream))


def pararnn_debug_hooks(wait_limit_ns, stall_first_tile):
    return load().pararnn_debug_hooks(wait_limit_ns, int(stall_first_tile))


def pararnn_newton_forward_noalloc(cell, B, T, D, px_dtype, preacts, diag_w, h0, K, H_out, resid_hist, wait_status,
                                   stream):
    return load().pararnn_newton_forward_noalloc(cell, B, T, D, px_dtype, _ptr(preacts), _ptr(diag_w), _ptr(h0), K,
                                                 _ptr(H_out), _ptr(resid_hist), int(wait_status), _stream(stream))


def pararnn_newton_forward_host_workspace_bytes(cell, B, T, D, K, px_dtype, rows_per_slice, channels_per_slice=0):
    return load().pararnn_newton_forward_host_workspace_bytes(cell, B, T, D, K, px_dtype, rows_per_slice,
                                                              channels_per_slice)


def pararnn_newton_forward_host(cell, B, T, D, px_dtype, preacts_host, diag_w, h0, K, H_host, workspace, ws_bytes,
                                rows_per_slice, channels_per_slice, stream):
    return load().pararnn_newton_forward_host(cell, B, T, D, px_dtype, _ptr(preacts_host), _ptr(diag_w), _ptr(h0), K,
                                              _ptr(H_host), _ptr(workspace), ws_bytes, rows_per_slice,
                                              channels_per_slice, _stream(stream))


def pararnn_newton_step_host_workspace_bytes(cell, B, T, D, K, px_dtype, channels_per_slice=0):
    return load().pararnn_newton_step_host_workspace_bytes(cell, B, T, D, K, px_dtype, channels_per_slice)


def pararnn_newton_step_host(cell, B, T, D, px_dtype, preacts_host, diag_w, h0, K, dL_dH_host, H_host, dL_dpx_host,
                             dL_da, workspace, ws_bytes, channels_per_slice, stream):
    return load().pararnn_newton_step_host(cell, B, T, D, px_dtype, _ptr(preacts_host), _ptr(diag_w), _ptr(h0), K,
                                           _ptr(dL_dH_host), _ptr(H_host), _ptr(dL_dpx_host), _ptr(dL_da),
                                           _ptr(workspace), ws_bytes, channels_per_slice, _stream(stream))


def pararnn_head_gru_workspace_bytes(B, T, D, n_heads, K):
    return load().pararnn_head_gru_workspace_bytes(B, T, D, n_heads, K)


def pararnn_head_gru_forward(B, T, D, n_heads, px_dtype, preacts, U, h0, K, H_out, workspace, ws_bytes, resid_hist,
                             stream):
    return load().pararnn_head_gru_forward(B, T, D, n_heads, px_dtype, _ptr(preacts), _ptr(U), _ptr(h0), K,
                                           _ptr(H_out), _ptr(workspace), ws_bytes, _ptr(resid_hist),
                                           _stream(stream))


def pararnn_head_gru_backward_workspace_bytes(B, T, D, n_heads):
    return load().pararnn_head_gru_backward_workspace_bytes(B, T, D, n_heads)


def pararnn_head_gru_backward(B, T, D, n_heads, px_dtype, preacts, U, h0, H, dL_dH, dL_dpx, dL_dU, dL_dh0, workspace,
                              ws_bytes, stream):
    return load().pararnn_head_gru_backward(B, T, D, n_heads, px_dtype, _ptr(preacts), _ptr(U), _ptr(h0), _ptr(H),
                                            _ptr(dL_dH), _ptr(dL_dpx), _ptr(dL_dU), _ptr(dL_dh0), _ptr(workspace),
                                            ws_bytes, _stream(stream))


def pararnn_head_gru_unroll(B, T, D, n_heads, px_dtype, preacts, U, h0, H_out, workspace, ws_bytes, stream):
    return load().pararnn_head_gru_unroll(B, T, D, n_heads, px_dtype, _ptr(preacts), _ptr(U), _ptr(h0), _ptr(H_out),
                                          _ptr(workspace), ws_bytes, _stream(stream))


def pararnn_gated_scan_checkpoint_bytes(B, T, D, dtype):
    return load().pararnn_gated_scan_checkpoint_bytes(B, T, D, dtype)


def pararnn_gated_scan_forward(B, T, D, dtype, preacts, lam, decay, h0, reset, H_out, h_last, checkpoints, workspace,
                               ws_bytes, stream):
    return load().pararnn_gated_scan_forward(B, T, D, dtype, _ptr(preacts), _ptr(lam), decay, _ptr(h0), _ptr(reset),
                                             _ptr(H_out), _ptr(h_last), _ptr(checkpoints), _ptr(workspace), ws_bytes,
                                             _stream(stream))


def pararnn_gated_scan_workspace_bytes(B, T, D):
    return load().pararnn_gated_scan_workspace_bytes(B, T, D)


def pararnn_gated_scan_backward(B, T, D, dtype, preacts, lam, decay, reset, checkpoints, dL_dH, dL_dh_last, dL_dpx,
                                dL_dlam, dL_dh0, workspace, ws_bytes, stream):
    return load().pararnn_gated_scan_backward(B, T, D, dtype, _ptr(preacts), _ptr(lam), decay, _ptr(reset),
                                              _ptr(checkpoints), _ptr(dL_dH), _ptr(dL_dh_last), _ptr(dL_dpx),
                                              _ptr(dL_dlam), _ptr(dL_dh0), _ptr(workspace), ws_bytes, _stream(stream))


def pararnn_gated_scan_step(N, D, dtype, preacts, lam, decay, n_slots, slots, state, y, workspace, ws_bytes, stream):
    return load().pararnn_gated_scan_step(N, D, dtype, _ptr(preacts), _ptr(lam), decay, n_slots, _ptr(slots),
                                          _ptr(state), _ptr(y), _ptr(workspace), ws_bytes, _stream(stream))


def pararnn_layer_norm_forward(M, P, N, dtype, x, weight, bias, eps, y, mean, rstd, workspace, ws_bytes, stream):
    return load().pararnn_layer_norm_forward(M, P, N, dtype, _ptr(x), _ptr(weight), _ptr(bias), eps, _ptr(y),
                                             _ptr(mean), _ptr(rstd), _ptr(workspace), ws_bytes, _stream(stream))


def pararnn_layer_norm_workspace_bytes(M, P, N):
    return load().pararnn_layer_norm_workspace_bytes(M, P, N)


def pararnn_layer_norm_backward(M, P, N, dtype, x, weight, mean, rstd, dL_dy, dL_dx, dL_dweight, dL_dbias, workspace,
                                ws_bytes, stream):
    return load().pararnn_layer_norm_backward(M, P, N, dtype, _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd),
                                              _ptr(dL_dy), _ptr(dL_dx), _ptr(dL_dweight), _ptr(dL_dbias),
                                              _ptr(workspace), ws_bytes, _stream(stream))


# ---- tensor-level helpers (allocation through torch, compute in the library) ----

def _check(status, where):
    if status != OK:
        raise PararnnError(status, where, pararnn_last_error())


def _dtype_code(t):
    import torch

    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("pre-activations must be float32 or bfloat16, got %s" % t.dtype)


def _shape(cell, px):
    G = pararnn_num_gates(cell)
    if px.dim() != 4 or px.shape[2] != G:
        raise ValueError("preacts must be (B, T, %d, D), got %s" % (G, tuple(px.shape)))
    if not px.is_contiguous():
        raise ValueError("preacts must be contiguous")
    B, T, _, D = px.shape
    return B, T, D


def workspace_for(cell, B, T, D, K, device):
    """An uninitialised workspace: every call clears what it reads."""
    import torch

    n = pararnn_workspace_bytes(cell, B, T, D, K)
    return torch.empty(n, dtype=torch.uint8, device=device)


def newton_forward(cell, px, diag_w=None, h0=None, K=1, out=None, workspace=None, resid_hist=None, stream=None,
                   sync_status=True, picard_iters=0):
    """H = h^(K) of shape (B,T,S,D), float32, on px's device.  K=0 (or None)
    takes the measured K*(cell, T); picard_iters > 0 runs that many Picard
    sweeps before the Newton iterations."""
    import torch

    cell = CELLS.get(cell, cell)
    K = 0 if K is None else K
    B, T, D = _shape(cell, px)
    S = pararnn_state_width(cell)
    if out is None:
        out = torch.empty((B, T, S, D), dtype=torch.float32, device=px.device)
    if workspace is None:
        workspace = workspace_for(cell, B, T, D, K, px.device)
    st = stream if stream is not None else torch.cuda.current_stream(px.device)
    if picard_iters:
        _check(pararnn_newton_forward_picard(cell, B, T, D, _dtype_code(px), px, diag_w, h0, picard_iters, K, out,
                                             workspace, workspace.numel(), resid_hist, st),
               "pararnn_newton_forward_picard")
    else:
        _check(pararnn_newton_forward(cell, B, T, D, _dtype_code(px), px, diag_w, h0, K, out, workspace,
                                      workspace.numel(), resid_hist, st), "pararnn_newton_forward")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_newton_forward (device status)")
    return out


def unroll(cell, px, diag_w=None, h0=None, out=None, workspace=None, stream=None, sync_status=True):
    """The sequential recurrence on the GPU: H (B,T,S,D) float32."""
    import torch

    cell = CELLS.get(cell, cell)
    B, T, D = _shape(cell, px)
    S = pararnn_state_width(cell)
    if out is None:
        out = torch.empty((B, T, S, D), dtype=torch.float32, device=px.device)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=px.device)
    st = stream if stream is not None else torch.cuda.current_stream(px.device)
    _check(pararnn_unroll(cell, B, T, D, _dtype_code(px), px, diag_w, h0, out, workspace, workspace.numel(), st),
           "pararnn_unroll")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_unroll (device status)")
    return out


def newton_backward(cell, px, H, dL_dH, diag_w=None, h0=None, workspace=None, want_da=True, want_dh0=False,
                    stream=None, sync_status=True):
    """Returns (dL_dpx (B,T,G,D), dL_da (G,D) or None, dL_dh0 (B,S,D) or None), float32."""
    import torch

    cell = CELLS.get(cell, cell)
    B, T, D = _shape(cell, px)
    G, S = pararnn_num_gates(cell), pararnn_state_width(cell)
    dpx = torch.empty((B, T, G, D), dtype=torch.float32, device=px.device)
    da = torch.empty((G, D), dtype=torch.float32, device=px.device) if (want_da and cell != LINEAR) else None
    dh0 = torch.empty((B, S, D), dtype=torch.float32, device=px.device) if want_dh0 else None
    if workspace is None:
        workspace = workspace_for(cell, B, T, D, 1, px.device)
    st = stream if stream is not None else torch.cuda.current_stream(px.device)
    _check(pararnn_newton_backward(cell, B, T, D, _dtype_code(px), px, diag_w, h0, H, dL_dH, dpx, da, dh0,
                                   workspace, workspace.numel(), st), "pararnn_newton_backward")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_newton_backward (device status)")
    return dpx, da, dh0


def head_gru_forward(px, U, h0=None, K=1, out=None, workspace=None, resid_hist=None, stream=None, sync_status=True):
    """Head-wise GRU: px (B,T,3,D), U (3, n_heads, d, d) -> H = h^(K) (B,T,D), float32."""
    import torch

    if px.dim() != 4 or px.shape[2] != 3 or not px.is_contiguous():
        raise ValueError("preacts must be contiguous (B, T, 3, D), got %s" % (tuple(px.shape),))
    if U.dim() != 4 or U.shape[0] != 3 or U.shape[2] != U.shape[3] or not U.is_contiguous():
        raise ValueError("U must be contiguous (3, n_heads, d, d), got %s" % (tuple(U.shape),))
    B, T, _, D = px.shape
    nh = U.shape[1]
    if out is None:
        out = torch.empty((B, T, D), dtype=torch.float32, device=px.device)
    if workspace is None:
        n = pararnn_head_gru_workspace_bytes(B, T, D, nh, K)
        if n == 0:
            raise PararnnError(EINVAL, "pararnn_head_gru_workspace_bytes", "invalid sizes")
        workspace = torch.empty(n, dtype=torch.uint8, device=px.device)
    st = stream if stream is not None else torch.cuda.current_stream(px.device)
    _check(pararnn_head_gru_forward(B, T, D, nh, _dtype_code(px), px, U, h0, K, out, workspace, workspace.numel(),
                                    resid_hist, st), "pararnn_head_gru_forward")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_head_gru_forward (device status)")
    return out


def head_gru_backward(px, U, H, dL_dH, h0=None, want_dU=True, want_dh0=False, workspace=None, stream=None,
                      sync_status=True):
    """Head-wise GRU adjoint: returns (dL/dpx (B,T,3,D), dL/dU (3,n_heads,d,d) or None, dL/dh0 (B,D) or None)."""
    import torch

    B, T, _, D = px.shape
    nh = U.shape[1]
    dpx = torch.empty((B, T, 3, D), dtype=torch.float32, device=px.device)
    dU = torch.empty(tuple(U.shape), dtype=torch.float32, device=px.device) if want_dU else None
    dh0 = torch.empty((B, D), dtype=torch.float32, device=px.device) if want_dh0 else None
    if workspace is None:
        n = pararnn_head_gru_backward_workspace_bytes(B, T, D, nh)
        if n == 0:
            raise PararnnError(EINVAL, "pararnn_head_gru_backward_workspace_bytes", "invalid sizes")
        workspace = torch.empty(n, dtype=torch.uint8, device=px.device)
    st = stream if stream is not None else torch.cuda.current_stream(px.device)
    _check(pararnn_head_gru_backward(B, T, D, nh, _dtype_code(px), px, U, h0, H, dL_dH, dpx, dU, dh0, workspace,
                                     workspace.numel(), st), "pararnn_head_gru_backward")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_head_gru_backward (device status)")
    return dpx, dU, dh0


def head_gru_unroll(px, U, h0=None, out=None, workspace=None, stream=None, sync_status=True):
    """Head-wise GRU, sequential unroll on the GPU: px (B,T,3,D), U (3,n_heads,d,d) -> H (B,T,D), float32."""
    import torch

    if px.dim() != 4 or px.shape[2] != 3 or not px.is_contiguous():
        raise ValueError("preacts must be contiguous (B, T, 3, D), got %s" % (tuple(px.shape),))
    B, T, _, D = px.shape
    nh = U.shape[1]
    if out is None:
        out = torch.empty((B, T, D), dtype=torch.float32, device=px.device)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=px.device)
    st = stream if stream is not None else torch.cuda.current_stream(px.device)
    _check(pararnn_head_gru_unroll(B, T, D, nh, _dtype_code(px), px, U, h0, out, workspace, workspace.numel(), st),
           "pararnn_head_gru_unroll")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_head_gru_unroll (device status)")
    return out


def newton_forward_host(cell, px_host, diag_w=None, h0=None, K=1, out_host=None, rows_per_slice=1,
                        channels_per_slice=0, workspace=None, stream=None, sync_status=True):
    """The forward on host tensors (pinned for overlap): H (B,T,S,D) float32 on the host."""
    import torch

    cell = CELLS.get(cell, cell)
    B, T, D = _shape(cell, px_host)
    S = pararnn_state_width(cell)
    code = _dtype_code(px_host)
    if out_host is None:
        out_host = torch.empty((B, T, S, D), dtype=torch.float32, pin_memory=px_host.is_pinned())
    dev = diag_w.device if diag_w is not None else torch.device("cuda", torch.cuda.current_device())
    if workspace is None:
        n = pararnn_newton_forward_host_workspace_bytes(cell, B, T, D, K, code, rows_per_slice, channels_per_slice)
        if n == 0:
            raise PararnnError(EINVAL, "pararnn_newton_forward_host_workspace_bytes", "invalid arguments")
        workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(pararnn_newton_forward_host(cell, B, T, D, code, px_host, diag_w, h0, K, out_host, workspace,
                                       workspace.numel(), rows_per_slice, channels_per_slice, st),
           "pararnn_newton_forward_host")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_newton_forward_host (device status)")
    return out_host


def newton_step_host(cell, px_host, dL_dH_host, diag_w=None, h0=None, K=1, channels_per_slice=0, outs=None,
                     workspace=None, stream=None, sync_status=True):
    """Forward + adjoint on host tensors (pinned for overlap): returns
    (H, dL/dpx) on the host and dL/da (G, D) on the device (None for the
    linear cell)."""
    import torch

    cell = CELLS.get(cell, cell)
    B, T, D = _shape(cell, px_host)
    S, G = pararnn_state_width(cell), pararnn_num_gates(cell)
    code = _dtype_code(px_host)
    dev = diag_w.device if diag_w is not None else torch.device("cuda", torch.cuda.current_device())
    if outs is None:
        pin = px_host.is_pinned()
        outs = (torch.empty((B, T, S, D), dtype=torch.float32, pin_memory=pin),
                torch.empty((B, T, G, D), dtype=torch.float32, pin_memory=pin),
                None if cell == LINEAR else torch.empty((G, D), dtype=torch.float32, device=dev))
    H_host, dpx_host, da = outs
    if workspace is None:
        n = pararnn_newton_step_host_workspace_bytes(cell, B, T, D, K, code, channels_per_slice)
        if n == 0:
            raise PararnnError(EINVAL, "pararnn_newton_step_host_workspace_bytes", "invalid arguments")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(pararnn_newton_step_host(cell, B, T, D, code, px_host, diag_w, h0, K, dL_dH_host, H_host, dpx_host, da,
                                    workspace, workspace.numel(), channels_per_slice, st),
           "pararnn_newton_step_host")
    if sync_status:
        _check(pararnn_status_sync(workspace, st), "pararnn_newton_step_host (device status)")
    return H_host, dpx_host, da


# ---- gated linear recurrence and layer normalisation ------------------------
# These calls are short enough that a decoding loop is bound by the host: the
# checks below read each tensor's attributes once.

def _same_device(px, *tensors):
    """Every given tensor is contiguous and on px's CUDA device, whose index is returned."""
    dev = px.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device, got %s" % px.device)
    if not px.is_contiguous():
        raise ValueError("tensors must be contiguous, got strides %s" % (px.stride(),))
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise ValueError("tensors on different devices: %s and %s" % (px.device, t.device))
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous, got strides %s" % (t.stride(),))
    return dev


def _expect(name, t, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError("%s must be %s %s, got %s %s" % (name, tuple(shape), dtype, tuple(t.shape), t.dtype))


def _launch(where, fn, dev, stream, scratch, workspace, sync_status, args):
    """fn(*args, workspace, its bytes, stream) with device `dev` current, and its
    status.  Memory in `scratch` was allocated here on torch's current stream:
    when the call runs on another stream, the allocator is told, so that it is
    not handed out again before that stream is done with it."""
    import torch

    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _launch(where, fn, dev, stream, scratch, workspace, sync_status, args)
    cur = torch.cuda.current_stream(dev)
    handle = cur.cuda_stream if stream is None else (stream if isinstance(stream, int) else stream.cuda_stream)
    if handle != cur.cuda_stream:
        ext = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
        ext.wait_stream(cur)  # the memory may still be in use by earlier work of the stream it came from
        for t in scratch:
            if t is not None:
                t.record_stream(ext)
    if workspace is None:
        status = fn(*args, None, 0, handle)
    else:
        status = fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), handle)
    if status != OK:
        _check(status, where)
    if sync_status:
        _check(pararnn_status_sync(workspace, handle), where + " (device status)")


def _header(workspace, sync_status, like):
    """The workspace of a call that needs one only to record its status."""
    import torch

    if workspace is None and sync_status:
        return torch.empty(256, dtype=torch.uint8, device=like.device)
    return workspace


def _scan_shape(px, lam, ndim):
    import torch

    shape = px.shape
    if len(shape) != ndim or shape[-2] != 3:
        raise ValueError("preacts must be (%s3, D), got %s" % ("B, T, " if ndim == 4 else "N, ", tuple(shape)))
    _expect("lam", lam, (shape[-1],), torch.float32)
    return _dtype_code(px), shape


def _mask(reset, B, T):
    import torch

    if reset is None:
        return None
    if reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    _expect("reset", reset, (B, T), torch.uint8)
    return reset


def gated_scan_forward(px, lam, decay=8.0, h0=None, reset=None, want_grad=False, out=None, h_last=None,
                       workspace=None, stream=None, sync_status=True):
    """The gated linear recurrence: px (B,T,3,D) float32 or bfloat16, lam (D),
    h0 (B,D) or None, reset (B,T) bool or uint8 or None (steps that start from
    a zero state).  Returns (H (B,T,D) in px's dtype, the last state (B,D)
    float32, the checkpoints that gated_scan_backward takes, or None without
    want_grad).  With sync_status=False the call does not wait, and its status
    is read only from a workspace that is passed: >= 256 bytes, or
    pararnn_gated_scan_workspace_bytes for the speed of few long channels."""
    import torch

    code, (B, T, _, D) = _scan_shape(px, lam, 4)
    reset = _mask(reset, B, T)
    _expect("h0", h0, (B, D), torch.float32)
    _expect("out", out, (B, T, D), px.dtype)
    _expect("h_last", h_last, (B, D), torch.float32)
    dev = _same_device(px, lam, h0, reset, out, h_last, workspace)
    H = px.new_empty((B, T, D)) if out is None else out
    last = lam.new_empty((B, D)) if h_last is None else h_last
    ck = lam.new_empty(pararnn_gated_scan_checkpoint_bytes(B, T, D, code) // 4) if want_grad else None
    ws = workspace
    if ws is None and T > 2048 and B * ((D + 63) // 64) <= 16:  # few channels: scratch to cut T into ranges
        ws = torch.empty(pararnn_gated_scan_workspace_bytes(B, T, D), dtype=torch.uint8, device=px.device)
    ws = _header(ws, sync_status, px)
    _launch("pararnn_gated_scan_forward", load().pararnn_gated_scan_forward, dev, stream, (H, last, ck, ws), ws,
            sync_status, (B, T, D, code, px.data_ptr(), lam.data_ptr(), decay, _ptr(h0), _ptr(reset), H.data_ptr(),
                          last.data_ptr(), _ptr(ck)))
    return H, last, ck


def gated_scan_backward(px, lam, checkpoints, dL_dH, decay=8.0, reset=None, dL_dh_last=None, want_dlam=True,
                        want_dh0=False, workspace=None, stream=None, sync_status=True):
    """The adjoint of gated_scan_forward called with the same px, lam, decay, h0
    and reset: returns (dL/dpx in px's dtype, dL/dlam (D) or None, dL/dh0 (B,D)
    or None), the latter two float32.  dL_dH has px's dtype."""
    import torch

    code, (B, T, _, D) = _scan_shape(px, lam, 4)
    reset = _mask(reset, B, T)
    _expect("dL_dH", dL_dH, (B, T, D), px.dtype)
    _expect("dL_dh_last", dL_dh_last, (B, D), torch.float32)
    _expect("checkpoints", checkpoints, (pararnn_gated_scan_checkpoint_bytes(B, T, D, code) // 4,), torch.float32)
    dev = _same_device(px, lam, checkpoints, dL_dH, reset, dL_dh_last, workspace)
    dpx = torch.empty_like(px)
    dlam = lam.new_empty((D,)) if want_dlam else None
    dh0 = lam.new_empty((B, D)) if want_dh0 else None
    ws = workspace
    if ws is None:
        ws = torch.empty(pararnn_gated_scan_workspace_bytes(B, T, D), dtype=torch.uint8, device=px.device)
    _launch("pararnn_gated_scan_backward", load().pararnn_gated_scan_backward, dev, stream, (dpx, dlam, dh0, ws), ws,
            sync_status, (B, T, D, code, px.data_ptr(), lam.data_ptr(), decay, _ptr(reset), checkpoints.data_ptr(),
                          dL_dH.data_ptr(), _ptr(dL_dh_last), dpx.data_ptr(), _ptr(dlam), _ptr(dh0)))
    return dpx, dlam, dh0


def gated_scan_step(px, lam, state, decay=8.0, slots=None, out=None, workspace=None, stream=None, sync_status=True):
    """One token per row: px (N,3,D), state (n_slots,D) float32, updated in place,
    slots (N) int32 or None (row n on slot n).  Returns y (N,D) in px's dtype; the
    rows of padding (slot < 0) keep what `out` held (zeros if it is not given).
    Rows that name one slot are taken in order."""
    import torch

    code, (N, _, D) = _scan_shape(px, lam, 3)
    if state.dim() != 2:
        raise ValueError("state must be (n_slots, D), got %s" % (tuple(state.shape),))
    n_slots = state.shape[0]
    _expect("state", state, (n_slots, D), torch.float32)
    _expect("slots", slots, (N,), torch.int32)
    _expect("out", out, (N, D), px.dtype)
    dev = _same_device(px, lam, state, slots, out, workspace)
    y = out
    if y is None:
        y = px.new_empty((N, D)) if slots is None else px.new_zeros((N, D))
    ws = _header(workspace, sync_status, px)
    _launch("pararnn_gated_scan_step", load().pararnn_gated_scan_step, dev, stream, (y, ws), ws, sync_status,
            (N, D, code, px.data_ptr(), lam.data_ptr(), decay, n_slots, _ptr(slots), state.data_ptr(), y.data_ptr()))
    return y


def _norm_shape(x, shape, *params):
    """(M, P, N) of x for scales of `shape`, (N,) or (P..., N): x's last dimensions."""
    import torch

    full, n = x.shape, len(shape)
    if not full or full[-1] == 0:
        raise ValueError("x must have at least one value in its last dimension, got %s" % (tuple(full),))
    if not 1 <= n <= len(full) or full[len(full) - n:] != shape or 0 in shape:
        raise ValueError("weight and bias must have the shape of x's last dimensions, got %s for %s"
                         % (tuple(shape), tuple(full)))
    for t in params:
        _expect("weight and bias", t, shape, torch.float32)
    P, N = 1, shape[-1]
    for k in shape[:-1]:
        P *= k
    return x.numel() // (P * N), P, N


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, want_stats=False, out=None, workspace=None, stream=None,
                       sync_status=True):
    """Layer normalisation over x's last dimension, x float32 or bfloat16.
    weight and bias (float32) are (N,), or (P, N) and so on for a scale of each
    gate or head: the shape of x's last dimensions.  Returns (y in x's dtype,
    mean, rstd); mean and rstd (float32, None without want_stats) are what
    layer_norm_backward takes."""
    import torch

    code = _dtype_code(x)
    like = weight if weight is not None else bias
    M, P, N = _norm_shape(x, x.shape[-1:] if like is None else like.shape, weight, bias)
    _expect("out", out, x.shape, x.dtype)
    dev = _same_device(x, weight, bias, out, workspace)
    y = torch.empty_like(x) if out is None else out
    mean = rstd = None
    if want_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    ws = _header(workspace, sync_status, x)
    _launch("pararnn_layer_norm_forward", load().pararnn_layer_norm_forward, dev, stream, (y, mean, rstd, ws), ws,
            sync_status, (M, P, N, code, x.data_ptr(), _ptr(weight), _ptr(bias), eps, y.data_ptr(), _ptr(mean),
                          _ptr(rstd)))
    return y, mean, rstd


def layer_norm_backward(x, dL_dy, mean, rstd, weight=None, param_shape=None, want_dparams=True, workspace=None,
                        stream=None, sync_status=True):
    """The gradients of layer_norm_forward: (dL/dx in x's dtype, dL/dweight,
    dL/dbias), the latter two float32 in weight's shape (param_shape without a
    weight, (N,) if that is not given either), or None without want_dparams."""
    import torch

    code = _dtype_code(x)
    shape = weight.shape if weight is not None else torch.Size(param_shape) if param_shape is not None else x.shape[-1:]
    M, P, N = _norm_shape(x, shape, weight)
    _expect("dL_dy", dL_dy, x.shape, x.dtype)
    _expect("mean", mean, x.shape[:-1], torch.float32)
    _expect("rstd", rstd, x.shape[:-1], torch.float32)
    dev = _same_device(x, dL_dy, mean, rstd, weight, workspace)
    dx = torch.empty_like(x)
    dw = torch.empty(shape, dtype=torch.float32, device=x.device) if want_dparams else None
    db = torch.empty_like(dw) if want_dparams else None
    ws = workspace
    if ws is None:
        ws = torch.empty(pararnn_layer_norm_workspace_bytes(M, P, N), dtype=torch.uint8, device=x.device)
    _launch("pararnn_layer_norm_backward", load().pararnn_layer_norm_backward, dev, stream, (dx, dw, db, ws), ws,
            sync_status, (M, P, N, code, x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(),
                          dL_dy.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db)))
    return dx, dw, db
