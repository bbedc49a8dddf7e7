"""Thin ctypes binding over libgdn.so (``include/gdn.h``).

Argument marshalling only: every step of the recurrence runs in the
library's CUDA kernels.  Functions with the C names take torch CUDA tensors
(or raw integer device pointers) for every buffer, pass ``data_ptr()`` and the
current torch stream, and raise ``GDNError`` on a negative status.  There is
no CPU fallback: if the library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_ALIGNMENT = -3
GDN_ERR_CUDA = -4
GDN_ERR_TIMEOUT = -5
GDN_ERR_WORKSPACE = -6
GDN_ERR_DEVICE_BOUNDS = -7
GDN_WARN_ZERO_STATE = 1
GDN_WARN_NOT_CONVERGED = 2
GDN_WARN_RANK_DEFICIENT = 3

GDN_BF16 = 0
GDN_FP32 = 1

GDN_GATE_SCALAR = 0
GDN_GATE_KDA = 1
GDN_GATE_GDN2 = 2
GATES = {"gdn": GDN_GATE_SCALAR, "kda": GDN_GATE_KDA, "gdn2": GDN_GATE_GDN2}

GDN_NORM_RMS = 0
GDN_NORM_L2 = 1
NORMS = {"rms": GDN_NORM_RMS, "l2": GDN_NORM_L2}
GDN_PAIR_HALF = 0
GDN_PAIR_ADJACENT = 1
PAIRINGS = {"half": GDN_PAIR_HALF, "adjacent": GDN_PAIR_ADJACENT}

GDN_SCAN_DECAY = 0
GDN_SCAN_SIGMOID = 1
SCANS = {"decay": GDN_SCAN_DECAY, "sigmoid": GDN_SCAN_SIGMOID}
GDN_SCAN_BLOCK = 64  # tokens between the states that a scan keeps

GDN_SELFTEST_SCAN = 0
GDN_SELFTEST_SCAN_BACKWARD = 1
GDN_SELFTEST_NORM = 2
GDN_SELFTEST_NORM_SUM = 3
GDN_SELFTEST_NORM_ANSWER = 4
GDN_SELFTEST_NORM_BACKWARD = 5

EXPORTS = (
    "gdn_prefill",
    "gdn_prefill_workspace_size",
    "gdn_prefill_two_pass_workspace_size",
    "gdn_decode_step",
    "gdn_state_rank",
    "gdn_get_last_device_status",
    "gdn_status_string",
    "gdn_version",
    "gdn_selftest_wait_timeout",
    "gdn_selftest_lost_copy",
    "gdn_prefill_noalloc",
    "gdn_prefill_noalloc_max_workspace",
    "gdn_gather_normalize",
    "gdn_decode_step_gathered",
    "gdn_prefill_gated",
    "gdn_decode_step_gated",
    "gdn_state_truncate",
    "gdn_prefill_truncated",
    "gdn_channel_gram_workspace_size",
    "gdn_channel_gram",
    "gdn_drrqr_select",
    "gdn_prefill_host_workspace_size",
    "gdn_prefill_host",
    "gdn_prefill_gathered",
    "gdn_prefill_gathered_workspace_size",
    "gdn_prefill_gated_chunked",
    "gdn_prefill_gated_chunked_workspace_size",
    "gdn_qk_norm_rotate",
    "gdn_qk_norm_rotate_backward",
    "gdn_qk_norm_rotate_backward_workspace_size",
    "gdn_linear_prefill",
    "gdn_linear_prefill_workspace_size",
    "gdn_linear_backward",
    "gdn_linear_backward_workspace_size",
    "gdn_linear_decode_step",
    "gdn_scan_prefill",
    "gdn_scan_prefill_workspace_size",
    "gdn_scan_backward",
    "gdn_scan_backward_workspace_size",
    "gdn_scan_decode_step",
    "gdn_layer_norm",
    "gdn_layer_norm_backward",
    "gdn_layer_norm_backward_workspace_size",
)

_lock = threading.Lock()
_lib = None


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (built by ``gated_delta_rule_49_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"libgdn.so is not built ({path} missing): run "
                "`python -m gated_delta_rule_49_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(path)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.gdn_prefill.argtypes = [vp] * 8 + [i] * 6 + [vp, sz, vp]
        lib.gdn_prefill.restype = i
        lib.gdn_prefill_workspace_size.argtypes = [i] * 6
        lib.gdn_prefill_workspace_size.restype = sz
        lib.gdn_prefill_two_pass_workspace_size.argtypes = [i] * 6
        lib.gdn_prefill_two_pass_workspace_size.restype = sz
        lib.gdn_decode_step.argtypes = [vp] * 7 + [i] * 5 + [vp]
        lib.gdn_decode_step.restype = i
        lib.gdn_state_rank.argtypes = [vp, i, i, i, vp, vp, vp, i, f, vp]
        lib.gdn_state_rank.restype = i
        lib.gdn_get_last_device_status.argtypes = [vp]
        lib.gdn_get_last_device_status.restype = i
        lib.gdn_status_string.argtypes = [i]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_version.argtypes = []
        lib.gdn_version.restype = i
        lib.gdn_selftest_wait_timeout.argtypes = [ctypes.c_longlong, vp]
        lib.gdn_selftest_wait_timeout.restype = i
        lib.gdn_selftest_lost_copy.argtypes = [i] + [ctypes.c_longlong] * 2 + [vp, sz, i, i, i, vp]
        lib.gdn_selftest_lost_copy.restype = i
        lib.gdn_prefill_noalloc.argtypes = [vp] * 8 + [i] * 6 + [vp]
        lib.gdn_prefill_noalloc.restype = i
        lib.gdn_gather_normalize.argtypes = [vp, vp, vp, ctypes.c_longlong, i, i, i, i, vp]
        lib.gdn_gather_normalize.restype = i
        lib.gdn_decode_step_gathered.argtypes = [vp, vp, vp, i] + [vp] * 5 + [i] * 5 + [vp]
        lib.gdn_decode_step_gathered.restype = i
        lib.gdn_prefill_gated.argtypes = [vp] * 10 + [i] * 7 + [vp]
        lib.gdn_prefill_gated.restype = i
        lib.gdn_prefill_gated_chunked.argtypes = [vp] * 10 + [i] * 7 + [vp, sz, vp]
        lib.gdn_prefill_gated_chunked.restype = i
        lib.gdn_prefill_gated_chunked_workspace_size.argtypes = [i] * 7
        lib.gdn_prefill_gated_chunked_workspace_size.restype = sz
        lib.gdn_decode_step_gated.argtypes = [vp] * 9 + [i] * 6 + [vp]
        lib.gdn_decode_step_gated.restype = i
        lib.gdn_state_truncate.argtypes = [vp, i, i, i, i, vp, i, vp]
        lib.gdn_state_truncate.restype = i
        lib.gdn_prefill_truncated.argtypes = [vp] * 8 + [i] * 9 + [vp, sz, vp]
        lib.gdn_prefill_truncated.restype = i
        lib.gdn_channel_gram_workspace_size.argtypes = [i] * 4
        lib.gdn_channel_gram_workspace_size.restype = sz
        lib.gdn_channel_gram.argtypes = [vp, vp] + [i] * 5 + [vp, vp, sz, vp]
        lib.gdn_channel_gram.restype = i
        lib.gdn_drrqr_select.argtypes = [vp, i, i, i, f, i, vp, vp, vp, vp]
        lib.gdn_drrqr_select.restype = i
        lib.gdn_prefill_host_workspace_size.argtypes = [i] * 7
        lib.gdn_prefill_host_workspace_size.restype = sz
        lib.gdn_prefill_host.argtypes = [vp] * 8 + [i] * 7 + [vp, sz, vp]
        lib.gdn_prefill_host.restype = i
        lib.gdn_prefill_noalloc_max_workspace.argtypes = []
        lib.gdn_prefill_noalloc_max_workspace.restype = sz
        lib.gdn_prefill_gathered.argtypes = [vp, vp, vp, i] + [vp] * 6 + [i] * 6 + [vp, sz, vp]
        lib.gdn_prefill_gathered.restype = i
        lib.gdn_prefill_gathered_workspace_size.argtypes = [i] * 7
        lib.gdn_prefill_gathered_workspace_size.restype = sz
        ll = ctypes.c_longlong
        lib.gdn_qk_norm_rotate.argtypes = [vp] * 8 + [ll] + [i] * 4 + [ll] * 2 + [i, i, f, i, vp]
        lib.gdn_qk_norm_rotate.restype = i
        lib.gdn_qk_norm_rotate_backward.argtypes = (
            [vp] * 12 + [ll] + [i] * 4 + [ll] * 2 + [i, i, f, i, vp, sz, vp])
        lib.gdn_qk_norm_rotate_backward.restype = i
        lib.gdn_qk_norm_rotate_backward_workspace_size.argtypes = [ll, i, i, i]
        lib.gdn_qk_norm_rotate_backward_workspace_size.restype = sz
        lib.gdn_linear_prefill.argtypes = [vp] * 8 + [i] * 6 + [ll] * 3 + [f, i, vp, sz, vp]
        lib.gdn_linear_prefill.restype = i
        lib.gdn_linear_prefill_workspace_size.argtypes = [i] * 7
        lib.gdn_linear_prefill_workspace_size.restype = sz
        lib.gdn_linear_backward.argtypes = [vp] * 12 + [i] * 6 + [ll] * 3 + [f, i, vp, sz, vp]
        lib.gdn_linear_backward.restype = i
        lib.gdn_linear_backward_workspace_size.argtypes = [i] * 8
        lib.gdn_linear_backward_workspace_size.restype = sz
        lib.gdn_linear_decode_step.argtypes = [vp] * 7 + [i] * 5 + [f, i, vp]
        lib.gdn_linear_decode_step.restype = i
        lib.gdn_scan_prefill.argtypes = [vp] * 7 + [i] * 3 + [ll] * 2 + [i, i, vp, sz, vp]
        lib.gdn_scan_prefill.restype = i
        lib.gdn_scan_prefill_workspace_size.argtypes = [i] * 4
        lib.gdn_scan_prefill_workspace_size.restype = sz
        lib.gdn_scan_backward.argtypes = [vp] * 10 + [i] * 3 + [ll] * 2 + [i, i, vp, sz, vp]
        lib.gdn_scan_backward.restype = i
        lib.gdn_scan_backward_workspace_size.argtypes = [i] * 5
        lib.gdn_scan_backward_workspace_size.restype = sz
        lib.gdn_scan_decode_step.argtypes = [vp] * 5 + [i] * 2 + [ll] * 2 + [i, i, vp]
        lib.gdn_scan_decode_step.restype = i
        lib.gdn_layer_norm.argtypes = [vp] * 7 + [ll, i, ll, ll, f, i, vp]
        lib.gdn_layer_norm.restype = i
        lib.gdn_layer_norm_backward.argtypes = [vp] * 8 + [ll, i, ll, i, vp, sz, vp]
        lib.gdn_layer_norm_backward.restype = i
        lib.gdn_layer_norm_backward_workspace_size.argtypes = [ll, i]
        lib.gdn_layer_norm_backward_workspace_size.restype = sz
        _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load().gdn_status_string(int(status)).decode()
    except RuntimeError:
        return "libgdn.so not loaded"


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _stream(stream):
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", None)
            if get and device:  # a tenth of the time of a Stream object
                _raw_stream = lambda: get(device())  # noqa: E731
            else:
                _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# A call may be given another stream than torch's current one, where torch's
# allocator takes memory that is let go of for free at once: scratch memory comes
# from the other stream's pool, and new outputs, which belong to the caller's
# stream, are kept until the other stream is done with them.

def _other_stream(stream):
    """The torch stream of `stream` where it is not the current one, else None."""
    if stream is None:
        return None
    handle = _stream(stream)
    if handle == _stream(None):
        return None
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _scratch(need, device, stream):
    """`need` bytes of device memory for a call on the stream; None for 0."""
    if not need:
        return None
    import torch
    other = _other_stream(stream)
    if other is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    with torch.cuda.stream(other):
        return torch.empty(need, dtype=torch.uint8, device=device)


def _written_on(stream, *new):
    """Keeps what a call on the stream writes to (tensors or None) until it is written."""
    if stream is None:
        return
    other = _other_stream(stream)
    if other is not None:
        for x in new:
            if x is not None:
                x.record_stream(other)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_FP32
    raise GDNError(GDN_ERR_INVALID_ARG, f"dtype {t.dtype}")


def _check(status: int, where: str) -> int:
    if status < 0:
        raise GDNError(status, where)
    return status


def gdn_prefill(q, k, v, alpha, beta, S0, o, S_T, B, T, H, K, V, dtype, workspace=None,
                workspace_bytes=0, stream=None) -> int:
    st = load().gdn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                            _ptr(o), _ptr(S_T), B, T, H, K, V, dtype, _ptr(workspace),
                            workspace_bytes, _stream(stream))
    return _check(st, "gdn_prefill")


def gdn_prefill_noalloc(q, k, v, alpha, beta, S0, o, S_T, B, T, H, K, V, dtype,
                        stream=None) -> int:
    """gdn_prefill without a workspace argument: its scratch is a fixed array
    inside the library (for callers that cannot allocate device memory)."""
    st = load().gdn_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                                    _ptr(o), _ptr(S_T), B, T, H, K, V, dtype, _stream(stream))
    return _check(st, "gdn_prefill_noalloc")


def gdn_prefill_noalloc_max_workspace() -> int:
    return int(load().gdn_prefill_noalloc_max_workspace())


def gdn_prefill_workspace_size(B, T, H, K, V, dtype) -> int:
    return int(load().gdn_prefill_workspace_size(B, T, H, K, V, dtype))


def gdn_prefill_two_pass_workspace_size(B, T, H, K, V, dtype) -> int:
    return int(load().gdn_prefill_two_pass_workspace_size(B, T, H, K, V, dtype))


def gdn_decode_step(q, k, v, alpha, beta, S, o, B, H, K, V, dtype, stream=None) -> int:
    st = load().gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S),
                                _ptr(o), B, H, K, V, dtype, _stream(stream))
    return _check(st, "gdn_decode_step")


def gdn_state_rank(S, BH, V, K, fro2, sigma1, stable_rank, max_iter=500, tol=1e-7,
                   stream=None) -> int:
    st = load().gdn_state_rank(_ptr(S), BH, V, K, _ptr(fro2), _ptr(sigma1), _ptr(stable_rank),
                               max_iter, tol, _stream(stream))
    return _check(st, "gdn_state_rank")


def gdn_gather_normalize(x, idx, y, N, H, K_in, K_out, dtype, stream=None) -> int:
    st = load().gdn_gather_normalize(_ptr(x), _ptr(idx), _ptr(y), N, H, K_in, K_out, dtype,
                                     _stream(stream))
    return _check(st, "gdn_gather_normalize")


def gdn_decode_step_gathered(q_full, k_full, idx, K_in, v, alpha, beta, S, o, B, H, K, V, dtype,
                             stream=None) -> int:
    st = load().gdn_decode_step_gathered(_ptr(q_full), _ptr(k_full), _ptr(idx), K_in, _ptr(v),
                                         _ptr(alpha), _ptr(beta), _ptr(S), _ptr(o), B, H, K, V,
                                         dtype, _stream(stream))
    return _check(st, "gdn_decode_step_gathered")


def gdn_prefill_gated(q, k, v, alpha, beta, b, w, S0, o, S_T, B, T, H, K, V, gate, dtype,
                      stream=None) -> int:
    st = load().gdn_prefill_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(b),
                                  _ptr(w), _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, K, V, gate,
                                  dtype, _stream(stream))
    return _check(st, "gdn_prefill_gated")


def gdn_prefill_gated_chunked(q, k, v, alpha, beta, b, w, S0, o, S_T, B, T, H, K, V, gate,
                              dtype, workspace, workspace_bytes, stream=None) -> int:
    st = load().gdn_prefill_gated_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                          _ptr(b), _ptr(w), _ptr(S0), _ptr(o), _ptr(S_T), B, T,
                                          H, K, V, gate, dtype, _ptr(workspace), workspace_bytes,
                                          _stream(stream))
    return _check(st, "gdn_prefill_gated_chunked")


def gdn_prefill_gated_chunked_workspace_size(B, T, H, K, V, gate, dtype) -> int:
    return load().gdn_prefill_gated_chunked_workspace_size(B, T, H, K, V, gate, dtype)


def prefill_gated_chunked(q, k, v, alpha, beta=None, b=None, w=None, S0=None, gate="kda",
                          want_o=True, want_state=True, workspace=None, stream=None):
    """gdn_prefill_gated_chunked on torch CUDA tensors (gate "kda" or "gdn2",
    K = V = 128, bf16); allocates the workspace unless one is given.
    Returns (o, S_T)."""
    import torch
    B, T, H, K = k.shape
    V = v.shape[-1]
    o = torch.empty((B, T, H, V), dtype=v.dtype, device=v.device) if want_o else None
    ST = torch.empty((B, H, V, K), dtype=torch.float32, device=v.device) if want_state else None
    need = gdn_prefill_gated_chunked_workspace_size(B, T, H, K, V, GATES[gate], _dtype_code(v))
    if workspace is None:
        workspace = _scratch(max(need, 1), v.device, stream)
    gdn_prefill_gated_chunked(q, k, v, alpha, beta, b, w, S0, o, ST, B, T, H, K, V, GATES[gate],
                              _dtype_code(v), workspace, workspace.numel(), stream)
    _written_on(stream, o, ST)
    return o, ST


def gdn_decode_step_gated(q, k, v, alpha, beta, b, w, S, o, B, H, K, V, gate, dtype,
                          stream=None) -> int:
    st = load().gdn_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                      _ptr(b), _ptr(w), _ptr(S), _ptr(o), B, H, K, V, gate, dtype,
                                      _stream(stream))
    return _check(st, "gdn_decode_step_gated")


def prefill_gated(q, k, v, alpha, beta=None, b=None, w=None, S0=None, gate="kda",
                  want_o=True, want_state=True, stream=None):
    """gdn_prefill_gated on torch CUDA tensors: q, k [B,T,H,K]; v [B,T,H,V];
    alpha [B,T,H] (gate "gdn") or [B,T,H,K]; beta [B,T,H] ("gdn", "kda");
    b [B,T,H,K], w [B,T,H,V] ("gdn2").  Returns (o, S_T)."""
    import torch
    B, T, H, K = k.shape
    V = v.shape[-1]
    o = torch.empty((B, T, H, V), dtype=v.dtype, device=v.device) if want_o else None
    ST = torch.empty((B, H, V, K), dtype=torch.float32, device=v.device) if want_state else None
    gdn_prefill_gated(q, k, v, alpha, beta, b, w, S0, o, ST, B, T, H, K, V, GATES[gate],
                      _dtype_code(v), stream)
    _written_on(stream, o, ST)
    return o, ST


def gdn_state_truncate(S, BH, V, K, r, sigma=None, max_sweeps=30, stream=None) -> int:
    st = load().gdn_state_truncate(_ptr(S), BH, V, K, r, _ptr(sigma), max_sweeps,
                                   _stream(stream))
    return _check(st, "gdn_state_truncate")


def gdn_prefill_truncated(q, k, v, alpha, beta, S0, o, S_T, B, T, H, K, V, dtype, seg_len, r,
                          max_sweeps=30, workspace=None, workspace_bytes=0, stream=None) -> int:
    st = load().gdn_prefill_truncated(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                      _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, K, V, dtype,
                                      seg_len, r, max_sweeps, _ptr(workspace), workspace_bytes,
                                      _stream(stream))
    return _check(st, "gdn_prefill_truncated")


def state_truncate(S, r, want_sigma=False, max_sweeps=30, stream=None):
    """In-place rank-r truncation of S [..., V, K] (float32 CUDA); returns the
    singular values [..., min(V, K)] if asked."""
    import torch
    V, K = S.shape[-2:]
    BH = S.numel() // (V * K)
    sigma = (torch.empty(S.shape[:-2] + (min(V, K),), dtype=torch.float32, device=S.device)
             if want_sigma else None)
    gdn_state_truncate(S, BH, V, K, r, sigma, max_sweeps, stream)
    _written_on(stream, sigma)
    return sigma


def prefill_truncated(q, k, v, alpha, beta, S0=None, seg_len=256, r=32, max_sweeps=30,
                      stream=None):
    """gdn_prefill_truncated on torch CUDA tensors.  Returns (o, S_T)."""
    import torch
    B, T, H, K = k.shape
    V = v.shape[-1]
    o = torch.empty((B, T, H, V), dtype=v.dtype, device=v.device)
    ST = torch.empty((B, H, V, K), dtype=torch.float32, device=v.device)
    dt = _dtype_code(v)
    L = min(seg_len, T) if T > 0 else 0
    need = max([gdn_prefill_workspace_size(B, n, H, K, V, dt) for n in (L, T % seg_len) if n] + [0])
    ws = _scratch(need, v.device, stream)
    gdn_prefill_truncated(q, k, v, alpha, beta, S0, o, ST, B, T, H, K, V, dt, seg_len, r,
                          max_sweeps, ws, need, stream)
    _written_on(stream, o, ST)
    return o, ST


def gdn_channel_gram_workspace_size(B, T, H, K) -> int:
    return int(load().gdn_channel_gram_workspace_size(B, T, H, K))


def gdn_channel_gram(k, q, B, T, H, K, dtype, G, workspace, workspace_bytes,
                     stream=None) -> int:
    st = load().gdn_channel_gram(_ptr(k), _ptr(q), B, T, H, K, dtype, _ptr(G), _ptr(workspace),
                                 workspace_bytes, _stream(stream))
    return _check(st, "gdn_channel_gram")


def gdn_drrqr_select(G, H, n, k, f, max_swaps, idx, rho_max=None, swaps=None,
                     stream=None) -> int:
    st = load().gdn_drrqr_select(_ptr(G), H, n, k, ctypes.c_float(f), max_swaps, _ptr(idx),
                                 _ptr(rho_max), _ptr(swaps), _stream(stream))
    return _check(st, "gdn_drrqr_select")


def channel_gram(k, q, stream=None):
    """k, q [B, T, H, 128] bf16 CUDA -> G [H, 128, 128] float32."""
    import torch
    B, T, H, K = k.shape
    G = torch.empty((H, K, K), dtype=torch.float32, device=k.device)
    need = gdn_channel_gram_workspace_size(B, T, H, K)
    ws = _scratch(max(need, 1), k.device, stream)
    gdn_channel_gram(k, q, B, T, H, K, _dtype_code(k), G, ws, need, stream)
    _written_on(stream, G)
    return G


def drrqr_select(G, k, f=2.0, max_swaps=1000, stream=None):
    """G [H, n, n] float32 CUDA -> (idx [H, k] int32 in selection order,
    rho_max [H], swaps [H])."""
    import torch
    H, n, _ = G.shape
    idx = torch.empty((H, k), dtype=torch.int32, device=G.device)
    rho = torch.empty(H, dtype=torch.float32, device=G.device)
    sw = torch.empty(H, dtype=torch.int32, device=G.device)
    gdn_drrqr_select(G, H, n, k, f, max_swaps, idx, rho, sw, stream)
    _written_on(stream, idx, rho, sw)
    return idx, rho, sw


def gdn_prefill_host_workspace_size(B, T, H, K, V, dtype, window) -> int:
    return int(load().gdn_prefill_host_workspace_size(B, T, H, K, V, dtype, window))


def gdn_prefill_host(q, k, v, alpha, beta, S0, o, S_T, B, T, H, K, V, dtype, window, workspace,
                     workspace_bytes, stream=None) -> int:
    """Host-buffer prefill: q .. S_T are (pinned) CPU tensors or host addresses;
    workspace is device memory."""
    st = load().gdn_prefill_host(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                                 _ptr(o), _ptr(S_T), B, T, H, K, V, dtype, window,
                                 _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "gdn_prefill_host")


def gdn_prefill_gathered_workspace_size(B, T, H, K_in, K, V, dtype) -> int:
    return int(load().gdn_prefill_gathered_workspace_size(B, T, H, K_in, K, V, dtype))


def gdn_prefill_gathered(q_full, k_full, idx, K_in, v, alpha, beta, S0, o, S_T, B, T, H, K, V,
                         dtype, workspace, workspace_bytes, stream=None) -> int:
    st = load().gdn_prefill_gathered(_ptr(q_full), _ptr(k_full), _ptr(idx), K_in, _ptr(v),
                                     _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T), B, T,
                                     H, K, V, dtype, _ptr(workspace), workspace_bytes,
                                     _stream(stream))
    return _check(st, "gdn_prefill_gathered")


def prefill_gathered(q_full, k_full, idx, v, alpha, beta, S0=None, want_o=True, want_state=True,
                     stream=None):
    """The pruned prefill from full-width q / k ([B, T, H, 128] bf16) and the kept
    channels idx ([H, 64] int32): returns (o, S_T) with S_T [B, H, 128, 64]."""
    import torch
    B, T, H, K_in = k_full.shape
    K, V = idx.shape[1], v.shape[-1]
    dt = _dtype_code(k_full)
    o = torch.empty((B, T, H, V), dtype=v.dtype, device=v.device) if want_o else None
    ST = torch.empty((B, H, V, K), dtype=torch.float32, device=v.device) if want_state else None
    need = gdn_prefill_gathered_workspace_size(B, T, H, K_in, K, V, dt)
    ws = _scratch(max(need, 1), v.device, stream)
    gdn_prefill_gathered(q_full, k_full, idx, K_in, v, alpha, beta, S0, o, ST, B, T, H, K, V, dt,
                         ws, need, stream)
    _written_on(stream, o, ST)
    return o, ST


def gather_normalize(x, idx, stream=None):
    """x [..., H, K_in] (bf16/fp32 CUDA); idx [H, K_out] int32 CUDA.  Returns
    the pruned, renormalised [..., H, K_out]."""
    import torch
    H, K_in = x.shape[-2:]
    K_out = idx.shape[-1]
    N = x.numel() // (H * K_in)
    y = torch.empty(x.shape[:-1] + (K_out,), dtype=x.dtype, device=x.device)
    gdn_gather_normalize(x, idx, y, N, H, K_in, K_out, _dtype_code(x), stream)
    _written_on(stream, y)
    return y


def gdn_qk_norm_rotate(q, k, wq, wk, pos, inv_freq, yq, yk, N, Hq, Hk, D, R, q_stride, k_stride,
                       norm, pairing, eps, dtype, stream=None) -> int:
    st = load().gdn_qk_norm_rotate(_ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(pos),
                                   _ptr(inv_freq), _ptr(yq), _ptr(yk), N, Hq, Hk, D, R, q_stride,
                                   k_stride, norm, pairing, eps, dtype, _stream(stream))
    return _check(st, "gdn_qk_norm_rotate")


def gdn_qk_norm_rotate_backward(q, k, wq, wk, pos, inv_freq, dyq, dyk, dq, dk, dwq, dwk, N, Hq,
                                Hk, D, R, q_stride, k_stride, norm, pairing, eps, dtype,
                                workspace=None, workspace_bytes=0, stream=None) -> int:
    st = load().gdn_qk_norm_rotate_backward(
        _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(pos), _ptr(inv_freq), _ptr(dyq), _ptr(dyk),
        _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk), N, Hq, Hk, D, R, q_stride, k_stride, norm,
        pairing, eps, dtype, _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "gdn_qk_norm_rotate_backward")


def gdn_qk_norm_rotate_backward_workspace_size(N, Hq, Hk, D) -> int:
    return int(load().gdn_qk_norm_rotate_backward_workspace_size(N, Hq, Hk, D))


def gdn_linear_prefill(q, k, v, alpha, S0, o, S_T, offsets, B, T, Hq, H, K, V, q_stride, k_stride,
                       v_stride, scale, dtype, workspace=None, workspace_bytes=0,
                       stream=None) -> int:
    st = load().gdn_linear_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(S0), _ptr(o),
                                   _ptr(S_T), _ptr(offsets), B, T, Hq, H, K, V, q_stride,
                                   k_stride, v_stride, scale, dtype, _ptr(workspace),
                                   workspace_bytes, _stream(stream))
    return _check(st, "gdn_linear_prefill")


def gdn_linear_prefill_workspace_size(B, T, H, K, V, packed, dtype) -> int:
    return int(load().gdn_linear_prefill_workspace_size(B, T, H, K, V, int(packed), dtype))


def gdn_linear_backward(q, k, v, alpha, dO, S0, dS_T, dq, dk, dv, dS0, offsets, B, T, Hq, H, K, V,
                        q_stride, k_stride, v_stride, scale, dtype, workspace=None,
                        workspace_bytes=0, stream=None) -> int:
    st = load().gdn_linear_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(dO), _ptr(S0),
                                    _ptr(dS_T), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dS0),
                                    _ptr(offsets), B, T, Hq, H, K, V, q_stride, k_stride,
                                    v_stride, scale, dtype, _ptr(workspace), workspace_bytes,
                                    _stream(stream))
    return _check(st, "gdn_linear_backward")


def gdn_linear_backward_workspace_size(B, T, Hq, H, K, V, packed, dtype) -> int:
    return int(load().gdn_linear_backward_workspace_size(B, T, Hq, H, K, V, int(packed), dtype))


def gdn_linear_decode_step(q, k, v, alpha, S, S_out, o, B, Hq, H, K, V, scale, dtype,
                           stream=None) -> int:
    st = load().gdn_linear_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(S),
                                       _ptr(S_out), _ptr(o), B, Hq, H, K, V, scale, dtype,
                                       _stream(stream))
    return _check(st, "gdn_linear_decode_step")


def gdn_scan_prefill(x, gate, h0, h, h_T, states, offsets, B, T, D, x_stride, gate_stride, kind,
                     dtype, workspace=None, workspace_bytes=0, stream=None) -> int:
    st = load().gdn_scan_prefill(_ptr(x), _ptr(gate), _ptr(h0), _ptr(h), _ptr(h_T), _ptr(states),
                                 _ptr(offsets), B, T, D, x_stride, gate_stride, kind, dtype,
                                 _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "gdn_scan_prefill")


def gdn_scan_prefill_workspace_size(B, T, D, packed) -> int:
    return int(load().gdn_scan_prefill_workspace_size(B, T, D, int(packed)))


def gdn_scan_backward(x, gate, dh, h0, dh_T, states, dx, dgate, dh0, offsets, B, T, D, x_stride,
                      gate_stride, kind, dtype, workspace=None, workspace_bytes=0,
                      stream=None) -> int:
    st = load().gdn_scan_backward(_ptr(x), _ptr(gate), _ptr(dh), _ptr(h0), _ptr(dh_T),
                                  _ptr(states), _ptr(dx), _ptr(dgate), _ptr(dh0), _ptr(offsets), B,
                                  T, D, x_stride, gate_stride, kind, dtype, _ptr(workspace),
                                  workspace_bytes, _stream(stream))
    return _check(st, "gdn_scan_backward")


def gdn_scan_backward_workspace_size(B, T, D, packed, kept) -> int:
    return int(load().gdn_scan_backward_workspace_size(B, T, D, int(packed), int(kept)))


def gdn_scan_decode_step(x, gate, h, h_out, y, B, D, x_stride, gate_stride, kind, dtype,
                         stream=None) -> int:
    st = load().gdn_scan_decode_step(_ptr(x), _ptr(gate), _ptr(h), _ptr(h_out), _ptr(y), B, D,
                                     x_stride, gate_stride, kind, dtype, _stream(stream))
    return _check(st, "gdn_scan_decode_step")


def gdn_layer_norm(x, residual, w, b, y, s, stats, N, D, x_stride, residual_stride, eps, dtype,
                   stream=None) -> int:
    st = load().gdn_layer_norm(_ptr(x), _ptr(residual), _ptr(w), _ptr(b), _ptr(y), _ptr(s),
                               _ptr(stats), N, D, x_stride, residual_stride, eps, dtype,
                               _stream(stream))
    return _check(st, "gdn_layer_norm")


def gdn_layer_norm_backward(s, dy, stats, w, ds, dx, dw, db, N, D, s_stride, dtype, workspace=None,
                            workspace_bytes=0, stream=None) -> int:
    st = load().gdn_layer_norm_backward(_ptr(s), _ptr(dy), _ptr(stats), _ptr(w), _ptr(ds),
                                        _ptr(dx), _ptr(dw), _ptr(db), N, D, s_stride, dtype,
                                        _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "gdn_layer_norm_backward")


def gdn_layer_norm_backward_workspace_size(N, D) -> int:
    return int(load().gdn_layer_norm_backward_workspace_size(N, D))


def gdn_get_last_device_status(stream=None) -> int:
    return int(load().gdn_get_last_device_status(_stream(stream)))


def gdn_status_string(status: int) -> str:
    return status_string(status)


def gdn_selftest_wait_timeout(limit_cycles, stream=None) -> int:
    st = load().gdn_selftest_wait_timeout(int(limit_cycles), _stream(stream))
    return _check(st, "gdn_selftest_wait_timeout")


def gdn_selftest_lost_copy(call, limit_cycles, lost, buffer, bytes, rows, T, D, stream=None) -> int:
    st = load().gdn_selftest_lost_copy(call, int(limit_cycles), int(lost), _ptr(buffer), bytes, rows,
                                       T, D, _stream(stream))
    return _check(st, "gdn_selftest_lost_copy")


def gdn_version() -> int:
    return int(load().gdn_version())


# ---- tensor-level conveniences (allocate outputs with torch, then call) ----

def prefill(q, k, v, alpha, beta, S0=None, want_o=True, want_state=True, out_state=None,
            stream=None, two_pass=True):
    """q, k [B,T,H,K]; v [B,T,H,V] (bf16 or fp32 CUDA tensors); alpha, beta
    [B,T,H] fp32; S0 [B,H,V,K] fp32 or None.  Returns (o, S_T).  two_pass:
    allocate the workspace of the two-pass form where the problem has one
    (identical results; False runs the one-pass form)."""
    import torch
    B, T, H, K = k.shape
    V = v.shape[-1]
    dt = _dtype_code(k)
    o = torch.empty((B, T, H, V), dtype=k.dtype, device=k.device) if want_o else None
    ST = None
    if want_state:
        ST = out_state if out_state is not None else torch.empty(
            (B, H, V, K), dtype=torch.float32, device=k.device)
    ws_bytes = gdn_prefill_workspace_size(B, T, H, K, V, dt)
    if two_pass:
        ws_bytes = max(ws_bytes, gdn_prefill_two_pass_workspace_size(B, T, H, K, V, dt))
    ws = _scratch(ws_bytes, k.device, stream)
    gdn_prefill(q, k, v, alpha, beta, S0, o, ST, B, T, H, K, V, dt, ws, ws_bytes, stream)
    _written_on(stream, o, None if ST is out_state else ST)
    return o, ST


def decode_step(q, k, v, alpha, beta, S, o=None, stream=None):
    """One token: q, k [B,H,K]; v [B,H,V]; alpha, beta [B,H]; S [B,H,V,K]
    updated in place.  Returns o [B,H,V]."""
    import torch
    B, H, K = k.shape
    V = v.shape[-1]
    given = o
    if o is None:
        o = torch.empty((B, H, V), dtype=k.dtype, device=k.device)
    gdn_decode_step(q, k, v, alpha, beta, S, o, B, H, K, V, _dtype_code(k), stream)
    if given is None:
        _written_on(stream, o)
    return o


def state_rank(S, max_iter=500, tol=1e-7, stream=None):
    """S [..., V, K] fp32.  Returns (fro2, sigma1, stable_rank) shaped [...]."""
    import torch
    lead = S.shape[:-2]
    V, K = S.shape[-2:]
    BH = 1
    for d in lead:
        BH *= d
    outs = [torch.empty(lead, dtype=torch.float32, device=S.device) for _ in range(3)]
    gdn_state_rank(S, BH, V, K, *outs, max_iter=max_iter, tol=tol, stream=stream)
    _written_on(stream, *outs)
    return tuple(outs)


def _reject(where, what):
    e = GDNError(GDN_ERR_INVALID_ARG, where)
    e.args = (f"{e.args[0]}: {what}",)
    raise e


def _token_stride(where, name, x, dtype, device):
    """Elements between consecutive tokens of x [..., heads, channels]: a
    token's heads and channels are dense, and the leading dimensions step
    evenly, as in a part of a wider projection."""
    if x.dtype is not dtype or x.get_device() != device:
        _reject(where, f"{name} is {x.dtype} on {x.device}")
    heads, D = x.shape[-2:]
    if x.is_contiguous():
        return heads * D
    st = x.stride()
    if st[-1] != 1 or (st[-2] != D and heads > 1):
        _reject(where, f"{name}'s heads and channels are not dense (strides {st})")
    step, span = None, 1  # of the tokens seen so far, innermost first
    for n, s in zip(reversed(x.shape[:-2]), reversed(st[:-2])):
        if n == 1:
            continue
        if step is None:
            step = s
        # a step of 0 (a broadcast) or of less than a token has no memory of its own for each
        if s != step * span or step < heads * D:
            _reject(where, f"{name}'s tokens do not lie evenly, a whole token apart (strides {st})")
        span *= n
    return heads * D if step is None else step


def _dense(where, name, x, dtype, device, shape):
    """x, if given, is contiguous, on the device (a number), of its type and shape."""
    if x is not None and (x.dtype is not dtype or x.get_device() != device or x.shape != shape
                          or not x.is_contiguous()):
        _reject(where, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                       f"device {device}; it is {x.dtype}, {tuple(x.shape)} on {x.device}")


_current_device = None


def _on_this_gpu(where, device):
    """The operands' device (a number; the last check of a call) is the GPU it runs on."""
    if device < 0:
        _reject(where, "its tensors are on the CPU, not on a GPU")
    global _current_device
    if _current_device is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    if device != _current_device():
        _reject(where, f"its tensors are on GPU {device}, not on the current one")


def _workspace(where, given, need, like, stream):
    """(workspace, its bytes): the one given, or a new one where one is needed."""
    if given is not None:
        if given.get_device() != like.get_device() or not given.is_contiguous():
            _reject(where, f"workspace must be contiguous on device {like.device}")
        return given, given.numel() * given.element_size()
    return _scratch(need, like.device, stream), need


def _qk_norm_args(where, q, k, pos, inv_freq, wq, wk, norm, pairing):
    import torch
    if norm not in NORMS or pairing not in PAIRINGS:
        _reject(where, f"norm {norm!r}, pairing {pairing!r}")
    dt, dev, lead = q.dtype, q.get_device(), q.shape[:-2]
    Hq, D = q.shape[-2:]
    Hk = ldk = 0
    ldq = _token_stride(where, "q", q, dt, dev)
    if k is not None:
        Hk = k.shape[-2]
        if k.shape[:-2] != lead or k.shape[-1] != D:
            _reject(where, f"q {tuple(q.shape)} and k {tuple(k.shape)}")
        ldk = _token_stride(where, "k", k, dt, dev)
    R = 0
    if inv_freq is not None:
        R = 2 * inv_freq.shape[0]
        _dense(where, "inv_freq", inv_freq, torch.float32, dev, (R // 2,))
    _dense(where, "pos", pos, torch.int64, dev, lead)
    _dense(where, "wq", wq, torch.float32, dev, (D,))
    _dense(where, "wk", wk, torch.float32, dev, (D,))
    return lead.numel(), Hq, Hk, D, R, ldq, ldk, NORMS[norm], PAIRINGS[pairing]


def _new(x):
    """A new dense tensor of x's shape and type."""
    import torch
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def qk_norm_rotate(q, k, pos=None, inv_freq=None, wq=None, wk=None, norm="rms", pairing="half",
                   eps=1e-6, out=None, stream=None):
    """Norms of q [..., Hq, D] and k [..., Hk, D] (or None) for each head, and
    the rotation of their first 2 len(inv_freq) channels by pos * inv_freq, in
    one pass (gdn_qk_norm_rotate).  pos [...] int64; wq, wk [D] float32 or None;
    norm "rms" or "l2"; pairing "half" (i with i + R/2) or "adjacent".  q and k
    may be slices of one projection.  Returns (yq, yk), new dense tensors or
    `out` (which may hold dense q and k themselves)."""
    where = "qk_norm_rotate"
    N, Hq, Hk, D, R, ldq, ldk, nrm, pair = _qk_norm_args(where, q, k, pos, inv_freq, wq, wk, norm,
                                                         pairing)
    if out is None:
        yq = _new(q)
        yk = None if k is None else _new(k)
    else:
        yq, yk = out
        _dense(where, "out[0]", yq, q.dtype, q.get_device(), q.shape)
        if k is not None:
            _dense(where, "out[1]", yk, q.dtype, q.get_device(), k.shape)
    _on_this_gpu(where, q.get_device())
    gdn_qk_norm_rotate(q, k, wq, wk, pos, inv_freq, yq, yk, N, Hq, Hk, D, R, ldq, ldk, nrm, pair,
                       eps, _dtype_code(q), stream)
    if out is None:
        _written_on(stream, yq, yk)
    return yq, yk


def qk_norm_rotate_backward(q, k, pos, inv_freq, dyq, dyk, wq=None, wk=None, norm="rms",
                            pairing="half", eps=1e-6, workspace=None, stream=None):
    """Gradients of qk_norm_rotate from its inputs and dyq, dyk (dense).
    Returns (dq, dk, dwq, dwk); a weight that was not given has None."""
    where = "qk_norm_rotate_backward"
    N, Hq, Hk, D, R, ldq, ldk, nrm, pair = _qk_norm_args(where, q, k, pos, inv_freq, wq, wk, norm,
                                                         pairing)
    _dense(where, "dyq", dyq, q.dtype, q.get_device(), q.shape)
    if k is not None:
        _dense(where, "dyk", dyk, q.dtype, q.get_device(), k.shape)
    _on_this_gpu(where, q.get_device())
    dq = _new(q)
    dk = None if k is None else _new(k)
    dwq = None if wq is None else _new(wq)
    dwk = None if wk is None else _new(wk)
    need = 0
    if wq is not None or wk is not None:
        need = gdn_qk_norm_rotate_backward_workspace_size(N, Hq, Hk, D)
    workspace, need = _workspace(where, workspace, need, q, stream)
    gdn_qk_norm_rotate_backward(q, k, wq, wk, pos, inv_freq, dyq, dyk, dq, dk, dwq, dwk, N, Hq, Hk,
                                D, R, ldq, ldk, nrm, pair, eps, _dtype_code(q), workspace, need,
                                stream)
    _written_on(stream, dq, dk, dwq, dwk)
    return dq, dk, dwq, dwk


def _linear_args(where, q, k, v, alpha, offsets):
    """Sizes, token strides and (type, device) of q, k [B, T, Hq, K], v [B, T, H, V]; with
    offsets, of q, k [tokens, Hq, K], v [tokens, H, V]."""
    import torch
    qs, vs = q.shape, v.shape
    dims = 4 if offsets is None else 3
    if len(qs) != dims or k.shape != qs or len(vs) != dims or vs[:-2] != qs[:-2]:
        _reject(where, f"q {tuple(qs)}, k {tuple(k.shape)}, v {tuple(vs)}"
                       + ("" if offsets is None else " with offsets"))
    dt, dev = v.dtype, v.get_device()
    Hq, K = qs[-2:]
    H, V = vs[-2:]
    if offsets is None:
        B, T = qs[:2]
    else:
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            _reject(where, "offsets must be [sequences + 1]")
        B, T = offsets.shape[0] - 1, qs[0]
        _dense(where, "offsets", offsets, torch.int32, dev, (B + 1,))
    _dense(where, "alpha", alpha, torch.float32, dev, (H,))
    ldq = _token_stride(where, "q", q, dt, dev)
    ldk = _token_stride(where, "k", k, dt, dev)
    ldv = _token_stride(where, "v", v, dt, dev)
    return B, T, Hq, H, K, V, ldq, ldk, ldv


def linear_prefill(q, k, v, alpha, S0=None, scale=1.0, offsets=None, want_o=True, want_state=True,
                   out_state=None, workspace=None, stream=None):
    """Linear attention with a decay for each head, S_t = alpha S_{t-1} + v_t k_t^T and
    o_t = scale S_t q_t (gdn_linear_prefill): q, k [B, T, Hq, K], v [B, T, H, V] (bf16 or fp32;
    H a multiple of Hq; slices of one projection will do), alpha [H] fp32, S0 [B, H, V, K] fp32 or
    None.  With offsets [B + 1] int32 the sequences lie packed: q, k [tokens, Hq, K],
    v [tokens, H, V]; outputs of tokens of no sequence are not written.  Returns (o, S_T);
    out_state may be S0."""
    import torch
    where = "linear_prefill"
    B, T, Hq, H, K, V, ldq, ldk, ldv = _linear_args(where, q, k, v, alpha, offsets)
    dev, shape = v.get_device(), (B, H, V, K)
    _dense(where, "S0", S0, torch.float32, dev, shape)
    _dense(where, "out_state", out_state, torch.float32, dev, shape)
    _on_this_gpu(where, dev)
    dt = _dtype_code(v)
    o = _new(v) if want_o else None
    ST = out_state
    if want_state and ST is None:
        ST = torch.empty(shape, dtype=torch.float32, device=v.device)
    workspace, need = _workspace(where, workspace, gdn_linear_prefill_workspace_size(
        B, T, H, K, V, offsets is not None, dt), v, stream)
    gdn_linear_prefill(q, k, v, alpha, S0, o, ST, offsets, B, T, Hq, H, K, V, ldq, ldk, ldv, scale,
                       dt, workspace, need, stream)
    _written_on(stream, o, None if ST is out_state else ST)
    return o, ST


def linear_backward(q, k, v, alpha, do, S0=None, dS_T=None, scale=1.0, offsets=None,
                    want_dS0=None, workspace=None, stream=None):
    """Gradients of linear_prefill from its inputs, do (dense, as v) and dS_T (fp32 or None).
    Returns (dq, dk, dv, dS0); dS0 is formed if S0 is given or want_dS0 is true, else None.
    alpha is a constant and has none.  Gradients of tokens of no sequence are not written."""
    import torch
    where = "linear_backward"
    B, T, Hq, H, K, V, ldq, ldk, ldv = _linear_args(where, q, k, v, alpha, offsets)
    dev, shape = v.get_device(), (B, H, V, K)
    _dense(where, "S0", S0, torch.float32, dev, shape)
    _dense(where, "dS_T", dS_T, torch.float32, dev, shape)
    _dense(where, "do", do, v.dtype, dev, v.shape)
    _on_this_gpu(where, dev)
    dt = _dtype_code(v)
    dq, dk, dv = _new(q), _new(k), _new(v)
    dS0 = None
    if want_dS0 or (want_dS0 is None and S0 is not None):
        dS0 = torch.empty(shape, dtype=torch.float32, device=v.device)
    workspace, need = _workspace(where, workspace, gdn_linear_backward_workspace_size(
        B, T, Hq, H, K, V, offsets is not None, dt), v, stream)
    gdn_linear_backward(q, k, v, alpha, do, S0, dS_T, dq, dk, dv, dS0, offsets, B, T, Hq, H, K, V,
                        ldq, ldk, ldv, scale, dt, workspace, need, stream)
    _written_on(stream, dq, dk, dv, dS0)
    return dq, dk, dv, dS0


def linear_decode_step(q, k, v, alpha, S, scale=1.0, S_out=None, o=None, stream=None):
    """One token of linear_prefill: q, k [B, Hq, K]; v [B, H, V]; alpha [H]; S [B, H, V, K],
    updated in place unless S_out is given.  Returns o [B, H, V]."""
    import torch
    where = "linear_decode_step"
    qs, vs = q.shape, v.shape
    if len(qs) != 3 or len(vs) != 3 or qs[0] != vs[0]:
        _reject(where, f"q {tuple(qs)}, v {tuple(vs)}")
    B, Hq, K = qs
    H, V = vs[1:]
    dt, dev, shape = v.dtype, v.get_device(), (B, H, V, K)
    if S_out is None:
        S_out = S
    given = o
    if o is None:
        o = torch.empty_like(v)
    _dense(where, "q", q, dt, dev, qs)
    _dense(where, "k", k, dt, dev, qs)
    _dense(where, "v", v, dt, dev, vs)
    _dense(where, "o", o, dt, dev, vs)
    _dense(where, "alpha", alpha, torch.float32, dev, (H,))
    _dense(where, "S", S, torch.float32, dev, shape)
    _dense(where, "S_out", S_out, torch.float32, dev, shape)
    _on_this_gpu(where, dev)
    gdn_linear_decode_step(q, k, v, alpha, S, S_out, o, B, Hq, H, K, V, scale, _dtype_code(v),
                           stream)
    if given is None:
        _written_on(stream, o)
    return o


def _row_stride(where, name, x, dtype, device):
    """Elements between consecutive rows of x [..., D]: a row is dense, and the leading dimensions
    step evenly, as in a part of a wider projection."""
    if x.is_contiguous() and x.dtype is dtype and x.get_device() == device:
        return x.shape[-1]
    return _token_stride(where, name, x.unsqueeze(-2), dtype, device)


def _scan_args(where, x, gate, kind, offsets):
    """B, T, D and the token strides of x and gate, [B, T, D] or with offsets [tokens, D]."""
    import torch
    if kind not in SCANS:
        _reject(where, f"kind {kind!r}")
    xs = x.shape
    if len(xs) != (3 if offsets is None else 2) or gate.shape != xs:
        _reject(where, f"x {tuple(xs)}, gate {tuple(gate.shape)}"
                       + ("" if offsets is None else " with offsets"))
    dev = x.get_device()
    if offsets is None:
        B, T, D = xs
    else:
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            _reject(where, "offsets must be [sequences + 1]")
        B, (T, D) = offsets.shape[0] - 1, xs
        _dense(where, "offsets", offsets, torch.int32, dev, (B + 1,))
    ldx = _row_stride(where, "x", x, x.dtype, dev)
    ldg = _row_stride(where, "gate", gate, torch.float32 if kind == "decay" else x.dtype, dev)
    return B, T, D, ldx, ldg


def _states_shape(B, T, D, packed):
    blocks = -(-T // GDN_SCAN_BLOCK)
    return (blocks, D) if packed else (B, blocks, D)


def scan_prefill(x, gate, h0=None, kind="sigmoid", offsets=None, want_h=True, want_state=True,
                 out_state=None, keep_states=False, workspace=None, stream=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + b_t x_t, channel by channel
    (gdn_scan_prefill): x, gate [B, T, D] (slices of one projection will do); kind "sigmoid":
    a = sigmoid(gate), b = 1 - a, gate of x's type (bf16 or fp32); "decay": a = gate, fp32, b = 1.
    h0 [B, D] fp32 or None.  With offsets [B + 1] int32 the sequences lie packed: x, gate
    [tokens, D]; outputs of tokens of no sequence are not written.  Returns (h, h_T, states): h as
    x, h_T [B, D] fp32 (out_state may be h0), and with keep_states what scan_backward starts from
    (the state before every 64th token, fp32), else None."""
    import torch
    where = "scan_prefill"
    B, T, D, ldx, ldg = _scan_args(where, x, gate, kind, offsets)
    dev = x.get_device()
    _dense(where, "h0", h0, torch.float32, dev, (B, D))
    _dense(where, "out_state", out_state, torch.float32, dev, (B, D))
    _on_this_gpu(where, dev)
    packed = offsets is not None
    h = _new(x) if want_h else None
    h_T = out_state
    if want_state and h_T is None:
        h_T = torch.empty((B, D), dtype=torch.float32, device=x.device)
    states = None
    if keep_states:
        states = torch.empty(_states_shape(B, T, D, packed), dtype=torch.float32, device=x.device)
    need = gdn_scan_prefill_workspace_size(B, T, D, packed) if packed else 0
    workspace, need = _workspace(where, workspace, need, x, stream)
    gdn_scan_prefill(x, gate, h0, h, h_T, states, offsets, B, T, D, ldx, ldg, SCANS[kind],
                     _dtype_code(x), workspace, need, stream)
    _written_on(stream, h, None if h_T is out_state else h_T, states)
    return h, h_T, states


def scan_backward(x, gate, dh, h0=None, dh_T=None, states=None, kind="sigmoid", offsets=None,
                  want_dh0=None, workspace=None, stream=None):
    """Gradients of scan_prefill from its inputs, dh (dense, as x) and dh_T [B, D] (fp32 or None).
    states: as the forward pass kept them for the same inputs, or None (formed again).  Returns
    (dx, dgate, dh0), dgate as gate; dh0 is formed if h0 is given or want_dh0 is true, else None.
    Gradients of tokens of no sequence are not written."""
    import torch
    where = "scan_backward"
    B, T, D, ldx, ldg = _scan_args(where, x, gate, kind, offsets)
    dev, packed = x.get_device(), offsets is not None
    _dense(where, "h0", h0, torch.float32, dev, (B, D))
    _dense(where, "dh_T", dh_T, torch.float32, dev, (B, D))
    _dense(where, "dh", dh, x.dtype, dev, x.shape)
    _dense(where, "states", states, torch.float32, dev, _states_shape(B, T, D, packed))
    _on_this_gpu(where, dev)
    dx, dgate, dh0 = _new(x), _new(gate), None
    if want_dh0 or (want_dh0 is None and h0 is not None):
        dh0 = torch.empty((B, D), dtype=torch.float32, device=x.device)
    need = 0
    if packed or states is None:
        need = gdn_scan_backward_workspace_size(B, T, D, packed, states is not None)
    workspace, need = _workspace(where, workspace, need, x, stream)
    gdn_scan_backward(x, gate, dh, h0, dh_T, states, dx, dgate, dh0, offsets, B, T, D, ldx, ldg,
                      SCANS[kind], _dtype_code(x), workspace, need, stream)
    _written_on(stream, dx, dgate, dh0)
    return dx, dgate, dh0


def scan_decode_step(x, gate, h, kind="sigmoid", h_out=None, y=None, stream=None):
    """One token of scan_prefill: x, gate [B, D] (slices of one projection will do); h [B, D] fp32,
    updated in place unless h_out is given.  Returns y [B, D], the new state rounded to x's type."""
    import torch
    where = "scan_decode_step"
    if kind not in SCANS or x.dim() != 2 or gate.shape != x.shape:
        _reject(where, f"kind {kind!r}, x {tuple(x.shape)}, gate {tuple(gate.shape)}")
    B, D = x.shape
    dev = x.get_device()
    if h_out is None:
        h_out = h
    ldx = _row_stride(where, "x", x, x.dtype, dev)
    ldg = _row_stride(where, "gate", gate, torch.float32 if kind == "decay" else x.dtype, dev)
    _dense(where, "h", h, torch.float32, dev, x.shape)
    _dense(where, "h_out", h_out, torch.float32, dev, x.shape)
    _dense(where, "y", y, x.dtype, dev, x.shape)
    _on_this_gpu(where, dev)
    given = y
    if y is None:
        y = _new(x)
    gdn_scan_decode_step(x, gate, h, h_out, y, B, D, ldx, ldg, SCANS[kind], _dtype_code(x), stream)
    if given is None:
        _written_on(stream, y)
    return y


def layer_norm(x, w=None, b=None, residual=None, eps=1e-5, want_stats=False, out=None,
               stream=None):
    """y = (s - mean) / sqrt(var + eps) * w + b over the channels of s = x [..., D], or of
    s = x + residual rounded to x's type (gdn_layer_norm); w, b [D] fp32 or None.  x and residual
    may be slices of a projection.  Returns (y, s, stats): s None without a residual, stats
    [..., 2] fp32 (what layer_norm_backward needs) or None.  out: (y, s) to write to, dense; they
    may hold dense x and residual themselves."""
    import torch
    where = "layer_norm"
    dev, D, lead = x.get_device(), x.shape[-1], x.shape[:-1]
    ldx = _row_stride(where, "x", x, x.dtype, dev)
    ldr = 0
    if residual is not None:
        if residual.shape != x.shape:
            _reject(where, f"x {tuple(x.shape)}, residual {tuple(residual.shape)}")
        ldr = _row_stride(where, "residual", residual, x.dtype, dev)
    _dense(where, "w", w, torch.float32, dev, (D,))
    _dense(where, "b", b, torch.float32, dev, (D,))
    if out is not None:
        y, s = out
        if y is None or (s is None) != (residual is None):
            _reject(where, "out must be (y, s), with s None where there is no residual")
        _dense(where, "out[0]", y, x.dtype, dev, x.shape)
        _dense(where, "out[1]", s, x.dtype, dev, x.shape)
    _on_this_gpu(where, dev)
    if out is None:
        y = _new(x)
        s = None if residual is None else _new(x)
    stats = None
    if want_stats:
        stats = torch.empty(lead + (2,), dtype=torch.float32, device=x.device)
    gdn_layer_norm(x, residual, w, b, y, s, stats, lead.numel(), D, ldx, ldr, eps, _dtype_code(x),
                   stream)
    if out is None:
        _written_on(stream, y, s, stats)
    else:
        _written_on(stream, stats)
    return y, s, stats


def layer_norm_backward(s, dy, stats, w=None, ds=None, want_db=False, workspace=None, stream=None):
    """Gradients of layer_norm from s (x where there was no residual), dy (dense), its stats and
    ds, the gradient that reaches s past the norm (dense, or None).  Returns (dx, dw, db): dx is
    the gradient of x and of the residual; dw None unless w is given, db None unless wanted."""
    import torch
    where = "layer_norm_backward"
    dev, D, lead = s.get_device(), s.shape[-1], s.shape[:-1]
    lds = _row_stride(where, "s", s, s.dtype, dev)
    _dense(where, "dy", dy, s.dtype, dev, s.shape)
    _dense(where, "ds", ds, s.dtype, dev, s.shape)
    _dense(where, "stats", stats, torch.float32, dev, lead + (2,))
    _dense(where, "w", w, torch.float32, dev, (D,))
    _on_this_gpu(where, dev)
    N = lead.numel()
    dx = _new(s)
    dw = None if w is None else _new(w)
    db = torch.empty(D, dtype=torch.float32, device=s.device) if want_db else None
    need = 0
    if w is not None or want_db:
        need = gdn_layer_norm_backward_workspace_size(N, D)
    workspace, need = _workspace(where, workspace, need, s, stream)
    gdn_layer_norm_backward(s, dy, stats, w, ds, dx, dw, db, N, D, lds, _dtype_code(s), workspace,
                            need, stream)
    _written_on(stream, dx, dw, db)
    return dx, dw, db
