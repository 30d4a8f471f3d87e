"""Thin torch binding of libdllm.so: the C entry points of include/dllm.h under the
same names, taking torch tensors.  Only argument marshalling happens here (shape
and dtype checks, pointers, the current CUDA stream, workspace tensors); every
step of the refresh runs in the library's kernels.  Nothing falls back to another
implementation: a missing library or a failed call raises.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libdllm.so")

DLLM_F32, DLLM_BF16, DLLM_E4M3 = 0, 1, 2
STATUS_TIMEOUT, STATUS_COUNT_CLAMP, STATUS_PAGE = 1, 2, 8

_lock = threading.Lock()
_lib = None


class DllmError(RuntimeError):
    pass


class dllm_layer(C.Structure):
    _fields_ = [("w_qkv", C.c_void_p), ("w_o", C.c_void_p), ("w_gu", C.c_void_p),
                ("w_down", C.c_void_p), ("gamma1", C.c_void_p), ("gamma2", C.c_void_p),
                ("rope_inv_freq", C.c_void_p),
                ("d", C.c_int), ("n_q", C.c_int), ("n_kv", C.c_int), ("hd", C.c_int), ("F", C.c_int),
                ("eps", C.c_float), ("rope_theta", C.c_float), ("use_rope", C.c_int),
                ("dtype", C.c_int)]


_SIGS = {
    "dllm_last_error": (C.c_char_p, []),
    "dllm_version": (C.c_int, []),
    "dllm_check_status": (C.c_int, [C.POINTER(C.c_uint), C.c_int]),
    "dllm_proxy_score": (C.c_int, [C.c_void_p] * 5 + [C.c_int] * 5 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_proxy_workspace_bytes": (C.c_size_t, [C.c_int] * 5),
    "dllm_kl_drift_workspace_bytes": (C.c_size_t, [C.c_int, C.c_int]),
    "dllm_kl_drift": (C.c_int, [C.c_void_p] * 3 + [C.c_int] * 3 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_ce_step": (C.c_int, [C.c_void_p] * 6 + [C.c_int] * 2 + [C.c_float] * 5 + [C.c_int, C.c_float, C.c_void_p]),
    "dllm_polestar_commit": (C.c_int, [C.c_void_p] * 7 + [C.c_int] * 2 + [C.c_float] * 2 + [C.c_void_p]),
    "dllm_spherical_kmeans": (C.c_int, [C.c_void_p] * 4 + [C.c_int] * 5 + [C.c_void_p]),
    "dllm_cluster_residual": (C.c_int, [C.c_void_p] * 5 + [C.c_int] * 4 + [C.c_void_p]),
    "dllm_nvfp4_quantize": (C.c_int, [C.c_void_p, C.c_float, C.c_void_p, C.c_void_p, C.c_long, C.c_int, C.c_void_p]),
    "dllm_nvfp4_dequantize": (C.c_int, [C.c_void_p, C.c_void_p, C.c_float, C.c_void_p, C.c_long, C.c_int, C.c_void_p]),
    "dllm_cluster_select": (C.c_int, [C.c_void_p] * 3 + [C.c_int] + [C.c_void_p] * 2 + [C.c_int] * 4 + [C.c_void_p]),
    "dllm_select_topk": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_float,
                                   C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p]),
    "dllm_layer_rho": (C.c_double, [C.c_int] + [C.c_double] * 5),
    "dllm_layer_budget": (C.c_int, [C.c_double, C.c_int]),
    "dllm_packed_layer_bytes": (C.c_size_t, [C.c_int] * 6),
    "dllm_pack_layer": (C.c_int, [C.c_void_p] * 9 + [C.c_int] * 5 + [C.c_float, C.c_float,
                                                                      C.c_int, C.c_int, C.c_void_p,
                                                                      C.c_size_t,
                                                                      C.POINTER(dllm_layer),
                                                                      C.c_void_p]),
    "dllm_refresh_workspace_bytes": (C.c_size_t, [C.POINTER(dllm_layer), C.c_int, C.c_int, C.c_int]),
    "dllm_sparse_layer_refresh": (C.c_int, [C.POINTER(dllm_layer), C.c_void_p, C.c_void_p,
                                            C.c_void_p, C.c_int, C.c_void_p, C.c_void_p,
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int,
                                            C.c_int, C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_layer_step_workspace_bytes": (C.c_size_t, [C.POINTER(dllm_layer)] + [C.c_int] * 5),
    "dllm_layer_step": (C.c_int, [C.POINTER(dllm_layer)] + [C.c_void_p] * 6 + [C.c_int] * 2 + [C.c_float]
                        + [C.c_void_p] * 5 + [C.c_int] * 3 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_set_pdl": (C.c_int, [C.c_int]),
    "dllm_timer_start": (C.c_int, [C.c_int, C.c_int]),
    "dllm_timer_stop": (C.c_int, [C.POINTER(C.c_double), C.POINTER(C.c_int)]),
    "dllm_launch_count": (C.c_ulonglong, []),
    "dllm_gemm_bf16": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                 C.c_int, C.c_void_p]),
    "dllm_gemm_plan": (C.c_int, [C.c_int] * 6 + [C.c_void_p]),
    "dllm_attention_workspace_bytes": (C.c_size_t, [C.c_int] * 6),
    "dllm_attention": (C.c_int, [C.c_void_p] * 6 + [C.c_int] * 7 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_embed": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_void_p] + [C.c_int] * 5
                   + [C.c_void_p]),
    "dllm_rows_rmsnorm": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_void_p, C.c_float, C.c_void_p]
                          + [C.c_int] * 4 + [C.c_void_p]),
    "dllm_check_wait_timeout": (C.c_int, [C.c_void_p, C.c_void_p]),
    "dllm_gather_rows": (C.c_int, [C.c_void_p] * 5 + [C.c_int] * 3 + [C.c_void_p]),
    "dllm_gather_rows_n": (C.c_int, [C.c_int] + [C.c_void_p] * 5 + [C.c_int] * 3 + [C.c_void_p]),
    "dllm_paged_append": (C.c_int, [C.c_void_p] * 3 + [C.c_longlong] * 3 + [C.c_void_p] * 2 + [C.c_float]
                          + [C.c_void_p] * 4 + [C.c_int] + [C.c_void_p] * 3 + [C.c_int] * 9 + [C.c_void_p]),
    "dllm_paged_append_at": (C.c_int, [C.c_void_p] * 3 + [C.c_longlong] * 3 + [C.c_void_p] * 2 + [C.c_float]
                             + [C.c_void_p] * 5 + [C.c_int] + [C.c_void_p] * 3 + [C.c_int] * 9 + [C.c_void_p]),
    "dllm_paged_append_f8": (C.c_int, [C.c_void_p] * 3 + [C.c_longlong] * 3 + [C.c_void_p] * 2 + [C.c_float]
                             + [C.c_void_p] * 5 + [C.c_int] + [C.c_void_p] * 5 + [C.c_int] * 8 + [C.c_void_p]),
    "dllm_paged_attention_f8_workspace_bytes": (C.c_size_t, [C.c_int] * 6),
    "dllm_paged_attention_f8": (C.c_int, [C.c_void_p, C.c_longlong] + [C.c_void_p] * 7 + [C.c_int] * 3 + [C.c_float]
                                + [C.c_void_p] * 2 + [C.c_int] * 7 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_paged_weights": (C.c_int, [C.c_void_p, C.c_longlong] + [C.c_void_p] * 5 + [C.c_int] * 3 + [C.c_float]
                           + [C.c_void_p] * 5 + [C.c_int] * 9 + [C.c_void_p]),
    "dllm_paged_evict_workspace_bytes": (C.c_size_t, [C.c_int] * 4),
    "dllm_paged_evict": (C.c_int, [C.c_void_p] * 6 + [C.c_int, C.c_void_p, C.c_int] + [C.c_void_p] * 3 + [C.c_int]
                         + [C.c_void_p] * 4 + [C.c_int] * 6 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_paged_attention_workspace_bytes": (C.c_size_t, [C.c_int] * 7),
    "dllm_paged_attention": (C.c_int, [C.c_void_p, C.c_longlong] + [C.c_void_p] * 5 + [C.c_int] * 3 + [C.c_float]
                             + [C.c_void_p] * 2 + [C.c_int] * 8 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_sample_workspace_bytes": (C.c_size_t, [C.c_int] * 3),
    "dllm_sample": (C.c_int, [C.c_void_p] * 9 + [C.c_int] * 4 + [C.c_void_p, C.c_size_t, C.c_void_p]),
    "dllm_commit_entropy_noalloc": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                              C.c_float, C.c_float] + [C.c_void_p] * 6),
    "dllm_commit_workspace_bytes": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "dllm_lmhead_workspace_bytes": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "dllm_lmhead_commit": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p] + [C.c_int] * 4 +
                           [C.c_float, C.c_float] + [C.c_void_p] * 6 + [C.c_size_t, C.c_void_p]),
    "dllm_commit_entropy": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                      C.c_float, C.c_float] + [C.c_void_p] * 6 +
                            [C.c_size_t, C.c_void_p]),
}


def exported_symbols():
    """Names of every entry point the binding expects the library to export."""
    return list(_SIGS)


def lib():
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise DllmError(f"libdllm.so not built ({LIB_PATH}); run __graft_entry__.build()")
            L = C.CDLL(LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = lib().dllm_last_error().decode(errors="replace")
        raise DllmError(f"{what} failed ({rc}): {msg}")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(device=None):
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DLLM_BF16
    if t.dtype == torch.float32:
        return DLLM_F32
    raise DllmError(f"unsupported dtype {t.dtype}")


def _cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise DllmError("tensors must be on a CUDA device")
            if not t.is_contiguous():
                raise DllmError("tensors must be contiguous")


_ws_cache: dict = {}


def _workspace(nbytes: int, device, tag: str) -> torch.Tensor:
    """Caller-side scratch buffer (the library itself never allocates).  One buffer is kept
    per (entry point, device) and reused by every call that passes no `ws`, so calls that
    are ordered on one stream share it safely; calls of the same entry point that may run
    concurrently (different streams without ordering, or different host threads, whose
    calls' launches may be interleaved on one stream) must each pass their own `ws`."""
    key = (tag, device.index if device.index is not None else torch.cuda.current_device())
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


# --------------------------------------------------------------------------- status
def check_status(reset: bool = True) -> int:
    st = C.c_uint(0)
    rc = lib().dllm_check_status(C.byref(st), 1 if reset else 0)
    if rc == -5:
        raise DllmError(f"device status 0x{st.value:x}: a kernel wait timed out")
    _check(rc, "dllm_check_status")
    return st.value


def dllm_check_wait_timeout():
    """Runs the library's bounded-wait diagnostic (about one second on the device) and
    returns (threads whose wait gave up, the return code of dllm_check_status after it,
    the status bits); the status word is cleared."""
    dev = torch.cuda.current_device()
    out = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(lib().dllm_check_wait_timeout(_ptr(out), _stream(dev)), "dllm_check_wait_timeout")
    st = C.c_uint(0)
    rc = lib().dllm_check_status(C.byref(st), 1)
    return int(out.item()), rc, st.value


# --------------------------------------------------------------------------- measurement
KERNELS = {"proxy_gemm": 1, "cosine": 2, "select": 3, "gather": 4, "qkv": 5, "attention": 6,
           "oproj": 7, "rmsnorm2": 8, "gateup": 9, "down": 10, "vocab": 11, "gemm": 12,
           "kl_drift": 13, "ce": 14, "polestar": 15, "cluster": 16, "paged_append": 17,
           "paged_attention": 18, "sample": 19, "paged_weights": 20, "paged_evict": 21}


def dllm_timer_start(kernel: str, max_launches: int) -> None:
    _check(lib().dllm_timer_start(KERNELS[kernel], int(max_launches)), "dllm_timer_start")


def dllm_timer_stop():
    """-> (total milliseconds over the timed launches, number of timed launches)."""
    ms, n = C.c_double(0), C.c_int(0)
    _check(lib().dllm_timer_stop(C.byref(ms), C.byref(n)), "dllm_timer_stop")
    return ms.value, n.value


def dllm_launch_count() -> int:
    return int(lib().dllm_launch_count())


def dllm_set_pdl(enable: bool) -> bool:
    """Programmatic dependent launch between the library's kernels (default on)."""
    return bool(lib().dllm_set_pdl(1 if enable else 0))


# --------------------------------------------------------------------------- proxy
def dllm_proxy_score(H, Pt, proxy_cache, proxy_cur=None, drift=None, ws=None):
    """H [B,N,d] (bf16|f32), Pt [r,d] same dtype, proxy_cache [B,N,r] f32 ->
    (proxy_cur [B,N,r] f32, drift [B,N] f32)."""
    B, N, d = H.shape
    r = Pt.shape[0]
    if Pt.shape != (r, d) or Pt.dtype != H.dtype:
        raise DllmError("Pt must be [r, d] with H's dtype")
    if proxy_cur is None:
        proxy_cur = torch.empty((B, N, r), dtype=torch.float32, device=H.device)
    if drift is None:
        drift = torch.empty((B, N), dtype=torch.float32, device=H.device)
    _cuda(H, Pt, proxy_cache, proxy_cur, drift)
    need = int(lib().dllm_proxy_workspace_bytes(B, N, d, r, _dtype_code(H)))
    if ws is None and need > 0:
        ws = _workspace(need, H.device, "proxy")
    _check(lib().dllm_proxy_score(_ptr(H), _ptr(Pt), _ptr(proxy_cache), _ptr(proxy_cur), _ptr(drift),
                                  B, N, d, r, _dtype_code(H), _ptr(ws), 0 if ws is None else ws.numel(),
                                  _stream(H.device)), "dllm_proxy_score")
    return proxy_cur, drift


def dllm_kl_drift(proxy_cur, proxy_cache, drift=None, ws=None):
    """proxy_cur, proxy_cache [B,N,r] f32 -> drift [B,N] f32 = KL of the rows' proxy-attention
    distributions (this step against the cached proxies)."""
    B, N, r = proxy_cur.shape
    if proxy_cache.shape != (B, N, r) or proxy_cur.dtype != torch.float32 or proxy_cache.dtype != torch.float32:
        raise DllmError("proxy_cur and proxy_cache must both be [B, N, r] float32")
    if drift is None:
        drift = torch.empty((B, N), dtype=torch.float32, device=proxy_cur.device)
    _cuda(proxy_cur, proxy_cache, drift)
    need = int(lib().dllm_kl_drift_workspace_bytes(B, N))
    if ws is None:
        ws = _workspace(need, proxy_cur.device, "kl")
    _check(lib().dllm_kl_drift(_ptr(proxy_cur), _ptr(proxy_cache), _ptr(drift), B, N, r, _ptr(ws), ws.numel(),
                               _stream(proxy_cur.device)), "dllm_kl_drift")
    return drift


def dllm_ce_step(conf, seen, undecided, committed, state, early=None, q_l=1e-3, q_v=1e-3, R=1e-2,
                 p_v0=1e-2, z=1.645, h_max=4, c_min=0.9):
    """Confidence extrapolation step: conf [B,M] f32, seen/undecided/committed [B,M] uint8,
    state [B,M,5] f32 (updated in place) -> early [B,M] uint8."""
    B, M = conf.shape
    if state.shape != (B, M, 5) or state.dtype != torch.float32 or conf.dtype != torch.float32:
        raise DllmError("conf [B, M] and state [B, M, 5] must be float32")
    for t in (seen, undecided, committed):
        if t.shape != (B, M) or t.dtype != torch.uint8:
            raise DllmError("seen, undecided, committed must be [B, M] uint8")
    if early is None:
        early = torch.empty((B, M), dtype=torch.uint8, device=conf.device)
    _cuda(conf, seen, undecided, committed, state, early)
    _check(lib().dllm_ce_step(_ptr(conf), _ptr(seen), _ptr(undecided), _ptr(committed), _ptr(state),
                              _ptr(early), B, M, float(q_l), float(q_v), float(R), float(p_v0), float(z),
                              int(h_max), float(c_min), _stream(conf.device)), "dllm_ce_step")
    return early


def dllm_polestar_commit(drift, conf, undecided, suffix, selected, history, commit=None, alpha=1.0, tau_s=0.9):
    """Drift-aware commit: drift, conf [B,M] f32; undecided, suffix, selected [B,M] uint8;
    history [B,M,2] f32 (updated in place) -> commit [B,M] uint8."""
    B, M = drift.shape
    if conf.shape != (B, M) or history.shape != (B, M, 2) or history.dtype != torch.float32:
        raise DllmError("conf [B, M] f32 and history [B, M, 2] f32 expected")
    for t in (undecided, suffix, selected):
        if t.shape != (B, M) or t.dtype != torch.uint8:
            raise DllmError("undecided, suffix, selected must be [B, M] uint8")
    if commit is None:
        commit = torch.empty((B, M), dtype=torch.uint8, device=drift.device)
    _cuda(drift, conf, undecided, suffix, selected, history, commit)
    _check(lib().dllm_polestar_commit(_ptr(drift), _ptr(conf), _ptr(undecided), _ptr(suffix), _ptr(selected),
                                      _ptr(history), _ptr(commit), B, M, float(alpha), float(tau_s),
                                      _stream(drift.device)), "dllm_polestar_commit")
    return commit


def dllm_spherical_kmeans(X, C, iters: int, assign=None, xnorm=None):
    """X [B,N,D] f32, C [B,K,D] f32 (initial; refined in place) -> (assign [B,N] int32, xnorm [B,N] f32)."""
    B, N, D = X.shape
    K = C.shape[1]
    if C.shape != (B, K, D) or X.dtype != torch.float32 or C.dtype != torch.float32:
        raise DllmError("X [B, N, D] and C [B, K, D] must be float32")
    if assign is None:
        assign = torch.empty((B, N), dtype=torch.int32, device=X.device)
    if xnorm is None:
        xnorm = torch.empty((B, N), dtype=torch.float32, device=X.device)
    _cuda(X, C, assign, xnorm)
    _check(lib().dllm_spherical_kmeans(_ptr(X), _ptr(C), _ptr(assign), _ptr(xnorm), B, N, D, K, int(iters),
                                       _stream(X.device)), "dllm_spherical_kmeans")
    return assign, xnorm


def dllm_cluster_residual(X, C, assign, xnorm, R=None):
    B, N, D = X.shape
    K = C.shape[1]
    if R is None:
        R = torch.empty_like(X)
    _cuda(X, C, assign, xnorm, R)
    _check(lib().dllm_cluster_residual(_ptr(X), _ptr(C), _ptr(assign), _ptr(xnorm), _ptr(R), B, N, D, K,
                                       _stream(X.device)), "dllm_cluster_residual")
    return R


def dllm_nvfp4_quantize(R, g: float, codes=None, scales=None):
    """R [rows, D] f32 -> (codes [rows, D/2] uint8, scales [rows, D/16] uint8)."""
    R2 = R.reshape(-1, R.shape[-1])
    rows, D = R2.shape
    if codes is None:
        codes = torch.empty((rows, D // 2), dtype=torch.uint8, device=R.device)
    if scales is None:
        scales = torch.empty((rows, D // 16), dtype=torch.uint8, device=R.device)
    _cuda(R2, codes, scales)
    _check(lib().dllm_nvfp4_quantize(_ptr(R2), float(g), _ptr(codes), _ptr(scales), rows, D, _stream(R.device)),
           "dllm_nvfp4_quantize")
    return codes, scales


def dllm_nvfp4_dequantize(codes, scales, g: float, out=None):
    """codes [rows, D/2] uint8, scales [rows, D/16] uint8 -> out [rows, D] f32."""
    rows, half = codes.shape
    D = half * 2
    if out is None:
        out = torch.empty((rows, D), dtype=torch.float32, device=codes.device)
    _cuda(codes, scales, out)
    _check(lib().dllm_nvfp4_dequantize(_ptr(codes), _ptr(scales), float(g), _ptr(out), rows, D,
                                       _stream(codes.device)), "dllm_nvfp4_dequantize")
    return out


def dllm_cluster_select(C_now, C_prev, assign, kc: int, idx=None, count=None):
    """-> (idx [B,N] int32 ascending member rows of the kc most drifted clusters, -1 padded; count [B])."""
    B, K, D = C_now.shape
    N = assign.shape[1]
    if idx is None:
        idx = torch.empty((B, N), dtype=torch.int32, device=C_now.device)
    if count is None:
        count = torch.empty((B,), dtype=torch.int32, device=C_now.device)
    _cuda(C_now, C_prev, assign, idx, count)
    _check(lib().dllm_cluster_select(_ptr(C_now), _ptr(C_prev), _ptr(assign), int(kc), _ptr(idx), _ptr(count),
                                     B, N, D, K, _stream(C_now.device)), "dllm_cluster_select")
    return idx, count


# --------------------------------------------------------------------------- selection
def dllm_select_topk(drift, forced, k: int, min_drift: float = 1e-6, idx=None, count=None):
    """drift [B,N] f32, forced [B,F] int32 (-1 padded) or None ->
    (idx [B,N] int32 ascending, -1 padded;  count [B] int32)."""
    B, N = drift.shape
    F = 0 if forced is None else forced.shape[1]
    if idx is None:
        idx = torch.empty((B, N), dtype=torch.int32, device=drift.device)
    if count is None:
        count = torch.empty((B,), dtype=torch.int32, device=drift.device)
    _cuda(drift, forced, idx, count)
    _check(lib().dllm_select_topk(_ptr(drift), _ptr(forced), F, int(k), float(min_drift), _ptr(idx),
                                  _ptr(count), B, N, _stream(drift.device)), "dllm_select_topk")
    return idx, count


def dllm_layer_rho(l: int, base=0.05, peak=0.30, centre=16.0, sigma_left=6.0, sigma_right=6.0):
    return float(lib().dllm_layer_rho(int(l), base, peak, centre, sigma_left, sigma_right))


def dllm_layer_budget(rho: float, N: int) -> int:
    return int(lib().dllm_layer_budget(float(rho), int(N)))


# --------------------------------------------------------------------------- layer
class Layer:
    """Packed weights of one layer on the device plus the dllm_layer descriptor."""

    def __init__(self, packed: torch.Tensor, desc: dllm_layer):
        self.packed = packed
        self.desc = desc

    @property
    def dtype(self):
        return torch.bfloat16 if self.desc.dtype == DLLM_BF16 else torch.float32


def dllm_pack_layer(w: dict, n_q: int, n_kv: int, hd: int, eps: float = 1e-5,
                    rope_theta: float = 10000.0, use_rope: bool = True) -> Layer:
    """w: device tensors in nn.Linear layout (w_q, w_k, w_v, w_o, w_g, w_u, w_d, gamma1, gamma2)."""
    keys = ("w_q", "w_k", "w_v", "w_o", "w_g", "w_u", "w_d", "gamma1", "gamma2")
    ts = [w[k].contiguous() for k in keys]
    _cuda(*ts)
    dt = _dtype_code(ts[0])
    if any(t.dtype != ts[0].dtype for t in ts):
        raise DllmError("all weights must share one dtype")
    d = ts[7].shape[0]
    F = ts[4].shape[0]
    nbytes = lib().dllm_packed_layer_bytes(d, n_q, n_kv, hd, F, dt)
    packed = torch.empty(nbytes, dtype=torch.uint8, device=ts[0].device)
    desc = dllm_layer()
    _check(lib().dllm_pack_layer(*[_ptr(t) for t in ts], d, n_q, n_kv, hd, F, float(eps),
                                 float(rope_theta), 1 if use_rope else 0, dt, _ptr(packed), nbytes,
                                 C.byref(desc), _stream(ts[0].device)), "dllm_pack_layer")
    return Layer(packed, desc)


def dllm_refresh_workspace_bytes(layer: Layer, B: int, N: int, k_max: int) -> int:
    return int(lib().dllm_refresh_workspace_bytes(C.byref(layer.desc), B, N, k_max))


def dllm_sparse_layer_refresh(layer: Layer, H_in, idx, count, k_max: int, K_cache, V_cache,
                              H_out_cache, proxy_cache=None, proxy_cur=None, ws=None):
    """Refreshes the cache rows idx[b, :count[b]] in place (K_cache, V_cache,
    H_out_cache, and proxy_cache when given)."""
    B, N, d = H_in.shape
    r = 0 if proxy_cache is None else proxy_cache.shape[-1]
    _cuda(H_in, idx, count, K_cache, V_cache, H_out_cache, proxy_cache, proxy_cur)
    need = dllm_refresh_workspace_bytes(layer, B, N, k_max)
    if ws is None:
        ws = _workspace(need, H_in.device, "refresh")
    _check(lib().dllm_sparse_layer_refresh(C.byref(layer.desc), _ptr(H_in), _ptr(idx), _ptr(count),
                                           int(k_max), _ptr(K_cache), _ptr(V_cache),
                                           _ptr(H_out_cache), _ptr(proxy_cache), _ptr(proxy_cur), r,
                                           B, N, _ptr(ws), ws.numel(), _stream(H_in.device)),
           "dllm_sparse_layer_refresh")
    return K_cache, V_cache, H_out_cache


def dllm_layer_step_workspace_bytes(layer: Layer, B: int, N: int, r: int, F: int, k: int) -> int:
    return int(lib().dllm_layer_step_workspace_bytes(C.byref(layer.desc), B, N, r, F, k))


def dllm_layer_step(layer: Layer, Pt, H_in, proxy_cache, proxy_cur, drift, forced, k: int, idx, count,
                    K_cache, V_cache, H_out_cache, min_drift: float = 1e-6, ws=None):
    """One layer's sparse step (proxy + drift, selection with the forced rows, refresh of
    the selected rows) in one library call; writes proxy_cur, drift, idx, count and the
    refreshed cache rows in place."""
    B, N, d = H_in.shape
    r = proxy_cache.shape[-1]
    F = 0 if forced is None else forced.shape[1]
    _cuda(Pt, H_in, proxy_cache, proxy_cur, drift, forced, idx, count, K_cache, V_cache, H_out_cache)
    need = dllm_layer_step_workspace_bytes(layer, B, N, r, F, k)
    if ws is None:
        ws = _workspace(need, H_in.device, "layer_step")
    _check(lib().dllm_layer_step(C.byref(layer.desc), _ptr(Pt), _ptr(H_in), _ptr(proxy_cache), _ptr(proxy_cur),
                                 _ptr(drift), _ptr(forced), F, int(k), float(min_drift), _ptr(idx), _ptr(count),
                                 _ptr(K_cache), _ptr(V_cache), _ptr(H_out_cache), B, N, r, _ptr(ws), ws.numel(),
                                 _stream(H_in.device)), "dllm_layer_step")
    return idx, count


# --------------------------------------------------------------------------- attention alone
def dllm_attention(Q, K_cache, V_cache, idx, count, k_max: int, A=None, ws=None):
    """Q [B*k_max, n_q*hd], caches [B, N, n_kv, hd] -> A [B*k_max, n_q*hd] (zeros for rows
    that are not live)."""
    Bn, N, n_kv, hd = K_cache.shape
    n_q = Q.shape[1] // hd
    if A is None:
        A = torch.empty_like(Q)
    _cuda(Q, K_cache, V_cache, A, idx, count)
    dt = _dtype_code(Q)
    need = int(lib().dllm_attention_workspace_bytes(Bn, N, int(k_max), n_q, hd, dt))
    if ws is None and need > 0:
        ws = _workspace(need, Q.device, "attention")
    _check(lib().dllm_attention(_ptr(Q), _ptr(K_cache), _ptr(V_cache), _ptr(A), _ptr(idx), _ptr(count),
                                int(k_max), Bn, N, n_q, n_kv, hd, dt, _ptr(ws),
                                0 if ws is None else ws.numel(), _stream(Q.device)), "dllm_attention")
    return A


# --------------------------------------------------------------------------- embedding, final norm
def dllm_embed(E, tokens, H, rows=None):
    """H[b, i] = E[tokens[b, i]] for all i, or for the positions rows[b, :] only."""
    B, N, d = H.shape
    V = E.shape[0]
    R = 0 if rows is None else rows.shape[1]
    _cuda(E, tokens, H, rows)
    _check(lib().dllm_embed(_ptr(E), _ptr(tokens), _ptr(rows), R, _ptr(H), B, N, d, V,
                            _dtype_code(H), _stream(H.device)), "dllm_embed")
    return H


def dllm_rows_rmsnorm(H, rows, gamma, eps: float = 1e-5, out=None):
    """out [B*R, d] = RMSNorm(H[b, rows[b, j]]) * gamma."""
    B, N, d = H.shape
    R = rows.shape[1]
    if out is None:
        out = torch.empty((B * R, d), dtype=H.dtype, device=H.device)
    _cuda(H, rows, gamma, out)
    _check(lib().dllm_rows_rmsnorm(_ptr(H), _ptr(rows), R, _ptr(gamma), float(eps), _ptr(out), B, N,
                                   d, _dtype_code(H), _stream(H.device)), "dllm_rows_rmsnorm")
    return out


def dllm_gather_rows(src, idx, count, k_max: int, dst=None):
    """src [B, N, ...] (any row layout, rows of a multiple of 16 bytes) ->
    dst [B*k_max, ...]: the rows idx[b, :count[b]] packed per sequence, zeros after."""
    Bn, N = src.shape[0], src.shape[1]
    row_bytes = src[0, 0].numel() * src.element_size()
    if dst is None:
        dst = torch.empty((Bn * k_max,) + tuple(src.shape[2:]), dtype=src.dtype, device=src.device)
    if dst.numel() * dst.element_size() < Bn * k_max * row_bytes:
        raise DllmError("dst holds fewer than B*k_max rows")
    _cuda(src, idx, count, dst)
    _check(lib().dllm_gather_rows(_ptr(src), _ptr(idx), _ptr(count), int(k_max), _ptr(dst), Bn, N, row_bytes,
                                  _stream(src.device)), "dllm_gather_rows")
    return dst


def dllm_gather_rows_n(srcs, idx, count, k_max: int, dsts=None):
    """The rows idx[b, :count[b]] of several caches [B, N, ...] sharing one selection,
    packed per sequence in one launch -> list of dst [B*k_max, ...] (zeros after)."""
    srcs = list(srcs)
    if not 1 <= len(srcs) <= 4:
        raise DllmError("between 1 and 4 caches")
    Bn, N = srcs[0].shape[0], srcs[0].shape[1]
    if dsts is None:
        dsts = [torch.empty((Bn * k_max,) + tuple(s.shape[2:]), dtype=s.dtype, device=s.device) for s in srcs]
    rb = []
    for s_, d_ in zip(srcs, dsts):
        if s_.shape[:2] != (Bn, N):
            raise DllmError("the caches must share [B, N]")
        rb.append(s_[0, 0].numel() * s_.element_size())
        if d_.numel() * d_.element_size() < Bn * k_max * rb[-1]:
            raise DllmError("dst holds fewer than B*k_max rows")
    _cuda(*srcs, *dsts, idx, count)
    n = len(srcs)
    src_arr = (C.c_void_p * n)(*[_ptr(t) for t in srcs])
    dst_arr = (C.c_void_p * n)(*[_ptr(t) for t in dsts])
    rb_arr = (C.c_int * n)(*rb)
    _check(lib().dllm_gather_rows_n(n, src_arr, dst_arr, rb_arr, _ptr(idx), _ptr(count), int(k_max), Bn, N,
                                    _stream(srcs[0].device)), "dllm_gather_rows_n")
    return dsts


# --------------------------------------------------------------------------- plain GEMM
def dllm_gemm_bf16(X, W, out=None, splits: int = 0):
    """X [M, K] bf16, W [N_out, K] bf16 -> out [M, N_out] fp32 = X W^T (tensor cores)."""
    M, K = X.shape
    N_out = W.shape[0]
    if W.shape != (N_out, K) or X.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise DllmError("X [M,K] and W [N_out,K] must be bf16")
    if out is None:
        out = torch.empty((M, N_out), dtype=torch.float32, device=X.device)
    _cuda(X, W, out)
    _check(lib().dllm_gemm_bf16(_ptr(X), _ptr(W), _ptr(out), M, N_out, K, int(splits),
                                _stream(X.device)), "dllm_gemm_bf16")
    return out


PLAN_FIELDS = ("BN", "splits", "stages", "tok_tiles", "w_tiles", "xrows", "smem", "ctas_per_sm")


def dllm_gemm_plan(M: int, N_out: int, K: int, splits: int = 0, sms: int = 152, slices: int = 0):
    """The tensor-core GEMM's launch plan for this shape on `sms` SMs (host only, no GPU
    needed) -> dict of PLAN_FIELDS.  slices: 0 the plain GEMM, 1 the proxy projection's
    independent K slices, 2 the proxy projection with its drift in the epilogue."""
    info = (C.c_int32 * 8)()
    _check(lib().dllm_gemm_plan(int(M), int(N_out), int(K), int(splits), int(sms), int(slices), info),
           "dllm_gemm_plan")
    return dict(zip(PLAN_FIELDS, list(info)))


# --------------------------------------------------------------------------- vocab
def dllm_commit_entropy(logits, valid, conf_thresh: float = 0.9, tau: float = 2.0, out=None, ws=None):
    """logits [B,M,V] f32, valid [B,M] uint8 ->
    (token [B,M] int32, conf [B,M], entropy [B,M], max_entropy [B], full_next [B] int32)."""
    B, M, V = logits.shape
    dev = logits.device
    if out is None:
        out = (torch.empty((B, M), dtype=torch.int32, device=dev),
               torch.empty((B, M), dtype=torch.float32, device=dev),
               torch.empty((B, M), dtype=torch.float32, device=dev),
               torch.empty((B,), dtype=torch.float32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    tok, conf, ent, E, full = out
    _cuda(logits, valid, *out)
    need = int(lib().dllm_commit_workspace_bytes(B, M, V))
    if ws is None:
        ws = _workspace(need, dev, "commit")
    _check(lib().dllm_commit_entropy(_ptr(logits), _ptr(valid), B, M, V, float(conf_thresh),
                                     float(tau), _ptr(tok), _ptr(conf), _ptr(ent), _ptr(E),
                                     _ptr(full), _ptr(ws), ws.numel(), _stream(dev)),
           "dllm_commit_entropy")
    return out


def dllm_lmhead_commit(X, W_lm, valid, conf_thresh: float = 0.9, tau: float = 2.0, out=None, ws=None):
    """X [B*M, d] bf16 (normalised block rows), W_lm [V, d] bf16, valid [B, M] uint8 ->
    the outputs of dllm_commit_entropy on X W_lm^T, without materialising the logits."""
    B, M = valid.shape
    V, d = W_lm.shape
    if X.shape != (B * M, d) or X.dtype != torch.bfloat16 or W_lm.dtype != torch.bfloat16:
        raise DllmError("X [B*M, d] and W_lm [V, d] must be bf16")
    dev = X.device
    if out is None:
        out = (torch.empty((B, M), dtype=torch.int32, device=dev),
               torch.empty((B, M), dtype=torch.float32, device=dev),
               torch.empty((B, M), dtype=torch.float32, device=dev),
               torch.empty((B,), dtype=torch.float32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    tok, conf, ent, E, full = out
    _cuda(X, W_lm, valid, *out)
    need = int(lib().dllm_lmhead_workspace_bytes(B, M, V))
    if ws is None:
        ws = _workspace(need, dev, "lmhead")
    _check(lib().dllm_lmhead_commit(_ptr(X), _ptr(W_lm), _ptr(valid), B, M, V, d, float(conf_thresh),
                                    float(tau), _ptr(tok), _ptr(conf), _ptr(ent), _ptr(E), _ptr(full),
                                    _ptr(ws), ws.numel(), _stream(dev)),
           "dllm_lmhead_commit")
    return out


def dllm_commit_entropy_noalloc(logits, valid, conf_thresh: float = 0.9, tau: float = 2.0, out=None):
    """dllm_commit_entropy for callers that cannot allocate device memory: the library
    keeps the scratch in its own fixed device array (no workspace argument).  The caller
    still provides the output tensors (allocated here when `out` is None)."""
    B, M, V = logits.shape
    dev = logits.device
    if out is None:
        out = (torch.empty((B, M), dtype=torch.int32, device=dev),
               torch.empty((B, M), dtype=torch.float32, device=dev),
               torch.empty((B, M), dtype=torch.float32, device=dev),
               torch.empty((B,), dtype=torch.float32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    tok, conf, ent, E, full = out
    _cuda(logits, valid, *out)
    _check(lib().dllm_commit_entropy_noalloc(_ptr(logits), _ptr(valid), B, M, V, float(conf_thresh),
                                             float(tau), _ptr(tok), _ptr(conf), _ptr(ent), _ptr(E),
                                             _ptr(full), _stream(dev)),
           "dllm_commit_entropy_noalloc")
    return out


# --------------------------------------------------------------------------- paged cache, sampling
_NO_GUARD = contextlib.nullcontext()


class _Scratch(threading.local):
    """A host thread's scratch buffers: two threads that issue on one stream may have their calls'
    launches interleaved there, so they must not share one either."""

    def __init__(self):
        self.bufs: dict = {}


_scratch = _Scratch()


def _stream_workspace(nbytes: int, device, dev: int, tag: str) -> torch.Tensor:
    """Scratch of the paged attention and the sampling when the caller passes no `ws`: one buffer per (host
    thread, device, stream), so calls that may overlap do not share it.  Under capture each call gets its
    own from the graph's memory, which lives as long as the graph does."""
    if _getdev() != dev:
        with torch.cuda.device(dev):
            return _stream_workspace(nbytes, device, dev, tag)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    bufs, key = _scratch.bufs, (tag, dev, _rawstream(dev))
    buf = bufs.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = bufs[key] = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return buf


# The paged calls are made once per layer and token, where their own cost on the host is most of
# a small call's: checks are inline, devices compared as ints (-1 for the CPU), pointers passed
# as ints.
_CODE = {torch.bfloat16: DLLM_BF16, torch.float32: DLLM_F32}
_getdev = torch._C._cuda_getDevice
_rawstream = torch._C._cuda_getCurrentRawStream


def _run(fn, what: str, dev: int, args):
    """fn(*args, stream) with `dev` as the current device, on its current stream."""
    if _getdev() == dev:
        rc = fn(*args, _rawstream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _rawstream(dev))
    if rc != 0:
        _check(rc, what)


def _same(dev: int, ts):
    """Every tensor on CUDA device dev, and contiguous."""
    if dev < 0:
        raise DllmError("tensors must be on a CUDA device")
    for t in ts:
        if t.get_device() != dev:
            raise DllmError("tensors must be on one CUDA device")
        if not t.is_contiguous():
            raise DllmError("tensors must be contiguous")


def _row_stride(t, T: int, h: int, hd: int, what: str) -> int:
    """Stride between the rows of t [T, h, hd] (a slice of a wider one, maybe)."""
    s = t.stride()
    if s[2] != 1 or (h > 1 and s[1] != hd):
        raise DllmError(f"{what} must be [T, heads, hd] with each row's heads contiguous")
    return s[0] if T > 1 else h * hd   # (one row, or none: its stride is arbitrary)


def _paged_shapes(K_pages, V_pages, page_table, q_start, kv_len):
    sh, ts, i32 = K_pages.shape, page_table.shape, torch.int32
    if len(sh) != 4 or V_pages.shape != sh or V_pages.dtype != K_pages.dtype:
        raise DllmError("K_pages and V_pages must both be [n_pages, page, n_kv, hd] of one dtype")
    if (len(ts) != 2 or q_start.shape != (ts[0] + 1,) or kv_len.shape != ts[:1] or page_table.dtype != i32
            or q_start.dtype != i32 or kv_len.dtype != i32):
        raise DllmError("page_table [B, max_pages], q_start [B + 1], kv_len [B] int32 expected")
    return sh, ts


def _append_args(K, V, K_pages, V_pages, page_table, q_start, kv_len, Q, Q_out, gamma_q, gamma_k, inv_freq, pos_base, cdt):
    """The checked arguments that the appends share; cdt is the type of Q_out and the gains."""
    (n_pages, page, n_kv, hd), (B, max_pages) = _paged_shapes(K_pages, V_pages, page_table, q_start, kv_len)
    dt, dev, sh = K.dtype, K.get_device(), K.shape
    if len(sh) != 3 or sh[1] != n_kv or sh[2] != hd or V.shape != sh or V.dtype != dt:
        raise DllmError("K and V must both be [T, n_kv, hd] of one dtype")
    T = sh[0]
    dense = [K_pages, V_pages, page_table, q_start, kv_len]
    q = qo = gq = gk = freq = base = None
    qs = n_q = 0
    if Q is None:
        if Q_out is not None or gamma_q is not None:
            raise DllmError("Q_out and gamma_q need Q")
    else:
        sh = Q.shape
        if len(sh) != 3 or sh[0] != T or sh[2] != hd or Q.dtype != dt:
            raise DllmError("Q must be [T, n_q, hd] with K's dtype")
        n_q = sh[1]
        qs = _row_stride(Q, T, n_q, hd, "Q")
        if Q_out is None:
            Q_out = torch.empty((T, n_q, hd), dtype=cdt, device=K.device)
        elif Q_out.numel() != T * n_q * hd or Q_out.dtype != cdt:
            raise DllmError("Q_out must hold [T, n_q, hd] in the cache's dtype")
        if Q.get_device() != dev:
            raise DllmError("tensors must be on one CUDA device")
        q, qo = Q.data_ptr(), Q_out.data_ptr()
        dense.append(Q_out)
    if gamma_q is not None:
        if gamma_q.shape != (hd,) or gamma_q.dtype != cdt:
            raise DllmError("gamma_q must be [hd] in the cache's dtype")
        gq = gamma_q.data_ptr()
        dense.append(gamma_q)
    if gamma_k is not None:
        if gamma_k.shape != (hd,) or gamma_k.dtype != cdt:
            raise DllmError("gamma_k must be [hd] in the cache's dtype")
        gk = gamma_k.data_ptr()
        dense.append(gamma_k)
    if isinstance(inv_freq, Layer):
        if inv_freq.desc.hd != hd:
            raise DllmError("the layer's head dimension differs from the cache's")
        freq = inv_freq.desc.rope_inv_freq if inv_freq.desc.use_rope else None
        dense.append(inv_freq.packed)
    elif inv_freq is not None:
        if inv_freq.shape != (hd // 2,) or inv_freq.dtype != torch.float32:
            raise DllmError("inv_freq must be [hd/2] float32")
        freq = inv_freq.data_ptr()
        dense.append(inv_freq)
    if pos_base is not None:
        if pos_base.shape != (B,) or pos_base.dtype != torch.int32:
            raise DllmError("pos_base must be [B] int32")
        base = pos_base.data_ptr()
        dense.append(pos_base)
    _same(dev, dense)
    if V.get_device() != dev:
        raise DllmError("tensors must be on one CUDA device")
    if dt not in _CODE or cdt not in _CODE:
        raise DllmError(f"unsupported dtype {dt}, {cdt}")
    head = (q, K.data_ptr(), V.data_ptr(), qs, _row_stride(K, T, n_kv, hd, "K"), _row_stride(V, T, n_kv, hd, "V"), gq, gk)
    at = (q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), max_pages, qo, K_pages.data_ptr(), V_pages.data_ptr())
    return Q_out, dev, head, freq, base, at, (T, B, n_q, n_kv, hd, page, n_pages, _CODE[dt])


def dllm_paged_append(K, V, K_pages, V_pages, page_table, q_start, kv_len, Q=None, Q_out=None, gamma_q=None,
                      gamma_k=None, eps: float = 1e-5, inv_freq=None, pos_base=None):
    """The new rows' keys and values [T, n_kv, hd] (f32, or the cache's dtype) into their pages and
    the queries Q [T, n_q, hd] into Q_out (cache's dtype): per-head RMS norm with gamma_q, gamma_k
    [hd] when given, rotation by inv_freq ([hd/2] f32, or a packed Layer's table) when given, at the slot's
    index plus pos_base[b] ([B] int32, None = 0).  Rows may be slices of one wider projection output.
    -> Q_out (None without Q)."""
    cdt = K_pages.dtype
    Q_out, dev, head, freq, base, at, sizes = _append_args(K, V, K_pages, V_pages, page_table, q_start, kv_len, Q, Q_out,
                                                           gamma_q, gamma_k, inv_freq, pos_base, cdt)
    L = _lib or lib()
    if base is None:
        _run(L.dllm_paged_append, "dllm_paged_append", dev, (*head, eps, freq, *at, *sizes, _CODE[cdt]))
    else:
        _run(L.dllm_paged_append_at, "dllm_paged_append_at", dev, (*head, eps, freq, base, *at, *sizes, _CODE[cdt]))
    return Q_out


# (a torch without one of them serves the calls that need neither)
_E4M3, _E8M0 = getattr(torch, "float8_e4m3fn", None), getattr(torch, "float8_e8m0fnu", None)


def _scales(K_pages, *scales):
    """8-bit pages and the scales that go with them."""
    if _E4M3 is None or _E8M0 is None:
        raise DllmError("8-bit pages need a torch with float8_e4m3fn and float8_e8m0fnu")
    if K_pages.dtype != _E4M3:
        raise DllmError("8-bit pages must be float8_e4m3fn")
    want = K_pages.shape[::2][:2] if K_pages.dim() == 4 else None
    for t in scales:
        if t is None or t.shape != want or t.dtype != _E8M0:
            raise DllmError("scales must be [n_pages, n_kv] float8_e8m0fnu")


def dllm_paged_append_f8(K, V, K_pages, V_pages, K_scale, V_scale, page_table, q_start, kv_len, Q=None, Q_out=None,
                         gamma_q=None, gamma_k=None, eps: float = 1e-5, inv_freq=None, pos_base=None):
    """dllm_paged_append into 8-bit pages: K_pages, V_pages [n_pages, page, n_kv, hd] float8_e4m3fn with
    K_scale, V_scale [n_pages, n_kv] float8_e8m0fnu.  The rows are f32 or bf16; gains and Q_out bf16."""
    _scales(K_pages, K_scale, V_scale)
    Q_out, dev, head, freq, base, at, sizes = _append_args(K, V, K_pages, V_pages, page_table, q_start, kv_len, Q, Q_out,
                                                           gamma_q, gamma_k, inv_freq, pos_base, torch.bfloat16)
    _same(dev, (K_scale, V_scale))
    _run((_lib or lib()).dllm_paged_append_f8, "dllm_paged_append_f8", dev,
         (*head, eps, freq, base, *at, K_scale.data_ptr(), V_scale.data_ptr(), *sizes))
    return Q_out


def dllm_paged_attention_workspace_bytes(T: int, B: int, max_new: int, n_q: int, n_kv: int, hd: int, dtype) -> int:
    code = DLLM_BF16 if dtype == torch.bfloat16 else DLLM_F32
    return int(lib().dllm_paged_attention_workspace_bytes(T, B, max_new, n_q, n_kv, hd, code))


def dllm_paged_attention(Q, K_pages, V_pages, page_table, q_start, kv_len, max_new: int, mask_block: int = 0,
                         scale: float | None = None, A=None, lse=None, ws=None):
    """Attention of the new rows Q [T, n_q, hd] (rows may be strided) over the pages -> A [T, n_q, hd].
    mask_block: 0 all keys, 1 causal, m blocks of m positions.  lse [T, n_q] f32 (optional) receives
    the rows' log-sum-exp.  max_new: host upper bound on a sequence's new rows."""
    (n_pages, page, n_kv, hd), (B, max_pages) = _paged_shapes(K_pages, V_pages, page_table, q_start, kv_len)
    sh, dt, dev = Q.shape, Q.dtype, Q.get_device()
    if len(sh) != 3 or sh[2] != hd or dt != K_pages.dtype or dt not in _CODE:
        raise DllmError("Q must be [T, n_q, hd] with the cache's dtype")
    T, n_q, _ = sh
    if A is None:
        A = torch.empty((T, n_q, hd), dtype=dt, device=Q.device)
    elif A.numel() != T * n_q * hd or A.dtype != dt:
        raise DllmError("A must hold [T, n_q, hd] in Q's dtype")
    dense = [K_pages, V_pages, page_table, q_start, kv_len, A]
    if lse is not None:
        if lse.shape != (T, n_q) or lse.dtype != torch.float32:
            raise DllmError("lse must be [T, n_q] float32")
        dense.append(lse)
    if ws is not None:
        dense.append(ws)
    _same(dev, dense)
    L, code = _lib or lib(), _CODE[dt]
    if ws is None:
        with torch.cuda.device(dev) if _getdev() != dev else _NO_GUARD:
            ws = _stream_workspace(L.dllm_paged_attention_workspace_bytes(T, B, max_new, n_q, n_kv, hd, code), Q.device,
                                   dev, "paged_attention")
    _run(L.dllm_paged_attention, "dllm_paged_attention", dev,
         (Q.data_ptr(), _row_stride(Q, T, n_q, hd, "Q"), K_pages.data_ptr(), V_pages.data_ptr(), q_start.data_ptr(),
          kv_len.data_ptr(), page_table.data_ptr(), max_pages, max_new, mask_block,
          1.0 / hd ** 0.5 if scale is None else scale, A.data_ptr(), None if lse is None else lse.data_ptr(), T, B, n_q,
          n_kv, hd, page, n_pages, code, ws.data_ptr(), ws.numel() * ws.element_size()))
    return A


def dllm_paged_attention_f8_workspace_bytes(T: int, B: int, max_new: int, n_q: int, n_kv: int, hd: int) -> int:
    return int(lib().dllm_paged_attention_f8_workspace_bytes(T, B, max_new, n_q, n_kv, hd))


def dllm_paged_attention_f8(Q, K_pages, V_pages, K_scale, V_scale, page_table, q_start, kv_len, max_new: int,
                            mask_block: int = 0, scale: float | None = None, A=None, lse=None, ws=None):
    """dllm_paged_attention over 8-bit pages (float8_e4m3fn with float8_e8m0fnu scales [n_pages, n_kv]); Q, A bf16."""
    _scales(K_pages, K_scale, V_scale)
    (n_pages, page, n_kv, hd), (B, max_pages) = _paged_shapes(K_pages, V_pages, page_table, q_start, kv_len)
    sh, dt, dev = Q.shape, Q.dtype, Q.get_device()
    if len(sh) != 3 or sh[2] != hd or dt != torch.bfloat16:
        raise DllmError("Q must be [T, n_q, hd] bfloat16")
    T, n_q, _ = sh
    if A is None:
        A = torch.empty((T, n_q, hd), dtype=dt, device=Q.device)
    elif A.numel() != T * n_q * hd or A.dtype != dt:
        raise DllmError("A must hold [T, n_q, hd] in Q's dtype")
    dense = [K_pages, V_pages, K_scale, V_scale, page_table, q_start, kv_len, A]
    if lse is not None:
        if lse.shape != (T, n_q) or lse.dtype != torch.float32:
            raise DllmError("lse must be [T, n_q] float32")
        dense.append(lse)
    if ws is not None:
        dense.append(ws)
    _same(dev, dense)
    L = _lib or lib()
    if ws is None:
        with torch.cuda.device(dev) if _getdev() != dev else _NO_GUARD:
            ws = _stream_workspace(L.dllm_paged_attention_f8_workspace_bytes(T, B, max_new, n_q, n_kv, hd), Q.device, dev,
                                   "paged_attention_f8")
    _run(L.dllm_paged_attention_f8, "dllm_paged_attention_f8", dev,
         (Q.data_ptr(), _row_stride(Q, T, n_q, hd, "Q"), K_pages.data_ptr(), V_pages.data_ptr(), K_scale.data_ptr(),
          V_scale.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), max_pages, max_new, mask_block,
          1.0 / hd ** 0.5 if scale is None else scale, A.data_ptr(), None if lse is None else lse.data_ptr(), T, B, n_q,
          n_kv, hd, page, n_pages, ws.data_ptr(), ws.numel() * ws.element_size()))
    return A


_PAGE_CODE = {torch.bfloat16: DLLM_BF16, torch.float32: DLLM_F32, _E4M3: DLLM_E4M3}


def _slot_arrays(B: int, n_kv: int, scores, tags):
    """score-like and slot_pos-like arrays [B, n_kv, slots] -> slots."""
    sh = scores[0].shape
    if len(sh) != 3 or sh[0] != B or sh[1] != n_kv:
        raise DllmError("score must be [B, n_kv, slots] float32")
    for t in scores:
        if t.shape != sh or t.dtype != torch.float32:
            raise DllmError("score and score_out must both be [B, n_kv, slots] float32")
    for t in tags:
        if t.shape != sh or t.dtype != torch.int32:
            raise DllmError("slot_pos must be [B, n_kv, slots] int32, as score")
    return sh[2]


def dllm_paged_weights(Q, K_pages, page_table, q_start, kv_len, max_new: int, lse, score, slot_pos=None, K_scale=None,
                       mask_block: int = 0, scale: float | None = None, pos_base=None, score_out=None):
    """Adds the attention weights of the new rows Q [T, n_q, hd], with their lse [T, n_q] f32 from the attention, to the
    keys' score [B, n_kv, slots] f32 (into score_out when given, else in place) -> score_out.  The new rows' own keys
    start from 0, and their positions go to slot_pos [B, n_kv, slots] int32.  Pages bf16, f32, or 8-bit with K_scale."""
    (n_pages, page, n_kv, hd), (B, max_pages) = _paged_shapes(K_pages, K_pages, page_table, q_start, kv_len)
    sh, dt, dev = Q.shape, K_pages.dtype, Q.get_device()
    if dt not in _PAGE_CODE:
        raise DllmError(f"unsupported dtype {dt}")
    if len(sh) != 3 or sh[2] != hd or Q.dtype != (torch.bfloat16 if dt == _E4M3 else dt):
        raise DllmError("Q must be [T, n_q, hd] with the cache's dtype (bfloat16 for 8-bit pages)")
    T, n_q, _ = sh
    if dt == _E4M3:
        _scales(K_pages, K_scale)
    elif K_scale is not None:
        raise DllmError("K_scale goes with 8-bit pages")
    if lse.shape != (T, n_q) or lse.dtype != torch.float32:
        raise DllmError("lse must be [T, n_q] float32")
    if score_out is None:
        score_out = score
    slots = _slot_arrays(B, n_kv, (score, score_out), () if slot_pos is None else (slot_pos,))
    dense = [K_pages, page_table, q_start, kv_len, lse, score, score_out]
    dense += [t for t in (slot_pos, K_scale, pos_base) if t is not None]
    if pos_base is not None and (pos_base.shape != (B,) or pos_base.dtype != torch.int32):
        raise DllmError("pos_base must be [B] int32")
    _same(dev, dense)
    _run((_lib or lib()).dllm_paged_weights, "dllm_paged_weights", dev,
         (Q.data_ptr(), _row_stride(Q, T, n_q, hd, "Q"), K_pages.data_ptr(), None if K_scale is None else K_scale.data_ptr(),
          q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), max_pages, max_new, mask_block,
          1.0 / hd ** 0.5 if scale is None else scale, lse.data_ptr(), None if pos_base is None else pos_base.data_ptr(),
          score.data_ptr(), score_out.data_ptr(), None if slot_pos is None else slot_pos.data_ptr(), slots, T, B, n_q, n_kv,
          hd, page, n_pages, _PAGE_CODE[dt]))
    return score_out


def dllm_paged_evict_workspace_bytes(B: int, n_kv: int, slots: int, dtype) -> int:
    return int(lib().dllm_paged_evict_workspace_bytes(B, n_kv, slots, _PAGE_CODE[dtype]))


def dllm_paged_evict(K_pages, V_pages, page_table, kv_len, keep, score, slot_pos, recent: int = 0, pos_base=None,
                     K_scale=None, V_scale=None, out=None, ws=None):
    """Gives up slots of the lowest score in every sequence and key head until keep [B] int32 are left (the keys of the
    last `recent` positions go last); later ones that stay move into them.  -> out = (score, slot_pos, kv_len, pos_base)
    after it, written in place when `out` is None (pos_base None if it was).  Masks go by slots: attend with mask_block =
    m > 1 afterwards only if the number of slots given up is a multiple of m in every sequence."""
    sh, ts, i32 = K_pages.shape, page_table.shape, torch.int32
    if len(sh) != 4 or V_pages.shape != sh or V_pages.dtype != K_pages.dtype:
        raise DllmError("K_pages and V_pages must both be [n_pages, page, n_kv, hd] of one dtype")
    n_pages, page, n_kv, hd = sh
    B, max_pages = ts if len(ts) == 2 else (-1, 0)
    dt, dev = K_pages.dtype, K_pages.get_device()
    if dt not in _PAGE_CODE:
        raise DllmError(f"unsupported dtype {dt}")
    if dt == _E4M3:
        _scales(K_pages, K_scale, V_scale)
    elif K_scale is not None or V_scale is not None:
        raise DllmError("scales go with 8-bit pages")
    if out is None:
        out = (score, slot_pos, kv_len, pos_base)
    score_out, pos_out, len_out, base_out = out
    each = (kv_len, keep, len_out) + (() if pos_base is None else (pos_base,)) + (() if base_out is None else (base_out,))
    if page_table.dtype != i32 or any(t.shape != (B,) or t.dtype != i32 for t in each):
        raise DllmError("page_table [B, max_pages], kv_len, keep and pos_base [B] int32 expected")
    if (pos_base is None) != (base_out is None):
        raise DllmError("pos_base must be given and returned, or neither")
    slots = _slot_arrays(B, n_kv, (score, score_out), (slot_pos, pos_out))
    dense = [K_pages, V_pages, page_table, score, score_out, slot_pos, pos_out, *each]
    dense += [t for t in (K_scale, V_scale, ws) if t is not None]
    _same(dev, dense)
    L, code = _lib or lib(), _PAGE_CODE[dt]
    if ws is None:
        ws = _stream_workspace(L.dllm_paged_evict_workspace_bytes(B, n_kv, slots, code), K_pages.device, dev, "paged_evict")
    ptr = lambda t: None if t is None else t.data_ptr()   # noqa: E731
    _run(L.dllm_paged_evict, "dllm_paged_evict", dev,
         (K_pages.data_ptr(), V_pages.data_ptr(), ptr(K_scale), ptr(V_scale), kv_len.data_ptr(), page_table.data_ptr(),
          max_pages, keep.data_ptr(), recent, ptr(pos_base), score.data_ptr(), slot_pos.data_ptr(), slots,
          score_out.data_ptr(), pos_out.data_ptr(), len_out.data_ptr(), ptr(base_out), B, n_kv, hd, page, n_pages, code,
          ws.data_ptr(), ws.numel() * ws.element_size()))
    return out


def dllm_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, valid=None, out=None, ws=None):
    """logits [B, M, V] (f32 or bf16), u [B, M] f32 in [0, 1); temperature, top_p, min_p [B] f32 and top_k
    [B] int32 (None = off); valid [B, M] uint8 or None -> (token [B, M] int32, prob [B, M] f32)."""
    sh, f32, dev = logits.shape, torch.float32, logits.get_device()
    if len(sh) != 3 or logits.dtype not in _CODE:
        raise DllmError("logits must be [B, M, V] float32 or bfloat16")
    B, M, V = sh
    rows, each = sh[:2], sh[:1]
    if u.shape != rows or u.dtype != f32:
        raise DllmError("u must be [B, M] float32")
    dense = [logits, u]
    ptrs = []
    for t in (temperature, top_k, top_p, min_p):
        if t is None:
            ptrs.append(None)
            continue
        if t.shape != each or t.dtype != (torch.int32 if t is top_k else f32):
            raise DllmError("temperature, top_p and min_p must be [B] float32, top_k [B] int32")
        ptrs.append(t.data_ptr())
        dense.append(t)
    if valid is not None:
        if valid.shape != rows or valid.dtype != torch.uint8:
            raise DllmError("valid must be [B, M] uint8")
        dense.append(valid)
    if out is None:
        out = (torch.empty(rows, dtype=torch.int32, device=logits.device), torch.empty(rows, dtype=f32, device=logits.device))
    tok, prob = out
    if tok.shape != rows or tok.dtype != torch.int32 or prob.shape != rows or prob.dtype != f32:
        raise DllmError("out must be (token [B, M] int32, prob [B, M] float32)")
    dense += out
    if ws is not None:
        dense.append(ws)
    _same(dev, dense)
    L = _lib or lib()
    if ws is None:
        ws = _stream_workspace(L.dllm_sample_workspace_bytes(B, M, V), logits.device, dev, "sample")
    _run(L.dllm_sample, "dllm_sample", dev,
         (logits.data_ptr(), u.data_ptr(), *ptrs, None if valid is None else valid.data_ptr(), tok.data_ptr(),
          prob.data_ptr(), B, M, V, _CODE[logits.dtype], ws.data_ptr(), ws.numel() * ws.element_size()))
    return out
