"""Python binding of libkda (ctypes).  Argument marshalling only: every step of
the computation runs in the library's CUDA kernels.

The entry points mirror ``include/kda.h``:

* ``chunk_fwd``   -> ``kda_chunk_fwd``   (chunkwise prefill)
* ``chunk_fwd_noalloc`` -> ``kda_chunk_fwd_noalloc`` (the same prefill over a fixed
  scratch array: no device allocation)
* ``chunk_fwd_varlen`` -> ``kda_chunk_fwd_varlen`` (packed batch of sequences, cu_seqlens)
* ``decode_step`` -> ``kda_decode_step`` (one recurrent step, state in place)
* ``chunk_fwd_raw`` / ``decode_step_raw`` -> ``kda_chunk_fwd_raw`` / ``kda_decode_step_raw``
  (raw projections in: the gate prologue and the q/k normalisation run in the kernels)
* ``stream_status`` -> ``kda_stream_status``
* ``workspace_bytes`` / ``release_workspace`` -> ``kda_chunk_fwd_workspace_bytes`` /
  ``kda_release_workspace``

* ``paged_attn`` -> ``kda_paged_attn`` (attention of new tokens over a paged cache: the
  full-attention layers of a hybrid stack); ``pages_reserve``, ``pages_fork``, ``pages_free``,
  ``pages_compact``, ``pages_copy`` -> ``kda_pages_*`` (that cache's pages, and pools of
  recurrent states)

* ``chunk_fwd_host`` -> ``kda_chunk_fwd_host`` (the prefill on host tensors, pinned for
  overlap: the library streams pieces of the token axis up, through the prefill and back)

If ``libkda.so`` is missing the calls raise; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "libkda_debug.so")

(KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_ALIGNMENT, KDA_ERR_CUDA, KDA_ERR_TIMEOUT,
 KDA_ERR_SCRATCH_LIMIT, KDA_ERR_BOUNDS) = range(8)
EXPORTED = ("kda_chunk_fwd", "kda_chunk_fwd_noalloc", "kda_chunk_fwd_host", "kda_chunk_fwd_host_debug_piece", "kda_chunk_fwd_varlen", "kda_decode_step",
            "kda_gdn_chunk_fwd", "kda_gdn_decode_step", "kda_chunk_fwd_raw", "kda_decode_step_raw",
            "kda_chunk_bwd", "kda_chunk_bwd_workspace_bytes",
            "kda_chunk_fwd_workspace_bytes", "kda_chunk_fwd_varlen_workspace_bytes", "kda_release_workspace",
            "kda_status_string", "kda_stream_status", "kda_chunk_fwd_debug_wait_limit",
            "kda_chunk_fwd_debug_inject_timeout", "kda_chunk_fwd_debug_force_exact", "kda_chunk_fwd_debug_block_refs", "kda_chunk_fwd_debug_record_cap", "kda_chunk_fwd_debug_parts",
            "kda_debug_kernel_timing", "kda_debug_kernel_times", "kda_debug_kernel_launches",
            "kda_paged_attn", "kda_paged_attn_workspace_bytes", "kda_pages_reserve", "kda_pages_fork",
            "kda_pages_free", "kda_pages_compact", "kda_pages_compact_workspace_bytes", "kda_pages_compact_pool",
            "kda_pages_copy", "kda_abi_version")

_lib = None          # the library the calls below go through
_libs = {}           # path -> loaded library


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def load():
    """The library the binding's calls go through: libkda.so (built in-tree by
    ``gated_delta_rule_100_b200.build``) unless ``use_debug_library(True)``."""
    global _lib
    if _lib is None:
        _lib = _open(LIB_PATH)
    return _lib


def use_debug_library(enable: bool) -> None:
    """Route every call through libkda_debug.so (device-side index checks that
    report KDA_ERR_BOUNDS) or back through libkda.so.  The two libraries have
    separate device state (status word, workspace)."""
    global _lib
    _lib = _open(DEBUG_LIB_PATH if enable else LIB_PATH)


def _open(path):
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m gated_delta_rule_100_b200.build`")
    lib = ctypes.CDLL(path)
    vp, fp, i, f = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd.restype = i
    lib.kda_chunk_fwd_noalloc.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_noalloc.restype = i
    lib.kda_chunk_fwd_host.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_host.restype = i
    lib.kda_chunk_fwd_host_debug_piece.argtypes = [i]
    lib.kda_chunk_fwd_host_debug_piece.restype = None
    lib.kda_chunk_bwd.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, vp, vp, vp, fp, fp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_bwd.restype = i
    lib.kda_chunk_bwd_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.kda_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_chunk_fwd_raw.argtypes = [vp, vp, vp, fp, fp, f, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_raw.restype = i
    lib.kda_decode_step_raw.argtypes = [vp, vp, vp, fp, fp, f, f, fp, vp, i, i, i, i, vp]
    lib.kda_decode_step_raw.restype = i
    lib.kda_chunk_fwd_varlen.argtypes = [vp, vp, vp, fp, fp, f, vp, i, fp, vp, fp, i, i, i, i, vp]
    lib.kda_chunk_fwd_varlen.restype = i
    lib.kda_chunk_fwd_varlen_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.kda_chunk_fwd_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_decode_step.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, i, i, i, i, vp]
    lib.kda_decode_step.restype = i
    lib.kda_gdn_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_gdn_chunk_fwd.restype = i
    lib.kda_gdn_decode_step.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, i, i, i, i, vp]
    lib.kda_gdn_decode_step.restype = i
    lib.kda_chunk_fwd_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.kda_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_release_workspace.argtypes = []
    lib.kda_release_workspace.restype = i
    lib.kda_status_string.argtypes = [i]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_stream_status.argtypes = [vp]
    lib.kda_stream_status.restype = i
    lib.kda_chunk_fwd_debug_wait_limit.argtypes = [ctypes.c_ulonglong]
    lib.kda_chunk_fwd_debug_wait_limit.restype = None
    lib.kda_chunk_fwd_debug_inject_timeout.argtypes = [ctypes.c_ulonglong]
    lib.kda_chunk_fwd_debug_inject_timeout.restype = None
    lib.kda_chunk_fwd_debug_parts.argtypes = [i]
    lib.kda_chunk_fwd_debug_parts.restype = None
    lib.kda_chunk_fwd_debug_record_cap.argtypes = [ctypes.c_ulonglong]
    lib.kda_chunk_fwd_debug_record_cap.restype = None
    lib.kda_chunk_fwd_debug_force_exact.argtypes = [i]
    lib.kda_chunk_fwd_debug_force_exact.restype = None
    lib.kda_chunk_fwd_debug_block_refs.argtypes = [i]
    lib.kda_chunk_fwd_debug_block_refs.restype = None
    lib.kda_debug_kernel_timing.argtypes = [i]
    lib.kda_debug_kernel_timing.restype = None
    lib.kda_debug_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong), i]
    lib.kda_debug_kernel_times.restype = i
    ll = ctypes.POINTER(ctypes.c_longlong)
    lib.kda_debug_kernel_launches.argtypes = [ctypes.POINTER(ctypes.c_int), ll, ll, i, ctypes.POINTER(ctypes.c_int)]
    lib.kda_debug_kernel_launches.restype = i
    ll, sz = ctypes.c_longlong, ctypes.c_size_t
    lib.kda_paged_attn.argtypes = [vp] * 9 + [f, vp, vp] + [i] * 10 + [ll] * 3 + [vp, i, vp, sz, vp]
    lib.kda_paged_attn_workspace_bytes.argtypes = [i] * 8
    lib.kda_paged_attn_workspace_bytes.restype = sz
    lib.kda_pages_reserve.argtypes = [vp] * 5 + [i, vp] + [i] * 4 + [vp]
    lib.kda_pages_fork.argtypes = [vp] * 5 + [i, vp, vp, vp] + [i] * 4 + [vp]
    lib.kda_pages_free.argtypes = [vp] * 4 + [i] * 5 + [vp]
    lib.kda_pages_compact.argtypes = [vp] * 6 + [i] * 4 + [vp, sz, vp]
    lib.kda_pages_compact_workspace_bytes.argtypes = [i]
    lib.kda_pages_compact_workspace_bytes.restype = sz
    lib.kda_pages_compact_pool.argtypes = [vp, ll, ll, ll, ll, i, vp, sz, vp]
    lib.kda_pages_copy.argtypes = [vp, ll, ll, ll, ll, i, vp, vp, i, vp]
    for name in ("kda_paged_attn", "kda_pages_reserve", "kda_pages_fork", "kda_pages_free", "kda_pages_compact",
                 "kda_pages_compact_pool", "kda_pages_copy"):
        getattr(lib, name).restype = i
    lib.kda_abi_version.restype = i
    _libs[path] = lib
    return lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype, shape):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def chunk_fwd(q, k, v, g, beta, scale, h0=None, *, out=None, hT=None, final_state=True, stream=None):
    """Chunkwise prefill.  q, k [B,T,H,dk] bf16; v [B,T,H,dv] bf16; g [B,T,H,dk] fp32;
    beta [B,T,H] fp32; h0 [B,H,dk,dv] fp32 or None.  Returns (out, hT); hT is None
    when ``final_state`` is False and no ``hT`` buffer was given."""
    return _prefill("kda_chunk_fwd", False, q, k, v, g, beta, scale, h0, out, hT, final_state, stream)


def gdn_chunk_fwd(q, k, v, g, beta, scale, h0=None, *, out=None, hT=None, final_state=True, stream=None):
    """Scalar-gate (Gated DeltaNet) prefill: as ``chunk_fwd`` with g [B,T,H] fp32, one
    log-decay per token and head shared by every key channel."""
    return _prefill("kda_gdn_chunk_fwd", True, q, k, v, g, beta, scale, h0, out, hT, final_state, stream)


def _prefill(symbol, scalar_gate, q, k, v, g, beta, scale, h0, out, hT, final_state, stream):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (B, T, H, dk))
    _check(k, "k", torch.bfloat16, (B, T, H, dk))
    _check(v, "v", torch.bfloat16, (B, T, H, dv))
    _check(g, "g", torch.float32, (B, T, H) if scalar_gate else (B, T, H, dk))
    _check(beta, "beta", torch.float32, (B, T, H))
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv))
    if out is None:
        out = torch.empty((B, T, H, dv), device=q.device, dtype=torch.bfloat16)
    _check(out, "out", torch.bfloat16, (B, T, H, dv))
    if hT is None and final_state:
        hT = torch.empty((B, H, dk, dv), device=q.device, dtype=torch.float32)
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, dk, dv))
    rc = getattr(load(), symbol)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                 _ptr(h0), _ptr(out), _ptr(hT), B, T, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, symbol)
    return out, hT


def chunk_bwd(q, k, v, g, beta, scale, h0=None, dout=None, dhT=None, *, want_dh0=True, stream=None):
    """Backward of ``chunk_fwd``: gradients of L given dL/dout (bf16 [B,T,H,dv]) and
    dL/dhT (fp32 [B,H,dk,dv]); either may be None (zero).  Returns a dict with dq, dk,
    dv (bf16), dg, dbeta and dh0 (fp32; None when ``want_dh0`` is False)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (B, T, H, dk))
    _check(k, "k", torch.bfloat16, (B, T, H, dk))
    _check(v, "v", torch.bfloat16, (B, T, H, dv))
    _check(g, "g", torch.float32, (B, T, H, dk))
    _check(beta, "beta", torch.float32, (B, T, H))
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv))
    if dout is not None:
        _check(dout, "dout", torch.bfloat16, (B, T, H, dv))
    if dhT is not None:
        _check(dhT, "dhT", torch.float32, (B, H, dk, dv))
    z = dict(device=q.device)
    r = dict(dq=torch.empty((B, T, H, dk), dtype=torch.bfloat16, **z),
             dk=torch.empty((B, T, H, dk), dtype=torch.bfloat16, **z),
             dv=torch.empty((B, T, H, dv), dtype=torch.bfloat16, **z),
             dg=torch.empty((B, T, H, dk), dtype=torch.float32, **z),
             dbeta=torch.empty((B, T, H), dtype=torch.float32, **z),
             dh0=torch.empty((B, H, dk, dv), dtype=torch.float32, **z) if want_dh0 else None)
    rc = load().kda_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(h0), _ptr(dout),
                              _ptr(dhT), _ptr(r["dq"]), _ptr(r["dk"]), _ptr(r["dv"]), _ptr(r["dg"]), _ptr(r["dbeta"]),
                              _ptr(r["dh0"]), B, T, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_bwd")
    return r


def chunk_fwd_raw(q, k, v, g_raw, beta_raw, gate_c, scale, h0=None, *, out=None, hT=None, final_state=True,
                  stream=None):
    """Prefill from raw projections: g = -gate_c softplus(g_raw), beta = sigmoid(beta_raw),
    q and k L2-normalised, all inside the kernels.  Shapes and dtypes as ``chunk_fwd``."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (B, T, H, dk))
    _check(k, "k", torch.bfloat16, (B, T, H, dk))
    _check(v, "v", torch.bfloat16, (B, T, H, dv))
    _check(g_raw, "g_raw", torch.float32, (B, T, H, dk))
    _check(beta_raw, "beta_raw", torch.float32, (B, T, H))
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv))
    if out is None:
        out = torch.empty((B, T, H, dv), device=q.device, dtype=torch.bfloat16)
    _check(out, "out", torch.bfloat16, (B, T, H, dv))
    if hT is None and final_state:
        hT = torch.empty((B, H, dk, dv), device=q.device, dtype=torch.float32)
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, dk, dv))
    rc = load().kda_chunk_fwd_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(beta_raw), float(gate_c),
                                  float(scale), _ptr(h0), _ptr(out), _ptr(hT), B, T, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_raw")
    return out, hT


def decode_step_raw(q, k, v, g_raw, beta_raw, gate_c, scale, state, *, out=None, stream=None):
    """One recurrent step from raw projections (see ``chunk_fwd_raw``); shapes as ``decode_step``."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (B, H, dk))
    _check(k, "k", torch.bfloat16, (B, H, dk))
    _check(v, "v", torch.bfloat16, (B, H, dv))
    _check(g_raw, "g_raw", torch.float32, (B, H, dk))
    _check(beta_raw, "beta_raw", torch.float32, (B, H))
    _check(state, "state", torch.float32, (B, H, dk, dv))
    if out is None:
        out = torch.empty((B, H, dv), device=q.device, dtype=torch.bfloat16)
    _check(out, "out", torch.bfloat16, (B, H, dv))
    rc = load().kda_decode_step_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(beta_raw), float(gate_c),
                                    float(scale), _ptr(state), _ptr(out), B, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step_raw")
    return out


def chunk_fwd_noalloc(q, k, v, g, beta, scale, h0=None, *, out, hT=None, stream=None):
    """``chunk_fwd`` through ``kda_chunk_fwd_noalloc``: the caller passes ``out``
    (and ``hT`` unless the final state is not wanted); the library allocates
    nothing.  Returns (out, hT)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (B, T, H, dk))
    _check(k, "k", torch.bfloat16, (B, T, H, dk))
    _check(v, "v", torch.bfloat16, (B, T, H, dv))
    _check(g, "g", torch.float32, (B, T, H, dk))
    _check(beta, "beta", torch.float32, (B, T, H))
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv))
    _check(out, "out", torch.bfloat16, (B, T, H, dv))
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, dk, dv))
    rc = load().kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                      _ptr(h0), _ptr(out), _ptr(hT), B, T, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_noalloc")
    return out, hT


def chunk_fwd_varlen(q, k, v, g, beta, scale, cu_seqlens, h0=None, *, out=None, hT=None, final_state=True,
                     stream=None):
    """Prefill of a packed batch.  q, k [T_total,H,dk] bf16; v [T_total,H,dv] bf16;
    g [T_total,H,dk] fp32; beta [T_total,H] fp32; cu_seqlens int32 [N+1] on the
    device; h0 [N,H,dk,dv] fp32 or None.  Returns (out [T_total,H,dv], hT [N,H,dk,dv]);
    hT is None when ``final_state`` is False and no ``hT`` buffer was given."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (T, H, dk))
    _check(k, "k", torch.bfloat16, (T, H, dk))
    _check(v, "v", torch.bfloat16, (T, H, dv))
    _check(g, "g", torch.float32, (T, H, dk))
    _check(beta, "beta", torch.float32, (T, H))
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
    N = cu_seqlens.numel() - 1
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv))
    if out is None:
        out = torch.empty((T, H, dv), device=q.device, dtype=torch.bfloat16)
    _check(out, "out", torch.bfloat16, (T, H, dv))
    if hT is None and final_state:
        hT = torch.empty((N, H, dk, dv), device=q.device, dtype=torch.float32)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv))
    rc = load().kda_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                     _ptr(cu_seqlens), N, _ptr(h0), _ptr(out), _ptr(hT), T, H, dk, dv,
                                     _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_varlen")
    return out, hT


def varlen_workspace_bytes(N: int, T_total: int, H: int, dk: int, dv: int) -> int:
    """Device memory ``chunk_fwd_varlen`` holds for these sizes (0 when unsupported)."""
    return int(load().kda_chunk_fwd_varlen_workspace_bytes(int(N), int(T_total), int(H), int(dk), int(dv)))


def set_parts(parts: int) -> None:
    """Test hook: parts of the two-level pass (0 = automatic, 1 = off, P >= 3 = forced)."""
    load().kda_chunk_fwd_debug_parts(int(parts))


def set_record_cap(nbytes: int) -> None:
    """Test hook: cap the chunk records the prefill workspace holds (0 = default)."""
    load().kda_chunk_fwd_debug_record_cap(int(nbytes))


def decode_step(q, k, v, g, beta, scale, state, *, out=None, stream=None):
    """One recurrent step.  q, k [B,H,dk] bf16; v [B,H,dv] bf16; g [B,H,dk] fp32;
    beta [B,H] fp32; state [B,H,dk,dv] fp32 (updated in place).  Returns out [B,H,dv] bf16."""
    return _decode("kda_decode_step", False, q, k, v, g, beta, scale, state, out, stream)


def gdn_decode_step(q, k, v, g, beta, scale, state, *, out=None, stream=None):
    """Scalar-gate (Gated DeltaNet) decode step: as ``decode_step`` with g [B,H] fp32."""
    return _decode("kda_gdn_decode_step", True, q, k, v, g, beta, scale, state, out, stream)


def _decode(symbol, scalar_gate, q, k, v, g, beta, scale, state, out, stream):
    B, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q", torch.bfloat16, (B, H, dk))
    _check(k, "k", torch.bfloat16, (B, H, dk))
    _check(v, "v", torch.bfloat16, (B, H, dv))
    _check(g, "g", torch.float32, (B, H) if scalar_gate else (B, H, dk))
    _check(beta, "beta", torch.float32, (B, H))
    _check(state, "state", torch.float32, (B, H, dk, dv))
    if out is None:
        out = torch.empty((B, H, dv), device=q.device, dtype=torch.bfloat16)
    _check(out, "out", torch.bfloat16, (B, H, dv))
    rc = getattr(load(), symbol)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                 _ptr(state), _ptr(out), B, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, symbol)
    return out


def workspace_bytes(B: int, T: int, H: int, dk: int, dv: int) -> int:
    """Device memory ``chunk_fwd`` holds for these sizes (0 when unsupported)."""
    return int(load().kda_chunk_fwd_workspace_bytes(int(B), int(T), int(H), int(dk), int(dv)))


def release_workspace() -> None:
    """Free the current device's prefill workspace (synchronises the device)."""
    rc = load().kda_release_workspace()
    if rc != KDA_OK:
        raise KdaError(rc, "kda_release_workspace")


def stream_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load().kda_stream_status(_stream(stream)))


def set_wait_limit(polls: int) -> None:
    """Test hook: polls a device-side wait makes before giving up (0 = default)."""
    load().kda_chunk_fwd_debug_wait_limit(int(polls))


def inject_timeout(polls: int) -> None:
    """Test hook: nonzero makes each prefill CTA first wait on a barrier nothing
    signals (at most ``polls`` polls) and take its timeout path; 0 = off."""
    load().kda_chunk_fwd_debug_inject_timeout(int(polls))


def force_exact(enable: bool) -> None:
    """Test hook: every prefill chunk takes the exact path (see ``kda.h``)."""
    load().kda_chunk_fwd_debug_force_exact(1 if enable else 0)


def block_refs(enable: bool) -> None:
    """Test hook: every prefill chunk is formed with its 16-token block
    references, mild decay or not (see ``kda.h``)."""
    load().kda_chunk_fwd_debug_block_refs(1 if enable else 0)


KERNEL_KINDS = ("prep", "chain", "exact", "fixup", "bwd")


def kernel_timing(enable: bool) -> None:
    """Measurement hook: every prefill and backward launch stamps its first CTA's
    start and last CTA's end (device globaltimer)."""
    load().kda_debug_kernel_timing(1 if enable else 0)


def kernel_times() -> dict:
    """{kind: (ms summed, launches)} of the launches timed since the last call."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_longlong * n)()
    rc = load().kda_debug_kernel_times(ms, cnt, n)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_debug_kernel_times")
    return {k: (ms[i], int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}


def kernel_launches(cap: int = 8192) -> list:
    """[(kind, start_ms, end_ms)] of the launches timed since the last read, in launch
    order, times relative to the first start (end < start: no stamp)."""
    kind = (ctypes.c_int * cap)()
    st, en = (ctypes.c_longlong * cap)(), (ctypes.c_longlong * cap)()
    cnt = ctypes.c_int(0)
    rc = load().kda_debug_kernel_launches(kind, st, en, cap, ctypes.byref(cnt))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_debug_kernel_launches")
    n = cnt.value
    t0 = min((st[i] for i in range(n) if en[i] >= st[i]), default=0)
    return [(KERNEL_KINDS[kind[i]] if 0 <= kind[i] < len(KERNEL_KINDS) else kind[i],
             (st[i] - t0) * 1e-6, (en[i] - t0) * 1e-6) for i in range(n)]


def _check_host(t, name, dtype, shape):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def chunk_fwd_host(q, k, v, g, beta, scale, h0=None, *, out, hT=None, stream=None):
    """``kda_chunk_fwd_host``: the prefill on HOST tensors (pinned, for overlapped copies),
    shapes and dtypes as ``chunk_fwd``; writes ``out`` (and ``hT`` when given) once
    ``stream`` reaches the end of the call's work.  Returns (bytes_h2d, bytes_d2h)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check_host(q, "q", torch.bfloat16, (B, T, H, dk))
    _check_host(k, "k", torch.bfloat16, (B, T, H, dk))
    _check_host(v, "v", torch.bfloat16, (B, T, H, dv))
    _check_host(g, "g", torch.float32, (B, T, H, dk))
    _check_host(beta, "beta", torch.float32, (B, T, H))
    _check_host(out, "out", torch.bfloat16, (B, T, H, dv))
    if h0 is not None:
        _check_host(h0, "h0", torch.float32, (B, H, dk, dv))
    if hT is not None:
        _check_host(hT, "hT", torch.float32, (B, H, dk, dv))
    rc = load().kda_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(h0),
                                   _ptr(out), _ptr(hT), B, T, H, dk, dv, _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_host")
    nin = sum(t.numel() * t.element_size() for t in (q, k, v, g, beta, h0) if t is not None)
    nout = sum(t.numel() * t.element_size() for t in (out, hT) if t is not None)
    return nin, nout


def set_host_piece(tokens: int) -> None:
    """Test hook: pieces of ``tokens`` tokens for ``chunk_fwd_host`` (0 = automatic)."""
    load().kda_chunk_fwd_host_debug_piece(int(tokens))


# ------------------------------------------------------------- paged cache ----
# A serving step makes many of these calls on little data, so what a call costs on the host
# counts: the checks compare whole shapes, and device and stream are only switched when they
# are not the current ones.
def _here(t, stream):
    """Whether the call runs on the current device and stream."""
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    return stream is None and torch._C._cuda_getDevice() == t.get_device()


def _there(t, stream):
    """Context of the tensor's device and of the stream that the call runs on, so that what
    the call allocates belongs to that stream."""
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


def _arr(t, name, dtype, shape, dev):
    """The address of a contiguous tensor that is what the call needs, on device index dev."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _check(t, name, dtype, shape)
        raise ValueError(f"{name} must be on device {dev}, got {t.device}")
    return t.data_ptr()


def _like(t, name, dtype, shape, dev):
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on device {dev}, got {t.device}")


def _token_stride(t, name, dtype, shape, dev):
    """Elements between the tokens of a [tokens, heads, d] tensor, which may lie apart (a slice
    of a fused projection)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _like(t, name, dtype, shape, dev)
    st, sh, sd = t.stride()
    n, h, d = shape
    if n and (sd != 1 or (h > 1 and sh != d)):
        raise ValueError(f"{name}: heads and channels must be contiguous")
    return st if n > 1 else h * d


def _page_strides(t, name, dtype, shape, dev):
    """Elements between the pages, tokens and heads of a pool of pages."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _like(t, name, dtype, shape, dev)
    sp, st, sh, sd = t.stride()
    n, ps, h, d = shape
    # a stride along one entry says nothing; give it the dense value
    if h == 1:
        sh = d
    if ps == 1:
        st = h * d
    if n == 1:
        sp = ps * h * d
    if sd != 1 or sh < d or st < d or sp < d:
        raise ValueError(f"{name}: channels must be contiguous, and tokens, heads and pages not overlap")
    return sp, st, sh


_attn_bytes = {}
_Strides = ctypes.c_longlong * 6


def paged_attn_workspace_bytes(N, total_q, max_q, Hq, Hkv, d, page_size, P) -> int:
    """Device memory that one ``paged_attn`` of these sizes uses while it runs."""
    return int(load().kda_paged_attn_workspace_bytes(N, total_q, max_q, Hq, Hkv, d, page_size, P))


def paged_attn(q, k_pages, v_pages, cu_q, page_table, length, scale, *, max_q, k_new=None, v_new=None, rows=None,
               out=None, lse=None, stream=None):
    """Attention of a packed batch of new tokens over a paged cache (see ``kda.h``).

    q [total_q,Hq,d] bf16 or fp16, its tokens contiguous or a slice of a wider row; k_pages,
    v_pages [num_pages,page_size,Hkv,d] of any strides with contiguous channels, under which (where
    the call writes) places do not overlap; cu_q int32
    [N+1]; page_table int32 [R,P]; length int32 [R], the rows' tokens with the new ones; rows
    int32 [N] or None (rows 0..N-1); max_q the most new tokens that a sequence has.  k_new,
    v_new [total_q,Hkv,d] are written to their pages first; without them the cache holds them.
    Returns out [total_q,Hq,d]; lse fp32 [total_q,Hq] is written when given."""
    dt, shape, pages, table, N = q.dtype, q.shape, k_pages.shape, page_table.shape, cu_q.numel() - 1
    if len(shape) != 3 or len(pages) != 4 or len(table) != 2 or cu_q.dim() != 1 or N < 1:
        raise ValueError("q must be [total_q,Hq,d], k_pages [num_pages,page_size,Hkv,d], page_table [R,P], cu_q [N+1]")
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError(f"q must be bfloat16 or float16, got {dt}")
    if not _here(q, stream):
        with _there(q, stream):
            return paged_attn(q, k_pages, v_pages, cu_q, page_table, length, scale, max_q=max_q, k_new=k_new, v_new=v_new,
                              rows=rows, out=out, lse=lse)
    dev, i32 = q.get_device(), torch.int32
    total, Hq, d = shape
    num_pages, ps, Hkv, dp = pages
    R, P = table
    if dp != d:
        raise ValueError(f"k_pages must have {d} channels, got {dp}")
    qs = _token_stride(q, "q", dt, shape, dev)
    strides = _page_strides(k_pages, "k_pages", dt, pages, dev) + _page_strides(v_pages, "v_pages", dt, pages, dev)
    cu = _arr(cu_q, "cu_q", i32, (N + 1,), dev)
    tab = _arr(page_table, "page_table", i32, table, dev)
    ln = _arr(length, "length", i32, (R,), dev)
    rw = None if rows is None else _arr(rows, "rows", i32, (N,), dev)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new come together")
    kp = vp = None
    ks = vs = Hkv * d
    if k_new is not None:
        new = (total, Hkv, d)
        ks, vs = _token_stride(k_new, "k_new", dt, new, dev), _token_stride(v_new, "v_new", dt, new, dev)
        kp, vp = k_new.data_ptr(), v_new.data_ptr()
    ls = None if lse is None else _arr(lse, "lse", torch.float32, (total, Hq), dev)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = out.data_ptr()
    else:
        op = _arr(out, "out", dt, shape, dev)
    lib = load()
    key = (dev, N, total, max_q, Hq, Hkv, d, ps, P)
    nbytes = _attn_bytes.get(key)
    if nbytes is None:  # a plan of sizes, the same for every call of them
        if len(_attn_bytes) > 4096:
            _attn_bytes.clear()
        nbytes = _attn_bytes[key] = paged_attn_workspace_bytes(*key[1:])
    ws = torch.empty(nbytes, device=q.device, dtype=torch.uint8) if nbytes else None
    rc = lib.kda_paged_attn(q.data_ptr(), kp, vp, k_pages.data_ptr(), v_pages.data_ptr(), cu, tab, ln, rw, scale, op, ls,
                            N, total, max_q, Hq, Hkv, d, ps, num_pages, P, R, qs, ks, vs, _Strides(*strides),
                            0 if dt is torch.bfloat16 else 1, ws.data_ptr() if nbytes else None, nbytes, _raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_paged_attn")
    return out


def _cache(table, length, ref, info, dev):
    """Addresses and sizes of a cache's table, length and ref, and of info (or None)."""
    if table.dim() != 2 or ref.dim() != 1:
        raise ValueError("table must be [R,P], ref [num_pages]")
    i32 = torch.int32
    R, P = shape = table.shape
    n = ref.numel()
    return (_arr(table, "table", i32, shape, dev), _arr(length, "length", i32, (R,), dev), _arr(ref, "ref", i32, (n,), dev),
            None if info is None else _arr(info, "info", i32, (1,), dev), R, P, n)


def _pool(t, num_pages, dev):
    """(pointer, outer, outer stride, page stride, page bytes) of a pool [outer, num_pages, ...]
    whose pages are contiguous; strides in bytes."""
    if t.get_device() != dev:
        raise ValueError(f"a pool must be on device {dev}, got {t.device}")
    shape, st = t.shape, t.stride()
    if len(shape) < 3 or shape[1] != num_pages:
        raise ValueError(f"a pool must be [outer, {num_pages}, ...], got {tuple(shape)}")
    want = 1
    for k in range(len(shape) - 1, 1, -1):
        if shape[k] != 1 and st[k] != want:
            raise ValueError("a pool's pages must be contiguous")
        want *= shape[k]
    es = t.element_size()
    page = want * es
    ps = st[1] * es if num_pages > 1 else page
    p, outer, os = t.data_ptr(), shape[0], st[0] * es if shape[0] > 1 else ps * num_pages
    apart = ps >= page and (os >= ps * num_pages or ps >= os * outer and os >= page)
    if (p | os | ps | page) & 15 or page < 1 or not apart or outer > 1 << 24:
        # refused here, before a call that changes the table has run
        rc = load().kda_pages_copy(p, outer, os, ps, page, num_pages, None, None, 0, None)
        if rc != KDA_OK:
            raise KdaError(rc, "kda_pages_copy")
    return p, outer, os, ps, page


def pages_reserve(table, length, ref, rows, new_length, page_size, *, info=None, stream=None):
    """Grows rows (int32 [n]) to new_length (int32 [n]), with the lowest-numbered free pages
    in the list's order; in place.  info int32 [1], when given, receives the free pages left,
    or minus the number missing, and then nothing has changed."""
    if not _here(table, stream):
        with _there(table, stream):
            return pages_reserve(table, length, ref, rows, new_length, page_size, info=info)
    dev, n = table.get_device(), rows.numel()
    t, ln, rf, inf, R, P, pages = _cache(table, length, ref, info, dev)
    rc = load().kda_pages_reserve(t, ln, rf, _arr(rows, "rows", torch.int32, (n,), dev),
                                  _arr(new_length, "new_length", torch.int32, (n,), dev), n, inf, R, P, pages, page_size,
                                  _raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_reserve")


def pages_fork(table, length, ref, src, dst, page_size, *, pools=(), info=None, stream=None):
    """Empty rows dst (int32 [n]) share the sequences of rows src: full pages by count, a
    partial last page copied in every pool [outer, num_pages, ...].  Returns int32 [2,n],
    the pages copied, from and to (-1, -1: none).  info as ``pages_reserve``."""
    if not _here(table, stream):
        with _there(table, stream):
            return pages_fork(table, length, ref, src, dst, page_size, pools=pools, info=info)
    dev, n = table.get_device(), src.numel()
    t, ln, rf, inf, R, P, pages = _cache(table, length, ref, info, dev)
    args = [_pool(x, pages, dev) for x in pools]
    a, b = _arr(src, "src", torch.int32, (n,), dev), _arr(dst, "dst", torch.int32, (n,), dev)
    pairs = torch.empty((2, n), device=table.device, dtype=torch.int32)
    lib, st, cs = load(), _raw_stream(dev), pairs.data_ptr()
    rc = lib.kda_pages_fork(t, ln, rf, a, b, n, cs, cs + 4 * n, inf, R, P, pages, page_size, st)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_fork")
    for x in args:
        rc = lib.kda_pages_copy(*x, pages, cs, cs + 4 * n, n, st)
        if rc != KDA_OK:
            raise KdaError(rc, "kda_pages_copy")
    return pairs


def pages_free(table, length, ref, rows, page_size, *, stream=None):
    """Ends the sequences of rows (int32 [n]), in place."""
    if not _here(table, stream):
        with _there(table, stream):
            return pages_free(table, length, ref, rows, page_size)
    dev, n = table.get_device(), rows.numel()
    t, ln, rf, _, R, P, pages = _cache(table, length, ref, None, dev)
    rc = load().kda_pages_free(t, ln, rf, _arr(rows, "rows", torch.int32, (n,), dev), n, R, P, pages, page_size,
                               _raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_free")


def pages_compact(table, length, ref, page_size, *, table_out=None, ref_out=None, pools=(), info=None, stream=None):
    """Moves the live pages of every pool [outer, num_pages, ...] to the front and renumbers
    table and ref, in place or into table_out and ref_out.  Returns (table, ref) as written;
    info int32 [1], when given, receives the number of free pages."""
    if not _here(table, stream):
        with _there(table, stream):
            return pages_compact(table, length, ref, page_size, table_out=table_out, ref_out=ref_out, pools=pools, info=info)
    dev = table.get_device()
    t, ln, rf, inf, R, P, pages = _cache(table, length, ref, info, dev)
    table_out = table if table_out is None else table_out
    ref_out = ref if ref_out is None else ref_out
    to, ro = _arr(table_out, "table_out", torch.int32, (R, P), dev), _arr(ref_out, "ref_out", torch.int32, (pages,), dev)
    args = [_pool(x, pages, dev) for x in pools]
    lib, st = load(), _raw_stream(dev)
    nbytes = lib.kda_pages_compact_workspace_bytes(pages)
    ws = torch.empty(nbytes, device=table.device, dtype=torch.uint8)
    rc = lib.kda_pages_compact(t, ln, rf, to, ro, inf, R, P, pages, page_size, ws.data_ptr(), nbytes, st)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_compact")
    for x in args:
        rc = lib.kda_pages_compact_pool(*x, pages, ws.data_ptr(), nbytes, st)
        if rc != KDA_OK:
            raise KdaError(rc, "kda_pages_compact_pool")
    return table_out, ref_out


def pages_copy(pool, src, dst, *, stream=None):
    """pool[:, dst[i]] = pool[:, src[i]] for int32 [n] src, dst, on a pool [outer, num_pages, ...]
    with contiguous pages: key/value pages of every layer, or recurrent states in slots.
    At most 2^21 pairs a call."""
    if not _here(pool, stream):
        with _there(pool, stream):
            return pages_copy(pool, src, dst)
    if pool.dim() < 3:
        raise ValueError("a pool must be [outer, num_pages, ...]")
    dev, pages, n = pool.get_device(), pool.shape[1], src.numel()
    rc = load().kda_pages_copy(*_pool(pool, pages, dev), pages, _arr(src, "src", torch.int32, (n,), dev),
                               _arr(dst, "dst", torch.int32, (n,), dev), n, _raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_copy")
