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
def _on(ref, stream):
    """Context of the tensors' device and of the stream that the call runs on, so that what
    the call allocates belongs to that stream; and the stream."""
    if not ref.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        stream = torch.cuda.current_stream(ref.device)
    elif stream.device != ref.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {ref.device}")
    return torch.cuda.stream(stream), stream


def _check_on(t, name, dtype, shape, device):
    _check(t, name, dtype, shape)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_heads(t, name, dtype, shape, device):
    """A [tokens, heads, d] tensor whose tokens may lie apart (a slice of a fused
    projection); returns the elements between them."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    n, h, d = shape
    if n == 0:
        return h * d
    if t.stride(2) != 1 or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: heads and channels must be contiguous")
    return t.stride(0) if n > 1 else h * d


def _pages_strides(t, name, dtype, shape, device):
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(3) != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    # a stride along one entry says nothing; give it the dense value
    d = shape[3]
    st = [t.stride(0), t.stride(1), t.stride(2)]
    for i, dense in ((2, d), (1, d * shape[2]), (0, d * shape[2] * shape[1])):
        if shape[i] == 1:
            st[i] = dense
        elif st[i] < d:
            raise ValueError(f"{name}: tokens, heads and pages must not overlap")
    return st


def paged_attn(q, k_pages, v_pages, cu_q, page_table, length, scale, *, max_q, k_new=None, v_new=None, rows=None,
               out=None, lse=None, stream=None):
    """Attention of a packed batch of new tokens over a paged cache (see ``kda.h``).

    q [total_q,Hq,d] bf16 or fp16, its tokens contiguous or a slice of a wider row; k_pages,
    v_pages [num_pages,page_size,Hkv,d] of any strides with contiguous channels; cu_q int32
    [N+1]; page_table int32 [R,P]; length int32 [R], the rows' tokens with the new ones; rows
    int32 [N] or None (rows 0..N-1); max_q the most new tokens that a sequence has.  k_new,
    v_new [total_q,Hkv,d] are written to their pages first; without them the cache holds them.
    Returns out [total_q,Hq,d]; lse fp32 [total_q,Hq] is written when given."""
    if q.dim() != 3 or k_pages.dim() != 4 or page_table.dim() != 2 or cu_q.dim() != 1 or cu_q.numel() < 2:
        raise ValueError("q must be [total_q,Hq,d], k_pages [num_pages,page_size,Hkv,d], page_table [R,P], cu_q [N+1]")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    ctx, stream = _on(q, stream)
    dev, dt = q.device, q.dtype
    total, Hq, d = q.shape
    num_pages, ps, Hkv, _ = k_pages.shape
    R, P = page_table.shape
    N = cu_q.numel() - 1
    qs = _check_heads(q, "q", dt, (total, Hq, d), dev)
    strides = _pages_strides(k_pages, "k_pages", dt, (num_pages, ps, Hkv, d), dev)
    strides += _pages_strides(v_pages, "v_pages", dt, (num_pages, ps, Hkv, d), dev)
    _check_on(cu_q, "cu_q", torch.int32, (N + 1,), dev)
    _check_on(page_table, "page_table", torch.int32, (R, P), dev)
    _check_on(length, "length", torch.int32, (R,), dev)
    if rows is not None:
        _check_on(rows, "rows", torch.int32, (N,), dev)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new come together")
    ks = vs = Hkv * d
    if k_new is not None:
        ks = _check_heads(k_new, "k_new", dt, (total, Hkv, d), dev)
        vs = _check_heads(v_new, "v_new", dt, (total, Hkv, d), dev)
    if lse is not None:
        _check_on(lse, "lse", torch.float32, (total, Hq), dev)
    with ctx:
        if out is None:
            out = torch.empty((total, Hq, d), device=dev, dtype=dt)
        _check_on(out, "out", dt, (total, Hq, d), dev)
        nbytes = paged_attn_workspace_bytes(N, total, max_q, Hq, Hkv, d, ps, P)
        ws = torch.empty(max(nbytes, 1), device=dev, dtype=torch.uint8)
        rc = load().kda_paged_attn(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages), _ptr(cu_q),
                                   _ptr(page_table), _ptr(length), _ptr(rows), float(scale), _ptr(out), _ptr(lse),
                                   N, total, int(max_q), Hq, Hkv, d, ps, num_pages, P, R, qs, ks, vs,
                                   (ctypes.c_longlong * 6)(*strides), 0 if dt == torch.bfloat16 else 1,
                                   _ptr(ws), nbytes, ctypes.c_void_p(stream.cuda_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_paged_attn")
    return out


def paged_attn_workspace_bytes(N, total_q, max_q, Hq, Hkv, d, page_size, P) -> int:
    """Device memory that one ``paged_attn`` of these sizes uses while it runs."""
    return int(load().kda_paged_attn_workspace_bytes(int(N), int(total_q), int(max_q), int(Hq), int(Hkv), int(d),
                                                     int(page_size), int(P)))


def _cache(table, length, ref, dev):
    if table.dim() != 2 or ref.dim() != 1:
        raise ValueError("table must be [R,P], ref [num_pages]")
    R, P = table.shape
    _check_on(table, "table", torch.int32, (R, P), dev)
    _check_on(length, "length", torch.int32, (R,), dev)
    _check_on(ref, "ref", torch.int32, (ref.numel(),), dev)
    return R, P, ref.numel()


def _pool(t, num_pages, dev):
    """(pointer, outer, outer stride, page stride, page bytes) of a pool [outer, num_pages, ...]
    whose pages are contiguous."""
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"a pool must be on {dev}")
    if t.dim() < 3 or t.shape[1] != num_pages:
        raise ValueError(f"a pool must be [outer, {num_pages}, ...], got {tuple(t.shape)}")
    want = 1
    for k in range(t.dim() - 1, 1, -1):
        if t.shape[k] != 1 and t.stride(k) != want:
            raise ValueError("a pool's pages must be contiguous")
        want *= t.shape[k]
    es = t.element_size()
    page = want * es
    ps = t.stride(1) * es if t.shape[1] > 1 else page
    os_ = t.stride(0) * es if t.shape[0] > 1 else ps * num_pages
    return _ptr(t), t.shape[0], os_, ps, page


def pages_reserve(table, length, ref, rows, new_length, page_size, *, info=None, stream=None):
    """Grows rows (int32 [n]) to new_length (int32 [n]), with the lowest-numbered free pages
    in the list's order; in place.  info int32 [1], when given, receives the free pages left,
    or minus the number missing, and then nothing has changed."""
    ctx, stream = _on(table, stream)
    dev = table.device
    R, P, num_pages = _cache(table, length, ref, dev)
    n = rows.numel()
    _check_on(rows, "rows", torch.int32, (n,), dev)
    _check_on(new_length, "new_length", torch.int32, (n,), dev)
    if info is not None:
        _check_on(info, "info", torch.int32, (1,), dev)
    with ctx:
        rc = load().kda_pages_reserve(_ptr(table), _ptr(length), _ptr(ref), _ptr(rows), _ptr(new_length), n, _ptr(info),
                                      R, P, num_pages, int(page_size), ctypes.c_void_p(stream.cuda_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_reserve")


def pages_fork(table, length, ref, src, dst, page_size, *, pools=(), info=None, stream=None):
    """Empty rows dst (int32 [n]) share the sequences of rows src: full pages by count, a
    partial last page copied in every pool [outer, num_pages, ...].  Returns (copy_src,
    copy_dst), int32 [n], the pages copied (-1, -1: none).  info as ``pages_reserve``."""
    ctx, stream = _on(table, stream)
    dev = table.device
    R, P, num_pages = _cache(table, length, ref, dev)
    n = src.numel()
    _check_on(src, "src", torch.int32, (n,), dev)
    _check_on(dst, "dst", torch.int32, (n,), dev)
    if info is not None:
        _check_on(info, "info", torch.int32, (1,), dev)
    args = [_pool(t, num_pages, dev) for t in pools]
    with ctx:
        pairs = torch.empty((2, n), device=dev, dtype=torch.int32)
        cs, cd = pairs[0], pairs[1]
        st = ctypes.c_void_p(stream.cuda_stream)
        rc = load().kda_pages_fork(_ptr(table), _ptr(length), _ptr(ref), _ptr(src), _ptr(dst), n, _ptr(cs), _ptr(cd),
                                   _ptr(info), R, P, num_pages, int(page_size), st)
        if rc != KDA_OK:
            raise KdaError(rc, "kda_pages_fork")
        for a in args:
            rc = load().kda_pages_copy(*a, num_pages, _ptr(cs), _ptr(cd), n, st)
            if rc != KDA_OK:
                raise KdaError(rc, "kda_pages_copy")
    return cs, cd


def pages_free(table, length, ref, rows, page_size, *, stream=None):
    """Ends the sequences of rows (int32 [n]), in place."""
    ctx, stream = _on(table, stream)
    dev = table.device
    R, P, num_pages = _cache(table, length, ref, dev)
    n = rows.numel()
    _check_on(rows, "rows", torch.int32, (n,), dev)
    with ctx:
        rc = load().kda_pages_free(_ptr(table), _ptr(length), _ptr(ref), _ptr(rows), n, R, P, num_pages, int(page_size),
                                   ctypes.c_void_p(stream.cuda_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_free")


def pages_compact(table, length, ref, page_size, *, table_out=None, ref_out=None, pools=(), info=None, stream=None):
    """Moves the live pages of every pool [outer, num_pages, ...] to the front and renumbers
    table and ref, in place or into table_out and ref_out.  Returns (table, ref) as written;
    info int32 [1], when given, receives the number of free pages."""
    ctx, stream = _on(table, stream)
    dev = table.device
    R, P, num_pages = _cache(table, length, ref, dev)
    table_out = table if table_out is None else table_out
    ref_out = ref if ref_out is None else ref_out
    _check_on(table_out, "table_out", torch.int32, (R, P), dev)
    _check_on(ref_out, "ref_out", torch.int32, (num_pages,), dev)
    if info is not None:
        _check_on(info, "info", torch.int32, (1,), dev)
    args = [_pool(t, num_pages, dev) for t in pools]
    with ctx:
        nbytes = int(load().kda_pages_compact_workspace_bytes(num_pages))
        ws = torch.empty(max(nbytes, 1), device=dev, dtype=torch.uint8)
        st = ctypes.c_void_p(stream.cuda_stream)
        rc = load().kda_pages_compact(_ptr(table), _ptr(length), _ptr(ref), _ptr(table_out), _ptr(ref_out), _ptr(info),
                                      R, P, num_pages, int(page_size), _ptr(ws), nbytes, st)
        if rc != KDA_OK:
            raise KdaError(rc, "kda_pages_compact")
        for a in args:
            rc = load().kda_pages_compact_pool(*a, num_pages, _ptr(ws), nbytes, st)
            if rc != KDA_OK:
                raise KdaError(rc, "kda_pages_compact_pool")
    return table_out, ref_out


def pages_copy(pool, src, dst, *, stream=None):
    """pool[:, dst[i]] = pool[:, src[i]] for int32 [n] src, dst, on a pool [outer, num_pages, ...]
    with contiguous pages: key/value pages of every layer, or recurrent states in slots."""
    ctx, stream = _on(pool, stream)
    dev = pool.device
    if pool.dim() < 3:
        raise ValueError("a pool must be [outer, num_pages, ...]")
    a = _pool(pool, pool.shape[1], dev)
    n = src.numel()
    _check_on(src, "src", torch.int32, (n,), dev)
    _check_on(dst, "dst", torch.int32, (n,), dev)
    with ctx:
        rc = load().kda_pages_copy(*a, pool.shape[1], _ptr(src), _ptr(dst), n, ctypes.c_void_p(stream.cuda_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_pages_copy")
