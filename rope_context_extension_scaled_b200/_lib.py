"""Binding of librcx.so (include/rcx.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
turns torch tensors into rcx_tensor views (data pointer, dtype, shape,
strides), passes the current CUDA stream, and maps status codes to
exceptions, through ctypes, or for the calls of a decoding step through the
extension module _rcx_torch.  PyTorch provides device memory and streams.  If the
library is missing, load() raises: there is no fallback path.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librcx.so")

RCX_OK, RCX_ERR_INVALID_ARG, RCX_ERR_UNSUPPORTED, RCX_ERR_ALIGNMENT, RCX_ERR_CUDA, RCX_ERR_DEVICE_TIMEOUT, \
    RCX_ERR_DEVICE_INDEX = 0, -1, -2, -3, -4, -5, -6
RCX_F32, RCX_BF16, RCX_I8, RCX_E4M3 = 0, 1, 2, 3
PLAIN, PI, NTK, DYN_NTK, NTK_PARTS, YARN = range(6)
ROTATE_Q, ROTATE_K = 1, 2
ROPE_HALVES, ROPE_INVERSE = 1, 2

# every symbol include/rcx.h declares
EXPORTS = (
    "rcx_abi_version", "rcx_status_string", "rcx_rope_freqs", "rcx_rope_apply",
    "rcx_attn_blockwise_fwd", "rcx_merge_partials", "rcx_ring_workspace_size",
    "rcx_ring_attn_fwd", "rcx_ring_attn_fwd_host", "rcx_device_status",
    "rcx_debug_inject_wait_timeout", "rcx_stats_enable_timing", "rcx_stats_reset", "rcx_stats_read",
    "rcx_ring_attn_fwd_noalloc", "rcx_rope_freqs_per_pair", "rcx_attn_decode_workspace_size",
    "rcx_attn_decode_fwd", "rcx_kv_quantize_int8", "rcx_attn_decode_int8_workspace_size",
    "rcx_attn_decode_int8_fwd", "rcx_attn_blockwise_merge_fwd", "rcx_release_staging",
    "rcx_rope_axes_map", "rcx_rope_axes_apply", "rcx_kv_block_append", "rcx_kv_block_read",
    "rcx_attn_kv_block_workspace_size", "rcx_attn_kv_block_fwd",
)
NOALLOC_SCRATCH_BYTES = 32 << 20   # RCX_NOALLOC_SCRATCH_BYTES in include/rcx.h
KERNEL_KINDS = {"rope_apply": 0, "attn_tc": 1, "attn_simt": 2, "merge": 3, "decode": 4}


class RcxError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class RcxTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class RcxKvBlocks(ctypes.Structure):
    _fields_ = [("k", RcxTensor), ("v", RcxTensor), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("B", ctypes.c_int64), ("width", ctypes.c_int64),
                ("table_stride", ctypes.c_int64)]


_lib = None


def load():
    """Load librcx.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run `python -m rope_context_extension_scaled_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    T = RcxTensor
    i64, f64, vp = ctypes.c_int64, ctypes.c_double, ctypes.c_void_p
    pd = ctypes.POINTER(ctypes.c_double)
    lib.rcx_abi_version.restype = ctypes.c_int
    lib.rcx_status_string.restype = ctypes.c_char_p
    lib.rcx_status_string.argtypes = [ctypes.c_int]
    lib.rcx_rope_freqs.argtypes = [ctypes.c_int, f64, ctypes.c_int, i64, i64, f64, f64, pd, pd]
    lib.rcx_rope_apply.argtypes = [T, T, T, T, vp, i64, pd, vp]
    lib.rcx_rope_freqs_per_pair.argtypes = [f64, ctypes.c_int, pd, pd]
    lib.rcx_rope_freqs_per_pair.restype = ctypes.c_int
    lib.rcx_attn_decode_workspace_size.argtypes = [T, T]
    lib.rcx_attn_decode_workspace_size.restype = i64
    lib.rcx_attn_decode_fwd.argtypes = [T, T, T, T, T, i64, i64, f64, i64, vp, i64, pd, ctypes.c_int, vp, i64, vp]
    lib.rcx_attn_decode_fwd.restype = ctypes.c_int
    lib.rcx_kv_quantize_int8.argtypes = [T, T, vp, vp]
    lib.rcx_attn_decode_int8_workspace_size.argtypes = [T, T]
    lib.rcx_attn_decode_int8_workspace_size.restype = i64
    lib.rcx_attn_decode_int8_fwd.argtypes = [T, T, vp, T, vp, T, T, i64, i64, f64, i64, vp, i64, pd, ctypes.c_int,
                                             vp, i64, vp]
    lib.rcx_attn_decode_int8_fwd.restype = ctypes.c_int
    lib.rcx_attn_blockwise_fwd.argtypes = [T, T, T, T, T, i64, i64, i64, f64, i64, i64, vp, i64, pd,
                                           ctypes.c_int, vp]
    lib.rcx_attn_blockwise_merge_fwd.argtypes = [T, T, T, T, T, T, T, i64, i64, i64, f64, i64, i64, vp, i64, pd,
                                                 ctypes.c_int, vp]
    lib.rcx_attn_blockwise_merge_fwd.restype = ctypes.c_int
    C = ctypes.POINTER(RcxKvBlocks)
    lib.rcx_rope_axes_map.argtypes = [ctypes.POINTER(i64), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.POINTER(ctypes.c_int32)]
    lib.rcx_rope_axes_apply.argtypes = [T, T, T, T, vp, ctypes.c_int, i64, i64, vp, vp, ctypes.c_int, vp]
    lib.rcx_kv_block_append.argtypes = [T, T, C, vp, vp, vp]
    lib.rcx_kv_block_read.argtypes = [C, vp, T, T, vp]
    lib.rcx_attn_kv_block_workspace_size.argtypes = [T, C]
    lib.rcx_attn_kv_block_workspace_size.restype = i64
    lib.rcx_attn_kv_block_fwd.argtypes = [T, C, vp, vp, T, T, i64, i64, f64, vp, i64, vp]
    lib.rcx_release_staging.argtypes = []
    lib.rcx_release_staging.restype = ctypes.c_int
    lib.rcx_merge_partials.argtypes = [T, T, T, T, T, T, vp]
    lib.rcx_ring_workspace_size.argtypes = [T, T, i64, ctypes.c_int]
    lib.rcx_ring_workspace_size.restype = i64
    lib.rcx_ring_attn_fwd.argtypes = [T, T, T, T, T, i64, i64, i64, f64, vp, i64, pd, ctypes.c_int, vp, i64, vp]
    lib.rcx_ring_attn_fwd_host.argtypes = [T, T, T, T, T, i64, i64, i64, f64, vp, i64, pd, ctypes.c_int, vp]
    lib.rcx_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.rcx_ring_attn_fwd_noalloc.argtypes = [T, T, T, T, T, i64, i64, i64, f64, vp, i64, pd, ctypes.c_int, vp]
    lib.rcx_ring_attn_fwd_noalloc.restype = ctypes.c_int
    lib.rcx_debug_inject_wait_timeout.argtypes = [i64]
    lib.rcx_stats_enable_timing.argtypes = [ctypes.c_int]
    lib.rcx_stats_read.argtypes = [ctypes.c_int, ctypes.POINTER(i64), ctypes.POINTER(f64)]
    for name in ("rcx_rope_freqs", "rcx_rope_apply", "rcx_attn_blockwise_fwd", "rcx_merge_partials",
                 "rcx_ring_attn_fwd", "rcx_ring_attn_fwd_host", "rcx_device_status",
                 "rcx_debug_inject_wait_timeout", "rcx_stats_enable_timing", "rcx_stats_reset",
                 "rcx_stats_read", "rcx_rope_axes_map", "rcx_rope_axes_apply", "rcx_kv_block_append",
                 "rcx_kv_block_read", "rcx_attn_kv_block_fwd"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(st):
    return load().rcx_status_string(int(st)).decode()


def _check(st, what):
    if st != RCX_OK:
        raise RcxError(st, what)


def _dtype_code(t: torch.Tensor):
    if t.dtype == torch.float32:
        return RCX_F32
    if t.dtype == torch.bfloat16:
        return RCX_BF16
    if t.dtype == torch.int8:
        return RCX_I8
    if t.dtype == torch.float8_e4m3fn:
        return RCX_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def view(t):
    """rcx_tensor of a [B, N, H, d] torch tensor (None -> null view)."""
    r = RcxTensor()
    if t is None:
        return r
    if t.dim() != 4:
        raise ValueError("expected a 4-D [B, N, H, d] tensor")
    r.ptr = t.data_ptr()
    r.dtype = _dtype_code(t)
    for i in range(4):
        r.shape[i] = t.shape[i]
        r.stride[i] = t.stride(i)
    return r


def lse_view(t):
    """rcx_tensor of a [B, H, N] fp32 LSE tensor (None -> null view)."""
    r = RcxTensor()
    if t is None:
        return r
    if t.dim() != 3 or t.dtype != torch.float32:
        raise ValueError("expected a 3-D [B, H, N] float32 tensor")
    r.ptr = t.data_ptr()
    r.dtype = RCX_F32
    for i in range(3):
        r.shape[i] = t.shape[i]
        r.stride[i] = t.stride(i)
    r.shape[3] = 1
    r.stride[3] = 1
    return r


def _freq_ptr(inv_freq):
    if inv_freq is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _pos(positions):
    if positions is None:
        return None, 0
    if positions.dtype != torch.int64:
        raise TypeError("positions must be int64")
    return ctypes.c_void_p(positions.data_ptr()), positions.numel()


# ----------------------------------------------------------------- entry points

def rope_freqs(scheme, base, d, L_train, L_target, alpha=1.0, beta=32.0):
    out = np.zeros(d // 2, dtype=np.float64)
    t = ctypes.c_double(0.0)
    st = load().rcx_rope_freqs(int(scheme), float(base), int(d), int(L_train), int(L_target), float(alpha),
                               float(beta), out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(t))
    _check(st, "rcx_rope_freqs")
    return out, t.value


def rope_freqs_per_pair(base, d, factors):
    """theta_i / factors[i] (per-plane rescaling); returns float64 [d/2]."""
    f = np.ascontiguousarray(np.asarray(factors, dtype=np.float64))
    if f.shape != (d // 2,):
        raise ValueError("need d/2 factors")
    out = np.zeros(d // 2, dtype=np.float64)
    st = load().rcx_rope_freqs_per_pair(float(base), int(d), f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                        out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)))
    _check(st, "rcx_rope_freqs_per_pair")
    return out


def rope_apply(q, k, inv_freq, positions=None, q_out=None, k_out=None):
    """Rotate q and/or k (either may be None).  Default: in place."""
    q_out = q if (q_out is None) else q_out
    k_out = k if (k_out is None) else k_out
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    dev = (q if q is not None else k).device
    st = load().rcx_rope_apply(view(q), view(k), view(q_out if q is not None else None),
                               view(k_out if k is not None else None), pp, npos, fp, _stream(dev))
    _check(st, "rcx_rope_apply")
    for x, y in ((q, q_out), (k, k_out)):
        if x is not None and not y.is_inference():
            torch.autograd.graph.increment_version(y)      # autograd sees that y has changed
    return q_out, k_out


def attn_blockwise_fwd(q, k, v, o=None, lse=None, kv_block=0, window=0, n_sink=0, temperature=1.0,
                       q_start=0, k_start=0, positions=None, inv_freq=None, rope_flags=0, want_lse=True,
                       out_dtype=None):
    B, N, H, D = q.shape
    if o is None:
        o = torch.empty(B, N, H, D, dtype=out_dtype or q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    st = load().rcx_attn_blockwise_fwd(view(q), view(k), view(v), view(o), lse_view(lse), int(kv_block),
                                       int(window), int(n_sink), float(temperature), int(q_start), int(k_start),
                                       pp, npos, fp, int(rope_flags), _stream(q.device))
    _check(st, "rcx_attn_blockwise_fwd")
    return o, lse


def attn_blockwise_merge_fwd(q, k, v, o, lse, acc, acc_lse, kv_block=0, window=0, n_sink=0, temperature=1.0,
                             q_start=0, k_start=0, positions=None, inv_freq=None, rope_flags=0):
    """Attention over this call's keys merged into the partial (acc, acc_lse)
    in the kernel's epilogue; o / lse may be acc / acc_lse (in place)."""
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    st = load().rcx_attn_blockwise_merge_fwd(view(q), view(k), view(v), view(o), lse_view(lse), view(acc),
                                             lse_view(acc_lse), int(kv_block), int(window), int(n_sink),
                                             float(temperature), int(q_start), int(k_start), pp, npos, fp,
                                             int(rope_flags), _stream(q.device))
    _check(st, "rcx_attn_blockwise_merge_fwd")
    return o, lse


def merge_partials(o_a, lse_a, o_b, lse_b, o_out=None, lse_out=None):
    st = load().rcx_merge_partials(view(o_a), lse_view(lse_a), view(o_b), lse_view(lse_b), view(o_out),
                                   lse_view(lse_out), _stream(o_a.device))
    _check(st, "rcx_merge_partials")
    return (o_a, lse_a) if o_out is None else (o_out, lse_out)


def ring_workspace_size(q, k, kv_block, rope_flags):
    n = load().rcx_ring_workspace_size(view(q), view(k), int(kv_block), int(rope_flags))
    if n < 0:
        raise RcxError(RCX_ERR_INVALID_ARG, "rcx_ring_workspace_size")
    return int(n)


def ring_attn_fwd(q, k, v, o=None, lse=None, kv_block=0, window=0, n_sink=0, temperature=1.0, positions=None,
                  inv_freq=None, rope_flags=0, workspace=None, want_lse=True):
    B, N, H, D = q.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    need = ring_workspace_size(q, k, kv_block, rope_flags)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    st = load().rcx_ring_attn_fwd(view(q), view(k), view(v), view(o), lse_view(lse), int(kv_block), int(window),
                                  int(n_sink), float(temperature), pp, npos, fp, int(rope_flags),
                                  ctypes.c_void_p(workspace.data_ptr()), workspace.numel(), _stream(q.device))
    _check(st, "rcx_ring_attn_fwd")
    return o, lse


def ring_attn_fwd_host(q, k, v, o, lse=None, kv_block=0, window=0, n_sink=0, temperature=1.0, positions=None,
                       inv_freq=None, rope_flags=0, stream=None):
    """Same as ring_attn_fwd on HOST tensors (pinned for full copy speed); synchronous."""
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = (None, 0) if positions is None else (ctypes.c_void_p(positions.data_ptr()), positions.numel())
    s = ctypes.c_void_p(stream.cuda_stream if stream is not None else torch.cuda.current_stream().cuda_stream)
    st = load().rcx_ring_attn_fwd_host(view(q), view(k), view(v), view(o), lse_view(lse), int(kv_block),
                                       int(window), int(n_sink), float(temperature), pp, npos, fp, int(rope_flags), s)
    _check(st, "rcx_ring_attn_fwd_host")
    return o, lse


def release_staging():
    """Return the staging memory rcx_ring_attn_fwd_host keeps between calls."""
    _check(load().rcx_release_staging(), "rcx_release_staging")


def device_status(device=None):
    v = ctypes.c_int(0)
    _check(load().rcx_device_status(_stream(device), ctypes.byref(v)), "rcx_device_status")
    return v.value


def debug_inject_wait_timeout(spins):
    _check(load().rcx_debug_inject_wait_timeout(int(spins)), "rcx_debug_inject_wait_timeout")


def stats_enable_timing(on=True):
    _check(load().rcx_stats_enable_timing(1 if on else 0), "rcx_stats_enable_timing")


def stats_reset():
    _check(load().rcx_stats_reset(), "rcx_stats_reset")


def stats_read():
    """{kind: (launches, elapsed_ms)} for every kernel kind."""
    out = {}
    for name, k in KERNEL_KINDS.items():
        n = ctypes.c_int64(0)
        ms = ctypes.c_double(0.0)
        _check(load().rcx_stats_read(k, ctypes.byref(n), ctypes.byref(ms)), "rcx_stats_read")
        out[name] = (n.value, ms.value)
    return out


def ring_attn_fwd_noalloc(q, k, v, o, lse=None, kv_block=0, window=0, n_sink=0, temperature=1.0, positions=None,
                          inv_freq=None, rope_flags=0):
    """rcx_ring_attn_fwd_noalloc: the ring forward with the library's static
    scratch instead of a caller workspace, for callers that cannot allocate
    device memory.  o (and lse) are caller-provided; nothing is allocated."""
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    st = load().rcx_ring_attn_fwd_noalloc(view(q), view(k), view(v), view(o), lse_view(lse), int(kv_block),
                                          int(window), int(n_sink), float(temperature), pp, npos, fp,
                                          int(rope_flags), _stream(q.device))
    _check(st, "rcx_ring_attn_fwd_noalloc")
    return o, lse


def kv_quantize_int8(x, codes=None, scale=None):
    """Int8 codes [B, N, H, 128] and fp32 scales [B, H, N] (head-major) of a bf16 cache x."""
    B, N, H, _ = x.shape
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(B, H, N, dtype=torch.float32, device=x.device)
    if not scale.is_contiguous() or scale.dtype != torch.float32 or tuple(scale.shape) != (B, H, N):
        raise ValueError("scale must be a contiguous float32 [B, H, N] tensor")
    st = load().rcx_kv_quantize_int8(view(x), view(codes), ctypes.c_void_p(scale.data_ptr()), _stream(x.device))
    _check(st, "rcx_kv_quantize_int8")
    return codes, scale


def attn_decode_int8_fwd(q, k, k_scale, v, v_scale, o=None, lse=None, window=0, n_sink=0, temperature=1.0,
                         q_index=None, positions=None, inv_freq=None, rope_flags=0, workspace=None, want_lse=True):
    """attn_decode_fwd over an int8 cache (codes k, v [B, Nk, Hkv, 128], scales [B, Hkv, Nk])."""
    B, _, H, D = q.shape
    if q_index is None:
        q_index = k.shape[1] - 1
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, 1, dtype=torch.float32, device=q.device)
    Bk, Nk, Hkv = k.shape[:3]
    for sc in (k_scale, v_scale):
        if not sc.is_contiguous() or sc.dtype != torch.float32 or tuple(sc.shape) != (Bk, Hkv, Nk):
            raise ValueError("scales must be contiguous float32 [B, Hkv, Nk] tensors")
    need = load().rcx_attn_decode_int8_workspace_size(view(q), view(k))
    if need < 0:
        raise RcxError(RCX_ERR_INVALID_ARG, "rcx_attn_decode_int8_workspace_size")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    st = load().rcx_attn_decode_int8_fwd(view(q), view(k), ctypes.c_void_p(k_scale.data_ptr()), view(v),
                                         ctypes.c_void_p(v_scale.data_ptr()), view(o), lse_view(lse), int(window),
                                         int(n_sink), float(temperature), int(q_index), pp, npos, fp,
                                         int(rope_flags), ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                         _stream(q.device))
    _check(st, "rcx_attn_decode_int8_fwd")
    return o, lse


def attn_decode_fwd(q, k, v, o=None, lse=None, window=0, n_sink=0, temperature=1.0, q_index=None, positions=None,
                    inv_freq=None, rope_flags=0, workspace=None, want_lse=True):
    """One query token per (batch, head) against a KV cache k, v [B, Nk, Hkv, 128].

    q: [B, 1, Hq, 128]; q_index defaults to Nk - 1 (the newest cached token)."""
    B, _, H, D = q.shape
    if q_index is None:
        q_index = k.shape[1] - 1
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, 1, dtype=torch.float32, device=q.device)
    need = load().rcx_attn_decode_workspace_size(view(q), view(k))
    if need < 0:
        raise RcxError(RCX_ERR_INVALID_ARG, "rcx_attn_decode_workspace_size")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    arr, fp = _freq_ptr(inv_freq)
    pp, npos = _pos(positions)
    st = load().rcx_attn_decode_fwd(view(q), view(k), view(v), view(o), lse_view(lse), int(window), int(n_sink),
                                    float(temperature), int(q_index), pp, npos, fp, int(rope_flags),
                                    ctypes.c_void_p(workspace.data_ptr()), workspace.numel(), _stream(q.device))
    _check(st, "rcx_attn_decode_fwd")
    return o, lse


# ------------------------------------------------- rotation by several axes
#
# The calls below serve decoding steps, whose kernels run for a few
# microseconds: their tensors are marshalled by _rcx_torch (csrc/torch_binding.cpp),
# which also checks types and devices, instead of through ctypes.

EXT_PATH = os.path.join(_PKG, "_rcx_torch.so")
_ext = None


def _fast():
    """Load _rcx_torch.so (built in-tree beside librcx.so); raise if it is missing."""
    global _ext
    if _ext is None:
        load()
        if not os.path.exists(EXT_PATH):
            raise RuntimeError(f"{EXT_PATH} is not built: run `python -m rope_context_extension_scaled_b200.build`")
        loader = importlib.machinery.ExtensionFileLoader("_rcx_torch", EXT_PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_rcx_torch", loader))
        loader.exec_module(ext)
        _ext = ext
    return _ext


def rope_axes_map(sections, interleaved=False):
    """The axis of each pair (int32 [sum(sections)]) when axis a owns sections[a]
    pairs: one section after another, or dealt out in turn (interleaved)."""
    sec = [int(x) for x in sections]
    out = np.zeros(max(sum(sec), 0), dtype=np.int32)
    st = load().rcx_rope_axes_map((ctypes.c_int64 * max(len(sec), 1))(*sec), len(sec), int(bool(interleaved)), out.size,
                                  out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    _check(st, "rcx_rope_axes_map")
    return out


def rope_axes_apply(q, k, inv_freq, axis, positions, halves=False, inverse=False, q_out=None, k_out=None):
    """Rotate q and/or k (either may be None) by positions on several axes.

    Pair i turns by positions[axis[i], b, n] * inv_freq[i]; the pair is (i, i + d/2)
    with halves, else (2i, 2i + 1); inverse turns back, which is the gradient of
    the rotation.  No autograd graph is recorded; an output that requires grad is
    refused while gradients are recorded, and a tensor that autograd has saved counts
    as changed when it is written.  inv_freq [d/2] and axis [d/2]
    are host arrays, positions an int64 [axes, B, N] tensor (axis and batch
    strides are free, 0 included).  Default: in place."""
    if q is None and k is None:
        return None, None
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    st = (_ext or _fast()).rope_axes_apply(q, k, q_out, k_out, np.asarray(inv_freq, np.float64),
                                           np.asarray(axis, np.int32), positions,
                                           (ROPE_HALVES if halves else 0) | (ROPE_INVERSE if inverse else 0))
    if st:
        _check(st, "rcx_rope_axes_apply")
    return q_out, k_out


# ------------------------------------------------- block-scaled 8-bit KV cache

class KvBlockCache:
    """A paged KV cache in 8 bits with one scale per block and head (rcx_kv_blocks).

    k, v: code pools [n_blocks, block, Hkv, d], int8 or float8_e4m3fn; block 16,
    32, 64 or 128; d 64 or 128; any strides with unit stride over d (the pools
    may be stored [n_blocks, Hkv, block, d]).  k_scale, v_scale: contiguous
    float32 [n_blocks, Hkv].  table: int32 [B, width], the block of each
    sequence's tokens j * block ..; entries behind a sequence's tokens are not
    read.  The handle keeps the tensors, not their contents: tables and pools
    are the caller's to fill and to change between calls; other tensors need
    another handle."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "table", "view", "address")

    def __setattr__(self, name, value):
        if hasattr(self, "address"):
            raise AttributeError(f"a KvBlockCache does not change: make another one for another {name}")
        object.__setattr__(self, name, value)

    def __init__(self, k, v, k_scale, v_scale, table):
        n, _, h, _ = k.shape
        for s in (k_scale, v_scale):
            if not s.is_contiguous() or s.dtype != torch.float32 or tuple(s.shape) != (n, h):
                raise ValueError(f"scales must be contiguous float32 [{n}, {h}] tensors")
        if table.dtype != torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be an int32 [B, width] tensor with unit stride over blocks")
        for x in (k, v, k_scale, v_scale, table):
            if not x.is_cuda or x.device != k.device:
                raise ValueError(f"expected CUDA tensors on one device, got {k.device} and {x.device}")
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.view = RcxKvBlocks(view(k), view(v), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(),
                                table.shape[0], table.shape[1], table.stride(0))
        self.address = ctypes.addressof(self.view)


def kv_block_append(k, v, cache, start, count=None):
    """Quantise tokens start[b] .. start[b] + count[b] - 1 (rows of k, v [B, N, Hkv,
    d], bf16 or fp32; count None: N each) into the cache's blocks."""
    st = (_ext or _fast()).kv_block_append(k, v, cache.k, cache.address, start, count)
    if st:
        _check(st, "rcx_kv_block_append")


def kv_block_read(cache, lengths, n, dtype=torch.bfloat16, k_out=None, v_out=None):
    """The first n tokens of each sequence as k, v [B, n, Hkv, d] in dtype (bf16 or
    fp32), zeros from token lengths[b] on."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}")
    st, k_out, v_out = (_ext or _fast()).kv_block_read(cache.k, cache.address, cache.view.B, lengths, n, k_out, v_out,
                                                       dtype == torch.bfloat16)
    if st:
        _check(st, "rcx_kv_block_read")
    return k_out, v_out


def attn_kv_block_workspace_size(q, cache):
    n = load().rcx_attn_kv_block_workspace_size(view(q), ctypes.byref(cache.view))
    if n < 0:
        raise RcxError(RCX_ERR_INVALID_ARG, "rcx_attn_kv_block_workspace_size")
    return int(n)


def attn_kv_block_fwd(q, cache, start, count=None, o=None, lse=None, window=0, n_sink=0, temperature=1.0,
                      workspace=None, want_lse=True):
    """Attention of tokens start[b] .. start[b] + count[b] - 1 (rows of q [B, N, Hq,
    d], bf16, rotated; count None: N each) over the cache, which holds them.

    Rows from count[b] on give O = 0, lse = -inf.  workspace: uint8 tensor of
    attn_kv_block_workspace_size(q, cache) bytes (None: a new one)."""
    st, o, lse = (_ext or _fast()).attn_kv_block_fwd(q, cache.k, cache.address, start, count, o, lse, window, n_sink,
                                                     temperature, workspace, want_lse)
    if st:
        _check(st, "rcx_attn_kv_block_fwd")
    return o, lse
