"""Thin ctypes binding of libmoe.so (include/moe.h), same function names.

Argument marshalling only: every step of the layer runs in the CUDA library.
Arrays may be passed as torch tensors (device or host), numpy arrays (host)
or raw integer addresses.  A status other than MOE_OK raises MoeError.  The
library must have been built (``python -m sparse_moe_expert_gemv_b200.build``);
importing this module without it raises ImportError -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_OOM", 3: "MOE_ERR_CUDA",
                4: "MOE_ERR_STATE", 5: "MOE_ERR_BAD_SLOT", 6: "MOE_ERR_DEVICE",
                7: "MOE_ERR_TIMEOUT", 8: "MOE_ERR_NOT_SUPPORTED"}
(MOE_ERR_INVALID_ARG, MOE_ERR_OOM, MOE_ERR_CUDA, MOE_ERR_STATE, MOE_ERR_BAD_SLOT,
 MOE_ERR_DEVICE, MOE_ERR_TIMEOUT, MOE_ERR_NOT_SUPPORTED) = range(1, 9)
MOE_Q4_SYM_G32_F16 = 1
MOE_Q2_ASYM_G64_F16 = 2
MOE_KV_BF16, MOE_KV_E4M3 = 1, 2

# every symbol include/moe.h declares
EXPORTS = ("moe_create", "moe_configure", "moe_destroy", "moe_load_experts",
           "moe_load_shared", "moe_set_router", "moe_set_norm", "moe_set_slots",
           "moe_route", "moe_bucket", "moe_forward", "moe_forward_delta",
           "moe_forward_stack", "moe_prefill", "moe_sync", "moe_get_stats",
           "moe_last_error", "moe_status_string", "moe_expert_bytes",
           "moe_debug_poke_slot", "moe_set_profiling", "moe_read_profile",
           "moe_set_trace", "moe_read_trace", "moe_route_static", "moe_prefill_delta",
           "moe_prefill_route", "moe_route_static_status", "moe_debug_last_h",
           "moe_debug_stall_next_decode", "moe_set_host_tier", "moe_tier_prepare",
           "moe_tier_prefetch", "moe_forward_tiered", "moe_tier_stats", "moe_tier_dump_trace",
           "moe_tier_sim_create", "moe_tier_sim_request", "moe_tier_sim_counts",
           "moe_tier_sim_destroy", "moe_rmsnorm", "moe_experts_given", "moe_ep_dispatch",
           "moe_ep_combine", "moe_experts_rows", "moe_attn_configure", "moe_qk_norm_rope",
           "moe_kv_append", "moe_attn_forward", "moe_attn_prefill")


class MoeError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class MoeStats(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
                ("near_ties", ctypes.c_int64), ("last_T", ctypes.c_int32),
                ("last_active", ctypes.c_int32), ("last_layer", ctypes.c_int32),
                ("E", ctypes.c_int32), ("expert_count", ctypes.POINTER(ctypes.c_int32))]


class _KvBatch(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("row_off", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_rows", ctypes.c_int32)]


class _QkNorm(ctypes.Structure):
    _fields_ = [("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p), ("eps", ctypes.c_float)]


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


def _load():
    if not os.path.exists(SO_PATH):
        raise ImportError(f"{SO_PATH} is missing: build it with "
                          "`python -m sparse_moe_expert_gemv_b200.build`")
    L = ctypes.CDLL(SO_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    I64 = ctypes.c_int64
    sig = {
        "moe_create": [I, I, I, I, I, ctypes.POINTER(P)],
        "moe_configure": [P, I, I, I, I],
        "moe_destroy": [P],
        "moe_load_experts": [P, I, I, I, P, P, P, I],
        "moe_load_shared": [P, I, P, P, P, I],
        "moe_set_router": [P, I, P, P, I],
        "moe_set_norm": [P, I, P, F],
        "moe_set_slots": [P, P],
        "moe_route": [P, I, P, I, P, P, P, P, P],
        "moe_bucket": [P, P, I, P, P, P],
        "moe_forward": [P, I, P, I, P],
        "moe_forward_delta": [P, I, P, I, P, P],
        "moe_forward_stack": [P, P, I, P],
        "moe_prefill": [P, I, P, I, P],
        "moe_prefill_delta": [P, I, P, I, P, P],
        "moe_prefill_route": [P, I, P, I, P, P, P, P, P],
        "moe_route_static_status": [ctypes.POINTER(I), P],
        "moe_debug_last_h": [P, P, I, P],
        "moe_debug_stall_next_decode": [P, ctypes.c_uint32],
        "moe_sync": [P, I],
        "moe_get_stats": [P, ctypes.POINTER(MoeStats)],
        "moe_debug_poke_slot": [P, I, I, ctypes.c_int32],
        "moe_set_profiling": [P, I],
        "moe_set_trace": [P, I],
        "moe_route_static": [P, I, I, I, I, P, P, P, P, P, P, P],
        "moe_read_trace": [P, ctypes.POINTER(ctypes.c_int64), I],
        "moe_read_profile": [P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)],
        "moe_set_host_tier": [P, I, I, ctypes.c_double],
        "moe_tier_prepare": [P, I, P, I, P],
        "moe_tier_prefetch": [P, I, P, I, P],
        "moe_forward_tiered": [P, I, P, I, P],
        "moe_tier_stats": [P, ctypes.POINTER(ctypes.c_int64)],
        "moe_tier_dump_trace": [P, ctypes.c_char_p],
        "moe_tier_sim_request": [P, ctypes.POINTER(ctypes.c_int64), I, I, ctypes.POINTER(I)],
        "moe_rmsnorm": [P, I, P, I, P, P],
        "moe_experts_given": [P, I, P, I, I, P, P, I, P, P],
        "moe_ep_dispatch": [P, P, I, I, P, P, P, P, ctypes.POINTER(ctypes.c_int32), P],
        "moe_ep_combine": [P, I, P, P, P, P, P, P, P],
        "moe_experts_rows": [P, I, P, I, P, P, P],
        "moe_attn_configure": [P, I, I, I, I, I],
        "moe_qk_norm_rope": [P, I, P, I64, P, I64, P, P, P, P, I64, P, I64, P],
        "moe_kv_append": [P, P, P, I64, P, I64, P, I64, P, P, P, I64, P],
        "moe_attn_forward": [P, P, P, I64, I, F, I, I, P, I64, P],
        "moe_attn_prefill": [P, P, P, I64, I, F, I, I, P, I64, P],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = I
    L.moe_last_error.argtypes = [P]
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [I]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_expert_bytes.argtypes = [I, I, I]
    L.moe_expert_bytes.restype = ctypes.c_int64
    L.moe_tier_sim_create.argtypes = [I, I, ctypes.c_double, ctypes.c_int64]
    L.moe_tier_sim_create.restype = P
    L.moe_tier_sim_counts.argtypes = [P, ctypes.POINTER(ctypes.c_int64)]
    L.moe_tier_sim_counts.restype = None
    L.moe_tier_sim_destroy.argtypes = [P]
    L.moe_tier_sim_destroy.restype = None
    return L


_lib = _load()


def lib():
    return _lib


def _ptr(a):
    """Address of a tensor / ndarray / int / None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return a.ctypes.data
    if hasattr(a, "data_ptr"):
        if not a.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return a.data_ptr()
    raise TypeError(f"cannot pass {type(a)} as a pointer")


def _is_dev(a):
    return bool(hasattr(a, "is_cuda") and a.is_cuda)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(ctx, rc):
    if rc != MOE_OK:
        msg = _lib.moe_last_error(ctx).decode() if ctx else ""
        raise MoeError(rc, msg)


# ------------------------------------------------------------------ C ABI
def moe_create(d, f, E, k, quant_fmt):
    out = ctypes.c_void_p()
    _check(None, _lib.moe_create(d, f, E, k, quant_fmt, ctypes.byref(out)))
    return out.value


def moe_configure(ctx, n_layers, n_shared, n_slots, max_tokens):
    _check(ctx, _lib.moe_configure(ctx, n_layers, n_shared, n_slots, max_tokens))


def moe_destroy(ctx):
    _attn.pop(ctx, None)
    _check(None, _lib.moe_destroy(ctx))


def moe_load_experts(ctx, layer, first_expert, n_experts, codes, scales, mins=None,
                     src_is_device=None):
    dev = _is_dev(codes) if src_is_device is None else bool(src_is_device)
    _check(ctx, _lib.moe_load_experts(ctx, layer, first_expert, n_experts, _ptr(codes),
                                      _ptr(scales), _ptr(mins), int(dev)))


def moe_load_shared(ctx, layer, codes, scales, mins=None, src_is_device=None):
    dev = _is_dev(codes) if src_is_device is None else bool(src_is_device)
    _check(ctx, _lib.moe_load_shared(ctx, layer, _ptr(codes), _ptr(scales), _ptr(mins), int(dev)))


def moe_set_router(ctx, layer, W, bias=None, src_is_device=None):
    dev = _is_dev(W) if src_is_device is None else bool(src_is_device)
    _check(ctx, _lib.moe_set_router(ctx, layer, _ptr(W), _ptr(bias), int(dev)))


def moe_set_norm(ctx, layer, gamma=None, eps=1e-6):
    _check(ctx, _lib.moe_set_norm(ctx, layer, _ptr(gamma), float(eps)))


def moe_set_slots(ctx, slot_of):
    a = np.ascontiguousarray(slot_of, dtype=np.int32)
    _check(ctx, _lib.moe_set_slots(ctx, _ptr(a)))


def moe_route(ctx, layer, h, T, idx, w, bucket_off=None, bucket_perm=None, stream=None):
    _check(ctx, _lib.moe_route(ctx, layer, _ptr(h), T, _ptr(idx), _ptr(w), _ptr(bucket_off),
                               _ptr(bucket_perm), _stream(stream)))


def moe_bucket(ctx, idx, T, bucket_off, bucket_perm, stream=None):
    _check(ctx, _lib.moe_bucket(ctx, _ptr(idx), T, _ptr(bucket_off), _ptr(bucket_perm),
                                _stream(stream)))


def moe_forward(ctx, layer, x, T, stream=None):
    _check(ctx, _lib.moe_forward(ctx, layer, _ptr(x), T, _stream(stream)))


def moe_forward_delta(ctx, layer, x, T, delta, stream=None):
    _check(ctx, _lib.moe_forward_delta(ctx, layer, _ptr(x), T, _ptr(delta), _stream(stream)))


def moe_forward_stack(ctx, x, T, stream=None):
    _check(ctx, _lib.moe_forward_stack(ctx, _ptr(x), T, _stream(stream)))


def moe_prefill(ctx, layer, x, N, stream=None):
    _check(ctx, _lib.moe_prefill(ctx, layer, _ptr(x), N, _stream(stream)))


def moe_prefill_delta(ctx, layer, x, N, delta, stream=None):
    _check(ctx, _lib.moe_prefill_delta(ctx, layer, _ptr(x), N, _ptr(delta), _stream(stream)))


def moe_prefill_route(ctx, layer, h, N, idx, w, bucket_off=None, bucket_perm=None, stream=None):
    _check(ctx, _lib.moe_prefill_route(ctx, layer, _ptr(h), N, _ptr(idx), _ptr(w),
                                       _ptr(bucket_off), _ptr(bucket_perm), _stream(stream)))


def moe_rmsnorm(ctx, layer, x, T, h, stream=None):
    _check(ctx, _lib.moe_rmsnorm(ctx, layer, _ptr(x), T, _ptr(h), _stream(stream)))


def moe_experts_given(ctx, layer, h, N, kk, idx, w, with_shared, delta, stream=None):
    _check(ctx, _lib.moe_experts_given(ctx, layer, _ptr(h), N, kk, _ptr(idx), _ptr(w),
                                       int(bool(with_shared)), _ptr(delta), _stream(stream)))


def moe_experts_rows(ctx, layer, h, M, e, y16, stream=None):
    _check(ctx, _lib.moe_experts_rows(ctx, layer, _ptr(h), M, _ptr(e), _ptr(y16), _stream(stream)))


def moe_ep_dispatch(ctx, idx, N, n_ranks, h, send_h, send_e, row_of, stream=None):
    """Returns the rows sent to each rank (a list of n_ranks ints)."""
    counts = (ctypes.c_int32 * n_ranks)()
    _check(ctx, _lib.moe_ep_dispatch(ctx, _ptr(idx), N, n_ranks, _ptr(h), _ptr(send_h),
                                     _ptr(send_e), _ptr(row_of), counts, _stream(stream)))
    return list(counts)


def moe_ep_combine(ctx, N, w, y, row_of, y_shared=None, x=None, delta=None, stream=None):
    _check(ctx, _lib.moe_ep_combine(ctx, N, _ptr(w), _ptr(y), _ptr(row_of), _ptr(y_shared),
                                    _ptr(x), _ptr(delta), _stream(stream)))


def moe_sync(ctx, timeout_ms=-1):
    _check(ctx, _lib.moe_sync(ctx, int(timeout_ms)))


def moe_get_stats(ctx):
    st = MoeStats()
    _check(ctx, _lib.moe_get_stats(ctx, ctypes.byref(st)))
    counts = np.ctypeslib.as_array(st.expert_count, shape=(st.E,)).copy() if st.E else None
    return dict(calls=st.calls, tokens=st.tokens, hits=st.hits, misses=st.misses,
                near_ties=st.near_ties, last_T=st.last_T, last_active=st.last_active,
                last_layer=st.last_layer, expert_count=counts)


def moe_last_error(ctx):
    return _lib.moe_last_error(ctx).decode()


def moe_status_string(status):
    return _lib.moe_status_string(status).decode()


def moe_expert_bytes(d, f, quant_fmt):
    return int(_lib.moe_expert_bytes(d, f, quant_fmt))


def moe_debug_poke_slot(ctx, layer, expert, slot):
    _check(ctx, _lib.moe_debug_poke_slot(ctx, layer, expert, slot))


def moe_debug_stall_next_decode(ctx, polls):
    _check(ctx, _lib.moe_debug_stall_next_decode(ctx, int(polls)))


def moe_debug_last_h(ctx, out, T, stream=None):
    _check(ctx, _lib.moe_debug_last_h(ctx, _ptr(out), T, _stream(stream)))


def moe_set_profiling(ctx, enable):
    _check(ctx, _lib.moe_set_profiling(ctx, int(enable)))


def moe_read_profile(ctx):
    """-> (route_ms, experts_ms, combine_ms, n_calls), summed over the calls."""
    ms = (ctypes.c_double * 3)(0.0, 0.0, 0.0)
    n = ctypes.c_int64(0)
    _check(ctx, _lib.moe_read_profile(ctx, ms, ctypes.byref(n)))
    return ms[0], ms[1], ms[2], n.value


TRACE_POINTS = ("route_start", "route_waited", "route_logits", "route_last_start", "route_topk",
                "route_bucket", "route_end", "gate_start", "gate_waited", "gate_first_item",
                "gate_end", "down_start", "down_waited", "down_end", "comb_start", "comb_end",
                "route_loaded", "route_selected")


def moe_set_trace(ctx, enable):
    _check(ctx, _lib.moe_set_trace(ctx, int(enable)))


def moe_read_trace(ctx):
    """-> {point: (earliest_ns, latest_ns)}; points no CTA reached are omitted."""
    n = 2 * len(TRACE_POINTS)
    buf = (ctypes.c_int64 * n)()
    _check(ctx, _lib.moe_read_trace(ctx, buf, n))
    k = len(TRACE_POINTS)
    return {name: (buf[i], buf[k + i]) for i, name in enumerate(TRACE_POINTS) if buf[i] != -1}


def moe_route_static(h, T, d, E, k, W, bias, idx, w, bucket_off, bucket_perm, stream=None):
    """Routing that allocates nothing (see include/moe.h)."""
    _check(None, _lib.moe_route_static(_ptr(h), T, d, E, k, _ptr(W), _ptr(bias), _ptr(idx),
                                       _ptr(w), _ptr(bucket_off), _ptr(bucket_perm),
                                       _stream(stream)))


def moe_route_static_status(stream=None):
    """Device status word of the last moe_route_static call on this device.
    Returns the word (0 = fine); raises MoeError when it is non-zero."""
    st = ctypes.c_int(0)
    rc = _lib.moe_route_static_status(ctypes.byref(st), _stream(stream))
    if rc not in (MOE_OK, 6):
        _check(None, rc)
    if rc == 6:
        raise MoeError(rc, f"moe_route_static device status 0x{st.value:x}")
    return st.value


# ------------------------------------------------------------- host tier
TIER_LRU, TIER_ADAPTIVE = 0, 1


def moe_set_host_tier(ctx, enable=1, policy=TIER_ADAPTIVE, half_life=64.0):
    """Backing copies in pinned host memory, the slot pool as an HBM cache
    (before moe_configure; see include/moe.h)."""
    _check(ctx, _lib.moe_set_host_tier(ctx, int(enable), int(policy), float(half_life)))


def moe_tier_prepare(ctx, layer, idx, T, stream=None):
    _check(ctx, _lib.moe_tier_prepare(ctx, layer, _ptr(idx), T, _stream(stream)))


def moe_tier_prefetch(ctx, layer, idx, T, stream=None):
    _check(ctx, _lib.moe_tier_prefetch(ctx, layer, _ptr(idx), T, _stream(stream)))


def moe_forward_tiered(ctx, layer, x, T, stream=None):
    _check(ctx, _lib.moe_forward_tiered(ctx, layer, _ptr(x), T, _stream(stream)))


def moe_tier_stats(ctx):
    """{"hits", "misses", "evictions", "bytes", "requests", "slots_used"}"""
    out = (ctypes.c_int64 * 6)()
    _check(ctx, _lib.moe_tier_stats(ctx, out))
    return dict(zip(("hits", "misses", "evictions", "bytes", "requests", "slots_used"), out))


def moe_tier_dump_trace(ctx, path):
    _check(ctx, _lib.moe_tier_dump_trace(ctx, os.fsencode(path)))


class TierSim:
    """Host-only model of the tier's replacement policy (moe_tier_sim_*)."""

    def __init__(self, n_slots, policy, half_life, n_keys):
        self.h = _lib.moe_tier_sim_create(n_slots, policy, float(half_life), n_keys)
        if not self.h:
            raise ValueError("moe_tier_sim_create: bad arguments")

    def request(self, keys, protect_prev=False):
        """(misses, slots) for one request of distinct keys; raises on -1 / -2."""
        n = len(keys)
        karr = (ctypes.c_int64 * max(n, 1))(*keys)
        sarr = (ctypes.c_int * max(n, 1))()
        r = _lib.moe_tier_sim_request(self.h, karr, n, int(protect_prev), sarr)
        if r == -1:
            raise ValueError("moe_tier_sim_request: bad arguments")
        if r == -2:
            raise MoeError(1, "the request needs more slots than may be taken")
        return r, list(sarr[:n])

    def counts(self):
        out = (ctypes.c_int64 * 3)()
        _lib.moe_tier_sim_counts(self.h, out)
        return dict(zip(("hits", "misses", "evictions"), out))

    def close(self):
        if self.h:
            _lib.moe_tier_sim_destroy(self.h)
            self.h = None

    def __del__(self):
        self.close()


# ------------------------------------------------------------- attention
# Geometry and device of the contexts configured for attention: the calls
# below take torch tensors and check their types, shapes, strides and device
# against it, since the library sees addresses only.
_attn = {}


class _Geometry:
    """Geometry of a context's attention, as the calls compare and pass it."""

    def __init__(self, n_q, n_kv, head_dim, page_size, cache_type, device):
        self.n_q, self.n_kv, self.dim, self.device = n_q, n_kv, head_dim, device
        self.batch = (n_kv, head_dim, page_size, cache_type, device)


@functools.cache
def _marshal():
    """The compiled marshalling of the attention calls, given their addresses."""
    import torch  # noqa: F401  (its libraries first)

    try:
        from . import _marshal as m
    except ImportError as e:
        raise ImportError("_marshal.so is missing or of another torch: build it with "
                          "`python -m sparse_moe_expert_gemv_b200.build`") from e
    m.set_calls(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        _lib.moe_qk_norm_rope, _lib.moe_kv_append, _lib.moe_attn_forward, _lib.moe_attn_prefill)))
    return m


def moe_attn_configure(ctx, n_q, n_kv, head_dim, page_size, cache_type):
    global _m
    _m = _marshal()
    _check(ctx, _lib.moe_attn_configure(ctx, n_q, n_kv, head_dim, page_size, cache_type))
    import torch
    _attn[ctx] = _Geometry(n_q, n_kv, head_dim, page_size, cache_type, torch.cuda.current_device())


def _no_geometry(ctx):
    raise MoeError(MOE_ERR_STATE, "moe_attn_configure comes first")


@functools.cache
def _dtype(name):
    import torch
    return getattr(torch, name)


def _dense(name, t, dtype, shape=None):
    """A dense CUDA tensor of this type (and shape); its address."""
    if not t.is_cuda or t.dtype is not _dtype(dtype) or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous CUDA tensor of {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, not {tuple(shape)}")
    return t.data_ptr()


def _stream_on(stream, device):
    """As _stream, with the current stream of `device` for None."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _raw_stream(device)


def _raw_stream(device):
    """The current stream's handle: torch's own accessor when it has one (a
    tenth of the time of building a Stream object)."""
    global _raw_stream
    import torch
    fast = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = fast or (lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


class KvBatch:
    """The rows of one call and the paged cache of one layer (moe_kv_batch).

    k, v: [n_pages, n_kv, page_size, head_dim] bfloat16 or float8_e4m3fn (with
    k_scale, v_scale: fp32 [n_kv] or None); page_table int32 [n_seqs,
    max_pages], row_off int32 [n_seqs + 1], kv_len int32 [n_seqs].  Holds the
    tensors; their contents are read when the calls run, so one batch object
    serves every step whose tables are updated in place."""

    def __init__(self, k, v, page_table, row_off, kv_len, n_rows, k_scale=None, v_scale=None):
        e4m3 = str(k.dtype) == "torch.float8_e4m3fn"
        kind = "float8_e4m3fn" if e4m3 else "bfloat16"
        if k.dim() != 4:
            raise ValueError("k: [n_pages, n_kv, page_size, head_dim]")
        n_pages, n_kv = k.shape[0], k.shape[1]
        if page_table.dim() != 2:
            raise ValueError("page_table: [n_seqs, max_pages]")
        n_seqs, max_pages = page_table.shape
        tensors = [k, v, page_table, row_off, kv_len, k_scale, v_scale]
        self.c = _KvBatch(
            _dense("k", k, kind), _dense("v", v, kind, k.shape),
            None if k_scale is None else _dense("k_scale", k_scale, "float32", (n_kv,)),
            None if v_scale is None else _dense("v_scale", v_scale, "float32", (n_kv,)),
            _dense("page_table", page_table, "int32"), _dense("row_off", row_off, "int32", (n_seqs + 1,)),
            _dense("kv_len", kv_len, "int32", (n_seqs,)), n_pages, n_seqs, max_pages, n_rows)
        device = k.get_device()
        self.geometry = (n_kv, k.shape[3], k.shape[2], MOE_KV_E4M3 if e4m3 else MOE_KV_BF16, device)
        if any(t is not None and t.get_device() != device for t in tensors):
            raise ValueError("the batch's tensors are on different devices")
        self.tensors = tensors
        self.n_rows = n_rows
        self.ref = ctypes.addressof(self.c)

class QkNorm:
    """RMSNorm of the query and key heads (moe_qk_norm): fp32 [head_dim] CUDA
    tensors or None (= 1)."""

    def __init__(self, q_gamma=None, k_gamma=None, eps=1e-6):
        self.tensors = [t for t in (q_gamma, k_gamma) if t is not None]
        kinds = {(t.numel(), t.get_device()) for t in self.tensors}
        if len(kinds) > 1:
            raise ValueError("q_gamma and k_gamma: of one length, on one device")
        self.geometry = kinds.pop() if kinds else None
        self.c = _QkNorm(None if q_gamma is None else _dense("q_gamma", q_gamma, "float32"),
                         None if k_gamma is None else _dense("k_gamma", k_gamma, "float32"), float(eps))
        self.ref = ctypes.addressof(self.c)

class Rope:
    """Rotary positions (moe_rope): inv_freq float64 [rot_dim / 2] on the GPU,
    radians per position."""

    def __init__(self, inv_freq, rot_dim, interleaved=False):
        self.tensors = [inv_freq]
        self.device = inv_freq.get_device()
        self.c = _Rope(_dense("inv_freq", inv_freq, "float64", (rot_dim // 2,)), rot_dim, int(bool(interleaved)))
        self.ref = ctypes.addressof(self.c)

def _batch_ref(batch, g):
    if batch.geometry != g.batch:
        raise ValueError(f"batch of (n_kv, head_dim, page_size, type, device) {batch.geometry}: the context has "
                         f"{g.batch}")
    return batch.ref


def _norm_ref(norm, g):
    if norm is None:
        return None
    if norm.geometry is not None and norm.geometry != (g.dim, g.device):
        raise ValueError(f"norm weights: [{g.dim}] on cuda:{g.device}")
    return norm.ref


def _rope_ref(rope, g):
    if rope is None:
        return None
    if rope.device != g.device:
        raise ValueError(f"inv_freq: on cuda:{g.device}")
    return rope.ref


def moe_qk_norm_rope(ctx, n_rows, q, k, pos, norm, rope, q_out, k_out, stream=None):
    g = _attn.get(ctx) or _no_geometry(ctx)
    rc = _m.qk_norm_rope(g.n_q, g.n_kv, g.dim, g.device, ctx, n_rows, q, k, pos, _norm_ref(norm, g),
                         _rope_ref(rope, g), q_out, k_out, _stream_on(stream, g.device))
    if rc:
        _check(ctx, rc)


def moe_kv_append(ctx, batch, q, k, v, norm, rope, q_out, stream=None):
    """q and q_out may both be None (keys and values only)."""
    g = _attn.get(ctx) or _no_geometry(ctx)
    rc = _m.kv_append(g.n_q, g.n_kv, g.dim, g.device, ctx, batch.n_rows, _batch_ref(batch, g), q, k, v,
                      _norm_ref(norm, g), _rope_ref(rope, g), q_out, _stream_on(stream, g.device))
    if rc:
        _check(ctx, rc)


def moe_attn_forward(ctx, batch, q, max_T, scale, window, n_sink, out, stream=None):
    g = _attn.get(ctx) or _no_geometry(ctx)
    rc = _m.attend(0, g.n_q, g.dim, g.device, ctx, batch.n_rows, _batch_ref(batch, g), q, max_T, scale, window,
                   n_sink, out, _stream_on(stream, g.device))
    if rc:
        _check(ctx, rc)


def moe_attn_prefill(ctx, batch, q, max_T, scale, window, n_sink, out, stream=None):
    g = _attn.get(ctx) or _no_geometry(ctx)
    rc = _m.attend(1, g.n_q, g.dim, g.device, ctx, batch.n_rows, _batch_ref(batch, g), q, max_T, scale, window,
                   n_sink, out, _stream_on(stream, g.device))
    if rc:
        _check(ctx, rc)
