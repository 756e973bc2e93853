"""ctypes binding of libpp's C ABI (include/pp.h): same names, argument marshalling only.

Every step of the path runs in the library's CUDA kernels. torch is used for device memory (tensors are passed as
raw device pointers) and for the current stream. There is no fallback: if libpp.so is missing or fails to load,
every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpp.so")

PP_OK = 0
PP_ERR_INVALID_ARG = -1
PP_ERR_UNSUPPORTED = -2
PP_ERR_CUDA = -3
PP_ERR_DEVICE_TIMEOUT = -4
PP_ERR_WORKSPACE = -5
PP_ERR_DEVICE_INPUT = -6
PP_BF16 = 0
PP_FP32 = 1
PP_E4M3 = 2
PP_INT8 = 3
PP_PASS_FWD = 0
PP_PASS_BWD = 1

STATUS_NAMES = {0: "PP_OK", -1: "PP_ERR_INVALID_ARG", -2: "PP_ERR_UNSUPPORTED", -3: "PP_ERR_CUDA",
                -4: "PP_ERR_DEVICE_TIMEOUT", -5: "PP_ERR_WORKSPACE", -6: "PP_ERR_DEVICE_INPUT"}

# exported symbol -> (restype, argtypes); the list mirrors include/pp.h
_VP, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_I64P = ctypes.POINTER(ctypes.c_int64)
SIGNATURES = {
    "pp_meta_bounds": (_I32, [_I32, _I32, _I64, _I32, _I32, _I64P]),
    "pp_build_meta": (_I32, [_VP, _I32, _VP, _I32, _I64, _I32, _I32, _VP, _VP, _I64, _VP]),
    "pp_meta_tiles": (_I32, [_VP, _I32, _VP, _I64, _VP, _VP]),
    "pp_meta_schedule": (_I32, [_VP, _I32, _VP, _I64, _VP, _VP]),
    "pp_rope": (_I32, [_VP, _VP, _VP, _I64, _I32, _I32, _I32, _F32, _I32, _I32, _VP]),
    "pp_workspace_bytes": (_I32, [_I32, _I64, _I32, _I32, _I32, _I64P]),
    "pp_attn_fwd": (_I32, [_VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _F32, _I32, _VP, _VP, _VP, _I64, _VP]),
    "pp_attn_bwd": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _F32, _VP, _VP, _VP, _VP,
                           _I64, _VP]),
    "pp_attn_bwd_noalloc": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _F32, _VP, _VP, _VP,
                                   _VP]),
    "pp_plan_batches": (_I32, [_VP, _I32, _I64, _I32, _VP, _VP, _VP]),
    "pp_decode_workspace_bytes": (_I32, [_VP, _I32, _VP, _I32, _I32, _I64P]),
    "pp_bwd_ds_bytes": (_I32, [_VP, _I32, _VP, _I32, _I32, _I32, _I64P]),
    "pp_decode_attn": (_I32, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I64, _I32, _I32, _I32, _F32, _VP, _VP, _VP, _I64,
                              _VP]),
    "pp_pack_batch": (_I32, [_VP, _VP, _I32, _VP, _VP, _I32, _VP, _I32, _VP, _I64, _VP, _VP, _VP, _VP, _VP]),
    "pp_response_logprobs": (_I32, [_VP, _I32, _I64, _VP, _VP, _I64, _F32, _VP, _VP]),
    "pp_qk_norm_rope": (_I32, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _F32, _F32, _I32, _VP, _VP,
                               _I64, _I64, _VP]),
    "pp_qk_norm_rope_bwd_bytes": (_I32, [_I64, _I32, _I32, _I32, _I64P]),
    "pp_qk_norm_rope_bwd": (_I32, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _F32, _F32, _I32, _VP,
                                   _VP, _I64, _I64, _VP, _VP, _I64, _I64, _VP, _VP, _VP, _I64, _VP]),
    "pp_pages_resize": (_I32, [_VP, _I32, _VP, _I32, _VP, _VP, _I32, _VP, _I64, _VP, _I32, _VP, _VP, _VP, _VP, _I64,
                               _VP, _VP]),
    "pp_cache_store": (_I32, [_VP, _VP, _I64, _I64, _I32, _VP, _I64, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _I32, _I32,
                              _VP]),
    "pp_paged_decode_bytes": (_I32, [_I32, _I32, _I32, _I64P]),
    "pp_paged_decode": (_I32, [_VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _VP, _I32, _VP, _I32, _VP, _VP, _I64, _I32,
                               _I32, _I32, _F32, _VP, _VP, _VP, _I64, _VP]),
    "pp_selftest_bounded_wait": (_I32, [_I64, _VP, _VP]),
    "pp_get_status": (_I32, [_VP]),
    "pp_last_error": (ctypes.c_char_p, []),
    "pp_version": (ctypes.c_char_p, []),
}

_lock = threading.Lock()
_lib = None


class PPError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def lib():
    """Load libpp.so once (no fallback: raises OSError if it is missing)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise OSError(f"libpp.so not built at {LIB_PATH}: run python -m shared_prefix_packed_b200.build")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _call(name, *args):
    st = getattr(lib(), name)(*args)
    if st != PP_OK:
        raise PPError(name, st, lib().pp_last_error().decode())
    return st


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return PP_BF16
    if t.dtype == torch.float32:
        return PP_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------------------------------------------------ calls
def pp_version() -> str:
    return lib().pp_version().decode()


def pp_meta_bounds(num_groups: int, num_segments: int, total_tokens: int, hq: int, hkv: int) -> int:
    out = ctypes.c_int64(0)
    _call("pp_meta_bounds", num_groups, num_segments, total_tokens, hq, hkv, ctypes.byref(out))
    return out.value


def pp_build_meta(groups_d, cu_seqlens_d, total_tokens: int, hq: int, hkv: int, pos_ids_d, meta_d, stream=None):
    """groups_d: int32 [G, 2] (prefix_len, num_suffixes); cu_seqlens_d: int32 [nseg+1]; all on the device."""
    G = groups_d.shape[0]
    nseg = cu_seqlens_d.shape[0] - 1
    _call("pp_build_meta", _ptr(groups_d), G, _ptr(cu_seqlens_d), nseg, total_tokens, hq, hkv, _ptr(pos_ids_d),
          _ptr(meta_d), meta_d.numel() * meta_d.element_size(), _stream(stream))


def pp_meta_tiles(meta_d, which: int, tiles_d, count_d, stream=None):
    cap = tiles_d.numel() // 3
    _call("pp_meta_tiles", _ptr(meta_d), which, _ptr(tiles_d), cap, _ptr(count_d), _stream(stream))


def pp_meta_schedule(meta_d, which: int, records_d, count_d, stream=None):
    cap = records_d.numel() // 5
    _call("pp_meta_schedule", _ptr(meta_d), which, _ptr(records_d), cap, _ptr(count_d), _stream(stream))


def pp_rope(q, k, pos_ids_d, hq: int, hkv: int, d: int, theta: float = 10000.0, inverse: bool = False,
            stream=None):
    ref = q if q is not None else k
    T = ref.shape[0]
    _call("pp_rope", _ptr(q), _ptr(k), _ptr(pos_ids_d), T, hq, hkv, d, float(theta), _dtype_code(ref),
          1 if inverse else 0, _stream(stream))


def pp_workspace_bytes(which: int, T: int, hq: int, hkv: int, d: int) -> int:
    out = ctypes.c_int64(0)
    _call("pp_workspace_bytes", which, T, hq, hkv, d, ctypes.byref(out))
    return out.value


def pp_attn_fwd(q, k, v, meta_d, o, lse, workspace, softmax_scale: float = 0.0, stream=None):
    T, hq, d = q.shape
    hkv = k.shape[1]
    _call("pp_attn_fwd", _ptr(q), _ptr(k), _ptr(v), _ptr(meta_d), T, hq, hkv, d, float(softmax_scale),
          _dtype_code(q), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
          _stream(stream))


def pp_plan_batches(group_tokens, capacity: int, sort_by_length: bool = True):
    """Host-side batch plan (see pp.h): returns (order, batch_of_group, n_batches) as a list, a list and an int."""
    import numpy as np
    toks = np.ascontiguousarray(np.asarray(group_tokens, dtype=np.int64))
    if toks.ndim != 1 or (toks.size and toks.min() < 0) or int(capacity) < 1:
        raise ValueError("group_tokens must be a 1-D array of non-negative counts and capacity >= 1")
    G = toks.size
    order = np.zeros(max(G, 1), dtype=np.int32)
    batch = np.zeros(max(G, 1), dtype=np.int32)
    nb = ctypes.c_int32(0)
    st = lib().pp_plan_batches(toks.ctypes.data_as(ctypes.c_void_p), G, int(capacity), 1 if sort_by_length else 0,
                               order.ctypes.data_as(ctypes.c_void_p), batch.ctypes.data_as(ctypes.c_void_p),
                               ctypes.byref(nb))
    if st != 0:
        raise PPError("pp_plan_batches", st, "invalid arguments")
    return order[:G].tolist(), batch[:G].tolist(), int(nb.value)


def pp_decode_workspace_bytes(groups_host, cu_host, hq: int) -> int:
    """groups_host: int32 [G, 2] CPU tensor; cu_host: int32 [nseg + 1] CPU tensor."""
    out = ctypes.c_int64(0)
    g = groups_host.contiguous()
    c = cu_host.contiguous()
    _call("pp_decode_workspace_bytes", ctypes.c_void_p(g.data_ptr()), g.shape[0], ctypes.c_void_p(c.data_ptr()),
          c.numel() - 1, hq, ctypes.byref(out))
    return out.value


def pp_bwd_ds_bytes(groups_host, cu_host, hq: int, hkv: int) -> int:
    """Extra backward workspace for the kept-dS path. groups_host: int32 [G, 2] CPU tensor; cu_host: int32 [nseg + 1]
    CPU tensor."""
    out = ctypes.c_int64(0)
    g = groups_host.contiguous()
    c = cu_host.contiguous()
    _call("pp_bwd_ds_bytes", ctypes.c_void_p(g.data_ptr()), g.shape[0], ctypes.c_void_p(c.data_ptr()), c.numel() - 1,
          hq, hkv, ctypes.byref(out))
    return out.value


def pp_decode_attn(q, k_cache, v_cache, groups_d, cu_d, o, lse, workspace, softmax_scale: float = 0.0, stream=None):
    T, hkv, d = k_cache.shape
    hq = q.shape[1]
    _call("pp_decode_attn", _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(groups_d), groups_d.shape[0], _ptr(cu_d),
          cu_d.numel() - 1, T, hq, hkv, d, float(softmax_scale), _ptr(o), _ptr(lse), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))


def pp_pack_batch(prompts, prompt_mask, responses, response_mask, uids, packed_ids, groups, cu_seqlens,
                  sample_offsets, counts, stream=None):
    bs, Lp = prompts.shape
    Lr = responses.shape[1]
    _call("pp_pack_batch", _ptr(prompts), _ptr(prompt_mask), Lp, _ptr(responses), _ptr(response_mask), Lr, _ptr(uids),
          bs, _ptr(packed_ids), packed_ids.numel(), _ptr(groups), _ptr(cu_seqlens), _ptr(sample_offsets),
          _ptr(counts), _stream(stream))


def pp_response_logprobs(logits, token_ids, meta_d, out, temperature: float = 1.0, stream=None):
    T, V = logits.shape
    _call("pp_response_logprobs", _ptr(logits), _dtype_code(logits), V, _ptr(token_ids), _ptr(meta_d), T,
          float(temperature), _ptr(out), _stream(stream))


def pp_attn_bwd(q, k, v, o, lse, dout, meta_d, dq, dk, dv, workspace, softmax_scale: float = 0.0, stream=None):
    T, hq, d = q.shape
    hkv = k.shape[1]
    _call("pp_attn_bwd", _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(meta_d), T, hq, hkv, d,
          float(softmax_scale), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))


def pp_attn_bwd_noalloc(q, k, v, o, lse, dout, meta_d, dq, dk, dv, softmax_scale: float = 0.0, stream=None):
    """pp_attn_bwd without a workspace argument: the library's built-in 64 MiB scratch is used instead."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    _call("pp_attn_bwd_noalloc", _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(meta_d), T, hq,
          hkv, d, float(softmax_scale), _ptr(dq), _ptr(dk), _ptr(dv), _stream(stream))


NOALLOC_SCRATCH_BYTES = 64 << 20


# ------------------------------------------------------------- q/k norm with the rotation, and the paged 8-bit cache
# These calls run once a layer on a few microseconds of GPU work. Their tensors are checked and the calls made in
# _bind.so (bind/pp_bind.cpp), which raises TypeError or ValueError and else returns the status.
_bind_module = None
_t = None


def _torch():
    global _t
    if _t is None:
        import torch
        _t = torch
    return _t


def _bind():
    global _bind_module
    if _bind_module is None:
        _torch()                                           # whose libraries it needs
        try:
            from . import _bind as m
        except ImportError as e:
            raise OSError(f"_bind.so is not built or does not load: run python -m shared_prefix_packed_b200.build ({e})")
        m.init(*(ctypes.cast(getattr(lib(), n), _VP).value for n in (
            "pp_qk_norm_rope", "pp_qk_norm_rope_bwd", "pp_pages_resize", "pp_cache_store", "pp_paged_decode")))
        _bind_module = m
    return _bind_module


def _done(name, st):
    if st != PP_OK:
        raise PPError(name, st, lib().pp_last_error().decode())


def stream_scope(device, stream):
    """A context in which torch allocates and launches on `stream` (None: the device's current stream), so that
    scratch and outputs belong to the stream that uses them. Raises ValueError for a stream of another device, whose
    scope would leave this device's own current stream in place."""
    torch = _torch()
    if stream is None:
        return torch.cuda.stream(None)                     # does nothing
    if not isinstance(stream, int):
        at = torch.cuda.current_device() if device.index is None else device.index
        if stream.device.index != at:
            raise ValueError(f"the stream is of cuda:{stream.device.index}, the tensors of cuda:{at}")
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream)


def pp_qk_norm_rope(q, k, wq, wk, pos_ids_d, q_out, k_out, eps: float = 1e-6, theta: float = 10000.0, stream=None):
    """q [T, hq, d], k [T, hkv, d] (views of a fused projection will do; either may be None): RMS norm of every head
    with weights wq, wk [d] (None: ones), rotated at pos_ids_d, into q_out, k_out."""
    _done("pp_qk_norm_rope", _bind().qk_norm_rope(q, k, wq, wk, pos_ids_d, q_out, k_out, eps, theta, stream))



@functools.lru_cache(maxsize=256)
def pp_qk_norm_rope_bwd_bytes(T: int, hq: int, hkv: int, d: int) -> int:
    out = ctypes.c_int64(0)
    _call("pp_qk_norm_rope_bwd_bytes", T, hq, hkv, d, ctypes.byref(out))
    return out.value


def pp_qk_norm_rope_bwd(q, k, wq, wk, pos_ids_d, gq, gk, dq, dk, dwq, dwk, workspace, eps: float = 1e-6,
                        theta: float = 10000.0, stream=None):
    """Gradients of pp_qk_norm_rope: gq, gk of its outputs -> dq, dk of its inputs and dwq, dwk (fp32 [d], or None)."""
    _done("pp_qk_norm_rope_bwd", _bind().qk_norm_rope_bwd(q, k, wq, wk, pos_ids_d, gq, gk, dq, dk, dwq, dwk, workspace,
                                                         eps, theta, stream))



def pp_pages_resize(group_start_d, seg_group_d, old_lens_d, new_lens_d, page_size: int, page_table_d, free_pages_d,
                    n_free_in, n_free_out, slots_d, pos_ids_d, counts_d, stream=None):
    """Give and take pages as the segments go from old_lens_d to new_lens_d tokens; slots and grouped positions of the
    new tokens. slots_d.numel() is the capacity, free_pages_d.numel() the pool's number of pages."""
    _done("pp_pages_resize", _bind().pages_resize(group_start_d, seg_group_d, old_lens_d, new_lens_d, page_size, page_table_d,
                                                 free_pages_d, n_free_in, n_free_out, slots_d, pos_ids_d, counts_d, stream))



def pp_cache_store(k, v, slots_d, k_pages, v_pages, k_scale, v_scale, stream=None):
    """Append rows k, v [n, hkv, d] at their slots: k_pages [num_pages, hkv, page_size, d], v_pages [num_pages, hkv, d,
    page_size] (float8_e4m3fn or int8), k_scale, v_scale fp32 [num_pages, hkv]. The rows of one page stand together: each
    within 256 rows of the one before, skipped rows (slot -1) between them and none of another page."""
    _done("pp_cache_store", _bind().cache_store(k, v, slots_d, k_pages, v_pages, k_scale, v_scale, stream))



@functools.lru_cache(maxsize=256)
def pp_paged_decode_bytes(n_resp: int, hq: int, hkv: int) -> int:
    out = ctypes.c_int64(0)
    _call("pp_paged_decode_bytes", n_resp, hq, hkv, ctypes.byref(out))
    return out.value


def pp_paged_decode(q, k_pages, v_pages, k_scale, v_scale, group_start_d, seg_group_d, lens_d, page_table_d, o, lse,
                    workspace, softmax_scale: float = 0.0, stream=None):
    """One decoding step of every response over a paged cache: q, o [n_resp, hq, d] bf16, lse [hq, n_resp] fp32."""
    _done("pp_paged_decode", _bind().paged_decode(q, k_pages, v_pages, k_scale, v_scale, group_start_d, seg_group_d, lens_d,
                                                 page_table_d, o, lse, workspace, softmax_scale, stream))



def pp_selftest_bounded_wait(limit_ns: int, waited_ns_d, stream=None):
    """Launch the bounded-wait self-test (a wait on an mbarrier nothing arrives on); waited_ns_d: int64 [1] device."""
    _call("pp_selftest_bounded_wait", int(limit_ns), _ptr(waited_ns_d), _stream(stream))


def pp_get_status(stream=None) -> int:
    """Synchronise the stream and read the device error word; raises PPError on a device-side error."""
    return _call("pp_get_status", _stream(stream))
