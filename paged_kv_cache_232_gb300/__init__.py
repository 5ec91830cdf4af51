"""Python binding of libpagedattn (include/pagedattn.h): argument marshalling only.

Every function here takes torch CUDA tensors, checks that they are contiguous and of
the expected dtypes, and forwards their device pointers and sizes to the C ABI through
ctypes on the caller's current CUDA stream.  All computation happens in the library's
CUDA kernels; there is no fallback of any kind.  If the shared library has not been
built, the first call builds it with nvcc (see _build.py) or raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from . import _build

PA_F16, PA_BF16 = 0, 1
PA_OK = 0
PA_DEVERR_SLOT, PA_DEVERR_BLOCK, PA_DEVERR_LENGTH, PA_DEVERR_TIMEOUT, PA_DEVERR_POSITION = 1, 2, 4, 8, 16
PA_DEVERR_SMEM = 32
PA_DEVERR_PATH, PA_DEVERR_FORK, PA_DEVERR_PAGES, PA_DEVERR_COUNT = 64, 128, 256, 512
DEFAULT_PARTITION_TOKENS = 256

# names the header declares; the CPU test checks that the library exports each one
EXPORTED = (
    "pa_reshape_and_cache", "pa_decode_workspace_size", "pa_decode", "pa_decode_plan", "pa_decode_v1",
    "pa_decode_splitk", "pa_prefill_chunk", "pa_device_errors", "pa_status_string", "pa_version",
    "pa_decode_splitk_static", "pa_rope_table", "pa_rope_reshape_and_cache", "pa_decode_shared_prefix",
    "pa_decode_shared_prefix_workspace_size", "pa_prefill_chunk_small_m", "pa_decode_write",
    "pa_norm_rope_reshape_and_cache", "pa_latent_rope_and_cache", "pa_latent_workspace_size", "pa_latent_decode",
    "pa_latent_prefill_chunk", "pa_tree_mask", "pa_tree_workspace_size", "pa_tree_decode", "pa_tree_commit",
    "pa_copy_pages", "pa_fork_pages", "pa_resize_workspace_size", "pa_resize_pages",
)
STATIC_SCRATCH_BYTES = 16 << 20


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.library_path()


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libpagedattn.so (building it first if needed)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libpagedattn is not built ({path}); run paged_kv_cache_232_gb300._build.build()")
        path = _build.build()
    L = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    L.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i64, i32, vp]
    L.pa_reshape_and_cache.restype = i32
    L.pa_rope_table.argtypes = [vp, i64, i32, ctypes.c_double]
    L.pa_rope_table.restype = i32
    L.pa_rope_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i64, i64, i32, vp]
    L.pa_rope_reshape_and_cache.restype = i32
    L.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.pa_decode_workspace_size.restype = sz
    L.pa_decode.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32, i32, vp, sz, vp]
    L.pa_decode.restype = i32
    L.pa_decode_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.pa_decode_plan.restype = i32
    L.pa_decode_write.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32, i32, vp, vp, vp,
                                  vp, sz, vp]
    L.pa_decode_write.restype = i32
    L.pa_decode_v1.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, f32, i32, vp]
    L.pa_decode_v1.restype = i32
    L.pa_decode_splitk.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32, i32, i32, vp,
                                   sz, vp]
    L.pa_decode_splitk.restype = i32
    L.pa_decode_splitk_static.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32, i32,
                                          i32, vp]
    L.pa_decode_splitk_static.restype = i32
    L.pa_decode_shared_prefix.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32, i32,
                                          i32, i32, vp, sz, vp]
    L.pa_decode_shared_prefix.restype = i32
    L.pa_decode_shared_prefix_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.pa_decode_shared_prefix_workspace_size.restype = sz
    L.pa_prefill_chunk.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i64, f32, i32, vp]
    L.pa_prefill_chunk.restype = i32
    L.pa_prefill_chunk_small_m.argtypes = L.pa_prefill_chunk.argtypes
    L.pa_prefill_chunk_small_m.restype = i32
    L.pa_norm_rope_reshape_and_cache.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, vp, vp, vp, vp,
                                                 i64, i32, i32, i32, i32, i64, i64, i32, vp]
    L.pa_norm_rope_reshape_and_cache.restype = i32
    L.pa_latent_rope_and_cache.argtypes = [vp, vp, i64, i64, vp, i64, vp, f32, vp, vp, vp, vp, i64, i32, i32, i32, i32,
                                           i64, i64, i32, i32, vp]
    L.pa_latent_rope_and_cache.restype = i32
    L.pa_latent_workspace_size.argtypes = [i32, i32, i32]
    L.pa_latent_workspace_size.restype = sz
    L.pa_latent_decode.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, f32, i32, vp, sz, vp]
    L.pa_latent_decode.restype = i32
    L.pa_latent_prefill_chunk.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i64, i32, i32, i32, i32, i64, f32, i32,
                                          vp, sz, vp]
    L.pa_latent_prefill_chunk.restype = i32
    L.pa_tree_mask.argtypes = [vp, vp, vp, i32, i32]
    L.pa_tree_mask.restype = i32
    L.pa_tree_workspace_size.argtypes = [i32, i32, i32, i32]
    L.pa_tree_workspace_size.restype = sz
    L.pa_tree_decode.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i64, i32, i32, i32, i32, i64, f32, i32,
                                 vp, sz, vp]
    L.pa_tree_decode.restype = i32
    L.pa_tree_commit.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, i32, vp, vp, i32, i64, i32, i64, vp]
    L.pa_tree_commit.restype = i32
    L.pa_copy_pages.argtypes = [vp, vp, i32, vp, i64, i64, i32, i64, vp]
    L.pa_copy_pages.restype = i32
    L.pa_fork_pages.argtypes = [vp, i32, vp, vp, i32, vp, i32, i64, vp]
    L.pa_fork_pages.restype = i32
    L.pa_resize_workspace_size.argtypes = [i32, i64]
    L.pa_resize_workspace_size.restype = sz
    L.pa_resize_pages.argtypes = [vp, vp, i32, vp, i32, vp, vp, i32, vp, vp, vp, i64, i32, i64, vp, sz, vp]
    L.pa_resize_pages.restype = i32
    L.pa_device_errors.argtypes = [i32]
    L.pa_device_errors.restype = i32
    L.pa_status_string.argtypes = [i32]
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_version.restype = i32
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().pa_status_string(status).decode()


# ------------------------------------------------------------------ marshalling helpers


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch, ty = _torch(), t.dtype
    if ty == torch.bfloat16:
        return PA_BF16
    if ty == torch.float16:
        return PA_F16
    raise TypeError(f"expected float16 or bfloat16, got {ty}")


def _dev(t, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream, device) -> int:
    if stream is None:
        stream = _torch().cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, what: str):
    if status != PA_OK:
        raise PagedAttnError(status, what)


def _cache_dims(k_cache):
    nb, bs, hkv, d = k_cache.shape
    return int(nb), int(bs), int(hkv), int(d)


# ------------------------------------------------------------------ entry points


def pa_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, stream=None) -> None:
    """Scatter key/value [N, Hkv, D] into the caches [NB, bs, Hkv, D] at slot_mapping [N] (int64, -1 skips)."""
    torch = _torch()
    dt = _dtype_code(key)
    nb, bs, hkv, d = _cache_dims(k_cache)
    n = int(key.shape[0])
    st = load().pa_reshape_and_cache(_dev(key, "key", key.dtype), _dev(value, "value", key.dtype),
                                     _dev(k_cache, "k_cache", key.dtype), _dev(v_cache, "v_cache", key.dtype),
                                     _dev(slot_mapping, "slot_mapping", torch.int64), n, hkv, d, bs, nb, dt,
                                     _stream(stream, key.device))
    _check(st, "pa_reshape_and_cache")


def pa_rope_table(max_position: int, head_dim: int, theta: float):
    """The float32 [max_position, head_dim] cos / sin table (host numpy array) the fused RoPE
    write reads; copy it to the device once."""
    import numpy as np
    out = np.empty((int(max_position), int(head_dim)), dtype=np.float32)
    _check(load().pa_rope_table(out.ctypes.data, int(max_position), int(head_dim), float(theta)), "pa_rope_table")
    return out


def rope_cos_sin(max_position: int, head_dim: int, theta: float, device="cuda"):
    """pa_rope_table's output as a device tensor."""
    return _torch().from_numpy(pa_rope_table(max_position, head_dim, theta)).to(device)


def pa_rope_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, q=None,
                              stream=None) -> None:
    """Rotate key [N, Hkv, D] by positions [N] (int64) with the cos_sin table [max_position, D]
    (float32) and scatter it, and value unchanged, into the caches at slot_mapping [N] (int64,
    -1 skips); q [N, Hq, D], if given, is rotated in place."""
    torch = _torch()
    dt = _dtype_code(key)
    nb, bs, hkv, d = _cache_dims(k_cache)
    n = int(key.shape[0])
    qp, hq = (None, 0) if q is None else (_dev(q, "q", key.dtype), int(q.shape[1]))
    st = load().pa_rope_reshape_and_cache(
        qp, _dev(key, "key", key.dtype), _dev(value, "value", key.dtype), _dev(k_cache, "k_cache", key.dtype),
        _dev(v_cache, "v_cache", key.dtype), _dev(slot_mapping, "slot_mapping", torch.int64),
        _dev(positions, "positions", torch.int64), _dev(cos_sin, "cos_sin", torch.float32), n, hq, hkv, d, bs, nb,
        int(cos_sin.shape[0]), dt, _stream(stream, key.device))
    _check(st, "pa_rope_reshape_and_cache")


def pa_decode_workspace_size(num_seqs: int, n_q_heads: int, head_dim: int, max_context_len: int,
                             partition_tokens: int = 0) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, n_q_heads, head_dim, max_context_len, partition_tokens))


def pa_decode_plan(num_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int, block_size: int,
                   max_context_len: int, dtype: int = PA_BF16):
    """(1 = one-pass kernel | 2 = split-K, partition_tokens) for these sizes on the current device."""
    pt = ctypes.c_int(0)
    r = load().pa_decode_plan(num_seqs, n_q_heads, n_kv_heads, head_dim, block_size, max_context_len, dtype,
                              ctypes.byref(pt))
    if r < 0:
        raise PagedAttnError(r, "pa_decode_plan")
    return r, pt.value


def _decode_common(out, q, k_cache, v_cache, block_tables, context_lens):
    torch = _torch()
    dt = _dtype_code(q)
    nb, bs, hkv, d = _cache_dims(k_cache)
    S, hq, d2 = (int(x) for x in q.shape)
    if d2 != d or tuple(out.shape) != tuple(q.shape):
        raise ValueError("q/out/cache head_dim mismatch")
    ptrs = (_dev(out, "out", q.dtype), _dev(q, "q", q.dtype), _dev(k_cache, "k_cache", q.dtype),
            _dev(v_cache, "v_cache", q.dtype), _dev(block_tables, "block_tables", torch.int32),
            _dev(context_lens, "context_lens", torch.int32))
    return dt, nb, bs, hkv, d, S, hq, int(block_tables.shape[1]), ptrs


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
              workspace=None, stream=None) -> None:
    """Decode attention with the library's dispatcher choosing one-pass or split-K."""
    dt, nb, bs, hkv, d, S, hq, mb, (po, pq, pk, pv, pbt, pcl) = _decode_common(out, q, k_cache, v_cache, block_tables,
                                                                             context_lens)
    wp, wb = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    st = load().pa_decode(po, pq, pk, pv, pbt, mb, pcl, int(max_context_len), S, hq, hkv, d, bs, nb, float(scale), dt,
                          wp, wb, _stream(stream, q.device))
    _check(st, "pa_decode")


def pa_decode_write(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
                    key, value, slot_mapping, workspace=None, stream=None) -> None:
    """One decode step: key / value [S, Hkv, D] (sequence s's new token) into the caches at
    slot_mapping [S] (int64, -1 skips; otherwise the slot of token context_lens[s] - 1), then the
    decode as pa_decode, over contexts that include those rows."""
    torch = _torch()
    dt, nb, bs, hkv, d, S, hq, mb, (po, pq, pk, pv, pbt, pcl) = _decode_common(out, q, k_cache, v_cache, block_tables,
                                                                             context_lens)
    if tuple(key.shape) != (S, hkv, d) or tuple(value.shape) != (S, hkv, d):
        raise ValueError("key / value must be [num_seqs, n_kv_heads, head_dim]")
    if tuple(slot_mapping.shape) != (S,):
        raise ValueError("slot_mapping must hold one slot per sequence")
    wp, wb = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    st = load().pa_decode_write(po, pq, pk, pv, pbt, mb, pcl, int(max_context_len), S, hq, hkv, d, bs, nb, float(scale),
                                dt, _dev(key, "key", q.dtype), _dev(value, "value", q.dtype),
                                _dev(slot_mapping, "slot_mapping", torch.int64), wp, wb, _stream(stream, q.device))
    _check(st, "pa_decode_write")


def pa_decode_v1(out, q, k_cache, v_cache, block_tables, context_lens, scale: float, stream=None) -> None:
    """One-pass decode: one CTA per (sequence, KV head) over the whole context."""
    dt, nb, bs, hkv, d, S, hq, mb, (po, pq, pk, pv, pbt, pcl) = _decode_common(out, q, k_cache, v_cache, block_tables,
                                                                             context_lens)
    st = load().pa_decode_v1(po, pq, pk, pv, pbt, mb, pcl, S, hq, hkv, d, bs, nb, float(scale), dt,
                             _stream(stream, q.device))
    _check(st, "pa_decode_v1")


def pa_decode_splitk(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
                     workspace, partition_tokens: int = 0, stream=None) -> None:
    """Split-K decode over partition_tokens-token pieces plus the merge kernel."""
    dt, nb, bs, hkv, d, S, hq, mb, (po, pq, pk, pv, pbt, pcl) = _decode_common(out, q, k_cache, v_cache, block_tables,
                                                                             context_lens)
    wp, wb = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    st = load().pa_decode_splitk(po, pq, pk, pv, pbt, mb, pcl, int(max_context_len), S, hq, hkv, d, bs, nb,
                                 float(scale), dt, int(partition_tokens), wp, wb, _stream(stream, q.device))
    _check(st, "pa_decode_splitk")


def pa_decode_splitk_static(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                            scale: float, partition_tokens: int = 0, stream=None) -> None:
    """Split-K decode for callers that cannot allocate device memory: the partials live in a
    fixed STATIC_SCRATCH_BYTES array inside the library (shared by all calls, so calls that
    overlap on the GPU race).  Raises PagedAttnError(PA_ERR_WORKSPACE) when the sizes need
    more than that."""
    dt, nb, bs, hkv, d, S, hq, mb, (po, pq, pk, pv, pbt, pcl) = _decode_common(out, q, k_cache, v_cache, block_tables,
                                                                             context_lens)
    st = load().pa_decode_splitk_static(po, pq, pk, pv, pbt, mb, pcl, int(max_context_len), S, hq, hkv, d, bs, nb,
                                        float(scale), dt, int(partition_tokens), _stream(stream, q.device))
    _check(st, "pa_decode_splitk_static")


def pa_decode_shared_prefix_workspace_size(num_seqs: int, n_q_heads: int, head_dim: int, max_context_len: int,
                                           prefix_tokens: int) -> int:
    return int(load().pa_decode_shared_prefix_workspace_size(num_seqs, n_q_heads, head_dim, max_context_len,
                                                             prefix_tokens))


def pa_decode_shared_prefix(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
                            prefix_tokens: int, workspace, prefix_piece_tokens: int = 0, stream=None) -> None:
    """Decode for sequences whose first prefix_tokens tokens are the same cache blocks: the prefix
    part once per KV head on the tensor cores, the rest per sequence, merged."""
    dt, nb, bs, hkv, d, S, hq, mb, (po, pq, pk, pv, pbt, pcl) = _decode_common(out, q, k_cache, v_cache, block_tables,
                                                                             context_lens)
    wp, wb = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    st = load().pa_decode_shared_prefix(po, pq, pk, pv, pbt, mb, pcl, int(max_context_len), S, hq, hkv, d, bs, nb,
                                        float(scale), dt, int(prefix_tokens), int(prefix_piece_tokens), wp, wb,
                                        _stream(stream, q.device))
    _check(st, "pa_decode_shared_prefix")


def pa_prefill_chunk(out, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens, max_q_len: int, scale: float,
                     stream=None, small_m: bool = False) -> None:
    """Prefill chunks (bottom-right causal over their cached context) on the tcgen05 tensor cores;
    small_m=True calls pa_prefill_chunk_small_m (M = 64 tiles for units of at most 64 rows)."""
    torch = _torch()
    dt = _dtype_code(q)
    nb, bs, hkv, d = _cache_dims(k_cache)
    T, hq, d2 = (int(x) for x in q.shape)
    if d2 != d or tuple(out.shape) != tuple(q.shape):
        raise ValueError("q/out/cache head_dim mismatch")
    C = int(seq_lens.shape[0])
    fn = load().pa_prefill_chunk_small_m if small_m else load().pa_prefill_chunk
    st = fn(_dev(out, "out", q.dtype), _dev(q, "q", q.dtype), _dev(k_cache, "k_cache", q.dtype),
            _dev(v_cache, "v_cache", q.dtype), _dev(block_tables, "block_tables", torch.int32),
            int(block_tables.shape[1]), _dev(query_start_loc, "query_start_loc", torch.int32),
            _dev(seq_lens, "seq_lens", torch.int32), C, int(max_q_len), hq, hkv, d, bs, nb,
            float(scale), dt, _stream(stream, q.device))
    _check(st, "pa_prefill_chunk_small_m" if small_m else "pa_prefill_chunk")


# The calls below run for microseconds on the GPU, so their checks are one pass over the tensors.


def _device(t) -> int:
    """Index of the device a call runs on: t's, which has to be the current one (the library launches there)."""
    at = t.get_device()
    if at < 0:
        raise ValueError("every tensor must be a CUDA tensor")
    dev = _torch().cuda.current_device()
    if at != dev:
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")
    return dev


def _refuse(t, name: str, dtype, shape, dev, what: str):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} like the other tensors, got {t.device}")
    raise ValueError(f"{name} must be {what}")


def _dims(t, name: str, shape: str, n: int):
    """t's sizes, n of them (shape: what the message calls them)."""
    dims = t.shape
    if len(dims) != n:
        raise ValueError(f"{name} must be {shape}, got {list(dims)}")
    return dims


def _rows(t, name: str, dtype, shape, dev):
    """Pointer and token stride (elements) of t [N, heads, dim], whose heads and columns are contiguous."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev, "")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        _refuse(t, name, dtype, shape, dev, "contiguous within a token")
    return t.data_ptr(), (s0 if n > 1 else h * d)


def _flat(t, name: str, dtype, shape, dev):
    """Pointer of a contiguous tensor of this type and shape."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, shape, dev, "contiguous")
    return t.data_ptr()


def _ptr(t, name: str, dtype, dev):
    """Pointer of a contiguous tensor of this type, whose own sizes the call takes."""
    if t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, t.shape, dev, "contiguous")
    return t.data_ptr()


def _raw_stream(stream, dev: int) -> int:
    """cudaStream_t of the given stream, or of the device's current one."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(dev)
    return _stream(stream, dev)


def pa_norm_rope_reshape_and_cache(q, key, value, q_weight, k_weight, k_cache, v_cache, slot_mapping, positions,
                                   cos_sin, eps: float = 1e-6, q_out=None, stream=None) -> None:
    """RMS norm of every head of q [N, Hq, D] (weight q_weight [D]) and key [N, Hkv, D] (k_weight),
    rotation by positions [N] (int64) with the cos_sin table [max_position, D] (float32), key and
    value into the caches at slot_mapping [N] (int64, -1 skips), q into q_out (default: in place).
    q, key, value and q_out may be slices of wider rows (contiguous within a token)."""
    torch = _torch()
    ty, dt = q.dtype, _dtype_code(q)
    nb, bs, hkv, d = _dims(k_cache, "k_cache", "[num_blocks, block_size, Hkv, D]", 4)
    n, hq, _ = _dims(q, "q", "[N, Hq, D]", 3)
    mp, _ = _dims(cos_sin, "cos_sin", "[max_position, D]", 2)
    dev = _device(q)
    qp, qs = _rows(q, "q", ty, (n, hq, d), dev)
    op, os_ = (qp, qs) if q_out is None else _rows(q_out, "q_out", ty, (n, hq, d), dev)
    kp, ks = _rows(key, "key", ty, (n, hkv, d), dev)
    vp, vs = _rows(value, "value", ty, (n, hkv, d), dev)
    _check(load().pa_norm_rope_reshape_and_cache(
        op, os_, qp, qs, kp, ks, vp, vs, _flat(q_weight, "q_weight", ty, (d,), dev),
        _flat(k_weight, "k_weight", ty, (d,), dev), float(eps), _flat(k_cache, "k_cache", ty, (nb, bs, hkv, d), dev),
        _flat(v_cache, "v_cache", ty, (nb, bs, hkv, d), dev), _flat(slot_mapping, "slot_mapping", torch.int64, (n,), dev),
        _flat(positions, "positions", torch.int64, (n,), dev), _flat(cos_sin, "cos_sin", torch.float32, (mp, d), dev),
        n, hq, hkv, d, bs, nb, mp, dt, _raw_stream(stream, dev)), "pa_norm_rope_reshape_and_cache")


LATENT_ROPE_DIM = 64


def _latent_dims(latent_cache):
    if latent_cache.dim() != 3 or int(latent_cache.shape[2]) <= LATENT_ROPE_DIM:
        raise ValueError("latent_cache must be [num_blocks, block_size, latent_dim + 64]")
    nb, bs, row = (int(x) for x in latent_cache.shape)
    return nb, bs, row - LATENT_ROPE_DIM


def pa_latent_rope_and_cache(kv, latent_cache, slot_mapping, positions, cos_sin, weight=None, eps: float = 1e-6,
                             q_pe=None, q=None, interleaved: bool = False, stream=None) -> None:
    """New tokens' rows of a paged latent cache [NB, bs, DL + 64]: kv [N, DL + 64] (rows may be strided),
    its first DL columns RMS-normalised with weight [DL] (None: unchanged), its last 64 rotated by
    positions [N] with the cos_sin table [max_position, 64], at slot_mapping [N] (-1 skips).  q_pe
    [N, H, 64] (strided rows, a token's heads before the next token's), if given, is rotated into the last 64 columns of
    q [N, H, DL + 64]; it may be that slice of q."""
    torch = _torch()
    ty, dt = kv.dtype, _dtype_code(kv)
    nb, bs, dl = _latent_dims(latent_cache)
    n, _ = _dims(kv, "kv", "[N, latent_dim + 64]", 2)
    mp, _ = _dims(cos_sin, "cos_sin", "[max_position, 64]", 2)
    row = dl + LATENT_ROPE_DIM
    if (q_pe is None) != (q is None):
        raise ValueError("q_pe and q come together")
    if q_pe is not None:
        _dims(q_pe, "q_pe", "[N, H, 64]", 3)
    dev = _device(kv)
    if kv.shape != (n, row) or kv.stride(1) != 1:
        raise ValueError("kv must be [N, latent_dim + 64] with contiguous rows")
    qp = pep = None
    h = pts = phs = 0
    if q_pe is not None:
        h = q_pe.shape[1]
        pts, phs, one = q_pe.stride()
        if q_pe.dtype != ty or q_pe.shape != (n, h, LATENT_ROPE_DIM) or one != 1 or q_pe.get_device() != dev:
            _refuse(q_pe, "q_pe", ty, (n, h, LATENT_ROPE_DIM), dev, "contiguous in its columns")
        qp, pep = _flat(q, "q", ty, (n, h, row), dev), q_pe.data_ptr()
        if h == 1:
            phs = LATENT_ROPE_DIM
        if n == 1:
            pts = (h - 1) * phs + LATENT_ROPE_DIM
    _check(load().pa_latent_rope_and_cache(
        qp, pep, pts, phs, kv.data_ptr(), kv.stride(0) if n > 1 else row,
        None if weight is None else _flat(weight, "weight", ty, (dl,), dev), float(eps),
        _flat(latent_cache, "latent_cache", ty, (nb, bs, row), dev),
        _flat(slot_mapping, "slot_mapping", torch.int64, (n,), dev), _flat(positions, "positions", torch.int64, (n,), dev),
        _flat(cos_sin, "cos_sin", torch.float32, (mp, LATENT_ROPE_DIM), dev), n, h, dl, LATENT_ROPE_DIM, bs, nb, mp,
        1 if interleaved else 0, dt, _raw_stream(stream, dev)), "pa_latent_rope_and_cache")


def pa_latent_workspace_size(n_heads: int, latent_dim: int, max_q_len: int = 1) -> int:
    return int(load().pa_latent_workspace_size(n_heads, latent_dim, max_q_len))


def _latent_common(out, q, latent_cache, block_tables, lens, workspace):
    torch = _torch()
    ty, dt = q.dtype, _dtype_code(q)
    nb, bs, dl = _latent_dims(latent_cache)
    rows, h, k = _dims(q, "q", "[rows, H, latent_dim + 64]", 3)
    if k != dl + LATENT_ROPE_DIM:
        raise ValueError("q must be [rows, H, latent_dim + 64]")
    n, mb = _dims(block_tables, "block_tables", "[sequences, max_blocks]", 2)
    dev = _device(q)
    wp = wb = 0
    if workspace is not None:
        wp, wb = _flat(workspace, "workspace", workspace.dtype, workspace.shape, dev), workspace.nbytes
    return ((_flat(out, "out", ty, (rows, h, dl), dev), _flat(q, "q", ty, (rows, h, k), dev),
             _flat(latent_cache, "latent_cache", ty, (nb, bs, k), dev),
             _flat(block_tables, "block_tables", torch.int32, (n, mb), dev), mb),
            _flat(lens, "lengths", torch.int32, (n,), dev), rows, n, (h, dl, LATENT_ROPE_DIM, bs, nb), dt, wp, wb, dev)


def pa_latent_decode(out, q, latent_cache, block_tables, context_lens, scale: float, workspace, stream=None) -> None:
    """Decode over a paged latent cache: out [S, H, DL], q [S, H, DL + 64]; workspace of at least
    pa_latent_workspace_size(H, DL) bytes."""
    args, lp, rows, n, dims, dt, wp, wb, dev = _latent_common(out, q, latent_cache, block_tables, context_lens, workspace)
    if n != rows:
        raise ValueError("block_tables and context_lens must hold one row per row of q")
    _check(load().pa_latent_decode(*args, lp, rows, *dims, float(scale), dt, wp, wb, _raw_stream(stream, dev)),
           "pa_latent_decode")


def pa_latent_prefill_chunk(out, q, latent_cache, block_tables, query_start_loc, seq_lens, max_q_len: int, scale: float,
                            workspace, stream=None) -> None:
    """Ragged chunks (bottom-right causal over their cached context) on a paged latent cache: out
    [T, H, DL], q [T, H, DL + 64], chunk c the rows query_start_loc[c] .. query_start_loc[c + 1];
    workspace of at least pa_latent_workspace_size(H, DL, max_q_len) bytes."""
    args, lp, rows, n, dims, dt, wp, wb, dev = _latent_common(out, q, latent_cache, block_tables, seq_lens, workspace)
    loc = _flat(query_start_loc, "query_start_loc", _torch().int32, (n + 1,), dev)
    _check(load().pa_latent_prefill_chunk(*args, loc, lp, n, int(max_q_len), rows, *dims, float(scale), dt, wp, wb,
                                          _raw_stream(stream, dev)), "pa_latent_prefill_chunk")


def tree_mask(parents, mask_words: int = 0):
    """(mask, depth) of a tree of drafted tokens as host numpy arrays: mask [n, words] int64 with the bits of each
    token and its ancestors (words: at least mask_words and enough for n), depth [n] int32.  parents[j] < j, or -1
    for a token that continues the context."""
    import numpy as np
    up = np.ascontiguousarray(parents, dtype=np.int32)
    if up.ndim != 1:
        raise ValueError(f"parents must be [num_tokens], got {list(up.shape)}")
    n = up.shape[0]
    words = max(int(mask_words), -(-n // 64))
    mask, depth = np.zeros((n, words), dtype=np.int64), np.zeros(n, dtype=np.int32)
    _check(load().pa_tree_mask(mask.ctypes.data, depth.ctypes.data, up.ctypes.data, n, words), "pa_tree_mask")
    return mask, depth


def pa_tree_workspace_size(n_q_heads: int, n_kv_heads: int, head_dim: int, max_q_len: int) -> int:
    return int(load().pa_tree_workspace_size(n_q_heads, n_kv_heads, head_dim, max_q_len))


def pa_tree_decode(out, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens, tree_mask, max_q_len: int, scale: float,
                   workspace, stream=None) -> None:
    """Attention of trees of drafted tokens over the paged cache: out, q [T, Hq, D], sequence s the rows
    query_start_loc[s] .. query_start_loc[s + 1], seq_lens [S] with the drafted tokens, tree_mask [T, words] int64 (bit k
    of a row: it sees the k-th drafted token); workspace of at least pa_tree_workspace_size(Hq, Hkv, D, max_q_len) bytes."""
    torch = _torch()
    ty, dt, i32 = q.dtype, _dtype_code(q), torch.int32
    cache = _dims(k_cache, "k_cache", "[num_blocks, block_size, Hkv, D]", 4)
    nb, bs, hkv, d = cache
    rows, hq, _ = _dims(q, "q", "[T, Hq, D]", 3)
    n, mb = _dims(block_tables, "block_tables", "[sequences, max_blocks]", 2)
    _, words = _dims(tree_mask, "tree_mask", "[T, words]", 2)
    dev = _device(q)
    wp, wb = _workspace(workspace, dev)
    _check(load().pa_tree_decode(
        _flat(out, "out", ty, (rows, hq, d), dev), _flat(q, "q", ty, (rows, hq, d), dev),
        _ptr(k_cache, "k_cache", ty, dev), _flat(v_cache, "v_cache", ty, cache, dev),
        _ptr(block_tables, "block_tables", i32, dev), mb,
        _flat(query_start_loc, "query_start_loc", i32, (n + 1,), dev), _flat(seq_lens, "seq_lens", i32, (n,), dev),
        _flat(tree_mask, "tree_mask", torch.int64, (rows, words), dev), words, n, int(max_q_len), rows, hq, hkv, d, bs, nb,
        float(scale), dt, wp, wb, _raw_stream(stream, dev)), "pa_tree_decode")


def _workspace(workspace, dev):
    if workspace is None:
        return 0, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(workspace, "workspace", workspace.dtype, workspace.shape, dev, "contiguous")
    return workspace.data_ptr(), workspace.nbytes


def _planes(k_cache, v_cache):
    """(k pointer, v pointer, layers, row bytes, block_size, num_blocks, device) of caches [NB, bs, Hkv, D] or, of all
    layers, [L, NB, bs, Hkv, D]; v_cache None: of one array a layer, [NB, bs, row] or [L, NB, bs, row]."""
    inner = 2 if v_cache is not None else 1
    shape = k_cache.shape
    if len(shape) not in (2 + inner, 3 + inner):
        raise ValueError("k_cache must be " + ("[num_blocks, block_size, Hkv, D]" if inner == 2 else "[num_blocks, block_size, row]")
                         + f" (layers before it where there are several), got {list(shape)}")
    _dtype_code(k_cache)
    dev = _device(k_cache)
    layers = shape[0] if len(shape) == 3 + inner else 1
    nb, bs = shape[-2 - inner], shape[-1 - inner]
    row = shape[-1] * (shape[-2] if inner == 2 else 1) * 2
    if not k_cache.is_contiguous():
        _refuse(k_cache, "k_cache", k_cache.dtype, shape, dev, "contiguous")
    vp = None if v_cache is None else _flat(v_cache, "v_cache", k_cache.dtype, shape, dev)
    return k_cache.data_ptr(), vp, layers, row, bs, nb, dev


def pa_tree_commit(k_cache, v_cache, block_tables, query_start_loc, seq_lens, path, num_accepted, new_lens, stream=None) -> None:
    """The accepted drafted tokens' rows moved to the front: row ctx + path[s][i] of every layer to ctx + i for i <
    num_accepted[s] (path [S, P] int32, rising), new_lens [S] = ctx + num_accepted.  Caches [NB, bs, Hkv, D] or, of all
    layers, [L, NB, bs, Hkv, D]; v_cache None with k_cache a latent cache [NB, bs, row] or [L, NB, bs, row]."""
    i32 = _torch().int32
    kp, vp, layers, row, bs, nb, dev = _planes(k_cache, v_cache)
    n, mb = _dims(block_tables, "block_tables", "[sequences, max_blocks]", 2)
    _, most = _dims(path, "path", "[sequences, max_path]", 2)
    _check(load().pa_tree_commit(
        kp, vp, layers, _ptr(block_tables, "block_tables", i32, dev), mb,
        _flat(query_start_loc, "query_start_loc", i32, (n + 1,), dev), _flat(seq_lens, "seq_lens", i32, (n,), dev),
        _flat(path, "path", i32, (n, most), dev), most, _flat(num_accepted, "num_accepted", i32, (n,), dev),
        _flat(new_lens, "new_lens", i32, (n,), dev), n, row, bs, nb, _raw_stream(stream, dev)), "pa_tree_commit")


def pa_copy_pages(k_cache, v_cache, pairs, stream=None) -> None:
    """Page pairs[i][0] copied to page pairs[i][1] (int32 [N, 2]; -1 skips) in all layers of the caches (as
    pa_tree_commit)."""
    kp, vp, layers, row, bs, nb, dev = _planes(k_cache, v_cache)
    n, _ = _dims(pairs, "pairs", "[N, 2]", 2)
    _check(load().pa_copy_pages(kp, vp, layers, _flat(pairs, "pairs", _torch().int32, (n, 2), dev), n, row, bs, nb,
                                _raw_stream(stream, dev)), "pa_copy_pages")


def pa_fork_pages(block_tables, seq_lens, parents, ref_counts, block_size: int, stream=None) -> None:
    """Empty sequences s with parents[s] >= 0 become forks of them: the same pages (counts + 1) and length."""
    i32 = _torch().int32
    n, mb = _dims(block_tables, "block_tables", "[sequences, max_blocks]", 2)
    nb, = _dims(ref_counts, "ref_counts", "[num_blocks]", 1)
    dev = _device(block_tables)
    _check(load().pa_fork_pages(
        _ptr(block_tables, "block_tables", i32, dev), mb, _flat(seq_lens, "seq_lens", i32, (n,), dev),
        _flat(parents, "parents", i32, (n,), dev), n, _ptr(ref_counts, "ref_counts", i32, dev), int(block_size), nb,
        _raw_stream(stream, dev)), "pa_fork_pages")


def pa_resize_workspace_size(num_seqs: int, num_blocks: int) -> int:
    return int(load().pa_resize_workspace_size(num_seqs, num_blocks))


def pa_resize_pages(k_cache, v_cache, block_tables, seq_lens, new_lens, ref_counts, free_list, free_count, workspace,
                    stream=None) -> None:
    """Sequences to new_lens [S] (-1: unchanged; seq_lens is updated): pages from and back to the free list, a shared
    last page copied before it is written.  Caches as pa_tree_commit; ref_counts and free_list [NB], free_count [1],
    all int32; workspace of at least pa_resize_workspace_size(S, NB) bytes."""
    i32 = _torch().int32
    kp, vp, layers, row, bs, nb, dev = _planes(k_cache, v_cache)
    n, mb = _dims(block_tables, "block_tables", "[sequences, max_blocks]", 2)
    wp, wb = _workspace(workspace, dev)
    _check(load().pa_resize_pages(
        kp, vp, layers, _ptr(block_tables, "block_tables", i32, dev), mb, _flat(seq_lens, "seq_lens", i32, (n,), dev),
        _flat(new_lens, "new_lens", i32, (n,), dev), n, _flat(ref_counts, "ref_counts", i32, (nb,), dev),
        _flat(free_list, "free_list", i32, (nb,), dev), _flat(free_count, "free_count", i32, (1,), dev), row, bs, nb, wp, wb,
        _raw_stream(stream, dev)), "pa_resize_pages")


def pa_device_errors(clear: bool = True) -> int:
    """PA_DEVERR_* bits recorded by the kernels on the current device (synchronises)."""
    r = load().pa_device_errors(1 if clear else 0)
    if r < 0:
        raise PagedAttnError(r, "pa_device_errors")
    return r


def version() -> int:
    return int(load().pa_version())
