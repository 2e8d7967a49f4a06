"""Packed variable-length GQA attention for GB300 (sm_103a).

A thin ctypes binding over ``libpva.so`` (declared in ``include/pva.h``):
the functions below only marshal arguments -- every step of the computation
runs in the library's CUDA kernels.  There is no CPU fallback: if the
compiled library is missing, every call raises.

PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading

import torch

from . import workloads  # noqa: F401  (seeded synthetic inputs)

__all__ = ["pva_forward", "pva_forward_local", "pva_forward_padded", "pva_gqa_kvcache",
           "pva_block_tables", "pva_rope_axes", "pva_norm_rope", "pva_norm_rope_backward", "pva_gqa_tree",
           "pva_gqa_prefix", "pva_kvcache_accept", "pva_kvcache_weights", "pva_kvcache_evict",
           "pva_get_status", "pva_schedule", "pva_status_string", "pva_last_error",
           "pva_release", "pva_version", "pva_profile", "pva_kernel_times", "pva_selftest_wait",
           "pva_selftest_give_up",
           "load_library", "build", "PvaError", "DTYPE_CODES", "DEV_FLAGS"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpva.so")

PVA_OK, PVA_ERR_INVALID_ARG, PVA_ERR_UNSUPPORTED, PVA_ERR_CUDA, PVA_ERR_OOM = 0, -1, -2, -3, -4
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}
DEV_FLAGS = {"cu_q_start": 0x1, "cu_kv_start": 0x2, "cu_q_order": 0x4, "cu_kv_order": 0x8,
             "too_many": 0x10, "null_tensor": 0x20, "kv_len": 0x40, "kv_cache": 0x80,
             "wait_timeout": 0x100, "tree": 0x200, "blocks": 0x400, "rope": 0x800,
             "prefix": 0x1000}

_lock = threading.Lock()
_lib = None


class PvaError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"pva error {code}: {message}")
        self.code = code


def build(force: bool = False) -> str:
    """Compile libpva.so in-tree (nvcc, sm_103a)."""
    from ._build import build as _b
    return _b(force=force)


def load_library(path: str | None = None):
    """Load libpva.so and declare its C signatures.  Raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise PvaError(PVA_ERR_CUDA, f"{p} not found: build it with "
                           "`python -m gqa_attention_cu_gb300._build`")
        lib = ctypes.CDLL(p)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.pva_forward.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i, vp]
        lib.pva_forward.restype = i
        lib.pva_forward_local.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i, i,
                                          vp]
        lib.pva_forward_from_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i,
                                              i, i, f, i, f, i, i, vp]
        lib.pva_forward_from_host.restype = i
        lib.pva_forward_local.restype = i
        lib.pva_forward_padded.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, f, i,
                                           vp]
        lib.pva_forward_padded.restype = i
        lib.pva_gqa_kvcache.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                        i, i, i, i, i, f, f, i, i, vp]
        lib.pva_gqa_kvcache.restype = i
        i64 = ctypes.c_int64
        lib.pva_block_tables.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i64, vp]
        lib.pva_block_tables.restype = i
        lib.pva_rope_axes.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i64, i64, i64, i64,
                                      i, i, i, i, vp, i, i, i, vp, i64, vp, vp, vp, i, i, i, vp]
        lib.pva_rope_axes.restype = i
        lib.pva_norm_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i64, i64, i64,
                                      i64, f, f, i, i, i, i, i, vp, i, i, vp, i64, vp, vp, vp, i, i,
                                      i, vp]
        lib.pva_norm_rope.restype = i
        lib.pva_norm_rope_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i,
                                               i, i, i64, i64, i64, i64, i64, i64, f, f, i, i, i, i, i,
                                               vp, i, i, i, vp]
        lib.pva_norm_rope_backward.restype = i
        lib.pva_gqa_tree.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i,
                                     i, i, i, i, i, i, i, i, vp, i, i, f, f, i, i, vp]
        lib.pva_gqa_tree.restype = i
        lib.pva_kvcache_accept.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i64, i, i, i, i, i,
                                           i, vp]
        lib.pva_kvcache_accept.restype = i
        lib.pva_gqa_prefix.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i,
                                       i, f, f, i, vp]
        lib.pva_gqa_prefix.restype = i
        lib.pva_kvcache_weights.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f,
                                            f, f, i, vp]
        lib.pva_kvcache_weights.restype = i
        lib.pva_kvcache_evict.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i64, i,
                                          i, i, i64, i, i, i, i, i, i, i, i, i, vp]
        lib.pva_kvcache_evict.restype = i
        lib.pva_get_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.pva_get_status.restype = i
        lib.pva_schedule.argtypes = [vp, vp, i, i, i, i, i, i, i,
                                     ctypes.POINTER(ctypes.c_int32), ctypes.c_size_t, vp]
        lib.pva_schedule.restype = i
        lib.pva_status_string.argtypes = [i]
        lib.pva_status_string.restype = ctypes.c_char_p
        lib.pva_last_error.argtypes = []
        lib.pva_last_error.restype = ctypes.c_char_p
        lib.pva_release.argtypes = []
        lib.pva_release.restype = None
        lib.pva_version.argtypes = []
        lib.pva_version.restype = i
        lib.pva_profile.argtypes = [i]
        lib.pva_profile.restype = i
        lib.pva_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_float), i]
        lib.pva_kernel_times.restype = i
        lib.pva_selftest_wait.argtypes = [ctypes.c_uint32, vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.pva_selftest_wait.restype = i
        lib.pva_selftest_give_up.argtypes = [ctypes.c_uint32]
        lib.pva_selftest_give_up.restype = i
        lib.pva_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i,
                                            vp, vp]
        lib.pva_forward_noalloc.restype = i
        if path is None:
            _lib = lib
        return lib


def _check(rc: int):
    if rc != PVA_OK:
        lib = load_library()
        raise PvaError(rc, f"{lib.pva_status_string(rc).decode()}: {lib.pva_last_error().decode()}")


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t) -> int:
    import torch
    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if t.dtype not in codes:
        raise PvaError(PVA_ERR_INVALID_ARG, f"dtype {t.dtype} not supported (f32, f16, bf16)")
    return codes[t.dtype]


def pva_forward(q, k, v, cu_seqlens_q, cu_seqlens_kv, out, B: int, num_heads: int,
                kv_num_heads: int, head_size: int, v_head_size: int, scale: float = 0.0,
                is_causal: int = 0, softcap: float = 0.0, dtype: int | None = None,
                stream=None) -> None:
    """Enqueue out = attention(q, k, v) on ``stream`` (torch stream, raw
    cudaStream_t int, or None for the current stream).  Tensors are CUDA
    tensors; their data pointers are passed as they are (contiguous layouts
    as in include/pva.h)."""
    lib = load_library()
    code = _dtype_code(q) if dtype is None else int(dtype)
    rc = lib.pva_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(),
                         cu_seqlens_kv.data_ptr(), out.data_ptr(), int(B), int(num_heads),
                         int(kv_num_heads), int(head_size), int(v_head_size), float(scale),
                         int(is_causal), float(softcap), code, _stream_ptr(stream))
    _check(rc)


def pva_forward_from_host(q_host, k_host, v_host, cu_seqlens_q_host, cu_seqlens_kv_host,
                          out_host, q_dev, k_dev, v_dev, out_dev, cu_dev, B: int,
                          num_heads: int, kv_num_heads: int, head_size: int, v_head_size: int,
                          scale: float = 0.0, is_causal: int = 0, softcap: float = 0.0,
                          chunks: int = 0, dtype: int | None = None, stream=None) -> None:
    """pva_forward on a batch in host memory (the *_host tensors, pinned for
    overlap; the offsets are host int32 tensors): the call copies it into the
    caller's device buffers (*_dev, cu_dev of >= 4 B + 34 int32) chunk by
    chunk, overlapping the copies with the attention, and copies the output
    back into out_host; ``stream`` completes after the last copy."""
    lib = load_library()
    code = _dtype_code(q_host) if dtype is None else int(dtype)
    rc = lib.pva_forward_from_host(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(),
                                   cu_seqlens_q_host.data_ptr(), cu_seqlens_kv_host.data_ptr(),
                                   out_host.data_ptr(), q_dev.data_ptr(), k_dev.data_ptr(),
                                   v_dev.data_ptr(), out_dev.data_ptr(), cu_dev.data_ptr(),
                                   int(B), int(num_heads), int(kv_num_heads), int(head_size),
                                   int(v_head_size), float(scale), int(is_causal),
                                   float(softcap), code, int(chunks), _stream_ptr(stream))
    _check(rc)


def pva_forward_local(q, k, v, cu_seqlens_q, cu_seqlens_kv, out, B: int, num_heads: int,
                      kv_num_heads: int, head_size: int, v_head_size: int, scale: float = 0.0,
                      is_causal: int = 0, softcap: float = 0.0, local_window: int = 0,
                      dtype: int | None = None, stream=None) -> None:
    """pva_forward with a local window: with local_window = W > 0 each query
    row also ignores keys before (its causal limit + 1 - W)."""
    lib = load_library()
    code = _dtype_code(q) if dtype is None else int(dtype)
    rc = lib.pva_forward_local(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                               cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(), out.data_ptr(),
                               int(B), int(num_heads), int(kv_num_heads), int(head_size),
                               int(v_head_size), float(scale), int(is_causal), float(softcap),
                               int(local_window), code, _stream_ptr(stream))
    _check(rc)


def pva_forward_padded(q, k, v, nonpad_kv_seqlen, out, B: int, q_seq: int, kv_seq: int,
                       num_heads: int, kv_num_heads: int, head_size: int, v_head_size: int,
                       scale: float = 0.0, is_causal: int = 0, softcap: float = 0.0,
                       dtype: int | None = None, stream=None) -> None:
    """The padded form: q [B, q_seq, H, d], k/v [B, kv_seq, Hkv, d/dv], out
    [B, q_seq, H, dv]; batch entry b's keys are the first
    ``nonpad_kv_seqlen[b]`` (CUDA int64 [B]) rows of its slot, and the causal
    limit of query row i is i + nonpad_kv_seqlen[b] - q_seq."""
    lib = load_library()
    code = _dtype_code(q) if dtype is None else int(dtype)
    rc = lib.pva_forward_padded(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                nonpad_kv_seqlen.data_ptr(), out.data_ptr(), int(B), int(q_seq),
                                int(kv_seq), int(num_heads), int(kv_num_heads), int(head_size),
                                int(v_head_size), float(scale), int(is_causal), float(softcap),
                                code, _stream_ptr(stream))
    _check(rc)


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


def pva_gqa_kvcache(q, k_new, v_new, k_cache, v_cache, seqlens_k, out, num_heads: int,
                    kv_num_heads: int, cos_cache=None, sin_cache=None, position_ids=None,
                    rotary_interleaved: bool = False, scale: float = 0.0, softcap: float = 0.0,
                    local_window: int = 0, dtype: int | None = None, stream=None) -> None:
    """One GroupQueryAttention step on a fixed-capacity BNSH cache: q
    [B, q_seq, H, d], k_new/v_new [B, k_seq, Hkv, d] (or None), caches
    [B, Hkv, capacity, d] (appended in place), seqlens_k int32 [B] (= keys
    after the step - 1), optional cos/sin tables [rows, rotary_dim/2] and
    position_ids int64 [B, q_seq]; out [B, q_seq, H, d]."""
    lib = load_library()
    code = _dtype_code(q) if dtype is None else int(dtype)
    B, q_seq, _, d = q.shape
    k_seq = 0 if k_new is None else int(k_new.shape[1])
    capacity = int(k_cache.shape[2])
    rot = rows = 0
    rot_code = 0
    if cos_cache is not None:
        rows, rot = int(cos_cache.shape[0]), 2 * int(cos_cache.shape[1])
        rot_code = _dtype_code(cos_cache)
    rc = lib.pva_gqa_kvcache(q.data_ptr(), _ptr_or_none(k_new), _ptr_or_none(v_new),
                             k_cache.data_ptr(), v_cache.data_ptr(), seqlens_k.data_ptr(),
                             _ptr_or_none(cos_cache), _ptr_or_none(sin_cache),
                             _ptr_or_none(position_ids), out.data_ptr(), int(B), int(q_seq),
                             k_seq, capacity, int(num_heads), int(kv_num_heads), int(d), rot,
                             rows, int(bool(rotary_interleaved)), rot_code, float(scale),
                             float(softcap), int(local_window), code, _stream_ptr(stream))
    _check(rc)


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise PvaError(PVA_ERR_INVALID_ARG, message)


def _device(first, *others) -> int:
    """Index of the device of ``first``, which has to be the current one if it is
    a GPU.  The ``_plain`` checks compare the other tensors' indices with it; on
    the host, where the index says little, ``others`` are compared in full."""
    at = first.get_device()
    if at < 0:
        for t in others:
            _need(t is None or t.device == first.device, "the tensors are on different devices")
    elif at != torch._C._cuda_getDevice():
        _need(False, f"the tensors are on cuda:{at}, which is not the current device")
    return at


def _stream_on(stream, device: int) -> int:
    """The given stream, or the device's current one (as a number: making a
    stream object costs more than the rest of a small call's checks)."""
    if stream is None:
        _need(device >= 0, "the tensors must be on a GPU")
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream_ptr(stream)


def _plain(t, name: str, dtype, shape, at: int):
    """The address of a contiguous tensor of this type and shape on device ``at``
    (None: none)."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == at):
        return t.data_ptr()
    _need(t.dtype is dtype, f"{name} must be {dtype}")
    _need(t.shape == shape, f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    _need(False, "the tensors are on different devices")


_sections = {}  # C arrays of the section lists met so far, by their numbers


def _rotary(cos_cache, sin_cache, sections, at: int):
    """(cos, sin, rotary_dim, table rows, table type code, host sections or None)."""
    _need(sin_cache is not None, "cos_cache and sin_cache come together")
    shape = cos_cache.shape
    _need(len(shape) == 2, "cos_cache must be [rows, rotary_dim / 2]")
    host = None
    if sections is not None:
        try:
            key = tuple(map(operator.index, sections))
        except TypeError:
            _need(False, "sections must be whole numbers")
        host = _sections.get(key)
        if host is None:
            _need(all(-2**31 <= x < 2**31 for x in key), "a section does not fit in int32")
            host = _sections[key] = (ctypes.c_int32 * len(key))(*key)
    dtype = cos_cache.dtype
    return (_plain(cos_cache, "cos_cache", dtype, shape, at),
            _plain(sin_cache, "sin_cache", dtype, shape, at), 2 * shape[1], shape[0],
            _type_code(cos_cache), host)


_TYPE_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _type_code(t) -> int:
    code = _TYPE_CODES.get(t.dtype)
    return _dtype_code(t) if code is None else code


def pva_block_tables(lens, block_table, held, free_blocks, free_count, page_size: int, cu_new=None,
                     slot_map=None, stream=None) -> None:
    """Give every sequence the blocks its length needs, on the device: lens,
    held int32 [B], block_table int32 [B, max_blocks], free_blocks int32 [pool]
    (a stack of *free_count int32 [1]* blocks).  With ``cu_new`` int32 [B + 1]
    and ``slot_map`` int64 [n], also the cache slot of every new packed token.
    See include/pva.h for the order and the errors (``blocks`` bit)."""
    _need(block_table.dim() == 2, "block_table must be [B, max_blocks]")
    B, width = block_table.shape
    i32 = torch.int32
    _need(free_blocks.dim() == 1, "free_blocks must be [pool]")
    _need((cu_new is None) == (slot_map is None), "cu_new and slot_map come together")
    slots = 0
    if slot_map is not None:
        _need(slot_map.dim() == 1, "slot_map must be [slots]")
        slots = slot_map.shape[0]
    at = _device(block_table, lens, held, free_blocks, free_count, cu_new, slot_map)
    _check((_lib or load_library()).pva_block_tables(
        _plain(lens, "lens", i32, (B,), at),
        _plain(block_table, "block_table", i32, (B, width), at),
        _plain(held, "held", i32, (B,), at),
        _plain(free_blocks, "free_blocks", i32, free_blocks.shape, at),
        _plain(free_count, "free_count", i32, (1,), at),
        _plain(cu_new, "cu_new", i32, (B + 1,), at),
        _plain(slot_map, "slot_map", torch.int64, (slots,), at), B, width, int(page_size),
        free_blocks.shape[0], slots, _stream_on(stream, at)))


def _token_rows(t, name: str, dtype, tokens: int, d: int, at: int):
    """Address, heads and token stride of a [tokens, heads, d] tensor whose tokens
    are each contiguous."""
    shape = t.shape
    if (len(shape) != 3 or t.dtype is not dtype or shape[0] != tokens or shape[2] != d
            or t.get_device() != at):
        _need(False, f"{name} must be [tokens, heads, head_size] of one type and device with the others")
    heads = shape[1]
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and heads > 1):
        _need(False, f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), heads, max(s0, heads * d) if tokens <= 1 else s0


def _positions(position_ids, sections, tokens: int, at: int):
    """Address and axes of position_ids [n_axes, tokens]."""
    _need(position_ids.dim() == 2, "position_ids must be [n_axes, tokens]")
    n_axes = position_ids.shape[0]
    _need(sections is None or len(sections) == n_axes, "sections needs one entry per axis")
    return _plain(position_ids, "position_ids", torch.int64, (n_axes, tokens), at), n_axes


def _cache_write(k, v, k_cache, v_cache, slot_map, dt, tokens: int, Hkv: int, d: int, at: int):
    """(v, its stride, caches, slots, blocks, page) of a write of k and v to the cache."""
    if k_cache is None:
        _need(v is None and v_cache is None and slot_map is None,
              "v, v_cache and slot_map come with k_cache")
        return None, 0, None, None, None, 0, 0
    _need(k is not None and v is not None and v_cache is not None and slot_map is not None,
          "the cache write needs k, v, both caches and slot_map")
    _need(k_cache.dim() == 4, "k_cache must be [n_blocks, kv_heads, page, head_size]")
    blocks, _, page, _ = k_cache.shape
    kc = _plain(k_cache, "k_cache", dt, (blocks, Hkv, page, d), at)
    vc = _plain(v_cache, "v_cache", dt, (blocks, Hkv, page, d), at)
    slots = _plain(slot_map, "slot_map", torch.int64, (tokens,), at)
    _need(v.shape == k.shape, "v must have k's shape")
    pv, _, vs = _token_rows(v, "v", dt, tokens, d, at)
    return pv, vs, kc, vc, slots, blocks, page


def pva_rope_axes(q, k, cos_cache, sin_cache, position_ids, q_out=None, k_out=None, sections=None,
                  rotary_interleaved: bool = False, axes_interleaved: bool = False,
                  inverse: bool = False, v=None, k_cache=None, v_cache=None, slot_map=None,
                  stream=None) -> None:
    """Rotate packed q [tokens, H, d] and/or k [tokens, Hkv, d] (token strides
    allowed) into q_out / k_out by cos/sin tables [rows, rotary_dim/2], with
    position_ids int64 [n_axes, tokens] and ``sections`` naming how many pairs
    turn with each axis.  ``inverse`` is the rotation's gradient.  With v, the
    caches [n_blocks, Hkv, page, d] and slot_map int64 [tokens], rotated keys
    and values are also written to the cache."""
    first = q if q is not None else k
    _need(first is not None, "q or k is needed")
    _need(first.dim() == 3, "q and k must be [tokens, heads, head_size]")
    tokens, _, d = first.shape
    dt = first.dtype
    at = _device(first, q_out, k, k_out, v, cos_cache, sin_cache, position_ids, k_cache, v_cache,
                 slot_map)
    H = Hkv = qs = ks = qos = kos = 0
    pq = pk = pqo = pko = None
    if q is not None:
        pq, H, qs = _token_rows(q, "q", dt, tokens, d, at)
        _need(q_out is not None and q_out.shape == q.shape, "q_out must have q's shape")
        pqo, _, qos = _token_rows(q_out, "q_out", dt, tokens, d, at)
    else:
        _need(q_out is None, "q and q_out come together")
    if k is not None:
        pk, Hkv, ks = _token_rows(k, "k", dt, tokens, d, at)
        if k_out is not None:
            _need(k_out.shape == k.shape, "k_out must have k's shape")
            pko, _, kos = _token_rows(k_out, "k_out", dt, tokens, d, at)
    else:
        _need(k_out is None, "k_out without k")
    pos, n_axes = _positions(position_ids, sections, tokens, at)
    pc, ps, rot, rows, code, host = _rotary(cos_cache, sin_cache, sections, at)
    pv, vs, kc, vc, slots, blocks, page = _cache_write(k, v, k_cache, v_cache, slot_map, dt, tokens, Hkv,
                                                       d, at)
    if tokens == 0:
        return
    _check((_lib or load_library()).pva_rope_axes(
        pq, pk, pqo, pko, pc, ps, pos, tokens, H, Hkv, d, qs, ks, qos, kos, rot, rows,
        1 if rotary_interleaved else 0, n_axes, host, 1 if axes_interleaved else 0,
        1 if inverse else 0, code, pv, vs, kc, vc, slots, blocks, page, _type_code(first),
        _stream_on(stream, at)))


def _norm_weights(q_weight, k_weight, dt, d: int, at: int):
    """(q_weight, k_weight, type code) of the gains [head_size], both of one type."""
    w = q_weight if q_weight is not None else k_weight
    if w is None:
        return None, None, 0
    _need(w.dtype is dt or w.dtype is torch.float32, "the weights must be f32 or of the rows' type")
    return (_plain(q_weight, "q_weight", w.dtype, (d,), at), _plain(k_weight, "k_weight", w.dtype, (d,), at),
            _type_code(w))


def pva_norm_rope(q, k, q_weight, k_weight, q_out=None, k_out=None, cos_cache=None, sin_cache=None,
                  position_ids=None, eps: float = 1e-6, weight_offset: float = 0.0, sections=None,
                  rotary_interleaved: bool = False, axes_interleaved: bool = False, v=None,
                  k_cache=None, v_cache=None, slot_map=None, stream=None) -> None:
    """Norm every head row of packed q [tokens, H, d] and/or k [tokens, Hkv, d] (token
    strides allowed), times ``weight_offset`` + weight [d] (f32 or the rows' type;
    None: gains of one), then rotate as pva_rope_axes does (no tables: norms only),
    into q_out / k_out and, with v, caches and slot_map, the cache."""
    first = q if q is not None else k
    _need(first is not None, "q or k is needed")
    _need(first.dim() == 3, "q and k must be [tokens, heads, head_size]")
    tokens, _, d = first.shape
    dt = first.dtype
    at = _device(first, q_out, k, k_out, q_weight, k_weight, v, cos_cache, sin_cache, position_ids, k_cache,
                 v_cache, slot_map)
    H = Hkv = qs = ks = qos = kos = 0
    pq = pk = pqo = pko = None
    if q is not None:
        pq, H, qs = _token_rows(q, "q", dt, tokens, d, at)
        _need(q_out is not None and q_out.shape == q.shape, "q_out must have q's shape")
        pqo, _, qos = _token_rows(q_out, "q_out", dt, tokens, d, at)
    else:
        _need(q_out is None, "q and q_out come together")
    if k is not None:
        pk, Hkv, ks = _token_rows(k, "k", dt, tokens, d, at)
        if k_out is not None:
            _need(k_out.shape == k.shape, "k_out must have k's shape")
            pko, _, kos = _token_rows(k_out, "k_out", dt, tokens, d, at)
    else:
        _need(k_out is None, "k_out without k")
    wq, wk, w_code = _norm_weights(q_weight, k_weight, dt, d, at)
    turn = _norm_rotary(cos_cache, sin_cache, position_ids, sections, tokens, at)
    pos, n_axes, pc, ps, rot, rows, code, host = turn
    pv, vs, kc, vc, slots, blocks, page = _cache_write(k, v, k_cache, v_cache, slot_map, dt, tokens, Hkv,
                                                       d, at)
    if tokens == 0:
        return
    _check((_lib or load_library()).pva_norm_rope(
        pq, pk, wq, wk, pqo, pko, pc, ps, pos, tokens, H, Hkv, d, qs, ks, qos, kos, float(eps),
        float(weight_offset), w_code, rot, rows, 1 if rotary_interleaved else 0, n_axes, host,
        1 if axes_interleaved else 0, code, pv, vs, kc, vc, slots, blocks, page, _type_code(first),
        _stream_on(stream, at)))


def _norm_rotary(cos_cache, sin_cache, position_ids, sections, tokens: int, at: int):
    """(positions, axes, cos, sin, rotary_dim, rows, table type, sections), or no rotation."""
    if cos_cache is None:
        _need(sin_cache is None and position_ids is None and sections is None,
              "positions and sections need the cos and sin tables")
        return None, 1, None, None, 0, 0, 0, None
    _need(position_ids is not None, "the rotation needs position_ids")
    return _positions(position_ids, sections, tokens, at) + _rotary(cos_cache, sin_cache, sections, at)


def pva_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, dq, dk, dq_weight=None,
                           dk_weight=None, cos_cache=None, sin_cache=None, position_ids=None,
                           eps: float = 1e-6, weight_offset: float = 0.0, sections=None,
                           rotary_interleaved: bool = False, axes_interleaved: bool = False,
                           stream=None) -> None:
    """The gradient of pva_norm_rope: from the gradients dq_out, dk_out of its
    outputs and the rows q, k that it read, dq and dk (which may take the place of
    dq_out and dk_out), and f32 dq_weight, dk_weight [d] where they are given.  One
    side may be None altogether."""
    first = q if q is not None else k
    _need(first is not None, "q or k is needed")
    _need(first.dim() == 3, "q and k must be [tokens, heads, head_size]")
    tokens, _, d = first.shape
    dt = first.dtype
    at = _device(first, dq_out, dk_out, k, dq, dk, q_weight, k_weight, dq_weight, dk_weight, cos_cache,
                 sin_cache, position_ids)

    def side(x, dy, dx, name):
        if x is None:
            _need(dy is None and dx is None, f"{name}, d{name}_out and d{name} come together")
            return None, None, None, 0, 0, 0, 0
        _need(dy is not None and dx is not None, f"{name}, d{name}_out and d{name} come together")
        _need(dy.shape == x.shape and dx.shape == x.shape, f"the gradients of {name} must have its shape")
        px, heads, sx = _token_rows(x, name, dt, tokens, d, at)
        py, _, sy = _token_rows(dy, f"d{name}_out", dt, tokens, d, at)
        pd, _, sd = _token_rows(dx, f"d{name}", dt, tokens, d, at)
        return px, py, pd, heads, sx, sy, sd

    pq, pqo, pdq, H, qs, qos, dqs = side(q, dq_out, dq, "q")
    pk, pko, pdk, Hkv, ks, kos, dks = side(k, dk_out, dk, "k")
    wq, wk, w_code = _norm_weights(q_weight, k_weight, dt, d, at)
    gq = _plain(dq_weight, "dq_weight", torch.float32, (d,), at)
    gk = _plain(dk_weight, "dk_weight", torch.float32, (d,), at)
    pos, n_axes, pc, ps, rot, rows, code, host = _norm_rotary(cos_cache, sin_cache, position_ids, sections,
                                                              tokens, at)
    _check((_lib or load_library()).pva_norm_rope_backward(
        pqo, pko, pq, pk, wq, wk, pdq, pdk, gq, gk, pc, ps, pos, tokens, H, Hkv, d, qos, kos, qs, ks, dqs,
        dks, float(eps), float(weight_offset), w_code, rot, rows, 1 if rotary_interleaved else 0, n_axes,
        host, 1 if axes_interleaved else 0, code, _type_code(first), _stream_on(stream, at)))


def pva_gqa_tree(q, k_new, v_new, k_cache, v_cache, past_lens, out, num_heads: int,
                 kv_num_heads: int, parents=None, tree_lens=None, block_table=None, cos_cache=None,
                 sin_cache=None, position_ids=None, sections=None,
                 rotary_interleaved: bool = False, axes_interleaved: bool = False,
                 scale: float = 0.0, softcap: float = 0.0, local_window: int = 0,
                 stream=None) -> None:
    """One GroupQueryAttention step of a tree of drafted tokens (``parents``
    int32 [B, T], -1 a root; None: a chain) on a KV cache: q [B, T, H, d],
    k_new/v_new [B, T, Hkv, d], caches [n_blocks, Hkv, page, d] with
    ``block_table`` int32 [B, max_blocks] (None: sequence b owns block b),
    past_lens int32 [B] rows before the step, tree_lens int32 [B] nodes in use;
    optional rotation by cos/sin tables with position_ids int64 [n_axes, B, T]
    (None: past + depth); out [B, T, H, d]."""
    _need(q.dim() == 4, "q must be [B, tokens, num_heads, head_size]")
    B, T, _, d = q.shape
    H, Hkv = int(num_heads), int(kv_num_heads)
    dt, i32 = q.dtype, torch.int32
    _need(k_cache.dim() == 4, "k_cache must be [n_blocks, kv_num_heads, page, head_size]")
    blocks, _, page, _ = k_cache.shape
    at = _device(q, k_new, v_new, k_cache, v_cache, past_lens, out, parents, tree_lens, block_table,
                 cos_cache, sin_cache, position_ids)
    rows_q, rows_k, cache = (B, T, H, d), (B, T, Hkv, d), (blocks, Hkv, page, d)
    width = 0
    if block_table is not None:
        _need(block_table.dim() == 2, "block_table must be [B, max_blocks]")
        width = block_table.shape[1]
    rot = rows = code = 0
    n_axes, pc, ps, pos, host = 1, None, None, None, None
    if cos_cache is not None:
        if position_ids is not None:
            _need(position_ids.dim() == 3, "position_ids must be [n_axes, B, tokens]")
            n_axes = position_ids.shape[0]
            pos = _plain(position_ids, "position_ids", torch.int64, (n_axes, B, T), at)
        elif sections is not None:
            n_axes = len(sections)
        _need(sections is None or len(sections) == n_axes, "sections needs one entry per axis")
        pc, ps, rot, rows, code, host = _rotary(cos_cache, sin_cache, sections, at)
    else:
        _need(sin_cache is None and position_ids is None and sections is None,
              "positions and sections need the cos and sin tables")
    _check((_lib or load_library()).pva_gqa_tree(
        _plain(q, "q", dt, rows_q, at), _plain(k_new, "k_new", dt, rows_k, at),
        _plain(v_new, "v_new", dt, rows_k, at), _plain(k_cache, "k_cache", dt, cache, at),
        _plain(v_cache, "v_cache", dt, cache, at), _plain(past_lens, "past_lens", i32, (B,), at),
        _plain(tree_lens, "tree_lens", i32, (B,), at), _plain(parents, "parents", i32, (B, T), at),
        _plain(block_table, "block_table", i32, (B, width), at), pc, ps, pos,
        _plain(out, "out", dt, rows_q, at), B, T, blocks, page, width, H, Hkv, d, rot, rows,
        1 if rotary_interleaved else 0, n_axes, host, 1 if axes_interleaved else 0, code,
        float(scale), float(softcap), int(local_window), _type_code(q), _stream_on(stream, at)))


def pva_kvcache_accept(k_cache, v_cache, past_lens, path, path_lens, new_lens, block_table=None,
                       stream=None) -> None:
    """Move the accepted path's rows of a drafted tree: cache row past + path[i]
    becomes row past + i for i < path_lens, for every head and layer.  Caches
    [n_blocks, Hkv, page, d] or [layers, n_blocks, Hkv, page, d], path int32
    [B, width], past_lens, path_lens, new_lens (= past + path_lens) int32 [B]."""
    _need(k_cache.dim() in (4, 5), "k_cache must be [layers,] [n_blocks, heads, page, head_size]")
    _need(path.dim() == 2, "path must be [B, width]")
    shape = k_cache.shape
    layers = shape[0] if len(shape) == 5 else 1
    blocks, Hkv, page, d = shape[-4:]
    B, width = path.shape
    i32, dt = torch.int32, k_cache.dtype
    table_width = 0
    if block_table is not None:
        _need(block_table.dim() == 2, "block_table must be [B, max_blocks]")
        table_width = block_table.shape[1]
    at = _device(k_cache, v_cache, past_lens, path, path_lens, new_lens, block_table)
    _check((_lib or load_library()).pva_kvcache_accept(
        _plain(k_cache, "k_cache", dt, shape, at), _plain(v_cache, "v_cache", dt, shape, at),
        _plain(past_lens, "past_lens", i32, (B,), at), _plain(path, "path", i32, (B, width), at),
        _plain(path_lens, "path_lens", i32, (B,), at),
        _plain(block_table, "block_table", i32, (B, table_width), at),
        _plain(new_lens, "new_lens", i32, (B,), at), B, width, layers, blocks * Hkv * page * d,
        blocks, Hkv, page, d, table_width, _type_code(k_cache), _stream_on(stream, at)))


def pva_gqa_prefix(q, k_cache, v_cache, lens, prefix_lens, out, num_heads: int, kv_num_heads: int,
                   prefix_start=None, q_lens=None, block_table=None, prefix_table=None, lse=None,
                   scale: float = 0.0, softcap: float = 0.0, stream=None) -> None:
    """Attention of q [B, T, H, d] over prefixes that sequences share and then over each
    one's own rows, lens int32 [B] of them with the tokens (q_lens int32 [B]; None: all)
    last.  Sequences prefix_start[p] .. prefix_start[p + 1] - 1 (int32 [P + 1]; None: all
    of one) have prefix p, prefix_lens int32 [P] rows.  Caches [n_blocks, Hkv, page, d]
    with block_table int32 [B, ...] and prefix_table int32 [P, ...] (None, both: sequence b
    owns block b, prefix p block B + p); out [B, T, H, d], lse f32 [B, T, H] or None."""
    _need(q.dim() == 4, "q must be [B, tokens, num_heads, head_size]")
    B, T, _, d = q.shape
    H, Hkv = int(num_heads), int(kv_num_heads)
    dt, i32 = q.dtype, torch.int32
    _need(k_cache.dim() == 4, "k_cache must be [n_blocks, kv_num_heads, page, head_size]")
    blocks, _, page, _ = k_cache.shape
    _need(prefix_lens.dim() == 1, "prefix_lens must be [prefixes]")
    P = prefix_lens.shape[0]
    at = _device(q, k_cache, v_cache, lens, prefix_lens, out, prefix_start, q_lens, block_table, prefix_table,
                 lse)
    rows, cache = (B, T, H, d), (blocks, Hkv, page, d)
    _need((block_table is None) == (prefix_table is None), "block_table and prefix_table come together")
    width = prefix_width = 0
    if block_table is not None:
        _need(block_table.dim() == 2 and prefix_table.dim() == 2,
              "block_table must be [B, max_blocks] and prefix_table [prefixes, max_blocks]")
        width, prefix_width = block_table.shape[1], prefix_table.shape[1]
    _check((_lib or load_library()).pva_gqa_prefix(
        _plain(q, "q", dt, rows, at), _plain(k_cache, "k_cache", dt, cache, at),
        _plain(v_cache, "v_cache", dt, cache, at), _plain(lens, "lens", i32, (B,), at),
        _plain(q_lens, "q_lens", i32, (B,), at), _plain(block_table, "block_table", i32, (B, width), at),
        _plain(prefix_lens, "prefix_lens", i32, (P,), at),
        _plain(prefix_start, "prefix_start", i32, (P + 1,), at),
        _plain(prefix_table, "prefix_table", i32, (P, prefix_width), at), _plain(out, "out", dt, rows, at),
        _plain(lse, "lse", torch.float32, (B, T, H), at), B, T, P, blocks, page, width, prefix_width, H, Hkv, d,
        float(scale), float(softcap), _type_code(q), _stream_on(stream, at)))


def pva_kvcache_weights(q, k_cache, lens, weights, num_heads: int, previous=None, decay: float = 1.0,
                        lse=None, q_lens=None, block_table=None, scale: float = 0.0,
                        softcap: float = 0.0, stream=None) -> None:
    """Add up the attention that queries [B, T, H, d] give to each cache row: weights
    f32 [B, Hkv, width] = decay * previous (may be weights; None: nothing) + the sum of
    exp(score - lse) over the tokens and heads of each group, row j < lens int32 [B].
    The tokens are the last rows (q_lens int32 [B] of them).  lse f32 [B, T, H] as
    pva_gqa_prefix gives it; None: over the sequence's own rows."""
    _need(q.dim() == 4, "q must be [B, tokens, num_heads, head_size]")
    B, T, _, d = q.shape
    H = int(num_heads)
    dt, i32, f32 = q.dtype, torch.int32, torch.float32
    _need(k_cache.dim() == 4, "k_cache must be [n_blocks, kv_num_heads, page, head_size]")
    blocks, Hkv, page, _ = k_cache.shape
    _need(weights.dim() == 3, "weights must be [B, kv_num_heads, width]")
    rows = (B, Hkv, weights.shape[2])
    at = _device(q, k_cache, lens, weights, previous, lse, q_lens, block_table)
    table_width = 0
    if block_table is not None:
        _need(block_table.dim() == 2, "block_table must be [B, max_blocks]")
        table_width = block_table.shape[1]
    _check((_lib or load_library()).pva_kvcache_weights(
        _plain(q, "q", dt, (B, T, H, d), at), _plain(k_cache, "k_cache", dt, (blocks, Hkv, page, d), at),
        _plain(lens, "lens", i32, (B,), at), _plain(q_lens, "q_lens", i32, (B,), at),
        _plain(block_table, "block_table", i32, (B, table_width), at),
        _plain(previous, "previous", f32, rows, at), _plain(lse, "lse", f32, (B, T, H), at),
        _plain(weights, "weights", f32, rows, at), B, T, blocks, page, table_width, H, Hkv, d, rows[2],
        float(decay), float(scale), float(softcap), _type_code(q), _stream_on(stream, at)))


def pva_kvcache_evict(k_cache, v_cache, weights, lens, keep, new_lens, first: int = 0, last: int = 0,
                      block_table=None, k_out=None, v_out=None, out_table=None, weights_out=None,
                      kept=None, stream=None) -> None:
    """Cut every sequence down to its ``keep`` int32 [B] heaviest cache rows (the
    ``first`` and ``last`` ones stay in any case), by f32 weights [layers,] [B, Hkv,
    width].  Caches [layers,] [n_blocks, Hkv, page, d]; in place, or to k_out, v_out
    and/or the blocks of out_table.  Written: new_lens int32 [B], the rows' weights
    (weights_out, may be weights) and their old numbers (kept, int32)."""
    _need(k_cache.dim() in (4, 5), "k_cache must be [layers,] [n_blocks, heads, page, head_size]")
    shape = k_cache.shape
    layers = shape[0] if len(shape) == 5 else 1
    blocks, Hkv, page, d = shape[-4:]
    _need(lens.dim() == 1, "lens must be [B]")
    B = lens.shape[0]
    _need(weights.dim() == len(shape) - 1 or (layers == 1 and weights.dim() in (3, 4)),
          "weights must be [layers,] [B, kv_heads, width]")
    width = weights.shape[-1]
    lead = weights.shape[:-3]
    _need(not lead or lead[0] == layers, "weights must be [layers,] [B, kv_heads, width]")
    rows = (*lead, B, Hkv, width)
    i32, f32, dt = torch.int32, torch.float32, k_cache.dtype
    at = _device(k_cache, v_cache, weights, lens, keep, new_lens, block_table, k_out, v_out, out_table,
                 weights_out, kept)

    def table(t, name):
        if t is None:
            return None, 0
        _need(t.dim() == 2, f"{name} must be [B, max_blocks]")
        return _plain(t, name, i32, (B, t.shape[1]), at), t.shape[1]

    ptable, table_width = table(block_table, "block_table")
    pout, out_width = table(out_table, "out_table")
    _need((k_out is None) == (v_out is None), "k_out and v_out come together")
    out_blocks = out_page = 0
    po = pvo = None
    if k_out is not None:
        out_shape = k_out.shape
        _need(len(out_shape) == len(shape) and out_shape[-1] == d and out_shape[-3] == Hkv
              and (len(shape) == 4 or out_shape[0] == layers), "k_out must be a pool like k_cache")
        out_blocks, out_page = out_shape[-4], out_shape[-2]
        po = _plain(k_out, "k_out", dt, out_shape, at)
        pvo = _plain(v_out, "v_out", dt, out_shape, at)
    _check((_lib or load_library()).pva_kvcache_evict(
        _plain(k_cache, "k_cache", dt, shape, at), _plain(v_cache, "v_cache", dt, shape, at),
        _plain(weights, "weights", f32, rows, at), _plain(lens, "lens", i32, (B,), at),
        _plain(keep, "keep", i32, (B,), at), _plain(new_lens, "new_lens", i32, (B,), at), ptable, po, pvo,
        pout, _plain(weights_out, "weights_out", f32, rows, at), _plain(kept, "kept", i32, rows, at), B,
        layers, blocks * Hkv * page * d, blocks, page, table_width, out_blocks * Hkv * out_page * d,
        out_blocks, out_page, out_width, Hkv, d, width, int(first), int(last), _type_code(k_cache),
        _stream_on(stream, at)))


def pva_forward_noalloc(q, k, v, cu_seqlens_q, cu_seqlens_kv, out, B: int, num_heads: int,
                        kv_num_heads: int, head_size: int, v_head_size: int, scale: float = 0.0,
                        is_causal: int = 0, softcap: float = 0.0, dtype: int | None = None,
                        device_status=None, stream=None) -> None:
    """pva_forward for callers that cannot allocate device memory at call
    time: the library uses its fixed 4 MiB per-device scratch array instead of
    a per-stream workspace (see include/pva.h for the limits and the rule that
    overlapping calls race).  ``device_status`` is an optional CUDA uint32
    tensor the call ORs its status bits into."""
    lib = load_library()
    code = _dtype_code(q) if dtype is None else int(dtype)
    st = device_status.data_ptr() if device_status is not None else None
    rc = lib.pva_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                 cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(),
                                 out.data_ptr(), int(B), int(num_heads), int(kv_num_heads),
                                 int(head_size), int(v_head_size), float(scale), int(is_causal),
                                 float(softcap), code, st, _stream_ptr(stream))
    _check(rc)


def pva_get_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) its latched device bits."""
    lib = load_library()
    flags = ctypes.c_uint32(0)
    _check(lib.pva_get_status(_stream_ptr(stream), ctypes.byref(flags)))
    return int(flags.value)


def pva_schedule(cu_seqlens_q, cu_seqlens_kv, B: int, num_heads: int, kv_num_heads: int,
                 head_size: int, v_head_size: int, is_causal: int, dtype: int, stream=None):
    """Run only the on-device scheduler; returns its int32 words as a list."""
    lib = load_library()
    n = 8 + 4 * int(B) + 2
    buf = (ctypes.c_int32 * n)()
    _check(lib.pva_schedule(cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(), int(B),
                            int(num_heads), int(kv_num_heads), int(head_size), int(v_head_size),
                            int(is_causal), int(dtype), buf, n, _stream_ptr(stream)))
    return list(buf)


def pva_status_string(code: int) -> str:
    return load_library().pva_status_string(int(code)).decode()


def pva_last_error() -> str:
    return load_library().pva_last_error().decode()


def pva_release() -> None:
    load_library().pva_release()


def pva_version() -> int:
    return int(load_library().pva_version())


def pva_selftest_give_up(limit_us: int) -> None:
    """Have the pipelines of later calls stall for limit_us microseconds and give up (0: no more)."""
    _check(load_library().pva_selftest_give_up(int(limit_us)))


def pva_selftest_wait(limit_us: int = 20000, stream=None) -> int:
    """Run the bounded-wait self-test; returns the device bits it latched."""
    lib = load_library()
    flags = ctypes.c_uint32(0)
    _check(lib.pva_selftest_wait(int(limit_us), _stream_ptr(stream), ctypes.byref(flags)))
    return int(flags.value)


def pva_profile(enable: bool) -> None:
    """Bracket each later launch (this thread) with CUDA events (benchmarks)."""
    _check(load_library().pva_profile(int(bool(enable))))


def pva_kernel_times():
    """Device durations (ms) of the last profiled call's launches:
    (scheduler, prefill, decode or -1)."""
    buf = (ctypes.c_float * 3)()
    _check(load_library().pva_kernel_times(buf, 3))
    return tuple(float(x) for x in buf)
