"""Python binding of the gfx950 paged MLA latent-K library (``include/mla_paged.h``).

Argument marshalling only: every step of every operation runs in the HIP
kernels of ``_build/libmla_paged.so``.  Tensors are torch tensors on the
current HIP device; the current torch stream is passed as the HIP stream.
There is no fallback: if the library has not been built, every call raises.

Entry points (same names as the C ABI):
  mla_decompress_k_paged       gather latent rows from a paged cache, up-project them
  mla_decompress_k_paged_fp8   the fp8 block-scaled form (1x128 activation, 128x128 weight scales)
  mla_decompress_k_paged_fp8_noalloc  the same without a workspace (for callers that cannot allocate)
  mla_decompress_kv_paged(_fp8)  one gather, K and V up-projections
  mla_decompress_k_paged_fp8_cache  the fp8 form on an e4m3 cache with per-128-column scales
  mla_write_latent_paged       RMSNorm + rope rotation of new tokens' rows into the cache pages
  mla_absorb_q(_fp8)           per-head product of the non-rope query columns with w_uk (decode)
  kv_matmul_paged              project hidden states and write them into K/V cache pages
  mla_gather_latent_paged      the gather step alone
  mla_latent_matmul            the up-projection step alone (rows already gathered)
  mla_rope_freqs               a freqs_cis table, with long-context scaling
  mla_rope_q                   rotation of every query head's rope columns at given positions
  mla_write_latent_paged(_fp8)_at  the latent writes with the rope position of each token given
  mla_tree_attention_paged(_fp8_cache)  attention of absorbed queries over cached and drafted rows
  mla_copy_pages, mla_fork_paged, mla_free_paged, mla_compact_paged  page upkeep
  mla_check_indices            debug validation of index arrays (synchronous)
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
import threading
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmla_paged.so")

MLA_DTYPE_F32, MLA_DTYPE_BF16, MLA_DTYPE_F8E4M3FN = 0, 1, 2
STATUS = {0: "MLA_OK", 1: "MLA_ERR_NULL_POINTER", 2: "MLA_ERR_INVALID_SHAPE",
          3: "MLA_ERR_INVALID_DTYPE", 4: "MLA_ERR_MISALIGNED", 5: "MLA_ERR_OUT_OF_RANGE",
          6: "MLA_ERR_WORKSPACE", 7: "MLA_ERR_UNSUPPORTED_DEVICE", 8: "MLA_ERR_HIP"}
EXPORTS = ("mla_paged_cache_default_strides", "mla_decompress_k_paged", "mla_gather_latent_paged",
           "mla_latent_matmul", "mla_decompress_k_paged_fp8_workspace_size", "mla_decompress_k_paged_fp8",
           "kv_matmul_paged", "mla_check_indices", "mla_status_string", "mla_last_hip_error",
           "mla_abi_version", "mla_decompress_kv_paged", "mla_decompress_kv_paged_fp8",
           "mla_write_latent_paged", "mla_decompress_k_paged_fp8_cache", "mla_absorb_q", "mla_absorb_q_fp8",
           "mla_write_latent_paged_fp8", "mla_decompress_kv_paged_fp8_cache", "mla_decompress_k_paged_fp8_noalloc",
           "mla_rope_freqs", "mla_rope_q", "mla_write_latent_paged_at", "mla_write_latent_paged_fp8_at",
           "mla_tree_attention_workspace_size", "mla_tree_attention_paged", "mla_tree_attention_paged_fp8_cache",
           "mla_copy_pages", "mla_fork_paged", "mla_free_paged", "mla_compact_paged")
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "by_parts": 2}
# mla_decompress_k_paged_fp8_noalloc's fixed device array (include/mla_paged.h)
MLA_FP8_NOALLOC_SCRATCH_BYTES = 33 << 20


class MlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class CacheDesc(ctypes.Structure):
    """Mirror of ``mla_paged_cache_t``."""
    _fields_ = [
        ("blocks", ctypes.c_void_p), ("dtype", ctypes.c_int32),
        ("num_layers", ctypes.c_uint32), ("num_pages", ctypes.c_uint32),
        ("page_size", ctypes.c_uint32), ("num_kv", ctypes.c_uint32),
        ("num_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32),
        ("stride_page", ctypes.c_int64), ("stride_layer", ctypes.c_int64),
        ("stride_kv", ctypes.c_int64), ("stride_token", ctypes.c_int64),
        ("page_table", ctypes.c_void_p), ("batch_size", ctypes.c_uint32),
        ("max_pages_per_seq", ctypes.c_uint32), ("cache_lengths", ctypes.c_void_p),
    ]


class ScalesDesc(ctypes.Structure):
    """Mirror of ``mla_cache_scales_t``."""
    _fields_ = [
        ("scales", ctypes.c_void_p), ("granularity", ctypes.c_uint32),
        ("stride_page", ctypes.c_int64), ("stride_layer", ctypes.c_int64),
        ("stride_kv", ctypes.c_int64), ("stride_token", ctypes.c_int64),
    ]


class RopeParams(ctypes.Structure):
    """Mirror of ``mla_rope_params_t``."""
    _fields_ = [
        ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("beta_fast", ctypes.c_double),
        ("beta_slow", ctypes.c_double), ("amplitude", ctypes.c_double), ("scaling", ctypes.c_int32),
        ("original_max_position", ctypes.c_int32),
    ]


_lock = threading.Lock()
_lib = None


def lib():
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"HIP library not built ({LIB_PATH}); run __graft_entry__.build() "
                                   "or python -m mla_paged_latent_page_amd.build")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
            L.mla_paged_cache_default_strides.argtypes = [ctypes.POINTER(CacheDesc)]
            L.mla_paged_cache_default_strides.restype = i32
            L.mla_decompress_k_paged.argtypes = [vp, vp, i32, vp, i32, i32, ctypes.POINTER(CacheDesc), u32,
                                                 vp, vp, vp]
            L.mla_decompress_k_paged.restype = i32
            L.mla_decompress_k_paged_fp8_workspace_size.argtypes = [i32, i32, i32]
            L.mla_decompress_k_paged_fp8_workspace_size.restype = sz
            L.mla_decompress_k_paged_fp8.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                                     ctypes.POINTER(CacheDesc), u32, vp, vp, vp, sz, vp]
            L.mla_decompress_k_paged_fp8.restype = i32
            L.mla_decompress_k_paged_fp8_noalloc.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                                             ctypes.POINTER(CacheDesc), u32, vp, vp, vp]
            L.mla_decompress_k_paged_fp8_noalloc.restype = i32
            L.mla_decompress_kv_paged.argtypes = [vp, vp, i32, vp, i32, vp, i32, i32, ctypes.POINTER(CacheDesc),
                                                  u32, vp, vp, vp, vp]
            L.mla_decompress_kv_paged.restype = i32
            L.mla_decompress_kv_paged_fp8.argtypes = [vp, vp, i32, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                                      ctypes.POINTER(CacheDesc), u32, vp, vp, vp, vp, sz, vp]
            L.mla_decompress_kv_paged_fp8.restype = i32
            L.mla_write_latent_paged.argtypes = [vp, vp, i32, vp, ctypes.c_float, vp, i32, i32,
                                                 ctypes.POINTER(CacheDesc), u32, vp]
            L.mla_write_latent_paged.restype = i32
            L.mla_write_latent_paged_fp8.argtypes = [vp, vp, i32, vp, ctypes.c_float, vp, i32, i32,
                                                     ctypes.POINTER(CacheDesc), ctypes.POINTER(ScalesDesc), u32, vp]
            L.mla_write_latent_paged_fp8.restype = i32
            L.mla_decompress_k_paged_fp8_cache.argtypes = [vp, vp, i32, vp, vp, i32, i32, ctypes.POINTER(CacheDesc),
                                                           ctypes.POINTER(ScalesDesc), u32, vp, vp, vp, vp]
            L.mla_decompress_k_paged_fp8_cache.restype = i32
            L.mla_decompress_kv_paged_fp8_cache.argtypes = [vp, vp, i32, vp, vp, i32, vp, vp, i32, i32,
                                                            ctypes.POINTER(CacheDesc), ctypes.POINTER(ScalesDesc), u32,
                                                            vp, vp, vp, vp, vp]
            L.mla_decompress_kv_paged_fp8_cache.restype = i32
            L.mla_absorb_q.argtypes = [vp, i32, i32, i32, i32, vp, i32, i32, vp, vp]
            L.mla_absorb_q.restype = i32
            L.mla_absorb_q_fp8.argtypes = [vp, i32, i32, i32, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp]
            L.mla_absorb_q_fp8.restype = i32
            i64, f32 = ctypes.c_int64, ctypes.c_float
            cd, sd = ctypes.POINTER(CacheDesc), ctypes.POINTER(ScalesDesc)
            L.mla_rope_freqs.argtypes = [ctypes.POINTER(RopeParams), i32, i32, i32, vp, vp]
            L.mla_rope_freqs.restype = i32
            L.mla_rope_q.argtypes = [vp, i64, i64, i32, i32, i32, i32, i32, vp, vp, i32, i32, vp, i64, i64, vp]
            L.mla_rope_q.restype = i32
            L.mla_write_latent_paged_at.argtypes = [vp, vp, i32, vp, vp, f32, vp, i32, i32, i32, cd, u32, vp]
            L.mla_write_latent_paged_at.restype = i32
            L.mla_write_latent_paged_fp8_at.argtypes = [vp, vp, i32, vp, vp, f32, vp, i32, i32, i32, cd, sd, u32, vp]
            L.mla_write_latent_paged_fp8_at.restype = i32
            L.mla_tree_attention_workspace_size.argtypes = [i32, i32, i32]
            L.mla_tree_attention_workspace_size.restype = sz
            L.mla_tree_attention_paged.argtypes = [vp, vp, i32, i32, vp, i32, f32, i32, cd, u32, vp, vp, vp, sz, vp]
            L.mla_tree_attention_paged.restype = i32
            L.mla_tree_attention_paged_fp8_cache.argtypes = [vp, vp, i32, i32, vp, i32, f32, i32, cd, sd, u32, vp, vp,
                                                             vp, sz, vp]
            L.mla_tree_attention_paged_fp8_cache.restype = i32
            L.mla_copy_pages.argtypes = [vp, vp, i32, cd, sd, vp]
            L.mla_copy_pages.restype = i32
            L.mla_fork_paged.argtypes = [vp, vp, vp, i32, vp, cd, sd, vp]
            L.mla_fork_paged.restype = i32
            L.mla_free_paged.argtypes = [vp, i32, vp, vp, vp, cd, vp]
            L.mla_free_paged.restype = i32
            L.mla_compact_paged.argtypes = [vp, vp, i32, cd, sd, vp]
            L.mla_compact_paged.restype = i32
            L.kv_matmul_paged.argtypes = [vp, vp, i32, i32, vp, ctypes.POINTER(CacheDesc), u32, vp]
            L.kv_matmul_paged.restype = i32
            L.mla_gather_latent_paged.argtypes = [vp, vp, i32, ctypes.POINTER(CacheDesc), u32, vp, vp]
            L.mla_gather_latent_paged.restype = i32
            L.mla_latent_matmul.argtypes = [vp, ctypes.c_int64, i32, vp, i32, i32, i32, vp, vp]
            L.mla_latent_matmul.restype = i32
            L.mla_check_indices.argtypes = [vp, vp, i32, ctypes.POINTER(CacheDesc),
                                            ctypes.POINTER(ctypes.c_int64), vp]
            L.mla_check_indices.restype = i32
            L.mla_status_string.argtypes = [i32]
            L.mla_status_string.restype = ctypes.c_char_p
            L.mla_last_hip_error.restype = i32
            L.mla_abi_version.restype = i32
            _lib = L
        return _lib


# ---------------------------------------------------------------------------
# cache descriptor from torch tensors
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class PagedKVCache:
    """A paged pool as torch tensors.

    pool          [num_pages, num_layers, num_kv, page_size, num_heads, head_dim]
                  (float32, bfloat16, or uint8 / float8_e4m3fn codes; may be a strided
                  view with contiguous token rows)
    page_table    int32/uint32 [batch, max_pages_per_seq] page ids (raw 32-bit values)
    cache_lengths int32/uint32 [batch] or None
    scales        fp8 pools only: float32 [num_pages, num_layers, num_kv, page_size, nblk],
                  one scale per scale_granularity columns of a token row
    """
    pool: "object"
    page_table: "object"
    cache_lengths: Optional["object"] = None
    scales: Optional["object"] = None
    scale_granularity: int = 128

    def descriptor(self) -> CacheDesc:
        p = self.pool
        if p.dim() != 6:
            raise ValueError("pool must be [pages, layers, kv, page_size, heads, head_dim]")
        pages, layers, kv, page_size, heads, head_dim = p.shape
        sp, sl, sk, st, sh, se = p.stride()
        if se != 1 or sh != head_dim:
            raise ValueError("token rows of the pool must be contiguous")
        pt = self.page_table
        if pt.dim() != 2 or not pt.is_contiguous() or pt.element_size() != 4:
            raise ValueError("page_table must be a contiguous 32-bit [batch, max_pages] tensor")
        batch, max_pages = pt.shape
        lengths = None
        if self.cache_lengths is not None:
            cl = self.cache_lengths
            if not cl.is_contiguous() or cl.element_size() != 4 or cl.numel() != batch:
                raise ValueError("cache_lengths must be a contiguous 32-bit [batch] tensor")
            lengths = cl.data_ptr()
        return CacheDesc(p.data_ptr(), _pool_dtypes().get(p.dtype, -1), layers, pages, page_size, kv, heads, head_dim,
                         sp, sl, sk, st, pt.data_ptr(), batch, max_pages, lengths)

    def scales_descriptor(self) -> ScalesDesc:
        import torch
        sc = self.scales
        if sc is None:
            raise ValueError("this cache has no scale pool")
        if sc.dim() != 5 or sc.dtype != torch.float32 or sc.stride(4) != 1:
            raise ValueError("scales must be float32 [pages, layers, kv, page_size, nblk] with contiguous rows")
        if tuple(sc.shape[:4]) != tuple(self.pool.shape[:4]):
            raise ValueError("scales must have the pool's pages, layers, kv halves and slots")
        d = ScalesDesc()
        d.scales = sc.data_ptr()
        d.granularity = int(self.scale_granularity)
        d.stride_page, d.stride_layer, d.stride_kv, d.stride_token = sc.stride(0), sc.stride(1), sc.stride(2), sc.stride(3)
        return d


def _stream(stream):
    import torch
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream() without the Stream object around the handle: it costs more
    # than a small call's kernel.
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _nbytes(t):
    return t.numel() * t.element_size()


def _buf(t, what, nbytes, dtypes=None):
    """Check a contiguous tensor of at least ``nbytes`` bytes (and, when given,
    one of ``dtypes``); returns its pointer.  Where it lives is checked by
    _gpu() once every shape, dtype and size check has passed."""
    if t is None:
        raise ValueError(f"{what} is required")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{what} must be of dtype {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if _nbytes(t) < nbytes:
        raise ValueError(f"{what} holds {_nbytes(t)} bytes; the call reads or writes {nbytes}")
    return t.data_ptr()


def _u32(t, what, entries=0):
    if t.element_size() != 4 or not t.is_contiguous() or t.dtype.is_floating_point:
        raise ValueError(f"{what} must be a contiguous 32-bit integer tensor")
    if t.numel() < entries:
        raise ValueError(f"{what} must have at least {entries} entries")
    return t.data_ptr()


def _gpu(cache=None, **tensors):
    """Every tensor a call hands to the library (the cache's too) must live on the current GPU;
    anything else (a host tensor, another GPU's tensor) is refused before any launch."""
    import torch
    items = tensors.items()
    if cache is not None:
        items = (*items, ("cache.pool", cache.pool), ("cache.page_table", cache.page_table),
                 ("cache.cache_lengths", cache.cache_lengths), ("cache.scales", cache.scales))
    current = None
    for name, t in items:
        if t is None:
            continue
        device = t.get_device() if isinstance(t, torch.Tensor) and t.is_cuda else -1
        if device >= 0:
            if current is None:
                current = torch._C._cuda_getDevice()
            if device == current:
                continue
        raise ValueError(f"{name} must be a tensor on the current GPU")


@functools.lru_cache(maxsize=None)
def _dtypes():
    import torch
    return {MLA_DTYPE_F32: (torch.float32,), MLA_DTYPE_BF16: (torch.bfloat16,),
            MLA_DTYPE_F8E4M3FN: (torch.uint8, torch.float8_e4m3fn)}


@functools.lru_cache(maxsize=None)
def _pool_dtypes():
    return {dtype: code for code, dtypes in _dtypes().items() for dtype in dtypes}


def _bytes_of(dtype_code):
    return {MLA_DTYPE_F32: 4, MLA_DTYPE_BF16: 2, MLA_DTYPE_F8E4M3FN: 1}.get(dtype_code, 1)


def _cache_desc(cache, scales=False):
    """The cache's descriptor(s)."""
    desc = cache.descriptor()
    if not scales:
        return desc
    return desc, cache.scales_descriptor()


def _index_args(buffer_row_offsets, cache_offsets, desc):
    B = desc.batch_size
    return (_u32(buffer_row_offsets, "buffer_row_offsets", B + 1), _u32(cache_offsets, "cache_offsets", B))


def _check_outputs(M, desc, N, k_latent_buffer, k_buffer, out_dtype=None):
    """k_latent_buffer holds M cache rows in the cache's dtype, k_buffer M rows of
    N values of ``out_dtype`` (default: the cache's dtype)."""
    dt = _dtypes()
    D = desc.num_heads * desc.head_dim
    eb = _bytes_of(desc.dtype)
    lat = _buf(k_latent_buffer, "k_latent_buffer", M * D * eb, dt.get(desc.dtype))
    odt = dt.get(desc.dtype) if out_dtype is None else out_dtype
    ob = _bytes_of(desc.dtype) if out_dtype is None else 2
    out = _buf(k_buffer, "k_buffer", M * N * ob, odt)
    return lat, out


def _check(status, what):
    if status != 0:
        if status == 8:
            raise MlaError(status, f"{what} (hipError {lib().mla_last_hip_error()})")
        raise MlaError(status, what)


# ---------------------------------------------------------------------------
# operations
# ---------------------------------------------------------------------------
def _weight(w, name, dtypes):
    if w is None or w.dim() != 2:
        raise ValueError(f"{name} must be a 2-D [N, K] tensor")
    N, K = w.shape
    return N, K, _buf(w, name, N * K * w.element_size(), dtypes)


def _f32(t, name, count):
    import torch
    return _buf(t, name, count * 4, (torch.float32,))


def mla_decompress_k_paged(buffer_row_offsets, cache_offsets, buffer_length: int, weight,
                           cache: PagedKVCache, layer_idx: int, k_latent_buffer, k_buffer,
                           stream=None) -> None:
    """k_latent_buffer[r] = paged cache row; k_buffer = k_latent_buffer[:, :K] @ weight.T."""
    desc = _cache_desc(cache)
    N, K, w = _weight(weight, "weight", _dtypes().get(desc.dtype))
    lat, out = _check_outputs(buffer_length, desc, N, k_latent_buffer, k_buffer)
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, weight=weight,
         k_latent_buffer=k_latent_buffer, k_buffer=k_buffer, cache=cache)
    st = lib().mla_decompress_k_paged(bro, co, int(buffer_length), w, N, K, ctypes.byref(desc), int(layer_idx),
                                      lat, out, _stream(stream))
    _check(st, "mla_decompress_k_paged")


def mla_gather_latent_paged(buffer_row_offsets, cache_offsets, buffer_length: int, cache: PagedKVCache,
                            layer_idx: int, k_latent_buffer, stream=None) -> None:
    """k_latent_buffer[r] = paged cache row (the gather step alone)."""
    desc = _cache_desc(cache)
    D = desc.num_heads * desc.head_dim
    lat = _buf(k_latent_buffer, "k_latent_buffer", buffer_length * D * _bytes_of(desc.dtype),
               _dtypes().get(desc.dtype))
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, k_latent_buffer=k_latent_buffer,
         cache=cache)
    st = lib().mla_gather_latent_paged(bro, co, int(buffer_length), ctypes.byref(desc), int(layer_idx), lat,
                                       _stream(stream))
    _check(st, "mla_gather_latent_paged")


def mla_latent_matmul(k_latent_buffer, buffer_length: int, weight, k_buffer, stream=None) -> None:
    """k_buffer[:M] = k_latent_buffer[:M, :K] @ weight.T (the up-projection step alone).
    k_latent_buffer is a 2-D tensor with unit column stride (its row stride is passed)."""
    import torch
    if weight is None or weight.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("weight must be a float32 or bfloat16 [N, K] tensor")
    N, K, w = _weight(weight, "weight", (weight.dtype,))
    M = int(buffer_length)
    if k_latent_buffer.dim() != 2 or k_latent_buffer.stride(1) != 1 or k_latent_buffer.shape[0] < M:
        raise ValueError("k_latent_buffer must be a [>= M, >= K] tensor with unit column stride")
    if k_latent_buffer.shape[1] < K or k_latent_buffer.dtype != weight.dtype or k_buffer.dtype != weight.dtype:
        raise ValueError("k_latent_buffer, weight and k_buffer must share a dtype, and K <= latent width")
    out = _buf(k_buffer, "k_buffer", M * N * weight.element_size(), (weight.dtype,))
    _gpu(k_latent_buffer=k_latent_buffer, weight=weight, k_buffer=k_buffer)
    lat = k_latent_buffer.data_ptr()
    dt = {torch.float32: MLA_DTYPE_F32, torch.bfloat16: MLA_DTYPE_BF16}[weight.dtype]
    st = lib().mla_latent_matmul(lat, k_latent_buffer.stride(0), M, w, N, K, dt, out, _stream(stream))
    _check(st, "mla_latent_matmul")


def mla_check_indices(row_offsets, cache_offsets, rows: int, cache: PagedKVCache, stream=None):
    """Debug validation of a call's index arrays (synchronous).  Returns
    (status, first failing request or -1); never raises on a failed check."""
    desc = _cache_desc(cache)
    bad = ctypes.c_int64(-1)
    _gpu(row_offsets=row_offsets, cache_offsets=cache_offsets, cache=cache)
    st = lib().mla_check_indices(_u32(row_offsets, "row_offsets", desc.batch_size + 1),
                                 _u32(cache_offsets, "cache_offsets", desc.batch_size)
                                 if cache_offsets is not None else None,
                                 int(rows), ctypes.byref(desc), ctypes.byref(bad), _stream(stream))
    if st in (1, 7, 8):
        _check(st, "mla_check_indices")
    return st, int(bad.value)


def mla_decompress_k_paged_fp8_workspace_size(buffer_length: int, K: int, k_gran: int = 128) -> int:
    return int(lib().mla_decompress_k_paged_fp8_workspace_size(int(buffer_length), int(K), int(k_gran)))


def _fp8_scale(sc, name, N, K, n_gran, k_gran):
    return _f32(sc, name, -(-N // n_gran) * -(-K // k_gran))


def _workspace(workspace):
    if workspace is None:
        raise ValueError("workspace is required")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), _nbytes(workspace)


def mla_decompress_k_paged_fp8(buffer_row_offsets, cache_offsets, buffer_length: int, weight_e4m3,
                               weight_scale, cache: PagedKVCache, layer_idx: int, k_latent_buffer,
                               k_buffer, workspace, m_gran: int = 1, n_gran: int = 128,
                               k_gran: int = 128, stream=None) -> None:
    """The fp8 block-scaled form; ``workspace`` is a device tensor of at least
    mla_decompress_k_paged_fp8_workspace_size(M, K) bytes."""
    import torch
    desc = _cache_desc(cache)
    N, K, w = _weight(weight_e4m3, "weight_e4m3", _dtypes()[MLA_DTYPE_F8E4M3FN])
    sw = _fp8_scale(weight_scale, "weight_scale", N, K, n_gran, k_gran)
    lat, out = _check_outputs(buffer_length, desc, N, k_latent_buffer, k_buffer, (torch.bfloat16,))
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    ws, ws_bytes = _workspace(workspace)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, weight_e4m3=weight_e4m3,
         weight_scale=weight_scale, k_latent_buffer=k_latent_buffer, k_buffer=k_buffer, workspace=workspace,
         cache=cache)
    st = lib().mla_decompress_k_paged_fp8(bro, co, int(buffer_length), w, sw, N, K, m_gran, n_gran, k_gran,
                                          ctypes.byref(desc), int(layer_idx), lat, out, ws, ws_bytes,
                                          _stream(stream))
    _check(st, "mla_decompress_k_paged_fp8")


def mla_decompress_k_paged_fp8_noalloc(buffer_row_offsets, cache_offsets, buffer_length: int, weight_e4m3,
                                       weight_scale, cache: PagedKVCache, layer_idx: int, k_latent_buffer,
                                       k_buffer, m_gran: int = 1, n_gran: int = 128, k_gran: int = 128,
                                       stream=None) -> None:
    """mla_decompress_k_paged_fp8 without a workspace: the library's fixed device
    array (MLA_FP8_NOALLOC_SCRATCH_BYTES per GPU) holds the activation codes and
    scales.  Calls that overlap on one GPU race on that array."""
    import torch
    desc = _cache_desc(cache)
    N, K, w = _weight(weight_e4m3, "weight_e4m3", _dtypes()[MLA_DTYPE_F8E4M3FN])
    sw = _fp8_scale(weight_scale, "weight_scale", N, K, n_gran, k_gran)
    lat, out = _check_outputs(buffer_length, desc, N, k_latent_buffer, k_buffer, (torch.bfloat16,))
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, weight_e4m3=weight_e4m3,
         weight_scale=weight_scale, k_latent_buffer=k_latent_buffer, k_buffer=k_buffer, cache=cache)
    st = lib().mla_decompress_k_paged_fp8_noalloc(bro, co, int(buffer_length), w, sw, N, K, m_gran, n_gran,
                                                  k_gran, ctypes.byref(desc), int(layer_idx), lat, out,
                                                  _stream(stream))
    _check(st, "mla_decompress_k_paged_fp8_noalloc")


def mla_decompress_kv_paged(buffer_row_offsets, cache_offsets, buffer_length: int, w_k, w_v,
                            cache: PagedKVCache, layer_idx: int, k_latent_buffer, k_buffer, v_buffer,
                            stream=None) -> None:
    """One gather, two up-projections: k_buffer = rows @ w_k.T, v_buffer = rows @ w_v.T."""
    desc = _cache_desc(cache)
    dt = _dtypes().get(desc.dtype)
    N_k, K, wk = _weight(w_k, "w_k", dt)
    N_v, K_v, wv = _weight(w_v, "w_v", dt)
    if K_v != K:
        raise ValueError("w_k and w_v must have the same K")
    lat, kout = _check_outputs(buffer_length, desc, N_k, k_latent_buffer, k_buffer)
    vout = _buf(v_buffer, "v_buffer", buffer_length * N_v * _bytes_of(desc.dtype), dt)
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, w_k=w_k, w_v=w_v,
         k_latent_buffer=k_latent_buffer, k_buffer=k_buffer, v_buffer=v_buffer, cache=cache)
    st = lib().mla_decompress_kv_paged(bro, co, int(buffer_length), wk, N_k, wv, N_v, K, ctypes.byref(desc),
                                       int(layer_idx), lat, kout, vout, _stream(stream))
    _check(st, "mla_decompress_kv_paged")


def mla_decompress_kv_paged_fp8(buffer_row_offsets, cache_offsets, buffer_length: int, w_k_e4m3, w_k_scale,
                                w_v_e4m3, w_v_scale, cache: PagedKVCache, layer_idx: int, k_latent_buffer,
                                k_buffer, v_buffer, workspace, m_gran: int = 1, n_gran: int = 128,
                                k_gran: int = 128, stream=None) -> None:
    """The fp8 block-scaled fused form (one gather and quantisation, two products)."""
    import torch
    desc = _cache_desc(cache)
    f8 = _dtypes()[MLA_DTYPE_F8E4M3FN]
    N_k, K, wk = _weight(w_k_e4m3, "w_k_e4m3", f8)
    N_v, K_v, wv = _weight(w_v_e4m3, "w_v_e4m3", f8)
    if K_v != K:
        raise ValueError("w_k_e4m3 and w_v_e4m3 must have the same K")
    sk = _fp8_scale(w_k_scale, "w_k_scale", N_k, K, n_gran, k_gran)
    sv = _fp8_scale(w_v_scale, "w_v_scale", N_v, K, n_gran, k_gran)
    lat, kout = _check_outputs(buffer_length, desc, N_k, k_latent_buffer, k_buffer, (torch.bfloat16,))
    vout = _buf(v_buffer, "v_buffer", buffer_length * N_v * 2, (torch.bfloat16,))
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    ws, ws_bytes = _workspace(workspace)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, w_k_e4m3=w_k_e4m3,
         w_k_scale=w_k_scale, w_v_e4m3=w_v_e4m3, w_v_scale=w_v_scale, k_latent_buffer=k_latent_buffer,
         k_buffer=k_buffer, v_buffer=v_buffer, workspace=workspace, cache=cache)
    st = lib().mla_decompress_kv_paged_fp8(bro, co, int(buffer_length), wk, sk, N_k, wv, sv, N_v, K,
                                           m_gran, n_gran, k_gran, ctypes.byref(desc), int(layer_idx),
                                           lat, kout, vout, ws, ws_bytes, _stream(stream))
    _check(st, "mla_decompress_kv_paged_fp8")


def _fp8_cache_buffers(desc, buffer_length, k_latent_buffer, k_latent_scales):
    import torch
    D = desc.num_heads * desc.head_dim
    nblk = -(-D // 128)
    lat = _buf(k_latent_buffer, "k_latent_buffer", buffer_length * D, _dtypes()[MLA_DTYPE_F8E4M3FN])
    lsc = _buf(k_latent_scales, "k_latent_scales", buffer_length * nblk * 4, (torch.float32,))
    return lat, lsc


def mla_decompress_k_paged_fp8_cache(buffer_row_offsets, cache_offsets, buffer_length: int, w_k_e4m3, w_k_scale,
                                     cache: PagedKVCache, layer_idx: int, k_latent_buffer, k_latent_scales, k_buffer,
                                     stream=None) -> None:
    """Gather e4m3 rows and their scales from an fp8 cache (bit copies into
    k_latent_buffer / k_latent_scales), then k_buffer = block-scaled rows @ w_k.T."""
    import torch
    desc, sdesc = _cache_desc(cache, scales=True)
    N, K, w = _weight(w_k_e4m3, "w_k_e4m3", _dtypes()[MLA_DTYPE_F8E4M3FN])
    sw = _fp8_scale(w_k_scale, "w_k_scale", N, K, 128, 128)
    lat, lsc = _fp8_cache_buffers(desc, buffer_length, k_latent_buffer, k_latent_scales)
    out = _buf(k_buffer, "k_buffer", buffer_length * N * 2, (torch.bfloat16,))
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, w_k_e4m3=w_k_e4m3,
         w_k_scale=w_k_scale, k_latent_buffer=k_latent_buffer, k_latent_scales=k_latent_scales,
         k_buffer=k_buffer, cache=cache)
    st = lib().mla_decompress_k_paged_fp8_cache(bro, co, int(buffer_length), w, sw, N, K, ctypes.byref(desc),
                                                ctypes.byref(sdesc), int(layer_idx), lat, lsc, out,
                                                _stream(stream))
    _check(st, "mla_decompress_k_paged_fp8_cache")


def mla_decompress_kv_paged_fp8_cache(buffer_row_offsets, cache_offsets, buffer_length: int, w_k_e4m3, w_k_scale,
                                      w_v_e4m3, w_v_scale, cache: PagedKVCache, layer_idx: int, k_latent_buffer,
                                      k_latent_scales, k_buffer, v_buffer, stream=None) -> None:
    """mla_decompress_k_paged_fp8_cache for K and, from the same gathered codes and
    scales, v_buffer = block-scaled rows @ w_v.T, in one gather and one product launch."""
    import torch
    desc, sdesc = _cache_desc(cache, scales=True)
    f8 = _dtypes()[MLA_DTYPE_F8E4M3FN]
    N, K, wk = _weight(w_k_e4m3, "w_k_e4m3", f8)
    Nv, Kv, wv = _weight(w_v_e4m3, "w_v_e4m3", f8)
    if Kv != K:
        raise ValueError("w_k_e4m3 and w_v_e4m3 must have the same K")
    sk = _fp8_scale(w_k_scale, "w_k_scale", N, K, 128, 128)
    sv = _fp8_scale(w_v_scale, "w_v_scale", Nv, K, 128, 128)
    lat, lsc = _fp8_cache_buffers(desc, buffer_length, k_latent_buffer, k_latent_scales)
    kout = _buf(k_buffer, "k_buffer", buffer_length * N * 2, (torch.bfloat16,))
    vout = _buf(v_buffer, "v_buffer", buffer_length * Nv * 2, (torch.bfloat16,))
    bro, co = _index_args(buffer_row_offsets, cache_offsets, desc)
    _gpu(buffer_row_offsets=buffer_row_offsets, cache_offsets=cache_offsets, w_k_e4m3=w_k_e4m3,
         w_k_scale=w_k_scale, w_v_e4m3=w_v_e4m3, w_v_scale=w_v_scale, k_latent_buffer=k_latent_buffer,
         k_latent_scales=k_latent_scales, k_buffer=k_buffer, v_buffer=v_buffer, cache=cache)
    st = lib().mla_decompress_kv_paged_fp8_cache(bro, co, int(buffer_length), wk, sk, N, wv, sv, Nv, K,
                                                 ctypes.byref(desc), ctypes.byref(sdesc), int(layer_idx),
                                                 lat, lsc, kout, vout, _stream(stream))
    _check(st, "mla_decompress_kv_paged_fp8_cache")


def _absorb_shapes(q, w, name, d_nope, copy_rope, q_latent):
    import torch
    if q is None or q.dim() != 3:
        raise ValueError("q must be a [T, H, d_nope + d_rope] tensor")
    if w is None or w.dim() != 3:
        raise ValueError(f"{name} must be a [H, kv_latent_dim, d_nope] tensor")
    T, H, Dq = q.shape
    if w.shape[0] != H or w.shape[2] != d_nope:
        raise ValueError(f"{name} must be [{H}, kv_latent_dim, {d_nope}]")
    L = w.shape[1]
    d_rope = Dq - d_nope
    Do = L + (d_rope if copy_rope else 0)
    if q_latent is None or tuple(q_latent.shape) != (T, H, Do):
        raise ValueError(f"q_latent must be a [{T}, {H}, {Do}] tensor")
    qp = _buf(q, "q", T * H * Dq * 2, (torch.bfloat16,))
    op = _buf(q_latent, "q_latent", T * H * Do * 2, (torch.bfloat16,))
    return T, H, L, d_rope, qp, op


def mla_absorb_q(q, w_uk, q_latent, d_nope: int = 128, copy_rope: bool = True, stream=None) -> None:
    """q_latent[t, h, :L] = q[t, h, :d_nope] @ w_uk[h].T per head (L = kv_latent_dim),
    then, with copy_rope, the rope columns q[t, h, d_nope:] after it."""
    import torch
    T, H, L, d_rope, qp, op = _absorb_shapes(q, w_uk, "w_uk", d_nope, copy_rope, q_latent)
    wp = _buf(w_uk, "w_uk", H * L * d_nope * 2, (torch.bfloat16,))
    _gpu(q=q, w_uk=w_uk, q_latent=q_latent)
    st = lib().mla_absorb_q(qp, T, H, int(d_nope), int(d_rope), wp, int(L), 1 if copy_rope else 0, op,
                            _stream(stream))
    _check(st, "mla_absorb_q")


def mla_absorb_q_fp8(q, w_uk_e4m3, w_uk_scale, q_latent, d_nope: int = 128, copy_rope: bool = True,
                     stream=None) -> None:
    """The fp8 form: each head's non-rope query part quantised per 1x128 block,
    times the e4m3 w_uk with its 128x128 block scales."""
    T, H, L, d_rope, qp, op = _absorb_shapes(q, w_uk_e4m3, "w_uk_e4m3", d_nope, copy_rope, q_latent)
    wp = _buf(w_uk_e4m3, "w_uk_e4m3", H * L * d_nope, _dtypes()[MLA_DTYPE_F8E4M3FN])
    sp = _f32(w_uk_scale, "w_uk_scale", H * (-(-L // 128)) * (-(-d_nope // 128)))
    _gpu(q=q, w_uk_e4m3=w_uk_e4m3, w_uk_scale=w_uk_scale, q_latent=q_latent)
    st = lib().mla_absorb_q_fp8(qp, T, H, int(d_nope), int(d_rope), wp, sp, int(L), 1, 128, 128,
                                1 if copy_rope else 0, op, _stream(stream))
    _check(st, "mla_absorb_q_fp8")


def _latent_write_args(kv_input, input_row_offsets, kv_norm_gamma, freqs_cis, K, desc):
    import torch
    if kv_input is None or kv_input.dim() != 2:
        raise ValueError("kv_input must be a [T, D_c] tensor")
    T, D = kv_input.shape
    if D != desc.num_heads * desc.head_dim:
        raise ValueError("kv_input rows must be as wide as the cache rows")
    x = _buf(kv_input, "kv_input", T * D * 2, (torch.bfloat16,))
    g = _f32(kv_norm_gamma, "kv_norm_gamma", int(K))
    if freqs_cis is not None:
        if freqs_cis.dim() != 2:
            raise ValueError("freqs_cis must be a [max_seq_len, qk_rope_head_dim] tensor")
        fr = _f32(freqs_cis, "freqs_cis", freqs_cis.shape[0] * freqs_cis.shape[1])
        max_seq = freqs_cis.shape[0]
    else:
        fr, max_seq = None, 0
    iro = _u32(input_row_offsets, "input_row_offsets", desc.batch_size + 1)
    return T, x, iro, g, fr, max_seq


def mla_write_latent_paged(kv_input, input_row_offsets, kv_norm_gamma, epsilon: float, freqs_cis, K: int,
                           cache: PagedKVCache, layer_idx: int, stream=None) -> None:
    """Append new tokens' rows (RMSNorm of the first K columns with kv_norm_gamma,
    the rest rotated by freqs_cis at each token's position) into the cache pages."""
    desc = _cache_desc(cache)
    T, x, iro, g, fr, max_seq = _latent_write_args(kv_input, input_row_offsets, kv_norm_gamma, freqs_cis, K, desc)
    _gpu(kv_input=kv_input, input_row_offsets=input_row_offsets, kv_norm_gamma=kv_norm_gamma,
         freqs_cis=freqs_cis, cache=cache)
    st = lib().mla_write_latent_paged(x, iro, T, g, float(epsilon), fr, int(max_seq), int(K), ctypes.byref(desc),
                                      int(layer_idx), _stream(stream))
    _check(st, "mla_write_latent_paged")


def mla_write_latent_paged_fp8(kv_input, input_row_offsets, kv_norm_gamma, epsilon: float, freqs_cis, K: int,
                               cache: PagedKVCache, layer_idx: int, stream=None) -> None:
    """mla_write_latent_paged into an e4m3 cache: the same fp32 rows, quantised
    per 128 columns (codes into the pool, fp32 scales into the cache's scale pool)."""
    desc, sdesc = _cache_desc(cache, scales=True)
    T, x, iro, g, fr, max_seq = _latent_write_args(kv_input, input_row_offsets, kv_norm_gamma, freqs_cis, K, desc)
    _gpu(kv_input=kv_input, input_row_offsets=input_row_offsets, kv_norm_gamma=kv_norm_gamma,
         freqs_cis=freqs_cis, cache=cache)
    st = lib().mla_write_latent_paged_fp8(x, iro, T, g, float(epsilon), fr, int(max_seq), int(K),
                                          ctypes.byref(desc), ctypes.byref(sdesc), int(layer_idx), _stream(stream))
    _check(st, "mla_write_latent_paged_fp8")


def kv_matmul_paged(hidden_state, input_row_offsets, weight, cache: PagedKVCache, layer_idx: int,
                    stream=None) -> None:
    """Append bf16(hidden_state @ weight) as K ([:HD]) and V ([HD:]) rows into the cache pages."""
    import torch
    if hidden_state is None or hidden_state.dim() != 2:
        raise ValueError("hidden_state must be a [T, hidden] tensor")
    T, Kd = hidden_state.shape
    desc = _cache_desc(cache)
    hd = desc.num_heads * desc.head_dim
    if weight is None or tuple(weight.shape) != (Kd, 2 * hd):
        raise ValueError(f"weight must be a [{Kd}, {2 * hd}] tensor")
    h = _buf(hidden_state, "hidden_state", T * Kd * 2, (torch.bfloat16,))
    w = _buf(weight, "weight", Kd * 2 * hd * 2, (torch.bfloat16,))
    if input_row_offsets.numel() != desc.batch_size + 1:
        raise ValueError("input_row_offsets must have batch_size + 1 entries")
    iro = _u32(input_row_offsets, "input_row_offsets", desc.batch_size + 1)
    _gpu(hidden_state=hidden_state, input_row_offsets=input_row_offsets, weight=weight, cache=cache)
    st = lib().kv_matmul_paged(h, iro, T, Kd, w, ctypes.byref(desc), int(layer_idx), _stream(stream))
    _check(st, "kv_matmul_paged")


def _rope_layout(layout):
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {', '.join(ROPE_LAYOUTS)}, not {layout!r}")
    return ROPE_LAYOUTS[layout]


def mla_rope_freqs(freqs_cis, theta: float = 10000.0, first_position: int = 0, scaling: str = "none",
                   factor: float = 1.0, original_max_position: int = 0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0, amplitude: float = 1.0, stream=None) -> None:
    """Fill freqs_cis[i] (a contiguous float32 [rows, d_rope] tensor) with amplitude * (cos, sin)
    of (first_position + i) times each pair's frequency, scaled "none", "linear" or "by_parts"."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}, not {scaling!r}")
    if freqs_cis is None or freqs_cis.dim() != 2:
        raise ValueError("freqs_cis must be a [rows, d_rope] tensor")
    for value, name in ((first_position, "first_position"), (original_max_position, "original_max_position")):
        if not -2 ** 31 <= value < 2 ** 31:     # (other bits would be cut off)
            raise ValueError(f"{name} must fit 32 bits, not {value}")
    rows, R = freqs_cis.shape
    fr = _f32(freqs_cis, "freqs_cis", rows * R)
    p = RopeParams(float(theta), float(factor), float(beta_fast), float(beta_slow), float(amplitude),
                   ROPE_SCALINGS[scaling], int(original_max_position))
    _gpu(freqs_cis=freqs_cis)
    st = lib().mla_rope_freqs(ctypes.byref(p), int(first_position), rows, R, fr, _stream(stream))
    _check(st, "mla_rope_freqs")


def _freqs(freqs_cis):
    if freqs_cis is None or freqs_cis.dim() != 2:
        raise ValueError("freqs_cis must be a [max_seq_len, qk_rope_head_dim] tensor")
    return _f32(freqs_cis, "freqs_cis", freqs_cis.shape[0] * freqs_cis.shape[1])


def mla_rope_q(q, positions, freqs_cis, q_out, d_nope: int = 128, layout: str = "interleaved", stream=None) -> None:
    """q_out[t, h] = q[t, h] with the columns from d_nope on rotated by freqs_cis[positions[t]].
    q and q_out are [T, H, d_nope + d_rope] bfloat16 or float32 tensors with unit column stride;
    passing q itself as q_out rotates in place."""
    import torch
    for t, name in ((q, "q"), (q_out, "q_out")):
        if t is None or t.dim() != 3 or t.stride(2) != 1:
            raise ValueError(f"{name} must be a [T, H, d_nope + d_rope] tensor with unit column stride")
    if q.dtype not in (torch.bfloat16, torch.float32) or q_out.dtype != q.dtype:
        raise ValueError("q and q_out must share a dtype, bfloat16 or float32")
    if q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    T, H, D = q.shape
    lay = _rope_layout(layout)
    fr = _freqs(freqs_cis)
    if freqs_cis.shape[1] != D - d_nope:
        raise ValueError("freqs_cis must be as wide as the rope part of q")
    pos = _u32(positions, "positions", T)
    _gpu(q=q, positions=positions, freqs_cis=freqs_cis, q_out=q_out)
    dt = MLA_DTYPE_F32 if q.dtype == torch.float32 else MLA_DTYPE_BF16

    def strides(t):   # the stride of a dimension of size 1 says nothing
        head = t.stride(1) if H > 1 else D
        return (t.stride(0) if T > 1 else H * head), head
    st = lib().mla_rope_q(q.data_ptr(), *strides(q), T, H, int(d_nope), D - int(d_nope), dt, pos, fr,
                          freqs_cis.shape[0], lay, q_out.data_ptr(), *strides(q_out), _stream(stream))
    _check(st, "mla_rope_q")


def mla_write_latent_paged_at(kv_input, input_row_offsets, positions, kv_norm_gamma, epsilon: float, freqs_cis,
                              K: int, cache: PagedKVCache, layer_idx: int, layout: str = "interleaved",
                              stream=None) -> None:
    """mla_write_latent_paged with the rope position of each token given (drafted tokens:
    their depth in the tree) and either layout of the rope columns."""
    desc = _cache_desc(cache)
    T, x, iro, g, fr, max_seq = _latent_write_args(kv_input, input_row_offsets, kv_norm_gamma, freqs_cis, K, desc)
    pos = _u32(positions, "positions", T)
    lay = _rope_layout(layout)
    _gpu(kv_input=kv_input, input_row_offsets=input_row_offsets, positions=positions, kv_norm_gamma=kv_norm_gamma,
         freqs_cis=freqs_cis, cache=cache)
    st = lib().mla_write_latent_paged_at(x, iro, T, pos, g, float(epsilon), fr, int(max_seq), int(K), lay,
                                         ctypes.byref(desc), int(layer_idx), _stream(stream))
    _check(st, "mla_write_latent_paged_at")


def mla_write_latent_paged_fp8_at(kv_input, input_row_offsets, positions, kv_norm_gamma, epsilon: float, freqs_cis,
                                  K: int, cache: PagedKVCache, layer_idx: int, layout: str = "interleaved",
                                  stream=None) -> None:
    """mla_write_latent_paged_at into an e4m3 cache."""
    desc, sdesc = _cache_desc(cache, scales=True)
    T, x, iro, g, fr, max_seq = _latent_write_args(kv_input, input_row_offsets, kv_norm_gamma, freqs_cis, K, desc)
    pos = _u32(positions, "positions", T)
    lay = _rope_layout(layout)
    _gpu(kv_input=kv_input, input_row_offsets=input_row_offsets, positions=positions, kv_norm_gamma=kv_norm_gamma,
         freqs_cis=freqs_cis, cache=cache)
    st = lib().mla_write_latent_paged_fp8_at(x, iro, T, pos, g, float(epsilon), fr, int(max_seq), int(K), lay,
                                             ctypes.byref(desc), ctypes.byref(sdesc), int(layer_idx),
                                             _stream(stream))
    _check(st, "mla_write_latent_paged_fp8_at")


def mla_tree_attention_workspace_size(total_tokens: int, num_heads: int, K: int = 512) -> int:
    return int(lib().mla_tree_attention_workspace_size(int(total_tokens), int(num_heads), int(K)))


def _attention_args(q_latent, input_row_offsets, tree_mask, K, desc, out_latent, lse, dtype):
    import torch
    if q_latent is None or q_latent.dim() != 3:
        raise ValueError("q_latent must be a [T, H, D_c] tensor")
    T, H, D = q_latent.shape
    if D != desc.num_heads * desc.head_dim:
        raise ValueError("q_latent rows must be as wide as the cache rows")
    eb = 4 if dtype == torch.float32 else 2
    q = _buf(q_latent, "q_latent", T * H * D * eb, (dtype,))
    if out_latent is None or tuple(out_latent.shape) != (T, H, K):
        raise ValueError(f"out_latent must be a [{T}, {H}, {K}] tensor")
    out = _buf(out_latent, "out_latent", T * H * K * eb, (dtype,))
    iro = _u32(input_row_offsets, "input_row_offsets", desc.batch_size + 1)
    mask, words = None, 0
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != T or tree_mask.dtype not in (torch.int64, torch.uint64):
            raise ValueError(f"tree_mask must be a 64-bit integer [{T}, mask_words] tensor")
        words = tree_mask.shape[1]
        mask = _buf(tree_mask, "tree_mask", T * words * 8)
    ls = None
    if lse is not None:
        if tuple(lse.shape) != (T, H):
            raise ValueError(f"lse must be a [{T}, {H}] tensor")
        ls = _f32(lse, "lse", T * H)
    return T, H, q, iro, mask, words, out, ls


def mla_tree_attention_paged(q_latent, input_row_offsets, tree_mask, scale: float, K: int, cache: PagedKVCache,
                             layer_idx: int, out_latent, workspace, lse=None, stream=None) -> None:
    """out_latent[t, h] = softmax(scale * q_latent[t, h] . rows) rows[:, :K] over the cached rows of the
    token's request and the drafted rows behind them that tree_mask (64-bit words per token; None: the
    tokens up to itself) names.  lse: optional float32 [T, H].  ``workspace``: a device tensor of at
    least mla_tree_attention_workspace_size(T, H, K) bytes."""
    import torch
    desc = _cache_desc(cache)
    dtype = torch.float32 if desc.dtype == MLA_DTYPE_F32 else torch.bfloat16
    T, H, q, iro, mask, words, out, ls = _attention_args(q_latent, input_row_offsets, tree_mask, K, desc, out_latent,
                                                         lse, dtype)
    ws, ws_bytes = _workspace(workspace)
    _gpu(q_latent=q_latent, input_row_offsets=input_row_offsets, tree_mask=tree_mask, out_latent=out_latent, lse=lse,
         workspace=workspace, cache=cache)
    st = lib().mla_tree_attention_paged(q, iro, T, H, mask, words, float(scale), int(K), ctypes.byref(desc),
                                        int(layer_idx), out, ls, ws, ws_bytes, _stream(stream))
    _check(st, "mla_tree_attention_paged")


def mla_tree_attention_paged_fp8_cache(q_latent, input_row_offsets, tree_mask, scale: float, K: int,
                                       cache: PagedKVCache, layer_idx: int, out_latent, workspace, lse=None,
                                       stream=None) -> None:
    """mla_tree_attention_paged over an e4m3 cache (codes times their block scales)."""
    import torch
    desc, sdesc = _cache_desc(cache, scales=True)
    T, H, q, iro, mask, words, out, ls = _attention_args(q_latent, input_row_offsets, tree_mask, K, desc, out_latent,
                                                         lse, torch.bfloat16)
    ws, ws_bytes = _workspace(workspace)
    _gpu(q_latent=q_latent, input_row_offsets=input_row_offsets, tree_mask=tree_mask, out_latent=out_latent, lse=lse,
         workspace=workspace, cache=cache)
    st = lib().mla_tree_attention_paged_fp8_cache(q, iro, T, H, mask, words, float(scale), int(K), ctypes.byref(desc),
                                                  ctypes.byref(sdesc), int(layer_idx), out, ls, ws, ws_bytes,
                                                  _stream(stream))
    _check(st, "mla_tree_attention_paged_fp8_cache")


def _page_descs(cache):
    """The cache's descriptor, and the scale pool's where it has one."""
    if cache.scales is None:
        return _cache_desc(cache), None
    desc, sdesc = _cache_desc(cache, scales=True)
    return desc, ctypes.byref(sdesc)


def mla_copy_pages(src_pages, dst_pages, cache: PagedKVCache, stream=None) -> None:
    """Page dst_pages[i] becomes a copy of page src_pages[i], in every layer."""
    desc, sdesc = _page_descs(cache)
    n = src_pages.numel()
    if dst_pages.numel() != n:
        raise ValueError("src_pages and dst_pages must have the same number of entries")
    src, dst = _u32(src_pages, "src_pages"), _u32(dst_pages, "dst_pages")
    _gpu(src_pages=src_pages, dst_pages=dst_pages, cache=cache)
    st = lib().mla_copy_pages(src, dst, n, ctypes.byref(desc), sdesc, _stream(stream))
    _check(st, "mla_copy_pages")


def mla_fork_paged(parents, children, new_pages, ref_counts, cache: PagedKVCache, stream=None) -> None:
    """Request children[i] becomes a copy of request parents[i]: whole pages shared (ref_counts + 1),
    the partly filled last page copied to new_pages[i]; writes the page table and the lengths."""
    desc, sdesc = _page_descs(cache)
    n = parents.numel()
    if children.numel() != n or new_pages.numel() != n:
        raise ValueError("parents, children and new_pages must have the same number of entries")
    pa, ch, pg = _u32(parents, "parents"), _u32(children, "children"), _u32(new_pages, "new_pages")
    refs = _u32(ref_counts, "ref_counts", desc.num_pages)
    _gpu(parents=parents, children=children, new_pages=new_pages, ref_counts=ref_counts, cache=cache)
    st = lib().mla_fork_paged(pa, ch, pg, n, refs, ctypes.byref(desc), sdesc, _stream(stream))
    _check(st, "mla_fork_paged")


def mla_free_paged(requests, ref_counts, free_list, free_count, cache: PagedKVCache, stream=None) -> None:
    """Drop the listed requests' references; pages left without any are appended to free_list at
    free_count[0] in ascending order.  Writes the page table and the lengths."""
    desc, _ = _page_descs(cache)
    req = _u32(requests, "requests")
    refs = _u32(ref_counts, "ref_counts", desc.num_pages)
    fl, fc = _u32(free_list, "free_list", desc.num_pages), _u32(free_count, "free_count", 1)
    _gpu(requests=requests, ref_counts=ref_counts, free_list=free_list, free_count=free_count,
         cache=cache)
    st = lib().mla_free_paged(req, requests.numel(), refs, fl, fc, ctypes.byref(desc), _stream(stream))
    _check(st, "mla_free_paged")


def mla_compact_paged(accepted, accepted_offsets, cache: PagedKVCache, stream=None) -> None:
    """Move the rows of each request's accepted drafted tokens (ascending positions in its draft)
    together behind its cached rows, in every layer.  The lengths are not updated."""
    desc, sdesc = _page_descs(cache)
    acc = _u32(accepted, "accepted")
    off = _u32(accepted_offsets, "accepted_offsets", desc.batch_size + 1)
    _gpu(accepted=accepted, accepted_offsets=accepted_offsets, cache=cache)
    st = lib().mla_compact_paged(acc, off, accepted.numel(), ctypes.byref(desc), sdesc, _stream(stream))
    _check(st, "mla_compact_paged")


def status_string(status: int) -> str:
    return lib().mla_status_string(int(status)).decode()


def abi_version() -> int:
    return int(lib().mla_abi_version())
