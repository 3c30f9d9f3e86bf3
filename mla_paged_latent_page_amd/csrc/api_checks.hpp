// Host-side argument checks shared by the C ABI's entry points.
#pragma once

#include <atomic>
#include <cstring>

#include "mla_paged.h"
#include "launch.hpp"

#define MLA_API extern "C" __attribute__((visibility("default")))

namespace mla {

inline thread_local int32_t g_last_hip_error = 0;

inline mla_status_t hip_failed(hipError_t e)
{
    g_last_hip_error = (int32_t)e;
    return MLA_ERR_HIP;
}

inline int elem_bytes(int32_t dtype)
{
    switch (dtype) {
    case MLA_DTYPE_F32: return 4;
    case MLA_DTYPE_BF16: return 2;
    case MLA_DTYPE_F8E4M3FN: return 1;
    default: return 0;
    }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device must be a gfx950; the answer is cached per device.
inline mla_status_t check_device()
{
    static std::atomic<int> verdict[64];  // 0 unknown, 1 gfx950, 2 other
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return MLA_ERR_UNSUPPORTED_DEVICE;
    if (dev < 64) {
        const int v = verdict[dev].load(std::memory_order_relaxed);
        if (v == 1)
            return MLA_OK;
        if (v == 2)
            return MLA_ERR_UNSUPPORTED_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return MLA_ERR_UNSUPPORTED_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64)
        verdict[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? MLA_OK : MLA_ERR_UNSUPPORTED_DEVICE;
}

// Checks of the cache descriptor shared by every call.  `row_check` holds
// the expected num_kv; `work` says whether device pointers must be present.
inline mla_status_t check_cache_shape(const mla_paged_cache_t* c, uint32_t num_kv)
{
    if (c->num_layers == 0 || c->num_pages == 0 || c->page_size == 0 || c->num_heads == 0 ||
        c->head_dim == 0 || c->batch_size == 0 || c->max_pages_per_seq == 0 || c->num_kv != num_kv)
        return MLA_ERR_INVALID_SHAPE;
    const int64_t row = (int64_t)c->num_heads * c->head_dim;
    if (c->stride_token < row || c->stride_page <= 0 || c->stride_layer < 0 || c->stride_kv < 0 ||
        (num_kv > 1 && c->stride_kv < row))
        return MLA_ERR_INVALID_SHAPE;
    return MLA_OK;
}

inline mla_status_t check_cache_alignment(const mla_paged_cache_t* c)
{
    const int eb = elem_bytes(c->dtype);
    if (!aligned16(c->blocks) || (c->stride_token * eb) % 16 || (c->stride_page * eb) % 16 ||
        (c->stride_layer * eb) % 16 || (c->stride_kv * eb) % 16 ||
        ((int64_t)c->num_heads * c->head_dim * eb) % 16)
        return MLA_ERR_MISALIGNED;
    return MLA_OK;
}

inline mla::PagedLayer layer_view(const mla_paged_cache_t* c, uint32_t layer)
{
    const int eb = elem_bytes(c->dtype);
    mla::PagedLayer L;
    L.base = static_cast<const char*>(c->blocks) + (int64_t)layer * c->stride_layer * eb;
    L.page_table = c->page_table;
    L.stride_page = c->stride_page * eb;
    L.stride_token = c->stride_token * eb;
    L.stride_kv = c->stride_kv * eb;
    L.num_pages = c->num_pages;
    L.page_size = c->page_size;
    L.max_pages = c->max_pages_per_seq;
    L.batch = c->batch_size;
    return L;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The product kernels address one 256-row tile of their operands and outputs
// through 32-bit byte offsets: a row of `width` elements of `eb` bytes times
// 256 rows must stay below 2^31 bytes.
inline bool tile_fits_32bit(int64_t width, int eb) { return width * eb * 256 < (int64_t(1) << 31); }

}  // namespace mla
