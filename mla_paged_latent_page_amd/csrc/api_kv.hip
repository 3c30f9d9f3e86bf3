// C ABI of the paged K/V cache's operators (include/mla_paged.h): writes, reads, attention.
// Host-side validation in the documented order, then one launcher of kv.hpp.
#include <cmath>

#include "api_checks.hpp"
#include "kv.hpp"

using namespace mla;

namespace {

constexpr int64_t k2G = int64_t(1) << 31;
constexpr int64_t kMostWidth = int64_t(1) << 20;   // columns of a token row

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

PagedLayer scales_view(const mla_paged_cache_t* cache, const mla_cache_scales_t* sc, uint32_t layer)
{
    PagedLayer L = layer_view(cache, layer);
    L.base = reinterpret_cast<const char*>(sc->scales + (int64_t)layer * sc->stride_layer);
    L.stride_page = sc->stride_page * 4;
    L.stride_token = sc->stride_token * 4;
    L.stride_kv = sc->stride_kv * 4;
    return L;
}

bool scales_shape_ok(const mla_cache_scales_t* sc, int64_t HD)
{
    const int64_t nblk = (HD + 127) / 128;
    return sc->granularity == 128 && sc->stride_token >= nblk && sc->stride_page > 0 && sc->stride_layer >= 0 &&
           sc->stride_kv >= nblk;
}

mla_status_t kv_write(const void* k, const void* v, int64_t k_stride_token, int64_t v_stride_token,
                      const uint32_t* input_row_offsets, int32_t total_tokens, const uint32_t* positions,
                      const float* freqs_cis, int32_t max_seq_len, int32_t d_rope, int32_t rope_layout,
                      const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales, bool fp8,
                      uint32_t layer_idx, void* stream)
{
    if (!cache || (fp8 && !cache_scales))
        return MLA_ERR_NULL_POINTER;
    const int32_t T = total_tokens;
    const bool work = T > 0;
    if (work && (!k || !v || !input_row_offsets || !cache->blocks || !cache->page_table || !cache->cache_lengths ||
                 (fp8 && !cache_scales->scales) || (d_rope > 0 && !freqs_cis)))
        return MLA_ERR_NULL_POINTER;
    if (mla_status_t st = check_cache_shape(cache, 2))
        return st;
    const int64_t HD = (int64_t)cache->num_heads * cache->head_dim;
    if (T < 0 || cache->head_dim % 8 || HD > kMostWidth || d_rope < 0 || d_rope > (int64_t)cache->head_dim ||
        d_rope % 8 || (d_rope > 0 && max_seq_len <= 0) ||
        (rope_layout != MLA_ROPE_INTERLEAVED && rope_layout != MLA_ROPE_HALF) ||
        (rope_layout == MLA_ROPE_HALF && d_rope % 16) || k_stride_token < 0 || v_stride_token < 0 ||
        (T > 1 && (k_stride_token < HD || v_stride_token < HD)) ||
        (fp8 && !scales_shape_ok(cache_scales, HD)))
        return MLA_ERR_INVALID_SHAPE;
    if (cache->dtype != (fp8 ? MLA_DTYPE_F8E4M3FN : MLA_DTYPE_BF16))
        return MLA_ERR_INVALID_DTYPE;
    if (!aligned16(k) || !aligned16(v) || k_stride_token % 8 || v_stride_token % 8 || !aligned16(freqs_cis) ||
        !aligned4(positions) || (fp8 && !aligned4(cache_scales->scales)))
        return MLA_ERR_MISALIGNED;
    if (mla_status_t st = check_cache_alignment(cache))
        return st;
    if (layer_idx >= cache->num_layers)
        return MLA_ERR_OUT_OF_RANGE;
    if (!work)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    KvWriteArgs a{};
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.k_st = k_stride_token * 2;
    a.v_st = v_stride_token * 2;
    a.iro = input_row_offsets;
    a.cache_len = cache->cache_lengths;
    a.pos = positions;
    a.freqs = freqs_cis;
    a.L = layer_view(cache, layer_idx);
    if (fp8)
        a.Ls = scales_view(cache, cache_scales, layer_idx);
    a.T = T;
    a.HD = (int)HD;
    a.D = (int)cache->head_dim;
    a.R = d_rope;
    a.max_seq = d_rope > 0 ? max_seq_len : 1;
    const hipError_t e = launch_kv_write(a, fp8, rope_layout == MLA_ROPE_HALF, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

mla_status_t kv_gather(const uint32_t* buffer_row_offsets, const uint32_t* cache_offsets, int32_t buffer_length,
                       const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales, bool fp8,
                       uint32_t layer_idx, void* k_buffer, void* v_buffer, void* stream)
{
    if (!cache || (fp8 && !cache_scales))
        return MLA_ERR_NULL_POINTER;
    const int32_t M = buffer_length;
    const bool work = M > 0;
    if (work && (!buffer_row_offsets || !cache_offsets || !k_buffer || !v_buffer || !cache->blocks ||
                 !cache->page_table || (fp8 && !cache_scales->scales)))
        return MLA_ERR_NULL_POINTER;
    if (mla_status_t st = check_cache_shape(cache, 2))
        return st;
    const int64_t HD = (int64_t)cache->num_heads * cache->head_dim;
    if (M < 0 || HD > kMostWidth || (fp8 && !scales_shape_ok(cache_scales, HD)))
        return MLA_ERR_INVALID_SHAPE;
    if (fp8 ? cache->dtype != MLA_DTYPE_F8E4M3FN : cache->dtype != MLA_DTYPE_BF16 && cache->dtype != MLA_DTYPE_F32)
        return MLA_ERR_INVALID_DTYPE;
    if (!aligned16(k_buffer) || !aligned16(v_buffer) || (fp8 && !aligned4(cache_scales->scales)))
        return MLA_ERR_MISALIGNED;
    if (mla_status_t st = check_cache_alignment(cache))
        return st;
    if (layer_idx >= cache->num_layers)
        return MLA_ERR_OUT_OF_RANGE;
    if (!work)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    KvGatherArgs a{};
    a.bro = buffer_row_offsets;
    a.co = cache_offsets;
    a.L = layer_view(cache, layer_idx);
    if (fp8)
        a.Ls = scales_view(cache, cache_scales, layer_idx);
    a.k = static_cast<char*>(k_buffer);
    a.v = static_cast<char*>(v_buffer);
    a.M = M;
    a.HD = (int)HD;
    const KvKind kind = fp8 ? KV_E4M3 : cache->dtype == MLA_DTYPE_F32 ? KV_F32 : KV_BF16;
    const hipError_t e = launch_kv_gather(a, kind, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

mla_status_t kv_attention(const void* q, int64_t q_stride_token, const uint32_t* input_row_offsets,
                          int32_t total_tokens, int32_t num_heads, float scale, int32_t window, int32_t sinks,
                          const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales, bool fp8,
                          uint32_t layer_idx, void* out, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream)
{
    if (!cache || (fp8 && !cache_scales))
        return MLA_ERR_NULL_POINTER;
    const int32_t T = total_tokens;
    const bool work = T > 0;
    if (work && (!q || !input_row_offsets || !out || !workspace || !cache->blocks || !cache->page_table ||
                 !cache->cache_lengths || (fp8 && !cache_scales->scales)))
        return MLA_ERR_NULL_POINTER;
    if (mla_status_t st = check_cache_shape(cache, 2))
        return st;
    const int64_t KH = cache->num_heads, D = cache->head_dim, HD = (int64_t)num_heads * D;
    if (T < 0 || num_heads <= 0 || num_heads % KH || D % 8 || D > 256 || !(std::fabs(scale) < 0x1p127f) || window < 0 ||
        sinks < 0 || (int64_t)T * num_heads >= k2G - 65536 || (T > 1 && q_stride_token < HD) || q_stride_token < 0 ||
        (int64_t)cache->max_pages_per_seq * cache->page_size >= k2G || (fp8 && !scales_shape_ok(cache_scales, KH * D)))
        return MLA_ERR_INVALID_SHAPE;
    if (fp8 ? cache->dtype != MLA_DTYPE_F8E4M3FN : cache->dtype != MLA_DTYPE_BF16 && cache->dtype != MLA_DTYPE_F32)
        return MLA_ERR_INVALID_DTYPE;
    const int eb = cache->dtype == MLA_DTYPE_F32 ? 4 : 2;
    if (!aligned16(q) || (q_stride_token * eb) % 16 || !aligned16(out) || !aligned4(lse) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) || (fp8 && !aligned4(cache_scales->scales)))
        return MLA_ERR_MISALIGNED;
    if (mla_status_t st = check_cache_alignment(cache))
        return st;
    if (layer_idx >= cache->num_layers)
        return MLA_ERR_OUT_OF_RANGE;
    if (work && workspace_bytes < kv_attention_workspace_size(T, num_heads, (int32_t)KH, (int32_t)D))
        return MLA_ERR_WORKSPACE;
    if (!work)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    KvAttentionArgs a{};
    a.q = static_cast<const char*>(q);
    a.q_st = q_stride_token * eb;
    a.iro = input_row_offsets;
    a.cache_len = cache->cache_lengths;
    a.out = out;
    a.lse = lse;
    a.ws = static_cast<float*>(workspace);
    a.L = layer_view(cache, layer_idx);
    if (fp8)
        a.Ls = scales_view(cache, cache_scales, layer_idx);
    a.scale = scale;
    a.T = T;
    a.H = num_heads;
    a.KH = (int)KH;
    a.D = (int)D;
    a.window = (uint32_t)window;
    a.sinks = (uint32_t)sinks;
    a.capacity = cache->max_pages_per_seq * cache->page_size;
    const KvKind kind = fp8 ? KV_E4M3 : cache->dtype == MLA_DTYPE_F32 ? KV_F32 : KV_BF16;
    const hipError_t e = launch_kv_attention(a, kind, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

}  // namespace

MLA_API mla_status_t kv_write_paged(const void* k, const void* v, int64_t k_stride_token, int64_t v_stride_token,
                                    const uint32_t* input_row_offsets, int32_t total_tokens,
                                    const uint32_t* positions, const float* freqs_cis, int32_t max_seq_len,
                                    int32_t d_rope, int32_t rope_layout, const mla_paged_cache_t* cache,
                                    uint32_t layer_idx, void* stream)
{
    return kv_write(k, v, k_stride_token, v_stride_token, input_row_offsets, total_tokens, positions, freqs_cis,
                    max_seq_len, d_rope, rope_layout, cache, nullptr, false, layer_idx, stream);
}

MLA_API mla_status_t kv_write_paged_fp8(const void* k, const void* v, int64_t k_stride_token, int64_t v_stride_token,
                                        const uint32_t* input_row_offsets, int32_t total_tokens,
                                        const uint32_t* positions, const float* freqs_cis, int32_t max_seq_len,
                                        int32_t d_rope, int32_t rope_layout, const mla_paged_cache_t* cache,
                                        const mla_cache_scales_t* cache_scales, uint32_t layer_idx, void* stream)
{
    return kv_write(k, v, k_stride_token, v_stride_token, input_row_offsets, total_tokens, positions, freqs_cis,
                    max_seq_len, d_rope, rope_layout, cache, cache_scales, true, layer_idx, stream);
}

MLA_API mla_status_t kv_gather_paged(const uint32_t* buffer_row_offsets, const uint32_t* cache_offsets,
                                     int32_t buffer_length, const mla_paged_cache_t* cache, uint32_t layer_idx,
                                     void* k_buffer, void* v_buffer, void* stream)
{
    return kv_gather(buffer_row_offsets, cache_offsets, buffer_length, cache, nullptr, false, layer_idx, k_buffer,
                     v_buffer, stream);
}

MLA_API mla_status_t kv_gather_paged_fp8_cache(const uint32_t* buffer_row_offsets, const uint32_t* cache_offsets,
                                               int32_t buffer_length, const mla_paged_cache_t* cache,
                                               const mla_cache_scales_t* cache_scales, uint32_t layer_idx,
                                               void* k_buffer, void* v_buffer, void* stream)
{
    return kv_gather(buffer_row_offsets, cache_offsets, buffer_length, cache, cache_scales, true, layer_idx, k_buffer,
                     v_buffer, stream);
}

MLA_API size_t kv_attention_workspace_size(int32_t total_tokens, int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim)
{
    if (total_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        head_dim > 256)
        return 0;
    const size_t piece = (size_t)kv_attention_row_groups(total_tokens, num_heads / num_kv_heads) * 32 * (head_dim + 2);
    return align256(2 * kKvGroups * piece * sizeof(float) + (kKvGroups + 1) * sizeof(KvCut));
}

MLA_API mla_status_t kv_attention_paged(const void* q, int64_t q_stride_token, const uint32_t* input_row_offsets,
                                        int32_t total_tokens, int32_t num_heads, float scale, int32_t window,
                                        int32_t sinks, const mla_paged_cache_t* cache, uint32_t layer_idx, void* out,
                                        float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    return kv_attention(q, q_stride_token, input_row_offsets, total_tokens, num_heads, scale, window, sinks, cache,
                        nullptr, false, layer_idx, out, lse, workspace, workspace_bytes, stream);
}

MLA_API mla_status_t kv_attention_paged_fp8_cache(const void* q, int64_t q_stride_token,
                                                  const uint32_t* input_row_offsets, int32_t total_tokens,
                                                  int32_t num_heads, float scale, int32_t window, int32_t sinks,
                                                  const mla_paged_cache_t* cache,
                                                  const mla_cache_scales_t* cache_scales, uint32_t layer_idx,
                                                  void* out, float* lse, void* workspace, size_t workspace_bytes,
                                                  void* stream)
{
    return kv_attention(q, q_stride_token, input_row_offsets, total_tokens, num_heads, scale, window, sinks, cache,
                        cache_scales, true, layer_idx, out, lse, workspace, workspace_bytes, stream);
}
