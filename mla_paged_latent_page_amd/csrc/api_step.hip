// C ABI of the speculative-decoding step (include/mla_paged.h): rotary positions,
// tree attention over the latent cache, page upkeep.  Host-side validation in the
// documented order, then one launcher of step.hpp.
#include <algorithm>
#include <cmath>

#include "api_checks.hpp"
#include "step.hpp"

using namespace mla;

namespace {

constexpr int64_t k2G = int64_t(1) << 31;
constexpr int32_t kMostPagePairs = int32_t(1) << 30;   // a launch's worth below 2^31, in ints

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

bool rope_layout_ok(int32_t layout) { return layout == MLA_ROPE_INTERLEAVED || layout == MLA_ROPE_HALF; }

PagedLayer scales_view(const mla_paged_cache_t* cache, const mla_cache_scales_t* sc, uint32_t layer)
{
    PagedLayer L = layer_view(cache, layer);
    L.base = reinterpret_cast<const char*>(sc->scales + (int64_t)layer * sc->stride_layer);
    L.stride_page = sc->stride_page * 4;
    L.stride_token = sc->stride_token * 4;
    L.stride_kv = sc->stride_kv * 4;
    return L;
}

bool scales_shape_ok(const mla_cache_scales_t* sc, int64_t D)
{
    return sc->granularity == 128 && sc->stride_token >= (D + 127) / 128 && sc->stride_page > 0 &&
           sc->stride_layer >= 0 && sc->stride_kv >= 0;
}

}  // namespace

MLA_API mla_status_t mla_rope_freqs(const mla_rope_params_t* params, int32_t first_position, int32_t rows,
                                    int32_t d_rope, float* freqs_cis, void* stream)
{
    if (!params || (rows > 0 && !freqs_cis))
        return MLA_ERR_NULL_POINTER;
    const mla_rope_params_t& p = *params;
    if (rows < 0 || first_position < 0 || (int64_t)first_position + rows > k2G || d_rope < 2 || d_rope % 2 ||
        d_rope > 2 * kMaxRopePairs || !std::isfinite(p.theta) || p.theta <= 0 || !std::isfinite(p.amplitude))
        return MLA_ERR_INVALID_SHAPE;
    const bool linear = p.scaling == MLA_ROPE_SCALING_LINEAR, parts = p.scaling == MLA_ROPE_SCALING_BY_PARTS;
    if (!linear && !parts && p.scaling != MLA_ROPE_SCALING_NONE)
        return MLA_ERR_INVALID_SHAPE;
    if ((linear || parts) && !(std::isfinite(p.factor) && p.factor > 0))
        return MLA_ERR_INVALID_SHAPE;
    if (parts && !(p.theta > 1 && p.original_max_position > 0 && std::isfinite(p.beta_fast) && p.beta_fast > 0 &&
                   std::isfinite(p.beta_slow) && p.beta_slow > 0))
        return MLA_ERR_INVALID_SHAPE;
    if (!aligned8(freqs_cis))
        return MLA_ERR_MISALIGNED;
    if (rows == 0)
        return MLA_OK;

    constexpr double kPi = 3.14159265358979323846;
    RopeFreqsArgs a{};
    a.out = freqs_cis;
    a.amplitude = p.amplitude;
    a.first = first_position;
    a.rows = rows;
    a.pairs = d_rope / 2;
    double low = 0, high = 0;
    if (parts) {
        auto pair = [&](double turns) {
            return d_rope * std::log(p.original_max_position / (2 * kPi * turns)) / (2 * std::log(p.theta));
        };
        low = std::fmax(std::floor(pair(p.beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair(p.beta_slow)), d_rope - 1.0);
    }
    for (int j = 0; j < a.pairs; ++j) {
        double f = std::pow(p.theta, -2.0 * j / d_rope);
        if (linear)
            f /= p.factor;
        if (parts) {
            const double r = std::fmin(std::fmax((j - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f / p.factor * r + f * (1 - r);
        }
        a.quarters[j] = f / (kPi / 2);
        // No angle of 2^50 quarter turns: two bits of it would be left.
        if (!(a.quarters[j] * ((double)first_position + (rows - 1)) < 0x1p50))
            return MLA_ERR_INVALID_SHAPE;
    }
    if (mla_status_t st = check_device())
        return st;
    const hipError_t e = launch_rope_freqs(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

MLA_API mla_status_t mla_rope_q(const void* q, int64_t q_stride_token, int64_t q_stride_head, int32_t total_tokens,
                                int32_t num_heads, int32_t d_nope, int32_t d_rope, int32_t dtype,
                                const uint32_t* positions, const float* freqs_cis, int32_t max_seq_len,
                                int32_t layout, void* q_out, int64_t out_stride_token, int64_t out_stride_head,
                                void* stream)
{
    const int32_t T = total_tokens;
    if (T > 0 && (!q || !positions || !freqs_cis || !q_out))
        return MLA_ERR_NULL_POINTER;
    const int64_t D = (int64_t)d_nope + d_rope;
    if (T < 0 || num_heads <= 0 || d_nope < 0 || d_nope > 4096 || d_rope < 8 || d_rope > 512 || d_rope % 8 ||
        max_seq_len <= 0 || !rope_layout_ok(layout) || (layout == MLA_ROPE_HALF && d_rope % 16) ||
        (int64_t)T * num_heads >= (int64_t(1) << 40) / D || q_stride_head < D || out_stride_head < D ||
        q_stride_token < 0 || out_stride_token < 0)
        return MLA_ERR_INVALID_SHAPE;
    // Heads of a token must not overlap those of the next (a stride of 0 is only
    // meaningful for one token); the output's rows are written, so theirs too.
    if (T > 1 && out_stride_token < D)
        return MLA_ERR_INVALID_SHAPE;
    if (dtype != MLA_DTYPE_BF16 && dtype != MLA_DTYPE_F32)
        return MLA_ERR_INVALID_DTYPE;
    const int eb = elem_bytes(dtype);
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(freqs_cis) || !aligned4(positions) ||
        (q_stride_token * eb) % 16 || (q_stride_head * eb) % 16 || (out_stride_token * eb) % 16 ||
        (out_stride_head * eb) % 16 || (d_nope * eb) % 16)
        return MLA_ERR_MISALIGNED;
    if (T == 0)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    RopeQArgs a{};
    a.q = static_cast<const char*>(q);
    a.out = static_cast<char*>(q_out);
    a.q_st = q_stride_token * eb;
    a.q_sh = q_stride_head * eb;
    a.o_st = out_stride_token * eb;
    a.o_sh = out_stride_head * eb;
    a.pos = positions;
    a.freqs = freqs_cis;
    a.T = T;
    a.H = num_heads;
    a.nope_bytes = d_nope * eb;
    a.R = d_rope;
    a.max_seq = max_seq_len;
    a.copy = !(q == q_out && a.q_st == a.o_st && a.q_sh == a.o_sh);
    const hipError_t e = launch_rope_q(a, dtype == MLA_DTYPE_F32, layout == MLA_ROPE_HALF,
                                       static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

namespace {

// Both _at writes; cache_scales is null for the bf16 cache.
mla_status_t latent_write_at(const void* kv_input, const uint32_t* input_row_offsets, int32_t total_tokens,
                             const uint32_t* positions, const float* kv_norm_gamma, float epsilon,
                             const float* freqs_cis, int32_t max_seq_len, int32_t K, int32_t rope_layout,
                             const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales, bool fp8,
                             uint32_t layer_idx, void* stream)
{
    if (!cache || (fp8 && !cache_scales))
        return MLA_ERR_NULL_POINTER;
    const bool work = total_tokens > 0;
    const int64_t D = (int64_t)cache->num_heads * cache->head_dim;
    const int64_t R = D - K;   // rope columns after the K latent ones
    if (work && (!kv_input || !input_row_offsets || !positions || !kv_norm_gamma || !cache->blocks ||
                 !cache->page_table || !cache->cache_lengths || (fp8 && !cache_scales->scales) || (R > 0 && !freqs_cis)))
        return MLA_ERR_NULL_POINTER;
    if (total_tokens < 0 || K <= 0 || K % (fp8 ? 128 : 8) || K > 512 || R < 0 || R % 8 || R > 512 ||
        (fp8 && D % 16) || (R > 0 && max_seq_len <= 0) || !(epsilon >= 0.0f) || !rope_layout_ok(rope_layout) ||
        (rope_layout == MLA_ROPE_HALF && R % 16) || (fp8 && !scales_shape_ok(cache_scales, D)))
        return MLA_ERR_INVALID_SHAPE;
    if (mla_status_t st = check_cache_shape(cache, 1))
        return st;
    if (cache->dtype != (fp8 ? MLA_DTYPE_F8E4M3FN : MLA_DTYPE_BF16))
        return MLA_ERR_INVALID_DTYPE;
    if (!aligned16(kv_input) || !aligned16(kv_norm_gamma) || !aligned16(freqs_cis) || !aligned4(positions) ||
        (fp8 && !aligned4(cache_scales->scales)))
        return MLA_ERR_MISALIGNED;
    if (mla_status_t st = check_cache_alignment(cache))
        return st;
    if (layer_idx >= cache->num_layers)
        return MLA_ERR_OUT_OF_RANGE;
    if (!work)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;

    LatentWriteAtArgs a{};
    a.X = static_cast<const uint16_t*>(kv_input);
    a.iro = input_row_offsets;
    a.cache_len = cache->cache_lengths;
    a.gamma = kv_norm_gamma;
    a.freqs = freqs_cis;
    a.eps = epsilon;
    a.L = layer_view(cache, layer_idx);
    if (fp8)
        a.Ls = scales_view(cache, cache_scales, layer_idx);
    a.T = total_tokens;
    a.K = K;
    a.R = (int)R;
    a.D = (int)D;
    a.max_seq = R > 0 ? max_seq_len : 1;
    a.pos = positions;
    a.half = rope_layout == MLA_ROPE_HALF;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = fp8 ? launch_latent_write_fp8_at(a, s) : launch_latent_write_at(a, s);
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

}  // namespace

MLA_API mla_status_t mla_write_latent_paged_at(const void* kv_input, const uint32_t* input_row_offsets,
                                               int32_t total_tokens, const uint32_t* positions,
                                               const float* kv_norm_gamma, float epsilon, const float* freqs_cis,
                                               int32_t max_seq_len, int32_t K, int32_t rope_layout,
                                               const mla_paged_cache_t* cache, uint32_t layer_idx, void* stream)
{
    return latent_write_at(kv_input, input_row_offsets, total_tokens, positions, kv_norm_gamma, epsilon, freqs_cis,
                           max_seq_len, K, rope_layout, cache, nullptr, false, layer_idx, stream);
}

MLA_API mla_status_t mla_write_latent_paged_fp8_at(const void* kv_input, const uint32_t* input_row_offsets,
                                                   int32_t total_tokens, const uint32_t* positions,
                                                   const float* kv_norm_gamma, float epsilon,
                                                   const float* freqs_cis, int32_t max_seq_len, int32_t K,
                                                   int32_t rope_layout, const mla_paged_cache_t* cache,
                                                   const mla_cache_scales_t* cache_scales, uint32_t layer_idx,
                                                   void* stream)
{
    return latent_write_at(kv_input, input_row_offsets, total_tokens, positions, kv_norm_gamma, epsilon, freqs_cis,
                           max_seq_len, K, rope_layout, cache, cache_scales, true, layer_idx, stream);
}

MLA_API size_t mla_tree_attention_workspace_size(int32_t total_tokens, int32_t num_heads, int32_t K)
{
    if (total_tokens < 0 || num_heads <= 0 || K <= 0 || K > 512)
        return 0;
    // Two partial results per workgroup: whole waves of 32 rows of K sums, a maximum and a sum each.
    const int64_t rows = (std::min<int64_t>((int64_t)total_tokens * num_heads, kAttnRows) + 31) / 32 * 32;
    return align256((size_t)(2 * kAttnGroups * rows * (K + 2)) * sizeof(float) + kAttnGroups * kAttnCutBytes);
}

namespace {

mla_status_t tree_attention(const void* q_latent, const uint32_t* input_row_offsets, int32_t total_tokens,
                            int32_t num_heads, const uint64_t* tree_mask, int32_t mask_words, float scale, int32_t K,
                            const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales, bool fp8,
                            uint32_t layer_idx, void* out_latent, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    if (!cache || (fp8 && !cache_scales))
        return MLA_ERR_NULL_POINTER;
    const int32_t T = total_tokens;
    const bool work = T > 0;
    if (work && (!q_latent || !input_row_offsets || !out_latent || !workspace || !cache->blocks ||
                 !cache->page_table || !cache->cache_lengths || (fp8 && !cache_scales->scales)))
        return MLA_ERR_NULL_POINTER;
    if (T < 0 || num_heads <= 0 || K <= 0 || K % 8 || K > 512 || !std::isfinite(scale) || mask_words < 0 ||
        (tree_mask && mask_words == 0) || (!tree_mask && mask_words != 0) || (int64_t)T * mask_words >= k2G)
        return MLA_ERR_INVALID_SHAPE;
    if (mla_status_t st = check_cache_shape(cache, 1))
        return st;
    const int64_t D = (int64_t)cache->num_heads * cache->head_dim, R = D - K;
    if (R < 0 || R % 8 || R > 512 || (int64_t)T * num_heads >= k2G / D ||
        (int64_t)cache->max_pages_per_seq * cache->page_size >= k2G || (fp8 && (D % 16 || !scales_shape_ok(cache_scales, D))))
        return MLA_ERR_INVALID_SHAPE;
    if (fp8 ? cache->dtype != MLA_DTYPE_F8E4M3FN : cache->dtype != MLA_DTYPE_BF16 && cache->dtype != MLA_DTYPE_F32)
        return MLA_ERR_INVALID_DTYPE;
    if (!aligned16(q_latent) || !aligned16(out_latent) || !aligned4(lse) || !aligned8(tree_mask) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) || (fp8 && !aligned4(cache_scales->scales)))
        return MLA_ERR_MISALIGNED;
    if (mla_status_t st = check_cache_alignment(cache))
        return st;
    if (layer_idx >= cache->num_layers)
        return MLA_ERR_OUT_OF_RANGE;
    if (work && workspace_bytes < mla_tree_attention_workspace_size(T, num_heads, K))
        return MLA_ERR_WORKSPACE;
    if (!work)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;

    TreeAttentionArgs a{};
    a.q = q_latent;
    a.iro = input_row_offsets;
    a.cache_len = cache->cache_lengths;
    a.mask = tree_mask;
    a.words = mask_words;
    a.out = out_latent;
    a.lse = lse;
    a.ws = static_cast<float*>(workspace);
    a.L = layer_view(cache, layer_idx);
    if (fp8)
        a.Ls = scales_view(cache, cache_scales, layer_idx);
    a.scale = scale;
    a.T = T;
    a.H = num_heads;
    a.K = K;
    a.D = (int)D;
    a.capacity = cache->max_pages_per_seq * cache->page_size;
    const AttnKind kind = fp8 ? ATTN_E4M3 : cache->dtype == MLA_DTYPE_F32 ? ATTN_F32 : ATTN_BF16;
    const hipError_t e = launch_tree_attention(a, kind, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

}  // namespace

MLA_API mla_status_t mla_tree_attention_paged(const void* q_latent, const uint32_t* input_row_offsets,
                                              int32_t total_tokens, int32_t num_heads, const uint64_t* tree_mask,
                                              int32_t mask_words, float scale, int32_t K,
                                              const mla_paged_cache_t* cache, uint32_t layer_idx, void* out_latent,
                                              float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    return tree_attention(q_latent, input_row_offsets, total_tokens, num_heads, tree_mask, mask_words, scale, K,
                          cache, nullptr, false, layer_idx, out_latent, lse, workspace, workspace_bytes, stream);
}

MLA_API mla_status_t mla_tree_attention_paged_fp8_cache(const void* q_latent, const uint32_t* input_row_offsets,
                                                        int32_t total_tokens, int32_t num_heads,
                                                        const uint64_t* tree_mask, int32_t mask_words, float scale,
                                                        int32_t K, const mla_paged_cache_t* cache,
                                                        const mla_cache_scales_t* cache_scales, uint32_t layer_idx,
                                                        void* out_latent, float* lse, void* workspace,
                                                        size_t workspace_bytes, void* stream)
{
    return tree_attention(q_latent, input_row_offsets, total_tokens, num_heads, tree_mask, mask_words, scale, K,
                          cache, cache_scales, true, layer_idx, out_latent, lse, workspace, workspace_bytes, stream);
}

namespace {

// Validation and descriptors shared by the page upkeep calls.  `pointers` says whether the
// call's own device pointers are all there; blocks: the call touches the pools.
mla_status_t page_call(const mla_paged_cache_t* cache, const mla_cache_scales_t* sc, int32_t count, bool pointers,
                       bool blocks, bool lengths, PageArgs& a)
{
    if (!cache)
        return MLA_ERR_NULL_POINTER;
    const bool fp8 = cache->dtype == MLA_DTYPE_F8E4M3FN;
    if (blocks && fp8 && !sc)
        return MLA_ERR_NULL_POINTER;
    const bool work = count > 0;
    if (work && (!pointers || (blocks && !cache->blocks) || (lengths && (!cache->page_table || !cache->cache_lengths)) ||
                 (blocks && fp8 && !sc->scales)))
        return MLA_ERR_NULL_POINTER;
    if (count < 0 || count > kMostPagePairs || (cache->num_kv != 1 && cache->num_kv != 2))
        return MLA_ERR_INVALID_SHAPE;
    if (mla_status_t st = check_cache_shape(cache, cache->num_kv))
        return st;
    const int64_t D = (int64_t)cache->num_heads * cache->head_dim;
    const int eb = elem_bytes(cache->dtype);
    if (D * 4 >= k2G || (int64_t)cache->page_size * (D * (eb ? eb : 1) / 16 + 1) >= k2G ||
        (int64_t)cache->num_layers * cache->num_kv >= k2G || (blocks && fp8 && !scales_shape_ok(sc, D)) ||
        (blocks && !fp8 && sc))
        return MLA_ERR_INVALID_SHAPE;
    if (!eb)
        return MLA_ERR_INVALID_DTYPE;
    if (blocks) {
        if (fp8 && !aligned4(sc->scales))
            return MLA_ERR_MISALIGNED;
        if (mla_status_t st = check_cache_alignment(cache))
            return st;
    }
    a = PageArgs{};
    a.pool = static_cast<char*>(cache->blocks);
    a.page_table = const_cast<uint32_t*>(cache->page_table);
    a.cache_len = const_cast<uint32_t*>(cache->cache_lengths);
    a.sp = cache->stride_page * eb;
    a.sl = cache->stride_layer * eb;
    a.sk = cache->stride_kv * eb;
    a.st = cache->stride_token * eb;
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.max_pages = cache->max_pages_per_seq;
    a.batch = cache->batch_size;
    a.layers = cache->num_layers;
    a.kvs = cache->num_kv;
    a.granules = (int)(D * eb / 16);
    a.count = count;
    if (blocks && fp8) {
        a.scales = const_cast<float*>(sc->scales);
        a.ssp = sc->stride_page;
        a.ssl = sc->stride_layer;
        a.ssk = sc->stride_kv;
        a.sst = sc->stride_token;
        a.nblk = (int)((D + 127) / 128);
    }
    return MLA_OK;
}

}  // namespace

MLA_API mla_status_t mla_copy_pages(const uint32_t* src_pages, const uint32_t* dst_pages, int32_t count,
                                    const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales,
                                    void* stream)
{
    PageArgs a;
    if (mla_status_t st = page_call(cache, cache_scales, count, src_pages && dst_pages, true, false, a))
        return st;
    if (count == 0)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    a.a = src_pages;
    a.b = dst_pages;
    const hipError_t e = launch_copy_pages(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

MLA_API mla_status_t mla_fork_paged(const uint32_t* parents, const uint32_t* children, const uint32_t* new_pages,
                                    int32_t count, uint32_t* ref_counts, const mla_paged_cache_t* cache,
                                    const mla_cache_scales_t* cache_scales, void* stream)
{
    PageArgs a;
    if (mla_status_t st = page_call(cache, cache_scales, count, parents && children && new_pages && ref_counts, true,
                                    true, a))
        return st;
    if (count == 0)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    a.a = parents;
    a.b = children;
    a.c = new_pages;
    a.refs = ref_counts;
    const hipError_t e = launch_fork(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

MLA_API mla_status_t mla_free_paged(const uint32_t* requests, int32_t count, uint32_t* ref_counts,
                                    uint32_t* free_list, uint32_t* free_count, const mla_paged_cache_t* cache,
                                    void* stream)
{
    PageArgs a;
    if (mla_status_t st = page_call(cache, nullptr, count, requests && ref_counts && free_list && free_count, false,
                                    true, a))
        return st;
    if (count > 65536 || (int64_t)cache->num_pages >= k2G)
        return MLA_ERR_INVALID_SHAPE;
    if (count == 0)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    a.a = requests;
    a.refs = ref_counts;
    a.free_list = free_list;
    a.free_count = free_count;
    const hipError_t e = launch_free(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}

MLA_API mla_status_t mla_compact_paged(const uint32_t* accepted, const uint32_t* accepted_offsets,
                                       int32_t total_accepted, const mla_paged_cache_t* cache,
                                       const mla_cache_scales_t* cache_scales, void* stream)
{
    PageArgs a;
    if (mla_status_t st = page_call(cache, cache_scales, total_accepted, accepted && accepted_offsets, true, true, a))
        return st;
    if (total_accepted == 0)
        return MLA_OK;
    if (mla_status_t st = check_device())
        return st;
    a.a = accepted;
    a.b = accepted_offsets;
    const hipError_t e = launch_compact(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLA_OK : hip_failed(e);
}
