// Attention of absorbed queries over the paged latent cache for trees of drafted
// tokens: out = softmax(scale * q . row) rows[:, :K], a token seeing the cached
// rows of its request and the drafted rows its mask names.
//
// tree_attention_general: any supported shape and F32 caches.  SPLIT waves per token and
// head, each taking every SPLIT-th group of four rows; lane l holds columns 8l .. 8l+7 of
// the latent and of the rope part of the query, and of the output sum.  The four rows are
// loaded side by side, with no branch between them (it would wait for the loads before it);
// each score is a wave sum, with the running maximum and sum of the softmax in binary32, and
// the waves' results are joined in LDS.  Bound by its arithmetic: each row is read for one
// head at a time.
#include <algorithm>
#include <type_traits>

#include "step.hpp"

namespace mla {
namespace {

// The sum over all lanes, in every lane: by rotations within rows of 16 lanes, then by
// swaps of rows and of halves.
__device__ inline float wave_sum_all(float v)
{
    auto rotated = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                     0xF, 0xF, true));
    };
    v += rotated(v, std::integral_constant<int, 0x128>{});
    v += rotated(v, std::integral_constant<int, 0x124>{});
    v += rotated(v, std::integral_constant<int, 0x122>{});
    v += rotated(v, std::integral_constant<int, 0x121>{});
    const uint32_t x = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const uint32_t y = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Eight columns of a row piece as floats.
template <AttnKind KIND>
__device__ inline void load8(const char* row, int col, float scale, float (&x)[8])
{
    if constexpr (KIND == ATTN_F32) {
        const u32x4 a = ld16(row + (int64_t)col * 4), b = ld16(row + (int64_t)col * 4 + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(a[i]);
            x[4 + i] = __uint_as_float(b[i]);
        }
    } else if constexpr (KIND == ATTN_BF16) {
        const u32x4 a = ld16(row + (int64_t)col * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(a[i]);
            x[2 * i + 1] = bf16_hi(a[i]);
        }
    } else {
        const u32x2 a = *reinterpret_cast<const u32x2*>(row + col);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[i], false);
            const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[i], true);
            x[4 * i] = lo[0] * scale;
            x[4 * i + 1] = lo[1] * scale;
            x[4 * i + 2] = hi[0] * scale;
            x[4 * i + 3] = hi[1] * scale;
        }
    }
}

template <AttnKind KIND, int SPLIT>
__global__ void __launch_bounds__(64 * SPLIT) tree_attention_general(TreeAttentionArgs a, uint32_t first_pair)
{
    constexpr bool F32 = KIND == ATTN_F32;
    constexpr AttnKind QKIND = F32 ? ATTN_F32 : ATTN_BF16;
    constexpr int EB = F32 ? 4 : 2;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t pair = first_pair + blockIdx.x;   // below 2^31 / D
    const int t = pair / (uint32_t)a.H, h = pair % (uint32_t)a.H;
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    if ((uint32_t)t >= end)
        return;
    const uint32_t b = find_request(a.iro, a.L.batch, t);
    const uint32_t t0 = a.iro[b], n = min(a.iro[b + 1], end) - t0, i = t - t0;
    const uint32_t cached = min(a.cache_len[b], a.capacity);
    const uint32_t len = min(cached + n, a.capacity);   // both below 2^31
    const int R = a.D - a.K;
    const bool lat = lane * 8 < a.K, rot = lane * 8 < R;
    // Lanes without columns load those of the first lane, and their query is zero.
    const int lat_col = lat ? lane * 8 : 0, rot_col = rot ? a.K + lane * 8 : 0;

    const int64_t row_q = (int64_t)t * a.H + h;
    const char* q = static_cast<const char*>(a.q) + row_q * a.D * EB;
    float ql[8] = {}, qr[8] = {};
    if (lat)
        load8<QKIND>(q, lane * 8, 1.0f, ql);
    if (rot)
        load8<QKIND>(q, a.K + lane * 8, 1.0f, qr);

    float m = -INFINITY, l = 0.0f, o[8] = {};
    constexpr int U = 4;
    // Rows p0 .. p0 + 3, of which the token sees those that `sees` says (positions are below last).
    auto rows = [&](uint32_t p0, uint32_t last, auto sees) __attribute__((always_inline)) {
        float v[U][8], x[U][8], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t p = min(p0 + u, last - 1);
            const char* row = a.L.base + token_offset(a.L, b, p);
            float sl = 1.0f, sr = 1.0f;
            if constexpr (KIND == ATTN_E4M3) {
                const float* sc = reinterpret_cast<const float*>(a.Ls.base + token_offset(a.Ls, b, p));
                sl = sc[lat_col / 128];
                sr = sc[rot_col / 128];
            }
            load8<KIND>(row, lat_col, sl, v[u]);
            load8<KIND>(row, rot_col, sr, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool seen = p0 + u < last && sees(p0 + u);
            float d = 0.0f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                // (a row that is not seen may hold anything; lanes without columns, another lane's)
                v[u][c] = seen ? v[u][c] : 0.0f;
                d += lat ? ql[c] * v[u][c] : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
                d += rot ? qr[c] * x[u][c] : 0.0f;
            s[u] = wave_sum_all(d) * a.scale;
            s[u] = seen ? s[u] : -INFINITY;
        }
        float mx = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            mx = fmaxf(mx, s[u]);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        const float keep = expf(m - ref);
        l *= keep;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            o[c] *= keep;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = expf(s[u] - ref);
            l += w;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                o[c] += w * v[u][c];
        }
        m = mx;
    };
    for (uint32_t p0 = wave * U; p0 < cached; p0 += SPLIT * U)
        rows(p0, cached, [](uint32_t) { return true; });
    const uint32_t drafted = a.mask ? n : i + 1;
    for (uint32_t j0 = wave * U; j0 < drafted && cached + j0 < len; j0 += SPLIT * U)
        rows(cached + j0, len, [&](uint32_t p) {
            const uint32_t j = p - cached;
            return a.mask ? j < 64u * (uint32_t)a.words && (a.mask[(int64_t)t * a.words + j / 64] >> (j & 63)) & 1 : j <= i;
        });

    __shared__ float part[SPLIT][10][64];
    float(*mine)[64] = part[wave];
#pragma unroll
    for (int c = 0; c < 8; ++c)
        mine[c][lane] = o[c];
    mine[8][lane] = m;
    mine[9][lane] = l;
    __syncthreads();
    if (wave > 0)
        return;
    for (int k = 1; k < SPLIT; ++k)
        m = fmaxf(m, part[k][8][lane]);
    const float ref = m == -INFINITY ? 0.0f : m;
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        o[c] = 0.0f;
    for (int k = 0; k < SPLIT; ++k) {
        const float f = expf(part[k][8][lane] - ref);
        l += part[k][9][lane] * f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            o[c] += part[k][c][lane] * f;
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    if (lat) {
        char* dst = static_cast<char*>(a.out) + (row_q * a.K + lane * 8) * EB;
        if constexpr (F32) {
            st16(dst, u32x4{__float_as_uint(o[0] * inv), __float_as_uint(o[1] * inv), __float_as_uint(o[2] * inv),
                            __float_as_uint(o[3] * inv)});
            st16(dst + 16, u32x4{__float_as_uint(o[4] * inv), __float_as_uint(o[5] * inv), __float_as_uint(o[6] * inv),
                                 __float_as_uint(o[7] * inv)});
        } else {
            st16(dst, u32x4{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                            pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv)});
        }
    }
    if (a.lse && lane == 0)
        a.lse[row_q] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

hipError_t launch_tree_attention(const TreeAttentionArgs& a, AttnKind kind, hipStream_t s)
{
    if (tree_attention_mfma_fits(a, kind))
        return launch_tree_attention_mfma(a, kind, s);
    // Few tokens and heads: more waves for each.  16 / 4 waves, us, F32 rows of 576 columns: 16 pairs
    // of a token and a head over 4096 rows 141 / 296, 256 pairs 209 / 320, 1024 pairs over 2048 rows
    // 429 / 442, 2048 pairs 754 / 748, 8192 pairs over 1024 rows 1351 / 1202.
    const int64_t pairs = (int64_t)a.T * a.H;
    const bool many = pairs <= 1024;
    const unsigned threads = many ? 1024 : 256;
    auto pick = [&](auto k) {
        constexpr AttnKind kd = decltype(k)::value;
        return many ? tree_attention_general<kd, 16> : tree_attention_general<kd, 4>;
    };
    auto* kernel = kind == ATTN_F32    ? pick(std::integral_constant<AttnKind, ATTN_F32>{})
                   : kind == ATTN_BF16 ? pick(std::integral_constant<AttnKind, ATTN_BF16>{})
                                       : pick(std::integral_constant<AttnKind, ATTN_E4M3>{});
    // A launch holds less than 2^32 threads in a dimension, and drops those past them without an error.
    constexpr int64_t kMostBlocks = int64_t(1) << 23;
    for (int64_t first = 0; first < pairs; first += kMostBlocks) {
        const unsigned blocks = (unsigned)std::min(pairs - first, kMostBlocks);
        log_launch("tree_attention_general", blocks, threads, "T=%d H=%d K=%d D=%d kind=%d", a.T, a.H, a.K, a.D, (int)kind);
        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), 0, s, a, (uint32_t)first);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    return hipSuccess;
}

}  // namespace mla
