// Attention of new tokens over a paged K/V cache, the cached rows and their own: causal, with
// or without a sliding window and first tokens that stay visible.
//
//   p = cache_lengths[b] + i;  k seen if k <= p and (no window or p - k < window or k < sinks)
//   out = sum_k exp(s_k) V_k / sum_k exp(s_k),  s_k = scale * q . K_k,  query head h with key head h / (H / KH)
//
// kv_attention_general: any head of up to 256 columns, F32 caches.  A block takes one token and up to
// HEADS query heads of one key head; L lanes hold a row, 8 columns each, so a wave has 64 / L rows at
// once and four times as many in flight.  Every group of L lanes keeps a running maximum, a sum and output
// sums of its own in binary32; they are joined at the end, first across the wave, then in LDS.  A context is
// not split over blocks, and the workspace is not used.  Bound by waiting: 35 tokens x 12 binary32 heads of 80
// columns with a window of 500 take 16.8 us at 1.0 TB/s and 1.5 TFLOP/s, the chain offsets -> length -> page -> row
// and two passes of 256 rows, then the join of 16 waves; waves wait 63 % of their time, the vector units are busy 30 %.
// The matrix cores' binary32 products (32x32x2) are not used.
#include <algorithm>
#include <type_traits>

#include "kv.hpp"

namespace mla {
namespace {

// Eight columns of a row as floats.
template <KvKind KIND>
__device__ inline void load8(const char* row, uint32_t col, float scale, float (&x)[8])
{
    if constexpr (KIND == KV_F32) {
        const u32x4 a = ld16(row + (int64_t)col * 4), b = ld16(row + (int64_t)col * 4 + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(a[i]);
            x[4 + i] = __uint_as_float(b[i]);
        }
    } else if constexpr (KIND == KV_BF16) {
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

// Sum over groups of L lanes, in every lane.
template <int L>
__device__ inline float group_sum(float v)
{
    if constexpr (L >= 2)
        v += dpp_f32<0xB1>(v);    // quad_perm [1, 0, 3, 2]
    if constexpr (L >= 4)
        v += dpp_f32<0x4E>(v);    // quad_perm [2, 3, 0, 1]
    if constexpr (L >= 8)
        v += dpp_f32<0x141>(v);   // row_half_mirror
    if constexpr (L >= 16)
        v += dpp_f32<0x140>(v);   // row_mirror
    if constexpr (L >= 32)
        v += __shfl_xor(v, 16, 64);
    return v;
}

template <KvKind KIND, int L, int HEADS, int SPLIT>
__global__ void __launch_bounds__(64 * SPLIT) kv_attention_general(KvAttentionArgs a, uint32_t first)
{
    constexpr bool F32 = KIND == KV_F32;
    constexpr KvKind QKIND = F32 ? KV_F32 : KV_BF16;
    constexpr int EB = F32 ? 4 : 2;
    constexpr int CB = F32 ? 4 : KIND == KV_BF16 ? 2 : 1;   // bytes of a cached element
    constexpr int ROWS = 64 / L;                            // of a wave at a time
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t G = a.H / a.KH, parts = (G + HEADS - 1) / HEADS, per_token = a.KH * parts;
    const uint32_t id = first + blockIdx.x, t = id / per_token, kh = id % per_token / parts;
    const uint32_t g0 = id % per_token % parts * HEADS;     // first query head of the group
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    if (t >= end)
        return;
    const uint32_t b = find_request(a.iro, a.L.batch, t);
    const uint32_t i = t - a.iro[b];
    const uint32_t p = min(a.cache_len[b], 0x80000000u) + i;              // (below 2^32)
    const uint32_t top = min(p, a.capacity - 1) + 1;                      // rows below it may be seen
    uint32_t low = a.window && p + 1 > a.window ? p + 1 - a.window : 0;
    low = min(low, top);
    const uint32_t sunk = min(a.sinks, low);                              // first rows, then those from low on
    const uint32_t count = sunk + (top - low);

    const uint32_t sub = lane % L, grp = lane / L, col = sub * 8 < (uint32_t)a.D ? sub * 8 : 0;
    const bool on = sub * 8 < (uint32_t)a.D;
    float q[HEADS][8];
#pragma unroll
    for (int g = 0; g < HEADS; ++g) {
        const uint32_t h = kh * G + min(g0 + g, G - 1);
        load8<QKIND>(a.q + (int64_t)t * a.q_st + (int64_t)h * a.D * EB, col, 1.0f, q[g]);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            q[g][c] = on ? q[g][c] : 0.0f;
    }
    float m[HEADS], l[HEADS], o[HEADS][8];
#pragma unroll
    for (int g = 0; g < HEADS; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            o[g][c] = 0.0f;
    }
    constexpr int U = HEADS > 1 ? 2 : 4;
    const uint32_t wide = kh * a.D + col;                                 // column in the token row
    for (uint32_t r0 = wave * ROWS * U; r0 < count; r0 += SPLIT * ROWS * U) {
        float k[U][8], v[U][8];
        bool seen[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + u * ROWS + grp;
            seen[u] = r < count;
            const uint32_t rr = min(r, count - 1), at = rr < sunk ? rr : low + (rr - sunk);
            const char* row = a.L.base + token_offset(a.L, b, at);
            float sk = 1.0f, sv = 1.0f;
            if constexpr (KIND == KV_E4M3) {
                const char* sc = a.Ls.base + token_offset(a.Ls, b, at) + wide / 128 * 4;
                sk = *reinterpret_cast<const float*>(sc);
                sv = *reinterpret_cast<const float*>(sc + a.Ls.stride_kv);
            }
            load8<KIND>(row + (int64_t)wide * CB, 0, sk, k[u]);
            load8<KIND>(row + a.L.stride_kv + (int64_t)wide * CB, 0, sv, v[u]);
        }
#pragma unroll
        for (int g = 0; g < HEADS; ++g) {
            float s[U], mx = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float d = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    d += on ? q[g][c] * k[u][c] : 0.0f;   // (lanes without columns hold another lane's)
                s[u] = group_sum<L>(d) * a.scale;
                s[u] = seen[u] ? s[u] : -INFINITY;
                mx = fmaxf(mx, s[u]);
            }
            const float ref = mx == -INFINITY ? 0.0f : mx, keep = expf(m[g] - ref);
            l[g] *= keep;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                o[g][c] *= keep;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = expf(s[u] - ref);
                l[g] += w;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    o[g][c] += w * (seen[u] ? v[u][c] : 0.0f);   // (a repeated row may hold anything)
            }
            m[g] = mx;
        }
    }

    // The wave's groups, then the waves.
    __shared__ float part[SPLIT][10][L];
#pragma unroll
    for (int g = 0; g < HEADS; ++g) {
        float mx = m[g];
#pragma unroll
        for (int d = L; d < 64; d *= 2)
            mx = fmaxf(mx, __shfl_xor(mx, d, 64));
        const float f = expf(m[g] - (mx == -INFINITY ? 0.0f : mx));
        float x[9];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            x[c] = o[g][c] * f;
        x[8] = l[g] * f;
#pragma unroll
        for (int c = 0; c < 9; ++c)
#pragma unroll
            for (int d = L; d < 64; d *= 2)
                x[c] += __shfl_xor(x[c], d, 64);
        __syncthreads();
        if (lane < L) {
#pragma unroll
            for (int c = 0; c < 9; ++c)
                part[wave][c][lane] = x[c];
            part[wave][9][lane] = mx;
        }
        __syncthreads();
        if (wave == 0 && lane < L && g0 + g < G) {
            mx = -INFINITY;
            for (int w = 0; w < SPLIT; ++w)
                mx = fmaxf(mx, part[w][9][lane]);
            float y[9] = {};
            for (int w = 0; w < SPLIT; ++w) {
                const float e = expf(part[w][9][lane] - (mx == -INFINITY ? 0.0f : mx));
    #pragma unroll
                for (int c = 0; c < 9; ++c)
                    y[c] += part[w][c][lane] * e;
            }
            const float sum = y[8], inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
            const int64_t head = (int64_t)t * a.H + kh * G + g0 + g;
            if (on) {
                char* dst = static_cast<char*>(a.out) + (head * a.D + col) * EB;
                if constexpr (F32) {
                    st16(dst, u32x4{__float_as_uint(y[0] * inv), __float_as_uint(y[1] * inv), __float_as_uint(y[2] * inv),
                                    __float_as_uint(y[3] * inv)});
                    st16(dst + 16, u32x4{__float_as_uint(y[4] * inv), __float_as_uint(y[5] * inv),
                                         __float_as_uint(y[6] * inv), __float_as_uint(y[7] * inv)});
                } else {
                    st16(dst, u32x4{pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv),
                                    pack_bf16x2(y[4] * inv, y[5] * inv), pack_bf16x2(y[6] * inv, y[7] * inv)});
                }
            }
            if (a.lse && lane == 0)
                a.lse[head] = sum == 0.0f ? -INFINITY : mx + logf(sum);
        }
    }
}

template <KvKind KIND, int L, int HEADS>
hipError_t launch_general(const KvAttentionArgs& a, hipStream_t s)
{
    const int64_t parts = (a.H / a.KH + HEADS - 1) / HEADS, blocks = (int64_t)a.T * a.KH * parts;
    // Few blocks: more waves for each.  16 against 4 waves: 96 blocks of 2,000 binary32 rows 33 against 63 us, 1,152 of
    // them 288 against 294, 4,800 blocks of 500 rows 173 against 124.
    const bool many = blocks <= 1024;
    auto* kernel = many ? kv_attention_general<KIND, L, HEADS, 16> : kv_attention_general<KIND, L, HEADS, 4>;
    const unsigned threads = many ? 1024 : 256;
    // A launch holds less than 2^32 threads in a dimension, and drops those past them without an error.
    constexpr int64_t kMostBlocks = int64_t(1) << 23;
    for (int64_t first = 0; first < blocks; first += kMostBlocks) {
        const unsigned grid = (unsigned)std::min(blocks - first, kMostBlocks);
        log_launch("kv_attention_general", grid, threads, "T=%d H=%d KH=%d D=%d kind=%d", a.T, a.H, a.KH, a.D, (int)KIND);
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, s, a, (uint32_t)first);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    return hipSuccess;
}

template <KvKind KIND>
hipError_t launch_kind(const KvAttentionArgs& a, hipStream_t s)
{
    // Several query heads read the rows of one key head: four at a time in a block against one, 64 tokens x 16 heads on
    // 4 key heads of 80 columns, 2,000 bf16 rows, 80 against 154 us; 32 on 8 of 128, 1,000 binary32 rows, 139 against 295.
    const bool shared = a.H > a.KH;
    if (a.D <= 64)
        return shared ? launch_general<KIND, 8, 4>(a, s) : launch_general<KIND, 8, 1>(a, s);
    if (a.D <= 128)
        return shared ? launch_general<KIND, 16, 4>(a, s) : launch_general<KIND, 16, 1>(a, s);
    return shared ? launch_general<KIND, 32, 4>(a, s) : launch_general<KIND, 32, 1>(a, s);
}

}  // namespace

hipError_t launch_kv_attention(const KvAttentionArgs& a, KvKind kind, hipStream_t s)
{
    if (kv_attention_mfma_fits(a, kind))
        return launch_kv_attention_mfma(a, kind, s);
    return kind == KV_F32 ? launch_kind<KV_F32>(a, s) : kind == KV_BF16 ? launch_kind<KV_BF16>(a, s)
                                                                       : launch_kind<KV_E4M3>(a, s);
}

}  // namespace mla
