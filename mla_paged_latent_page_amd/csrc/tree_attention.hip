// Attention of absorbed queries over the paged latent cache for trees of drafted
// tokens: out = softmax(scale * q . row) rows[:, :K], a token seeing the cached
// rows of its request and the drafted rows its mask names.
//
// tree_attention_general: any supported shape and F32 caches.  One wave per token
// and head; lane l holds columns 8l .. 8l+7 of the latent and of the rope part of
// the query, and of the output sum.  Rows are taken four at a time (four loads in
// flight), each score a wave sum, with the running maximum and sum of the softmax
// in binary32.  What the token does not see is not loaded.
#include "step.hpp"

namespace mla {
namespace {

__device__ inline float wave_sum_all(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
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

template <AttnKind KIND>
__global__ void __launch_bounds__(256) tree_attention_general(TreeAttentionArgs a)
{
    constexpr bool F32 = KIND == ATTN_F32;
    constexpr AttnKind QKIND = F32 ? ATTN_F32 : ATTN_BF16;
    constexpr int EB = F32 ? 4 : 2;
    const int lane = threadIdx.x & 63;
    const int head_groups = (a.H + 3) / 4;
    const int t = blockIdx.x / head_groups;
    const int h = (blockIdx.x % head_groups) * 4 + (threadIdx.x >> 6);
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    if ((uint32_t)t >= end || h >= a.H)
        return;
    const uint32_t b = find_request(a.iro, a.L.batch, t);
    const uint32_t t0 = a.iro[b], n = min(a.iro[b + 1], end) - t0, i = t - t0;
    const uint32_t cached = min(a.cache_len[b], a.capacity);
    const uint32_t len = min(cached + n, a.capacity);   // both below 2^31
    const int R = a.D - a.K;
    const bool lat = lane * 8 < a.K, rot = lane * 8 < R;

    const int64_t row_q = (int64_t)t * a.H + h;
    const char* q = static_cast<const char*>(a.q) + row_q * a.D * EB;
    float ql[8] = {}, qr[8] = {};
    if (lat)
        load8<QKIND>(q, lane * 8, 1.0f, ql);
    if (rot)
        load8<QKIND>(q, a.K + lane * 8, 1.0f, qr);

    float m = -INFINITY, l = 0.0f, o[8] = {};
    constexpr int U = 4;
    for (uint32_t p0 = 0; p0 < len; p0 += U) {
        float v[U][8], s[U];
        bool vis[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t p = p0 + u;
            bool seen = p < len;
            if (seen && p >= cached) {
                const uint32_t j = p - cached;
                if (a.mask)
                    seen = j < 64u * (uint32_t)a.words && ((a.mask[(int64_t)t * a.words + j / 64] >> (j & 63)) & 1);
                else
                    seen = j <= i;
            }
            vis[u] = seen;
            s[u] = 0.0f;
            float x[8] = {};
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[u][c] = 0.0f;
            if (seen) {
                const char* row = a.L.base + token_offset(a.L, b, p);
                float sl = 1.0f, sr = 1.0f;
                if constexpr (KIND == ATTN_E4M3) {
                    const float* sc = reinterpret_cast<const float*>(a.Ls.base + token_offset(a.Ls, b, p));
                    sl = lat ? sc[lane * 8 / 128] : 0.0f;
                    sr = rot ? sc[(a.K + lane * 8) / 128] : 0.0f;
                }
                if (lat)
                    load8<KIND>(row, lane * 8, sl, v[u]);
                if (rot)
                    load8<KIND>(row, a.K + lane * 8, sr, x);
                float d = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    d += ql[c] * v[u][c];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    d += qr[c] * x[c];
                s[u] = d;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            s[u] = vis[u] ? wave_sum_all(s[u]) * a.scale : -INFINITY;
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
    const dim3 grid((unsigned)a.T * ((a.H + 3) / 4));
    log_launch("tree_attention_general", grid.x, 256, "T=%d H=%d K=%d D=%d kind=%d", a.T, a.H, a.K, a.D, (int)kind);
    if (kind == ATTN_F32)
        hipLaunchKernelGGL(tree_attention_general<ATTN_F32>, grid, dim3(256), 0, s, a);
    else if (kind == ATTN_BF16)
        hipLaunchKernelGGL(tree_attention_general<ATTN_BF16>, grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(tree_attention_general<ATTN_E4M3>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace mla
