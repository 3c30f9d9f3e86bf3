// Writes of new tokens' keys and values into the pages of a K/V cache: the last d_rope columns
// of every key head rotated at the token's position, the rest as it is, as bf16 or as e4m3
// codes with a scale per 128 columns of the token row.
//
//   y = x, or (x0 c - x1 s, x0 s + x1 c) for the pairs of rotated columns  (binary32)
//   bf16: round(y);  e4m3: s = amax / 448 (1 where amax is 0), code = e4m3(y * (448 / amax))
// An amax below 448 * 2^-126 counts as that: 448 / amax would overflow.
//
// Memory-bound: 4 HD bytes read, 4 HD (bf16) or 2 HD + 8 HD / 128 (e4m3) written per token.  A
// lane holds 8 columns, 16 lanes a block of 128, so that a block's amax is four DPP steps.  The
// pieces of all tokens (keys, then values) are one flat run, of which a wave takes 256 (e4m3 128): four
// loads in flight per lane (two) before the chain offsets -> length -> page -> store begins, which
// one lane per token walks for the wave (up to nine tokens, their requests counted by ballots).
// Measured from memory: 16,372 tokens into bf16 pages 33.3 us = 4.3 TB/s, 36,257 into e4m3 pages 61 us = 3.8 TB/s;
// a large copy reaches 5.1.
#include "kv.hpp"

namespace mla {
namespace {

// Pieces of a lane.  bf16: 4 against 2, 16,372 tokens of 8 heads of 128 columns 23.3 against 24.0 us; e4m3: 2 against 4,
// 36,257 tokens 56 against 58 us, and 61 against 65 where the inputs come from memory (fewer registers, more waves
// under the rotation, the divisions and the packing); 1 takes 70.
template <bool FP8>
constexpr int kPieces = FP8 ? 2 : 4;
constexpr int WAVES = 4;

__device__ inline uint64_t shfl64(uint64_t v, int lane)
{
    return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, lane, 64) |
           ((uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), lane, 64) << 32);
}

template <bool FP8, bool HALF>
__global__ void __launch_bounds__(64 * WAVES) kv_write_kernel(KvWriteArgs a, uint32_t first_token, uint32_t tokens)
{
    constexpr int U = kPieces<FP8>, PIECES = 64 * U;   // of a lane, of a wave
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t nblk = (a.HD + 127) / 128, per_half = nblk * 16, per_token = 2 * per_half;
    const uint32_t base = (blockIdx.x * WAVES + wave) * PIECES;   // below 2^31: see the launch
    const uint32_t j0 = base / per_token, r0 = base - j0 * per_token;
    if (j0 >= tokens)
        return;
    const uint32_t t0 = first_token + j0, end = a.iro[a.L.batch];

    // The lane's pieces: token (counted from t0), key or value, columns; its input.
    uint32_t tok[U], col[U], rc[U];
    bool val[U], on[U], rot[U], upper[U];
    u32x4 x[U], other[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t f = r0 + u * 64 + lane;
        tok[u] = f / per_token;
        const uint32_t g = f - tok[u] * per_token;
        val[u] = g >= per_half;
        col[u] = (val[u] ? g - per_half : g) * 8;
        const bool live = j0 + tok[u] < tokens;
        on[u] = live && col[u] < (uint32_t)a.HD;
        const uint32_t hc = col[u] % (uint32_t)a.D, nope = a.D - a.R;
        rot[u] = on[u] && !val[u] && hc >= nope;
        rc[u] = rot[u] ? hc - nope : 0;               // column among the rotated ones
        upper[u] = HALF && rc[u] * 2 >= (uint32_t)a.R;
        x[u] = other[u] = u32x4{0u, 0u, 0u, 0u};
        const char* src = (val[u] ? a.v + (int64_t)(t0 + tok[u]) * a.v_st : a.k + (int64_t)(t0 + tok[u]) * a.k_st) +
                          (int64_t)col[u] * 2;
        if (on[u])
            x[u] = ld16(src);
        if (HALF && rot[u])
            other[u] = ld16(src + (upper[u] ? -a.R : a.R));   // R / 2 columns away
    }

    // Lane j: request, page and slot of token t0 + j.  Offsets <= t form a prefix; its last
    // index is the request (empty requests are skipped by taking the last).
    const uint32_t last = min((r0 + PIECES - 1) / per_token, tokens - 1 - j0);
    uint32_t cnt = 0;
    for (uint32_t c = 0; c < a.L.batch; c += 256) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t k = c + i * 64 + lane;
            o[i] = k < a.L.batch ? a.iro[k] : 0xFFFFFFFFu;
        }
        for (uint32_t j = 0; j <= last; ++j) {
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                n += (uint32_t)__popcll(__ballot(o[i] <= t0 + j));
            cnt += (uint32_t)lane == j ? n : 0;
        }
    }
    uint64_t off = ~0ull, soff = 0;
    uint32_t row = 0;
    if ((uint32_t)lane <= last) {
        const uint32_t t = t0 + lane;
        const uint32_t b = cnt == 0 ? 0u : min(cnt, a.L.batch) - 1;
        const uint32_t cached = a.cache_len[b], p = cached + (t - a.iro[b]);
        // -1: no slot for this position, nothing is stored; nor is it past 2^32, or behind the last request
        off = (uint64_t)(store_offset(a.L, b, p) | -(int64_t)(p < cached || t >= end));
        if (FP8)
            soff = (uint64_t)store_offset(a.Ls, b, p);
        const uint32_t pr = a.pos ? a.pos[t] : p;
        row = min(pr, (uint32_t)a.max_seq - 1);
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t to = (int64_t)shfl64(off, (int)tok[u]);
        const uint32_t fr = (uint32_t)__shfl((int)row, (int)tok[u], 64);
        const uint64_t sto = FP8 ? shfl64(soff, (int)tok[u]) : 0;
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = bf16_lo(x[u][i]);
            y[2 * i + 1] = bf16_hi(x[u][i]);
        }
        if (rot[u]) {
            const float* f = a.freqs + (int64_t)fr * a.R;
            if constexpr (!HALF) {
                const f32x4 f0 = *reinterpret_cast<const f32x4*>(f + rc[u]);
                const f32x4 f1 = *reinterpret_cast<const f32x4*>(f + rc[u] + 4);
                const float cs[8] = {f0[0], f0[1], f0[2], f0[3], f1[0], f1[1], f1[2], f1[3]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = y[2 * i], x1 = y[2 * i + 1], c = cs[2 * i], s = cs[2 * i + 1];
                    y[2 * i] = x0 * c - x1 * s;
                    y[2 * i + 1] = x0 * s + x1 * c;
                }
            } else {
                f += 2 * (rc[u] - (upper[u] ? a.R / 2 : 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 cs = *reinterpret_cast<const f32x4*>(f + 4 * i);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float c = cs[2 * k], s = cs[2 * k + 1], me = y[2 * i + k];
                        const float ot = k ? bf16_hi(other[u][i]) : bf16_lo(other[u][i]);
                        y[2 * i + k] = upper[u] ? ot * s + me * c : me * c - ot * s;
                    }
                }
            }
        }
        const bool store = on[u] && to >= 0;
        char* dst = const_cast<char*>(a.L.base) + to + (val[u] ? a.L.stride_kv : 0);
        if constexpr (!FP8) {
            if (store)
                st16(dst + (int64_t)col[u] * 2, u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                      pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])});
        } else {
            float am = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                am = fmaxf(am, fabsf(y[i]));
            am = max16(am);   // a token's blocks start at multiples of 16 lanes
            float s = 1.0f, inv = 1.0f;
            if (am > 0.0f) {
                am = fmaxf(am, 448.0f * 0x1p-126f);
                s = am / 448.0f;
                inv = 448.0f / am;
            }
            if (store) {
                *reinterpret_cast<u32x2*>(dst + col[u]) =
                    u32x2{pack_e4m3x2(y[0] * inv, y[1] * inv) | pack_e4m3x2(y[2] * inv, y[3] * inv) << 16,
                          pack_e4m3x2(y[4] * inv, y[5] * inv) | pack_e4m3x2(y[6] * inv, y[7] * inv) << 16};
                if ((lane & 15) == 0)
                    *reinterpret_cast<float*>(const_cast<char*>(a.Ls.base) + sto + (val[u] ? a.Ls.stride_kv : 0) +
                                              (col[u] / 128) * 4) = s;
            }
        }
    }
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs& a, bool fp8, bool half, hipStream_t s)
{
    auto* kernel = fp8 ? (half ? kv_write_kernel<true, true> : kv_write_kernel<true, false>)
                       : (half ? kv_write_kernel<false, true> : kv_write_kernel<false, false>);
    // Pieces of a launch are numbered in 32 bits.
    const int64_t per_token = 2 * ((a.HD + 127) / 128) * 16;
    const int64_t most = (int64_t(1) << 30) / per_token, per_block = 64 * WAVES * (fp8 ? kPieces<true> : kPieces<false>);
    for (int64_t first = 0; first < a.T; first += most) {
        const int64_t tokens = a.T - first < most ? a.T - first : most;
        const unsigned grid = (unsigned)((tokens * per_token + per_block - 1) / per_block);
        log_launch(fp8 ? "kv_write_kernel<e4m3>" : "kv_write_kernel<bf16>", grid, 64 * WAVES, "T=%d HD=%d R=%d half=%d",
                   a.T, a.HD, a.R, (int)half);
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * WAVES), 0, s, a, (uint32_t)first, (uint32_t)tokens);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    return hipSuccess;
}

}  // namespace mla
