// Rotary positions: freqs_cis tables and the rotation of query heads (page
// "mla_prefill_decode_graph_fp8", Args freqs_cis, q).
//
// rope_freqs_kernel: entry (p, j) is (cos, sin) of p * g_j.  A position of 10^6
// times a frequency of 1 has 20 bits before the binary point, so binary32 would
// leave four for the angle: the product with g_j in quarter turns, its reduction
// to [-1/2, 1/2] quarter turns and the Taylor sums of sine and cosine, which stop
// below 2^-30 at pi/4, are binary64, and the result, times the amplitude, is rounded
// once.  Bound by its stores all the same (262,144 rows of 128 columns: 27 us, 5.0
// TB/s; 8,191 rows of 64: 2.9 us); a thread divides once, then walks rows and pairs
// by the grid's step.
//
// rope_q_kernel: one block per token (and 64 heads).  A thread keeps one group of
// pairs of the rope part for every head it visits, so the token's (cos, sin) row is
// read once into registers.  Bound by memory: the nope columns are only copied, in
// 16-byte pieces that are all in flight before the first store.  8,300 tokens of 128
// heads: 158 us, 5.2 TB/s of reads and writes; 83 tokens of 16 heads: 3 us.
#include <algorithm>

#include "step.hpp"

namespace mla {
namespace {

__global__ void __launch_bounds__(256) rope_freqs_kernel(RopeFreqsArgs a, int step_rows, int step_pairs)
{
    const int64_t total = (int64_t)a.rows * a.pairs;
    const int64_t step = (int64_t)gridDim.x * 256;   // step_rows rows and step_pairs pairs
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int row = (int)(first / a.pairs);
    int j = (int)(first - (int64_t)row * a.pairs);
    double quarters = first < total ? a.quarters[j] : 0.0;
    for (int64_t i = first; i < total; i += step) {
        const double turn = (double)((uint32_t)a.first + (uint32_t)row) * quarters;
        // Rounded to an integer by a sum whose last place is 1, where its low bits are too.
        constexpr double kWhole = 0x1.8p52;
        const double whole = turn + kWhole;
        const uint32_t quadrant = (uint32_t)__builtin_bit_cast(uint64_t, whole);
        const double x = (turn - (whole - kWhole)) * 1.57079632679489661923, x2 = x * x;
        const double sx = x + x * x2 * (-1.0 / 6 + x2 * (1.0 / 120 + x2 * (-1.0 / 5040 + x2 * (1.0 / 362880 -
                          x2 * (1.0 / 39916800)))));
        const double cx = 1.0 + x2 * (-0.5 + x2 * (1.0 / 24 + x2 * (-1.0 / 720 + x2 * (1.0 / 40320 -
                          x2 * (1.0 / 3628800)))));
        const float sa = (float)(sx * a.amplitude), ca = (float)(cx * a.amplitude);
        const float s = (quadrant & 1) ? ca : sa, c = (quadrant & 1) ? sa : ca;
        const uint32_t s_sign = quadrant << 30 & 0x80000000u, c_sign = (quadrant + 1) << 30 & 0x80000000u;
        *reinterpret_cast<f32x2*>(a.out + 2 * i) = f32x2{__uint_as_float(__float_as_uint(c) ^ c_sign),
                                                         __uint_as_float(__float_as_uint(s) ^ s_sign)};
        row += step_rows;
        if (step_pairs) {
            j += step_pairs;
            if (j >= a.pairs)
                j -= a.pairs, ++row;
            quarters = a.quarters[j];
        }
    }
}

// Rotate E elements (interleaved pairs) held in one 16-byte piece; cs holds their pairs.
template <bool F32>
__device__ inline u32x4 rotate_pairs(u32x4 v, const float* cs)
{
    u32x4 y;
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x0 = __uint_as_float(v[2 * i]), x1 = __uint_as_float(v[2 * i + 1]);
            const float c = cs[2 * i], s = cs[2 * i + 1];
            y[2 * i] = __float_as_uint(x0 * c - x1 * s);
            y[2 * i + 1] = __float_as_uint(x0 * s + x1 * c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = bf16_lo(v[i]), x1 = bf16_hi(v[i]);
            const float c = cs[2 * i], s = cs[2 * i + 1];
            y[i] = pack_bf16x2(x0 * c - x1 * s, x0 * s + x1 * c);
        }
    }
    return y;
}

// Rotate the pairs (element i of lo, element i of hi); cs holds one pair per element.
template <bool F32>
__device__ inline void rotate_halves(u32x4& lo, u32x4& hi, const float* cs)
{
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = __uint_as_float(lo[i]), x1 = __uint_as_float(hi[i]);
            const float c = cs[2 * i], s = cs[2 * i + 1];
            lo[i] = __float_as_uint(x0 * c - x1 * s);
            hi[i] = __float_as_uint(x0 * s + x1 * c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a0 = bf16_lo(lo[i]), a1 = bf16_hi(lo[i]), b0 = bf16_lo(hi[i]), b1 = bf16_hi(hi[i]);
            const float* t = cs + 4 * i;
            lo[i] = pack_bf16x2(a0 * t[0] - b0 * t[1], a1 * t[2] - b1 * t[3]);
            hi[i] = pack_bf16x2(a0 * t[1] + b0 * t[0], a1 * t[3] + b1 * t[2]);
        }
    }
}

constexpr int HEADS_PER_BLOCK = 64;

template <bool F32, bool HALF>
__global__ void __launch_bounds__(256) rope_q_kernel(RopeQArgs a)
{
    constexpr int E = F32 ? 4 : 8;             // elements of a 16-byte piece
    constexpr int NCS = HALF ? 2 * E : E;      // table floats of a thread's pairs
    const int t = blockIdx.x;
    const int h0 = blockIdx.y * HEADS_PER_BLOCK;
    const int nh = min(a.H - h0, HEADS_PER_BLOCK);
    const char* q = a.q + (int64_t)t * a.q_st + (int64_t)h0 * a.q_sh;
    char* out = a.out + (int64_t)t * a.o_st + (int64_t)h0 * a.o_sh;
    const uint32_t p0 = a.pos[t];
    const uint32_t p = p0 < (uint32_t)a.max_seq ? p0 : (uint32_t)a.max_seq - 1;

    // Rope part: `units` pieces (pairs of pieces in the half layout) per head.
    const int units = a.R / (HALF ? 2 * E : E);
    const int per_pass = 256 / units;          // heads the block covers at once (units <= 128)
    const int g = threadIdx.x % units;
    const int hh = threadIdx.x / units;
    constexpr int U = 4;
    if (hh < per_pass && hh < nh) {
        float cs[NCS];
        const float* f = a.freqs + (int64_t)p * a.R + g * NCS;
#pragma unroll
        for (int i = 0; i < NCS / 4; ++i) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(f + 4 * i);
            cs[4 * i] = v[0], cs[4 * i + 1] = v[1], cs[4 * i + 2] = v[2], cs[4 * i + 3] = v[3];
        }
        const int at = a.nope_bytes + g * 16;
        const int hi_at = a.R * (16 / E) / 2;   // bytes between the halves
        for (int h = hh; h < nh; h += U * per_pass) {
            u32x4 v[U], w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hu = min(h + u * per_pass, nh - 1);
                v[u] = ld16(q + (int64_t)hu * a.q_sh + at);
                if constexpr (HALF)
                    w[u] = ld16(q + (int64_t)hu * a.q_sh + at + hi_at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hu = h + u * per_pass;
                if (hu < nh) {
                    char* o = out + (int64_t)hu * a.o_sh + at;
                    if constexpr (HALF) {
                        rotate_halves<F32>(v[u], w[u], cs);
                        st16(o, v[u]);
                        st16(o + hi_at, w[u]);
                    } else {
                        st16(o, rotate_pairs<F32>(v[u], cs));
                    }
                }
            }
        }
    }
    if (!a.copy)
        return;
    const uint32_t pieces = (uint32_t)a.nope_bytes / 16;
    const uint32_t total = pieces * (uint32_t)nh;
    for (uint32_t i = threadIdx.x; i < total; i += U * 256) {
        u32x4 v[U];
        int64_t o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = min(i + u * 256, total - 1);
            const uint32_t h = k / pieces, c = k - h * pieces;
            v[u] = ld16(q + (int64_t)h * a.q_sh + c * 16);
            o[u] = (int64_t)h * a.o_sh + c * 16;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * 256 < total)
                st16(out + o[u], v[u]);
    }
}

}  // namespace

hipError_t launch_rope_freqs(const RopeFreqsArgs& a, hipStream_t s)
{
    const int64_t total = (int64_t)a.rows * a.pairs;
    const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 256 * 16);
    log_launch("rope_freqs_kernel", grid, 256, "rows=%d pairs=%d", a.rows, a.pairs);
    hipLaunchKernelGGL(rope_freqs_kernel, dim3(grid), dim3(256), 0, s, a, (int)((int64_t)grid * 256 / a.pairs),
                       (int)((int64_t)grid * 256 % a.pairs));
    return hipGetLastError();
}

hipError_t launch_rope_q(const RopeQArgs& a, bool f32, bool half, hipStream_t s)
{
    // A launch holds less than 2^32 threads in a dimension, and drops those past them without an error;
    // 65,535 blocks is the portable limit of the second one.
    constexpr int kMostTokens = 1 << 23, kMostHeads = 65535 * HEADS_PER_BLOCK;
    auto* kernel = f32 ? (half ? rope_q_kernel<true, true> : rope_q_kernel<true, false>)
                       : (half ? rope_q_kernel<false, true> : rope_q_kernel<false, false>);
    for (int64_t t0 = 0; t0 < a.T; t0 += kMostTokens)
        for (int64_t h0 = 0; h0 < a.H; h0 += kMostHeads) {
            RopeQArgs c = a;
            c.T = (int)std::min<int64_t>(a.T - t0, kMostTokens);
            c.H = (int)std::min<int64_t>(a.H - h0, kMostHeads);
            c.q += t0 * a.q_st + h0 * a.q_sh;
            c.out += t0 * a.o_st + h0 * a.o_sh;
            c.pos += t0;
            const dim3 grid(c.T, (c.H + HEADS_PER_BLOCK - 1) / HEADS_PER_BLOCK);
            log_launch("rope_q_kernel", grid.x * grid.y, 256, "T=%d H=%d R=%d f32=%d half=%d", c.T, c.H, c.R, f32, half);
            hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, c);
            if (hipError_t e = hipGetLastError())
                return e;
        }
    return hipSuccess;
}

}  // namespace mla
