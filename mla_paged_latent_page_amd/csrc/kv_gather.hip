// Rows of a paged K/V cache read back into contiguous buffers of keys and values: a bit copy,
// or e4m3 codes times their scale (one per 128 columns of the token row) rounded to bf16.
//
// Memory-bound.  The 16-byte pieces of all rows (keys, then values) are one flat run, of which
// a wave takes 256; lane j walks offsets -> page of the wave's row j, and every lane then has
// four loads in flight before its first store.  36,039 rows of 8 heads of 128 columns from e4m3 pages 53 us = 4.2 TB/s
// from memory (2, 4 or 8 pieces a lane differ by 4 %); a large copy reaches 5.1.
#include "kv.hpp"

namespace mla {
namespace {

constexpr int U = 4;                  // pieces of a lane
constexpr int WAVES = 4;
constexpr int PIECES = 64 * U;        // of a wave
constexpr int LEAST = 4;              // pieces a half row counts at least, so that a wave has less than 64 rows

__device__ inline uint64_t shfl64(uint64_t v, int lane)
{
    return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, lane, 64) |
           ((uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), lane, 64) << 32);
}

template <bool FP8>
__global__ void __launch_bounds__(64 * WAVES) kv_gather_kernel(KvGatherArgs a, uint32_t first_row, uint32_t rows,
                                                               uint32_t granules)
{
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t per_half = max(granules, (uint32_t)LEAST), per_row = 2 * per_half;
    const uint32_t base = (blockIdx.x * WAVES + wave) * PIECES;   // below 2^31: see the launch
    const uint32_t j0 = base / per_row, r0 = base - j0 * per_row;
    if (j0 >= rows)
        return;
    const uint32_t row0 = first_row + j0;
    const uint32_t last = min((r0 + PIECES - 1) / per_row, rows - 1 - j0);

    // Lane j: where row row0 + j lies.
    uint32_t cnt = 0;
    for (uint32_t c = 0; c < a.L.batch; c += 256) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t k = c + i * 64 + lane;
            o[i] = k < a.L.batch ? a.bro[k] : 0xFFFFFFFFu;
        }
        for (uint32_t j = 0; j <= last; ++j) {
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                n += (uint32_t)__popcll(__ballot(o[i] <= row0 + j));
            cnt += (uint32_t)lane == j ? n : 0;
        }
    }
    uint64_t off = 0, soff = 0;
    if ((uint32_t)lane <= last) {
        const uint32_t b = cnt == 0 ? 0u : min(cnt, a.L.batch) - 1;
        const uint32_t p = a.co[b] + (row0 + lane - a.bro[b]);
        off = (uint64_t)token_offset(a.L, b, p);
        if (FP8)
            soff = (uint64_t)token_offset(a.Ls, b, p);
    }

    uint32_t row[U], gran[U];
    bool val[U], on[U];
    u32x4 x[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t f = r0 + u * 64 + lane;
        row[u] = f / per_row;
        const uint32_t g = f - row[u] * per_row;
        val[u] = g >= per_half;
        gran[u] = val[u] ? g - per_half : g;
        on[u] = row[u] <= last && gran[u] < granules;
        const char* src = a.L.base + shfl64(off, (int)(row[u] & 63)) + (val[u] ? a.L.stride_kv : 0) + (int64_t)gran[u] * 16;
        x[u] = on[u] ? ld16(src) : u32x4{0u, 0u, 0u, 0u};
        if constexpr (FP8) {
            const char* sc = a.Ls.base + shfl64(soff, (int)(row[u] & 63)) + (val[u] ? a.Ls.stride_kv : 0);
            scale[u] = on[u] ? *reinterpret_cast<const float*>(sc + gran[u] / 8 * 4) : 0.0f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!on[u])
            continue;
        char* dst = (val[u] ? a.v : a.k) + ((int64_t)(row0 + row[u]) * granules + gran[u]) * (FP8 ? 32 : 16);
        if constexpr (!FP8) {
            st16(dst, x[u]);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[u][i], false);
                const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[u][i], true);
                w[2 * i] = pack_bf16x2(lo[0] * scale[u], lo[1] * scale[u]);
                w[2 * i + 1] = pack_bf16x2(hi[0] * scale[u], hi[1] * scale[u]);
            }
            st16(dst, u32x4{w[0], w[1], w[2], w[3]});
            st16(dst + 16, u32x4{w[4], w[5], w[6], w[7]});
        }
    }
}

}  // namespace

hipError_t launch_kv_gather(const KvGatherArgs& a, KvKind kind, hipStream_t s)
{
    const bool fp8 = kind == KV_E4M3;
    const int64_t granules = (int64_t)a.HD * (fp8 ? 1 : kind == KV_F32 ? 4 : 2) / 16;
    auto* kernel = fp8 ? kv_gather_kernel<true> : kv_gather_kernel<false>;
    // Pieces of a launch are numbered in 32 bits.
    const int64_t per_row = 2 * (granules > LEAST ? granules : LEAST);
    const int64_t most = (int64_t(1) << 30) / per_row;
    for (int64_t first = 0; first < a.M; first += most) {
        const int64_t rows = a.M - first < most ? a.M - first : most;
        const unsigned grid = (unsigned)((rows * per_row + PIECES * WAVES - 1) / (PIECES * WAVES));
        log_launch(fp8 ? "kv_gather_kernel<e4m3>" : "kv_gather_kernel", grid, 64 * WAVES, "M=%d HD=%d", a.M, a.HD);
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * WAVES), 0, s, a, (uint32_t)first, (uint32_t)rows,
                           (uint32_t)granules);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    return hipSuccess;
}

}  // namespace mla
