// Tree attention on the matrix cores: rows of 576 columns (512 latent + 64 rope),
// bf16 cache (see tree_attention.hip for the operator and the general form).
#include <algorithm>

#include "step.hpp"

namespace mla {
namespace {

constexpr int D = 576, K = 512;              // row width, latent columns
constexpr int TILE = 32;                     // cache rows per step
constexpr int BLOCKS = D / 64;               // 64-column blocks of a tile: 32 rows x 128 bytes each
constexpr int BLOCK_BYTES = TILE * 128;
constexpr int STAGE = BLOCKS * BLOCK_BYTES;  // 36,864 bytes
constexpr int STAGES = 4;
constexpr int WAVES = 4;
constexpr int LOADS = BLOCKS;                // LDS loads per wave and tile
constexpr int PIECE_WAVE = 32 * (K + 2);     // floats of one wave's partial result: 32 rows, maximum, sum
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.0f;               // the reference maximum may lag by 2^8

typedef short v4i16 __attribute__((ext_vector_type(4)));

struct MfmaParams {
    TreeAttentionArgs a;
    uint32_t ps_magic, ps_shift;             // p / page_size = mulhi(p, magic) >> shift for p < 2^31
    uint32_t piece;                          // floats of a partial result slot
    int min_tiles;                           // least tiles of a workgroup's share
};

__device__ inline uint64_t uniform(uint64_t v)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
           ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32);
}
__device__ inline uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// Rows of a request and its share of the work: nm items of 128 query rows, nt tiles each.
struct Request {
    uint32_t b, t0, n, cached, len, nm, nt;
    uint64_t base;                           // tiles of all requests before it
};

__device__ inline Request request_at(const TreeAttentionArgs& a, uint32_t b)
{
    Request r;
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    r.b = b;
    r.t0 = min(a.iro[b], end);
    const uint32_t t1 = min(a.iro[b + 1], end);
    r.n = t1 > r.t0 ? t1 - r.t0 : 0;
    r.cached = min(a.cache_len[b], a.capacity);
    r.len = min(r.cached + r.n, a.capacity);
    r.nm = (uint32_t)(((uint64_t)r.n * a.H + kAttnRows - 1) / kAttnRows);
    r.nt = (r.len + TILE - 1) / TILE;
    return r;
}

__device__ inline uint64_t wave_inclusive(uint64_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t up = __shfl_up(v, d);
        v += lane >= d ? up : 0;
    }
    return v;
}

// Tiles of all requests (every wave computes it for itself).
__device__ inline uint64_t total_tiles(const TreeAttentionArgs& a, int lane)
{
    uint64_t sum = 0;
    for (uint32_t b0 = 0; b0 < a.L.batch; b0 += 64) {
        uint64_t v = 0;
        if (b0 + lane < a.L.batch) {
            const Request r = request_at(a, b0 + lane);
            v = (uint64_t)r.nm * r.nt;
        }
        sum += uniform(__shfl(wave_inclusive(v, lane), 63));
    }
    return sum;
}

// A wave-uniform request, in scalar registers.
__device__ inline Request uniform(Request r)
{
    return Request{uniform(r.b), uniform(r.t0), uniform(r.n), uniform(r.cached), uniform(r.len), uniform(r.nm),
                   uniform(r.nt), uniform(r.base)};
}

// The request that holds tile u (u < total).
__device__ inline Request find_tile(const TreeAttentionArgs& a, uint64_t u, int lane)
{
    uint64_t before = 0;
    for (uint32_t b0 = 0; b0 < a.L.batch; b0 += 64) {
        uint64_t v = 0;
        if (b0 + lane < a.L.batch) {
            const Request r = request_at(a, b0 + lane);
            v = (uint64_t)r.nm * r.nt;
        }
        const uint64_t scan = wave_inclusive(v, lane);
        const uint64_t all = uniform(__shfl(scan, 63));
        if (u < before + all) {
            const int k = __ffsll((unsigned long long)__ballot(u < before + scan)) - 1;
            Request r = request_at(a, b0 + k);
            r.base = before + __shfl(scan - v, k);
            return uniform(r);
        }
        before += all;
    }
    return Request{};
}

// The tiles are cut into `groups` equal shares.  A cut that falls within `snap` tiles of
// an item's end is moved there (the item is then not split for so little).
struct Cuts {
    uint64_t total;
    uint32_t groups, snap;
    __device__ uint64_t raw(uint32_t w) const { return total * w / groups; }
    // Cut w, where [lo, hi) is the item that raw(w) lies in.
    __device__ uint64_t at(uint64_t r, uint64_t lo, uint64_t hi) const
    {
        return r - lo <= snap ? lo : hi - r <= snap ? hi : r;
    }
};

__device__ inline Cuts make_cuts(const MfmaParams& P, int lane)
{
    Cuts c;
    c.total = total_tiles(P.a, lane);
    const uint64_t want = (c.total + P.min_tiles - 1) / P.min_tiles;
    c.groups = want < 1 ? 1u : want > kAttnGroups ? (uint32_t)kAttnGroups : (uint32_t)want;
    c.snap = (uint32_t)min(c.total / c.groups / 8, (uint64_t)1 << 20);
    return c;
}

__device__ inline v4i16 lds_tr16(const char* p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16*)(__attribute__((address_space(3))) void*)p);
}

__device__ inline float swap32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    // r[0]: lanes 32.. hold the low half's value; r[1]: lanes 0..31 hold the high half's
    return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
}

// 16 bytes per lane from a uniform base and a 32-bit lane offset into LDS at lds + 16 * lane.
__device__ inline void load_lds(const char* base, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory", "m0");
}

template <int N>
__device__ inline void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One product with its sums in ordinary registers: the output sums take all 256 accumulation
// registers, and the compiler would put these there too.  It does not see that this is a matrix
// instruction, so the last one of a chain waits for its result before anything can read it
// (12 wait states after 8 passes; back-to-back products into the same registers need none).
__device__ inline void mfma_first(f32x16& acc, bf16x8 x, bf16x8 y)
{
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(acc) : "v"(x), "v"(y));
}
__device__ inline void mfma_next(f32x16& acc, bf16x8 x, bf16x8 y)
{
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(acc) : "v"(x), "v"(y));
}
__device__ inline void mfma_last(f32x16& acc, bf16x8 x, bf16x8 y)
{
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0\n\ts_nop 13" : "+v"(acc) : "v"(x), "v"(y));
}

// Element e of an output sum times f, in its accumulation register (written out, as the
// compiler would otherwise keep all the sums in ordinary registers between the steps).
__device__ inline void scale_sum(f32x16& o, int e, float f)
{
    float x = o[e], t;
    asm("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1"
        : "+a"(x), "=&v"(t)
        : "v"(f));
    o[e] = x;
}

__device__ inline bool nonfinite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Final output of one lane pair's row: eight features per 16-byte store.
__device__ inline void store_row(uint16_t* out, const f32x16 (&o)[16], float inv, bool valid, int half)
{
#pragma unroll
    for (int fb = 0; fb < 16; ++fb)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            uint32_t x0 = pack_bf16x2(o[fb][i] * inv, o[fb][i + 1] * inv);
            uint32_t x1 = pack_bf16x2(o[fb][i + 2] * inv, o[fb][i + 3] * inv);
            uint32_t y0 = pack_bf16x2(o[fb][i + 4] * inv, o[fb][i + 5] * inv);
            uint32_t y1 = pack_bf16x2(o[fb][i + 6] * inv, o[fb][i + 7] * inv);
            const auto a = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
            if (valid)
                st16(out + fb * 32 + 2 * i + 8 * half, u32x4{a[0], b[0], a[1], b[1]});
            __builtin_amdgcn_sched_barrier(0);
        }
}

template <bool PAGE8>
__global__ void __launch_bounds__(64 * WAVES, 1) tree_attention_mfma(MfmaParams P)
{
    __shared__ __attribute__((aligned(1024))) char smem[STAGES * STAGE];
    const TreeAttentionArgs& a = P.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;

    const Cuts cuts = make_cuts(P, lane);
    // Neighbouring shares go to one XCD (block i runs on XCD i % 8): items of one request
    // then read the same rows through one L2.
    const uint32_t per = (cuts.groups + 7) / 8;
    const uint32_t w = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || w >= cuts.groups || cuts.total == 0)
        return;
    Request r = find_tile(a, cuts.raw(w), lane);
    uint64_t u, stop;
    {
        const uint64_t raw = cuts.raw(w), lo = r.base + (raw - r.base) / r.nt * r.nt;
        u = cuts.at(raw, lo, lo + r.nt);
        if (w + 1 == cuts.groups) {
            stop = cuts.total;
        } else {
            const uint64_t raw1 = cuts.raw(w + 1);
            const Request r1 = find_tile(a, raw1, lane);
            const uint64_t lo1 = r1.base + (raw1 - r1.base) / r1.nt * r1.nt;
            stop = cuts.at(raw1, lo1, lo1 + r1.nt);
        }
    }
    u = w == 0 ? 0 : uniform(u);
    stop = uniform(stop);

    // Lane-constant offsets.  A tile is stored as 9 blocks of 32 rows x 128 bytes; the
    // 16-byte granule g of row x sits at g ^ f(x), f(x) = 2 (x % 4) + (x / 4) % 2, which
    // spreads both the 8 rows of a phase of the 16-byte reads and the 4 rows of a phase
    // of the transposing reads over all banks.
    const uint32_t fx = (uint32_t)(((lane >> 3) & 3) << 1 | ((lane >> 5) & 1));   // row lane / 8
    const uint32_t load_off = (((uint32_t)lane & 7) ^ fx) * 16;
    const uint32_t fk = (uint32_t)((col & 3) << 1 | ((col >> 2) & 1));
    uint32_t k_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        k_off[s] = col * 128 + (((2 * s + half) ^ fk) * 16);
    // Transposing reads: lane c of a 16-lane group addresses row c / 4 and 8 bytes of columns.
    const uint32_t c16 = lane & 15, vrow = 4 * half + (c16 >> 2);
    const uint32_t fv = (uint32_t)(((c16 >> 2) & 3) << 1 | half);
    uint32_t v_off[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
        v_off[s] = vrow * 128 + (((uint32_t)(4 * s + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1)) ^ fv) * 16) + (c16 & 1) * 8;
    const uint32_t lds0 = lds_addr(smem) + wave * 1024;
    const float c = a.scale * kLog2e;

    while (u < stop) {
        while (u >= r.base + (uint64_t)r.nm * r.nt) {
            const uint64_t next = r.base + (uint64_t)r.nm * r.nt;
            r = request_at(a, r.b + 1);
            r.base = next;
            r = uniform(r);
        }
        const uint32_t m = uniform((uint32_t)((u - r.base) / r.nt));
        const uint64_t item = r.base + (uint64_t)m * r.nt;
        const uint32_t tile0 = uniform((uint32_t)(u - item));
        const uint32_t tile1 = uniform((uint32_t)(min(stop, item + r.nt) - item));
        u = uniform(item + tile1);
        const uint32_t n_tiles = tile1 - tile0;
        const uint32_t len = r.len, cached = r.cached;
        const uint32_t table_row = r.b * a.L.max_pages;   // checked on the host: below 2^32

        const uint32_t rows = r.n * (uint32_t)a.H;                 // below 2^31 / D
        const uint32_t row = m * kAttnRows + wave * 32 + col;
        const bool live = uniform(m * kAttnRows + wave * 32) < rows;
        const bool valid = row < rows;
        const uint32_t qrow = r.t0 * (uint32_t)a.H + min(row, rows - 1);
        const uint32_t tok = min(row, rows - 1) / (uint32_t)a.H;   // token of the request

        __syncthreads();   // the stages of the item before are no longer read

        // Loads of one tile: this wave fetches rows 8 wave .. 8 wave + 7, lane l granule l % 8
        // of every block of row l / 8.  Rows past the end repeat the last one.
        auto issue = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t stage = (t & (STAGES - 1)) * STAGE + lds0;
            const uint32_t p0 = (tile0 + t) * TILE + wave * 8;
            if constexpr (PAGE8) {
                uint32_t pg = p0 < len ? p0 : (len - 1) & ~7u;
                const uint32_t lp = __umulhi(pg, P.ps_magic) >> P.ps_shift;
                const uint32_t* entry = a.L.page_table + table_row + min(lp, a.L.max_pages - 1);
                uint32_t id = *(const __attribute__((address_space(4))) uint32_t*)(uint64_t)entry;
                id = min(id, a.L.num_pages - 1);
                const char* base = a.L.base + (int64_t)id * a.L.stride_page +
                                   (int64_t)(pg - lp * a.L.page_size) * a.L.stride_token;
                const uint32_t last = len - 1 - pg;
                const uint32_t voff = min((uint32_t)lane >> 3, last) * (uint32_t)a.L.stride_token + load_off;
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j)
                    load_lds(base, voff + j * 128, stage + j * BLOCK_BYTES);
            } else {
                const uint32_t p = min(p0 + ((uint32_t)lane >> 3), len - 1);
                const uint32_t lp = p / a.L.page_size;
                const uint32_t id = min(a.L.page_table[table_row + min(lp, a.L.max_pages - 1)], a.L.num_pages - 1);
                const char* src = a.L.base + (int64_t)id * a.L.stride_page +
                                  (int64_t)(p - lp * a.L.page_size) * a.L.stride_token + load_off;
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j)
                    asm_gld16_lds(src + j * 128, stage + j * BLOCK_BYTES);
            }
        };

        issue(0);
        if (n_tiles > 1)
            issue(1);
        if (n_tiles > 2)
            issue(2);

        // Start of step t: tile t + 1 has landed for every wave and every wave is done with
        // tile t - 1, whose stage takes tile t + 3.  Returns whether the tile has drafted rows.
        auto enter = [&](uint32_t t) __attribute__((always_inline)) {
            if (t + 2 < n_tiles)
                wait_loads<LOADS>();
            else
                wait_loads<0>();
            lds_barrier();
            if (t + 3 < n_tiles)
                issue(t + 3);
            const uint32_t p0 = (tile0 + t) * TILE;
            const bool masked = p0 + TILE > cached;
            if (masked && (r.n > 1 || a.mask)) {
                // Drafted rows may be hidden from some tokens and hold anything: a weight of 0
                // would turn their infinities and NaN into NaN, so those become 0 here (a token
                // that sees such a row has a NaN weight for it already).
                char* mine = smem + (t & (STAGES - 1)) * STAGE + wave * 1024 + lane * 16;
                if (p0 + wave * 8 + (lane >> 3) >= cached)
                    for (int j = 0; j < BLOCKS - 1; ++j) {
                        u32x4 v = lds_ld16(mine + j * BLOCK_BYTES);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = nonfinite16(v[e]) ? v[e] & 0xFFFF0000u : v[e];
                            v[e] = nonfinite16(v[e] >> 16) ? v[e] & 0xFFFFu : v[e];
                        }
                        lds_st16(mine + j * BLOCK_BYTES, v);
                    }
                lds_barrier();
            }
            return masked;
        };
        // Bits of the tile's rows that this lane's token sees.
        auto seen_rows = [&](uint32_t p0) __attribute__((always_inline)) {
            const uint32_t room = min(len - p0, (uint32_t)TILE);
            uint32_t seen;
            if (a.mask) {
                const int64_t* words = reinterpret_cast<const int64_t*>(a.mask) + (int64_t)(r.t0 + tok) * a.words;
                const int64_t j0 = (int64_t)p0 - cached;
                uint64_t bits;
                if (j0 < 0) {
                    bits = ((uint64_t)words[0] << -j0) | ((1ull << -j0) - 1);   // -32 < j0
                } else {
                    const uint32_t wd = (uint32_t)(j0 >> 6), sh = (uint32_t)j0 & 63;
                    bits = wd < (uint32_t)a.words ? (uint64_t)words[wd] >> sh : 0;
                    if (sh > 32 && wd + 1 < (uint32_t)a.words)
                        bits |= (uint64_t)words[wd + 1] << (64 - sh);
                }
                seen = (uint32_t)bits;
            } else {
                const int64_t upto = (int64_t)cached + tok + 1 - p0;
                seen = upto >= 32 ? ~0u : upto <= 0 ? 0u : (1u << upto) - 1;
            }
            return seen & (room >= 32 ? ~0u : (1u << room) - 1);
        };

        if (n_tiles > 2)
            wait_loads<2 * LOADS>();
        else if (n_tiles > 1)
            wait_loads<LOADS>();
        else
            wait_loads<0>();
        lds_barrier();
        if (!live) {
            // No query rows for this wave: it only loads.
            for (uint32_t t = 0; t < n_tiles; ++t)
                enter(t);
            continue;
        }

        // Query fragments: lane holds features 16 s + 8 half .. + 7 of its row.
        bf16x8 q[D / 16];
        {
            const char* src = static_cast<const char*>(a.q) + (int64_t)qrow * (D * 2) + half * 16;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                q[s] = as_bf16x8(ld16(src + s * 32));
        }
        f32x16 o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] = f32x16{0.f};
        float mref = -INFINITY, l = 0.0f;

        // Scores of tile t: lane (col, half) gets rows 8 (i / 4) + 4 half + i % 4 for its query.
        // `between(k)` is work done while the matrix cores run group k of 3 products.
        auto scores = [&](uint32_t t, auto between) __attribute__((always_inline)) {
            const char* st = smem + (t & (STAGES - 1)) * STAGE;
            auto frag = [&](int k) __attribute__((always_inline)) {
                return as_bf16x8(lds_ld16(st + k_off[k & 3] + (k >> 2) * BLOCK_BYTES));
            };
            f32x16 acc;
            bf16x8 f[2][3];
#pragma unroll
            for (int j = 0; j < 3; ++j)
                f[0][j] = frag(j);
#pragma unroll
            for (int k = 0; k < 12; ++k) {
                if (k < 11)
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        f[(k + 1) & 1][j] = frag(3 * (k + 1) + j);
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    if (k == 0 && j == 0)
                        mfma_first(acc, f[0][0], q[0]);
                    else if (k == 11 && j == 2)
                        mfma_last(acc, f[1][2], q[35]);
                    else
                        mfma_next(acc, f[k & 1][j], q[3 * k + j]);
                }
                between(k);
                __builtin_amdgcn_sched_barrier(0);
            }
            return acc;
        };
        f32x16 raw = scores(0, [](int) {});

        for (uint32_t t = 0; t < n_tiles; ++t) {
            const bool masked = enter(t);
            const uint32_t p0 = (tile0 + t) * TILE;
            float s[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = raw[i] * c;
            if (masked) {
                const uint32_t seen = seen_rows(p0);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] = (seen >> (8 * (i >> 2) + 4 * half + (i & 3))) & 1 ? s[i] : -INFINITY;
            }
            float mx = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i)
                mx = fmaxf(mx, s[i]);
            mx = fmaxf(mx, swap32(mx));
            if (__ballot(mx > mref + kSlack)) {
                const float next = fmaxf(mref, mx);
                const float keep = next == mref ? 1.0f : __builtin_amdgcn_exp2f(mref - next);
                mref = next;
                l *= keep;
#pragma unroll
                for (int i = 0; i < 16; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        scale_sum(o[i], e, keep);
            }
            const float ref = mref == -INFINITY ? 0.0f : mref;
            __builtin_amdgcn_sched_barrier(0);
            // The scores of the next tile; the weights of this one between them.  (The last
            // step computes scores that nobody uses, from whatever the stage holds.)
            uint32_t pk[8];
            float sum = 0.0f;
            raw = scores(t + 1, [&](int k) __attribute__((always_inline)) {
                if (k < 8) {
                    const float e0 = __builtin_amdgcn_exp2f(s[2 * k] - ref);
                    const float e1 = __builtin_amdgcn_exp2f(s[2 * k + 1] - ref);
                    sum += e0 + e1;
                    pk[k] = pack_bf16x2(e0, e1);
                }
            });
            l += sum;
            const bf16x8 pf[2] = {as_bf16x8(u32x4{pk[0], pk[1], pk[2], pk[3]}),
                                  as_bf16x8(u32x4{pk[4], pk[5], pk[6], pk[7]})};
            const char* st = smem + (t & (STAGES - 1)) * STAGE;
            auto vfrag = [&](int fb, int ks) __attribute__((always_inline)) {
                const char* v = st + v_off[fb & 1] + (fb >> 1) * BLOCK_BYTES + ks * 2048;
                const v4i16 lo = lds_tr16(v), hi = lds_tr16(v + 1024);
                return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            };
            bf16x8 vf[2][2];
            vf[0][0] = vfrag(0, 0);
            vf[0][1] = vfrag(0, 1);
#pragma unroll
            for (int fb = 0; fb < 16; ++fb) {
                if (fb < 15) {
                    vf[(fb + 1) & 1][0] = vfrag(fb + 1, 0);
                    vf[(fb + 1) & 1][1] = vfrag(fb + 1, 1);
                }
                o[fb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[fb & 1][0], pf[0], o[fb], 0, 0, 0);
                o[fb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[fb & 1][1], pf[1], o[fb], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        }

        l += swap32(l);
        if (tile0 == 0 && tile1 == r.nt) {
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            store_row(static_cast<uint16_t*>(a.out) + (int64_t)qrow * K, o, inv, valid, half);
            if (a.lse && valid && half == 0)
                a.lse[qrow] = l == 0.0f ? -INFINITY : mref * kLn2 + __logf(l);
        } else {
            // A share of the item: sums, maximum and sum as they are, in lane order.
            float* piece = a.ws + (size_t)(2 * w + (tile0 == 0 ? 1 : 0)) * P.piece + (size_t)wave * PIECE_WAVE;
#pragma unroll
            for (int fb = 0; fb < 16; ++fb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    *reinterpret_cast<f32x4*>(piece + ((fb * 4 + i) * 64 + lane) * 4) =
                        f32x4{o[fb][4 * i], o[fb][4 * i + 1], o[fb][4 * i + 2], o[fb][4 * i + 3]};
                    __builtin_amdgcn_sched_barrier(0);
                }
            if (half == 0) {
                piece[32 * K + col] = mref;
                piece[32 * K + 32 + col] = l;
            }
        }
    }
}

// Joins the pieces of split items.  Block (w, g): if cut w lies inside an item, rows 32 g ..
// of that item; the blocks of all cuts inside one item share its 64 column groups (quads of
// features in the lane order of the accumulators).
__global__ void __launch_bounds__(256) tree_attention_join(MfmaParams P)
{
    const TreeAttentionArgs& a = P.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const uint32_t w = 1 + (blockIdx.x >> 2), g = blockIdx.x & 3;
    const Cuts cuts = make_cuts(P, lane);
    if (w >= cuts.groups || cuts.total == 0)
        return;
    const uint64_t raw = cuts.raw(w);
    const Request r = find_tile(a, raw, lane);
    const uint32_t m = (uint32_t)((raw - r.base) / r.nt);
    const uint64_t lo = r.base + (uint64_t)m * r.nt, hi = lo + r.nt;
    if (cuts.at(raw, lo, hi) != raw || raw == lo)
        return;
    const uint32_t rows = r.n * (uint32_t)a.H;
    const uint32_t row = m * kAttnRows + g * 32 + col;
    if (m * kAttnRows + g * 32 >= rows)
        return;
    // First and last cut inside the item.
    uint32_t w0 = w, w1 = w;
    while (w0 > 1 && cuts.raw(w0 - 1) > lo && cuts.at(cuts.raw(w0 - 1), lo, hi) == cuts.raw(w0 - 1))
        --w0;
    while (w1 + 1 < cuts.groups && cuts.raw(w1 + 1) < hi && cuts.at(cuts.raw(w1 + 1), lo, hi) == cuts.raw(w1 + 1))
        ++w1;
    const uint32_t pieces = w1 - w0 + 2;
    // Piece 0 is the end of share w0 - 1, piece k the start of share w0 + k - 1.
    auto piece = [&](uint32_t k) __attribute__((always_inline)) {
        const uint32_t slot = k == 0 ? 2 * (w0 - 1) + 1 : 2 * (w0 + k - 1);
        return a.ws + (size_t)slot * P.piece + (size_t)g * PIECE_WAVE;
    };
    float mx = -INFINITY;
    for (uint32_t k = 0; k < pieces; ++k)
        mx = fmaxf(mx, piece(k)[32 * K + col]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    for (uint32_t k = 0; k < pieces; ++k)
        l += piece(k)[32 * K + 32 + col] * __builtin_amdgcn_exp2f(piece(k)[32 * K + col] - ref);
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const uint32_t qrow = r.t0 * (uint32_t)a.H + min(row, rows - 1);
    const uint32_t share = (w - w0) * 4 + wave, shares = (w1 - w0 + 1) * 4;
    if (a.lse && share == 0 && half == 0 && row < rows)
        a.lse[qrow] = l == 0.0f ? -INFINITY : mx * kLn2 + __logf(l);
    for (uint32_t quad = share; quad < 64; quad += shares) {
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        constexpr int U = 8;
        for (uint32_t k0 = 0; k0 < pieces; k0 += U) {
            f32x4 v[U];
            float f[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float* p = piece(min(k0 + i, pieces - 1));
                v[i] = *reinterpret_cast<const f32x4*>(p + (quad * 64 + lane) * 4);
                f[i] = p[32 * K + col];
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (k0 + i < pieces)
                    sum += v[i] * __builtin_amdgcn_exp2f(f[i] - ref);
        }
        sum *= inv;
        if (row < rows)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + (int64_t)qrow * K + (quad >> 2) * 32 +
                                      (quad & 3) * 8 + half * 4) =
                u32x2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
    }
}

}  // namespace

bool tree_attention_mfma_fits(const TreeAttentionArgs& a, AttnKind kind)
{
    return kind == ATTN_BF16 && a.D == D && a.K == K && a.L.stride_token < (int64_t(1) << 28) &&
           (uint64_t)a.L.batch * a.L.max_pages < (uint64_t(1) << 32);
}

hipError_t launch_tree_attention_mfma(const TreeAttentionArgs& a, hipStream_t s)
{
    MfmaParams P{};
    P.a = a;
    const uint32_t ps = a.L.page_size;
    if (ps % 8 == 0) {
        // ps >= 8, positions below 2^31: with 2^(s-1) < ps <= 2^s, ceil(2^(31+s) / ps) fits 32 bits
        // and mulhi(p, that) >> (s - 1) is the quotient.
        uint32_t sh = 3;
        while ((uint64_t(1) << sh) < ps)
            ++sh;
        P.ps_magic = (uint32_t)(((uint64_t(1) << (31 + sh)) + ps - 1) / ps);
        P.ps_shift = sh - 1;
    }
    const int64_t waves = (std::min<int64_t>((int64_t)a.T * a.H, kAttnRows) + 31) / 32;
    P.piece = (uint32_t)(waves * PIECE_WAVE);
    P.min_tiles = 4;
    log_launch("tree_attention_mfma", kAttnGroups, 64 * WAVES, "T=%d H=%d page_size=%u", a.T, a.H, ps);
    if (ps % 8 == 0)
        hipLaunchKernelGGL(tree_attention_mfma<true>, dim3(kAttnGroups), dim3(64 * WAVES), 0, s, P);
    else
        hipLaunchKernelGGL(tree_attention_mfma<false>, dim3(kAttnGroups), dim3(64 * WAVES), 0, s, P);
    if (hipError_t e = hipGetLastError())
        return e;
    log_launch("tree_attention_join", (kAttnGroups - 1) * 4, 256, "T=%d H=%d", a.T, a.H);
    hipLaunchKernelGGL(tree_attention_join, dim3((kAttnGroups - 1) * 4), dim3(256), 0, s, P);
    return hipGetLastError();
}

}  // namespace mla
