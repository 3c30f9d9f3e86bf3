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
    uint32_t base;                           // tiles of all requests before it
    uint32_t items;                          // items of all requests before it
};

__device__ inline Request request_at(const TreeAttentionArgs& a, uint32_t b)
{
    Request r{};
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    r.b = b;
    r.t0 = min(a.iro[b], end);
    const uint32_t t1 = min(a.iro[b + 1], end);
    r.n = t1 > r.t0 ? t1 - r.t0 : 0;
    r.cached = min(a.cache_len[b], a.capacity);
    r.len = min(r.cached + r.n, a.capacity);
    r.nm = (r.n * (uint32_t)a.H + kAttnRows - 1) / kAttnRows;   // n * H below 2^31 / D
    r.nt = (r.len + TILE - 1) / TILE;
    return r;
}

// A wave-uniform request, in scalar registers.
__device__ inline Request uniform(Request r)
{
    return Request{uniform(r.b), uniform(r.t0), uniform(r.n), uniform(r.cached), uniform(r.len), uniform(r.nm),
                   uniform(r.nt), uniform(r.base)};
}

__device__ inline uint32_t wave_inclusive(uint32_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(v, d);
        v += lane >= d ? up : 0u;
    }
    return v;
}

// The schedule: all tiles (of all items of all requests, in that order) in equal shares.
// A cut that falls within `snap` tiles of an item's end is moved there: the item is then
// not split for so little.  Every wave works it out for itself; the requests of the last 64
// looked at stay in its lanes.  The host has checked that the tiles number below 2^31.
struct Schedule {
    const TreeAttentionArgs& a;
    int lane;
    uint32_t total, groups, share, rest, snap;
    uint32_t first;                          // first request in the lanes
    uint32_t before;                         // tiles before it
    Request mine;
    uint32_t scan;                           // tiles up to and including mine, from `before`

    __device__ void load(uint32_t b0, uint32_t tiles_before)
    {
        first = b0;
        before = tiles_before;
        mine = Request{};
        if (b0 + lane < a.L.batch)
            mine = request_at(a, b0 + lane);
        scan = wave_inclusive(mine.nm * mine.nt, lane);
    }
    __device__ uint32_t loaded() const { return (uint32_t)__builtin_amdgcn_readlane((int)scan, 63); }

    __device__ Schedule(const TreeAttentionArgs& args, int l, uint32_t min_tiles) : a(args), lane(l)
    {
        load(0, 0);
        total = loaded();
        for (uint32_t b0 = 64; b0 < a.L.batch; b0 += 64) {
            load(b0, total);
            total += loaded();
        }
        if (a.L.batch > 64)
            load(0, 0);
        const uint32_t want = (total + min_tiles - 1) / min_tiles;
        groups = want < 1 ? 1u : want > kAttnGroups ? (uint32_t)kAttnGroups : want;
        share = total / groups;
        rest = total - share * groups;
        snap = share / 32;
    }
    // Cut w before snapping, and the first cut past position x.
    __device__ uint32_t raw(uint32_t w) const { return share * w + min(w, rest); }
    __device__ uint32_t first_cut_past(uint32_t x) const
    {
        return x < rest * (share + 1) ? x / (share + 1) + 1 : rest + (x - rest * (share + 1)) / share + 1;
    }
    // The request that holds tile u < total.
    __device__ Request find(uint32_t u)
    {
        if (u < before)
            load(0, 0);
        while (u >= before + loaded())
            load(first + 64, before + loaded());
        const int k = __ffsll((unsigned long long)__ballot(u < before + scan)) - 1;
        Request r;
        auto get = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, k); };
        r.b = first + k;
        r.t0 = get(mine.t0);
        r.n = get(mine.n);
        r.cached = get(mine.cached);
        r.len = get(mine.len);
        r.nm = get(mine.nm);
        r.nt = get(mine.nt);
        r.base = uniform(before + get(scan) - r.nm * r.nt);
        return r;
    }
    // Cut w, and the request it lies in.
    __device__ uint32_t cut(uint32_t w, Request& r)
    {
        const uint32_t x = raw(w);
        r = find(x);
        const uint32_t lo = r.base + (x - r.base) / r.nt * r.nt;
        return x - lo <= snap ? lo : lo + r.nt - x <= snap ? lo + r.nt : x;
    }
};

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

// 16 bytes per lane into LDS at lds + 16 * lane, by all lanes or (on = 0, else ~0) none: from a
// uniform base and a 32-bit lane offset, or from a lane address.
__device__ inline void load_lds(const char* base, uint32_t voff, uint32_t lds, uint32_t on)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(voff), "s"(base), "s"(on)
                 : "memory", "m0");
}
__device__ inline void load_lds(const char* src, uint32_t lds, uint32_t on)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(src), "s"(on)
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

    Schedule sched(a, lane, P.min_tiles);
    // Neighbouring shares go to one XCD (block i runs on XCD i % 8): items of one request
    // then read the same rows through one L2.
    const uint32_t per = (sched.groups + 7) / 8;
    const uint32_t w = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || w >= sched.groups || sched.total == 0)
        return;
    Request r;
    uint32_t stop = sched.total;
    if (w + 1 < sched.groups)
        stop = uniform(sched.cut(w + 1, r));
    uint32_t u = uniform(sched.cut(w, r));

    // Lane-constant offsets.  A tile is stored as 9 blocks of 32 rows x 128 bytes; the
    // 16-byte granule g of row x sits at g ^ f(x), where bits 2, 1 and 0 of f(x) are bits 1, 2
    // and 3 of x: 16 rows of the 16-byte reads (two rows fill the 256 bytes of all banks) and
    // 4 rows x 64 bytes of the transposing reads then fall on different banks.
    auto f = [](uint32_t x) { return (x >> 1 & 1) << 2 | (x >> 2 & 1) << 1 | (x >> 3 & 1); };
    const uint32_t load_off = (((uint32_t)lane & 7) ^ f(wave * 8 + (lane >> 3))) * 16;
    const uint32_t fk = f(col);
    uint32_t k_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        k_off[s] = col * 128 + (((2 * s + half) ^ fk) * 16);
    // Transposing reads: lane c of a 16-lane group addresses row c / 4 and 8 bytes of columns.
    const uint32_t c16 = lane & 15, vrow = 4 * half + (c16 >> 2);
    uint32_t v_off[2][2];   // [feature block parity][rows vrow or vrow + 8]
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v_off[s][h] = (vrow + 8 * h) * 128 + (c16 & 1) * 8 +
                          (((uint32_t)(4 * s + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1)) ^ f(vrow + 8 * h)) * 16);
    const uint32_t lds0 = lds_addr(smem) + wave * 1024;
    const float c = a.scale * kLog2e;

    while (u < stop) {
        while (u >= r.base + r.nm * r.nt) {
            const uint32_t next = r.base + r.nm * r.nt;
            r = request_at(a, r.b + 1);
            r.base = next;
            r = uniform(r);
        }
        const uint32_t m = uniform((u - r.base) / r.nt);
        const uint32_t item = r.base + m * r.nt;
        const uint32_t tile0 = u - item;
        const uint32_t tile1 = min(stop, item + r.nt) - item;
        u = item + tile1;
        const uint32_t n_tiles = tile1 - tile0;
        const uint32_t len = r.len, cached = r.cached;
        const uint32_t table_row = r.b * a.L.max_pages;   // checked on the host: below 2^32

        const uint32_t rows = r.n * (uint32_t)a.H;                 // below 2^31 / D
        const uint32_t row = m * kAttnRows + wave * 32 + col;
        const bool live = uniform(m * kAttnRows + wave * 32) < rows;
        const bool valid = row < rows;
        const uint32_t qrow = r.t0 * (uint32_t)a.H + min(row, rows - 1);
        const uint32_t tok = min(row, rows - 1) / (uint32_t)a.H;   // token of the request

        // Query fragments: lane holds features 16 s + 8 half .. + 7 of its row.
        bf16x8 q[D / 16];
        {
            const char* src = static_cast<const char*>(a.q) + (int64_t)qrow * (D * 2) + half * 16;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                q[s] = as_bf16x8(ld16(src + s * 32));
        }
        // The stages of the item before are no longer read (and no load into them is in flight:
        // the last step waited for all of them, and those behind the last tile are switched off).
        lds_barrier();

        // Loads of one tile: this wave fetches rows 8 wave .. 8 wave + 7, lane l granule l % 8
        // of every block of row l / 8.  Rows past the end repeat the last one.
        // The page id of a tile's rows (PAGE8: 8 rows starting at a multiple of 8 are in one page)
        // is asked for one tile early, when no LDS read is outstanding: a scalar load makes every
        // wait for LDS reads wait for all of them.
        [[maybe_unused]] uint32_t next_id = 0;
        [[maybe_unused]] const uint32_t* next_entry = a.L.page_table;
        auto group_start = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t p0 = (tile0 + t) * TILE + wave * 8;
            return p0 < len ? p0 : (len - 1) & ~7u;
        };
        auto entry_of = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t lp = __umulhi(group_start(t), P.ps_magic) >> P.ps_shift;
            return a.L.page_table + table_row + min(lp, a.L.max_pages - 1);
        };
        auto id_at = [&](const uint32_t* entry) __attribute__((always_inline)) {
            return *(const __attribute__((address_space(4))) uint32_t*)(uint64_t)entry;
        };

        // Where the loads of a tile come from and go to; then its 9 loads one by one: spread over
        // a step they never wait for one another (64 bytes per clock and CU).
        const char* src_base = nullptr;     // PAGE8: uniform; else the lane's address
        uint32_t src_off = 0, dst = 0, src_on = 0;
        uint32_t last_tile = n_tiles;
        asm("" : "+s"(last_tile));   // the switch below stays scalar arithmetic
        auto locate = [&](uint32_t t) __attribute__((always_inline)) {
            dst = (t & (STAGES - 1)) * STAGE + lds0;
            src_on = (uint32_t)((int32_t)(t - last_tile) >> 31);   // all ones while t < n_tiles
            if constexpr (PAGE8) {
                const uint32_t pg = group_start(t);
                const uint32_t slot = pg - (__umulhi(pg, P.ps_magic) >> P.ps_shift) * a.L.page_size;
                src_base = a.L.base + (int64_t)min(next_id, a.L.num_pages - 1) * a.L.stride_page +
                           (int64_t)slot * a.L.stride_token;
                const uint32_t last = len - 1 - pg;
                src_off = min((uint32_t)lane >> 3, last) * (uint32_t)a.L.stride_token + load_off;
            } else {
                const uint32_t p = min((tile0 + t) * TILE + wave * 8 + ((uint32_t)lane >> 3), len - 1);
                const uint32_t lp = p / a.L.page_size;
                const uint32_t id = min(a.L.page_table[table_row + min(lp, a.L.max_pages - 1)], a.L.num_pages - 1);
                src_base = a.L.base + (int64_t)id * a.L.stride_page +
                           (int64_t)(p - lp * a.L.page_size) * a.L.stride_token + load_off;
            }
        };
        auto load = [&](int j) __attribute__((always_inline)) {
            if constexpr (PAGE8)
                load_lds(src_base, src_off + j * 128, dst + j * BLOCK_BYTES, src_on);
            else
                load_lds(src_base + j * 128, dst + j * BLOCK_BYTES, src_on);
        };
        auto issue = [&](uint32_t t) __attribute__((always_inline)) {
            locate(t);
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                load(j);
        };

        if constexpr (PAGE8) {
            const uint32_t id0 = id_at(entry_of(0)), id1 = id_at(entry_of(1)), id2 = id_at(entry_of(2)),
                           id3 = id_at(entry_of(3));
            next_id = id0;
            issue(0);
            next_id = id1;
            issue(1);
            next_id = id2;
            issue(2);
            next_id = id3;
        } else {
            issue(0);
            issue(1);
            issue(2);
        }

        // Start of step t: tile t + 1 has landed for every wave and every wave is done with
        // tile t - 1, whose stage takes tile t + 3.
        auto enter = [&](uint32_t t) __attribute__((always_inline)) {
            if (t + 2 < n_tiles)
                wait_loads<LOADS>();
            else
                wait_loads<0>();
            lds_barrier();
            locate(t + 3);
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
            for (uint32_t t = 0; t < n_tiles; ++t) {
                enter(t);
#pragma unroll
                for (int j = 0; j < LOADS; ++j)
                    load(j);
                if constexpr (PAGE8)
                    next_id = id_at(entry_of(t + 4));
            }
            continue;
        }

        f32x16 o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] = f32x16{0.f};
        float mref = -INFINITY, l = 0.0f;

        // Scores of tile t: lane (col, half) gets rows 8 (i / 4) + 4 half + i % 4 for its query.
        // Fragments are read KD products ahead; `between(k)` is other work during product k.
        constexpr int KN = D / 16, KD = 6, VN = 2 * (K / 32), VD = 4;
        auto scores = [&](uint32_t t, auto between) __attribute__((always_inline)) {
            const char* st = smem + (t & (STAGES - 1)) * STAGE;
            auto frag = [&](int k) __attribute__((always_inline)) {
                return as_bf16x8(lds_ld16(st + k_off[k & 3] + (k >> 2) * BLOCK_BYTES));
            };
            f32x16 acc;
            bf16x8 kf[KD];
#pragma unroll
            for (int k = 0; k < KD; ++k)
                kf[k] = frag(k);
            between(-1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < KN; ++k) {
                if (k == 0)
                    mfma_first(acc, kf[0], q[0]);
                else if (k == KN - 1)
                    mfma_last(acc, kf[k % KD], q[k]);
                else
                    mfma_next(acc, kf[k % KD], q[k]);
                if (k + KD < KN)
                    kf[k % KD] = frag(k + KD);
                between(k);
                __builtin_amdgcn_sched_barrier(0);
            }
            return acc;
        };
        float s[16];        // scores of the tile at hand, in units of log2
        float mx;
        auto scaled_max = [&](const f32x16& raw, int i) __attribute__((always_inline)) {
            s[i] = raw[i] * c;
            mx = i == 0 ? s[0] : fmaxf(mx, s[i]);
        };
        // Masks the scores of tile t, and moves the reference maximum if it lags too far.
        auto settle = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t p0 = (tile0 + t) * TILE;
            if (p0 + TILE > cached) {
                const uint32_t seen = seen_rows(p0);
                mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[i] = (seen >> (8 * (i >> 2) + 4 * half + (i & 3))) & 1 ? s[i] : -INFINITY;
                    mx = fmaxf(mx, s[i]);
                }
                mx = fmaxf(mx, swap32(mx));
            }
            if (__ballot(mx > mref + kSlack)) {
                const float next = fmaxf(mref, mx);
                const float keep = next == mref ? 1.0f : __builtin_amdgcn_exp2f(mref - next);
                mref = next;
                l *= keep;
                asm volatile("s_nop 15");   // the last products' sums are in their registers
#pragma unroll
                for (int i = 0; i < 16; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        scale_sum(o[i], e, keep);
            }
        };
        {
            const f32x16 raw = scores(0, [](int) {});
#pragma unroll
            for (int i = 0; i < 16; ++i)
                scaled_max(raw, i);
            mx = fmaxf(mx, swap32(mx));
            settle(0);
        }

        for (uint32_t t = 0; t < n_tiles; ++t) {
            enter(t);
            const char* st = smem + (t & (STAGES - 1)) * STAGE;
            auto vfrag = [&](int v) __attribute__((always_inline)) {
                const int fb = v >> 1, ks = v & 1;
                const v4i16 lo = lds_tr16(st + v_off[fb & 1][0] + (fb >> 1) * BLOCK_BYTES + ks * 2048);
                const v4i16 hi = lds_tr16(st + v_off[fb & 1][1] + (fb >> 1) * BLOCK_BYTES + ks * 2048);
                return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            };
            const float ref = mref == -INFINITY ? 0.0f : mref;
            // The scores of the next tile, and the weights of this one while the matrix cores
            // run.  (The last step computes scores that nobody uses, from whatever the stage holds.)
            uint32_t pk[8];
            float sum = 0.0f;
            bf16x8 vf[VD];
            auto weights = [&](int k) __attribute__((always_inline)) {
                const float e0 = __builtin_amdgcn_exp2f(s[2 * k] - ref);
                const float e1 = __builtin_amdgcn_exp2f(s[2 * k + 1] - ref);
                sum += e0 + e1;
                pk[k] = pack_bf16x2(e0, e1);
            };
            const f32x16 raw = scores(t + 1, [&](int k) __attribute__((always_inline)) {
                if (k < 0) {
                    weights(0);
                    weights(1);
                } else if (k % 3 == 0 && k / 3 < 6) {
                    weights(2 + k / 3);
                }
                if (k >= 0 && k % 4 == 1)
                    load(k / 4);
                if (k >= KN - VD)
                    vf[k - (KN - VD)] = vfrag(k - (KN - VD));
            });
            l += sum;
            const bf16x8 pf[2] = {as_bf16x8(u32x4{pk[0], pk[1], pk[2], pk[3]}),
                                  as_bf16x8(u32x4{pk[4], pk[5], pk[6], pk[7]})};
#pragma unroll
            for (int v = 0; v < VN; ++v) {
                o[v >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[v % VD], pf[v & 1], o[v >> 1], 0, 0, 0);
                if (v + VD < VN)
                    vf[v % VD] = vfrag(v + VD);
                if (v >= 4 && v < 20)
                    scaled_max(raw, v - 4);
                if (v == 20)
                    mx = fmaxf(mx, swap32(mx));
                if constexpr (PAGE8)
                    if (v == 24)
                        next_entry = entry_of(t + 4);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (PAGE8)
                next_id = id_at(next_entry);
            if (t + 1 < n_tiles)
                settle(t + 1);
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
    Schedule sched(a, lane, P.min_tiles);
    if (w >= sched.groups || sched.total == 0)
        return;
    Request r;
    const uint32_t cut = sched.cut(w, r);
    if (cut != sched.raw(w))
        return;
    const uint32_t m = (cut - r.base) / r.nt;
    const uint32_t lo = r.base + m * r.nt, hi = lo + r.nt;
    if (cut == lo)
        return;
    const uint32_t rows = r.n * (uint32_t)a.H;
    const uint32_t row = m * kAttnRows + g * 32 + col;
    if (m * kAttnRows + g * 32 >= rows)
        return;
    // First and last cut inside the item (an end of an item may be a cut, within `snap` of it).
    const uint32_t w0 = sched.first_cut_past(lo + sched.snap);
    const uint32_t w1 = sched.first_cut_past(hi - sched.snap - 1) - 1;
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
           (uint64_t)a.L.batch * a.L.max_pages < (uint64_t(1) << 32) &&
           // items (at most one partly filled per request) times tiles
           ((uint64_t)a.T * a.H / kAttnRows + std::min<uint64_t>(a.L.batch, a.T)) * (a.capacity / TILE + 1) <
               (uint64_t(1) << 31);
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
