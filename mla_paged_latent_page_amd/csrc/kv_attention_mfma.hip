// Attention over a paged K/V cache on the matrix cores: heads of 64 or 128 columns, bf16 or e4m3
// cache (see kv_attention.hip for the operator and the general form).
//
// The query heads that share a key head are rows of one product: row r of a request is token r / G,
// head r % G.  A wave holds 32 rows and takes 32 cached positions at a time: scores S^T = K Q^T,
// weights P = exp(S - reference), O^T += V^T P^T (products of 32x32x16).  Transposed like this a lane has
// one query row throughout: its maximum, sum and rescaling need no exchange but one swap of the wave's
// halves, and P goes from the score layout into the next product's operand as it is.  The reference
// is the running maximum, let lag by up to 2^8 (the weights stay below 2^8 in binary32), so the sums
// are rescaled only now and then.  Weights are rounded to bf16 for the product, their sum is not.
//
// A workgroup is eight waves, two per SIMD, so that one's softmax runs under the other's products.
// It takes tiles of 64 positions, loaded into a ring in LDS.  Requests of more than 128 rows have
// items of 256 rows, 32 per wave; the others one item of up to 128, whose positions two groups of
// four waves share.
//
// Work: every workgroup takes an equal share of the estimated work of all items; shares that end
// inside an item leave their sums, maximum and sum in the workspace in binary32, and kv_attention_join
// adds them up in a fixed order.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv.hpp"

namespace mla {
namespace {

constexpr int WAVES = 8;
constexpr int TILE = 64;                     // positions of a step
constexpr int WIDE = 256, NARROW = 128;      // rows of an item
constexpr int STAGES = 4;
constexpr int PAGE_SLOTS = 1024;             // page ids held in LDS
constexpr uint32_t OVER = 128;               // an item counts as so many positions more than it has
constexpr uint32_t SNAP = 64;                // a cut so close to an end of an item is moved there
constexpr uint32_t LEAST = 256;              // positions of the smallest share
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;               // the reference maximum may lag by 2^8
constexpr float kNothing = -1e30f;           // the reference of a row that has seen nothing

typedef short v4i16 __attribute__((ext_vector_type(4)));

struct Params {
    KvAttentionArgs a;
    uint32_t G;                              // query heads of a key head
    uint32_t ps_magic, ps_shift;             // p / page_size = mulhi(p, magic) >> shift for p < 2^31 (page sizes of 8 and more)
    uint32_t ids;                            // page ids of a tile
    uint32_t piece;                          // floats of a partial result
    KvCut* cuts;                             // [kKvGroups]
};

__device__ inline uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ inline uint64_t uniform(uint64_t v)
{
    return (uint64_t)uniform((uint32_t)v) | (uint64_t)uniform((uint32_t)(v >> 32)) << 32;
}

// ---------------------------------------------------------------------------
// the schedule
// ---------------------------------------------------------------------------
// Rows of a request and its work.  Item m of a key head counts as OVER + min(first + slope (m + 1), most)
// positions: what its last rows see, without the rounding to tiles.
struct Request {
    uint32_t b, t0, n, cached, len, rows, R, nm;
    uint32_t first, slope;
    uint64_t most;
    uint64_t each;                           // work of all items of one key head
};

__device__ inline uint64_t work_before(const Request& r, uint32_t m)
{
    // items below `grow` are below the most
    const uint64_t room = r.most > r.first ? r.most - r.first : 0;
    const uint32_t grow = room >= (uint64_t)r.slope * r.nm ? r.nm : (uint32_t)((double)room / (double)r.slope);
    const uint64_t k = min(m, grow);
    return (uint64_t)m * OVER + k * r.first + r.slope * (k * (k + 1) / 2) + (m - k) * r.most;
}

__device__ inline Request request_at(const Params& P, uint32_t b)
{
    const KvAttentionArgs& a = P.a;
    Request r{};
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    r.b = b;
    r.t0 = min(a.iro[b], end);
    const uint32_t t1 = min(a.iro[b + 1], end);
    r.n = t1 > r.t0 ? t1 - r.t0 : 0;
    r.cached = min(a.cache_len[b], 0x80000000u);
    r.len = min(r.cached + r.n, a.capacity);
    r.rows = r.n * P.G;                      // below 2^31
    r.R = r.rows <= (uint32_t)NARROW ? NARROW : WIDE;
    r.nm = (r.rows + r.R - 1) / r.R;
    r.first = min(r.cached, a.capacity);
    r.slope = (r.R + P.G - 1) / P.G;
    r.most = a.window ? (uint64_t)a.window + a.sinks + TILE + r.slope : ~0ull;
    r.each = work_before(r, r.nm);
    return r;
}

// Positions that the rows of an item see: tiles 0 .. ns - 1, then those from lo on, nt in all.
struct Item {
    uint32_t b, kh, m;
    uint32_t nt, ns, lo;
    uint64_t cost;
};

__device__ inline Item item_at(const Params& P, const Request& r, uint32_t kh, uint32_t m)
{
    const KvAttentionArgs& a = P.a;
    Item it{};
    it.b = r.b;
    it.kh = kh;
    it.m = m;
    const uint32_t tok0 = m * r.R / P.G, tok1 = (min(r.rows, (m + 1) * r.R) - 1) / P.G;
    const uint32_t hi = min(r.cached + tok1 + 1, a.capacity), p = r.cached + tok0;
    const uint32_t low = a.window && p + 1 > a.window ? min(p + 1 - a.window, hi) : 0;
    const uint32_t end = (hi + TILE - 1) / TILE;
    it.lo = min(low / TILE, end - 1);        // (hi is at least 1; a tile even if no row sees it)
    it.ns = min((min(a.sinks, low) + TILE - 1) / TILE, it.lo);
    it.nt = it.ns + end - it.lo;
    it.cost = work_before(r, m + 1) - work_before(r, m);
    return it;
}

__device__ inline uint64_t shfl64(uint64_t v, int lane)
{
    return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, lane, 64) |
           ((uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), lane, 64) << 32);
}

struct Schedule {
    const Params& P;
    int lane;
    uint64_t total, share;
    uint32_t groups;
    uint32_t first;                          // first request in the lanes
    uint64_t before;                         // work before it
    uint64_t mine, scan;                     // this lane's request; sum up to and including it

    __device__ void load(uint32_t b0, uint64_t work)
    {
        first = b0;
        before = work;
        mine = 0;
        if (b0 + lane < P.a.L.batch)
            mine = request_at(P, b0 + lane).each * (uint32_t)P.a.KH;
        scan = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint64_t v = shfl64(scan, lane >= d ? lane - d : lane);
            scan += lane >= d ? v : 0;
        }
    }
    __device__ bool decreasing(uint32_t b0) const
    {
        return __ballot(b0 + lane < P.a.L.batch && P.a.iro[b0 + lane] > P.a.iro[b0 + lane + 1]) != 0;
    }
    __device__ uint64_t loaded() const { return uniform(shfl64(scan, 63)); }

    __device__ Schedule(const Params& p, int l) : P(p), lane(l)
    {
        load(0, 0);
        total = loaded();
        bool bad = decreasing(0);
        for (uint32_t b0 = 64; b0 < P.a.L.batch; b0 += 64) {
            load(b0, total);
            total += loaded();
            bad |= decreasing(b0);
        }
        if (bad)                             // (they could name a token in many requests)
            total = 0;
        if (P.a.L.batch > 64)
            load(0, 0);
        groups = (uint32_t)min((uint64_t)kKvGroups, total / LEAST + 1);
        share = total / groups;
    }
    // Where workgroup w's share begins (share w > 0), as a request, an item of it and a tile; the item
    // that follows where the cut is moved to the item's end.
    __device__ Item cut(uint32_t w, Request& r, uint32_t& tile)
    {
        const uint64_t x = share * w;        // below total
        if (x < before)
            load(0, 0);
        while (x >= before + loaded())
            load(first + 64, before + loaded());
        const int k = __ffsll((unsigned long long)__ballot(x < before + scan)) - 1;
        r = request_at(P, first + k);
        uint64_t off = x - uniform(before + shfl64(scan - mine, k));
        // key head: the largest with kh * each <= off, and the item likewise
        uint32_t kh = 0;
        for (uint32_t step = 1u << (31 - __clz(P.a.KH)); step; step >>= 1)
            if (kh + step < (uint32_t)P.a.KH && (kh + step) * r.each <= off)
                kh += step;
        off -= kh * r.each;
        uint32_t m = 0;
        for (uint32_t step = 1u << (31 - __clz((int)r.nm)); step; step >>= 1)
            if (m + step < r.nm && work_before(r, m + step) <= off)
                m += step;
        off -= work_before(r, m);
        Item it = item_at(P, r, kh, m);
        tile = 0;
        if (off > OVER + SNAP) {
            tile = it.nt;
            if (it.cost - off > SNAP)
                tile = min((uint32_t)((double)(off - OVER) * (double)it.nt / (double)(it.cost - OVER)), it.nt);
        }
        if (tile == it.nt) {
            tile = 0;
            it = next(r, it);
        }
        return it;
    }
    // The item behind it; b is the batch size behind the last.
    __device__ Item next(Request& r, const Item& it) const
    {
        if (it.m + 1 < r.nm)
            return item_at(P, r, it.kh, it.m + 1);
        if (it.kh + 1 < (uint32_t)P.a.KH)
            return item_at(P, r, it.kh + 1, 0);
        uint32_t b = it.b + 1;
        for (; b < P.a.L.batch; ++b) {
            r = request_at(P, b);
            if (r.nm)
                return item_at(P, r, 0, 0);
        }
        Item none{};
        none.b = b;
        return none;
    }
};

// Wave-uniform ones, in scalar registers.
__device__ inline Request uniform(const Request& r)
{
    return Request{uniform(r.b), uniform(r.t0), uniform(r.n), uniform(r.cached), uniform(r.len), uniform(r.rows),
                   uniform(r.R), uniform(r.nm), uniform(r.first), uniform(r.slope), uniform(r.most), uniform(r.each)};
}
__device__ inline Item uniform(const Item& i)
{
    return Item{uniform(i.b), uniform(i.kh), uniform(i.m), uniform(i.nt), uniform(i.ns), uniform(i.lo), uniform(i.cost)};
}

// ---------------------------------------------------------------------------
// small pieces
// ---------------------------------------------------------------------------
__device__ inline v4i16 lds_tr16(const char* p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16*)(__attribute__((address_space(3))) void*)p);
}
__device__ inline bf16x8 join8(v4i16 lo, v4i16 hi)
{
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return as_bf16x8(u32x4{a[0], a[1], b[0], b[1]});
}

// This lane's value and that of the lane 32 away, in the order of the halves.
__device__ inline f32x2 halves(float v)
{
    const uint32_t x = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return f32x2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

template <int N>
__device__ inline void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// At most `tiles` (up to 3) tiles' worth of loads, N each, may be in flight.
template <int N>
__device__ inline void wait_tiles(uint32_t tiles)
{
    if (tiles >= 3)
        wait_loads<3 * N>();
    else if (tiles == 2)
        wait_loads<2 * N>();
    else if (tiles == 1)
        wait_loads<N>();
    else
        wait_loads<0>();
}

// 16 bytes per lane from a uniform base and a lane offset into LDS at lds + 16 * lane (see asm_ld16_lds).
__device__ inline void load_lds16(const char* base, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory", "m0");
}
__device__ inline void load_lds4(const void* src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(src) : "memory", "m0");
}

// Four e4m3 codes as bf16 (every code's value is one).
__device__ inline u32x2 bf16_of_codes(uint32_t x)
{
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true))};
}

__device__ inline bool nonfinite2(uint32_t x) { return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u; }

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
// A tile in LDS: 64 rows of keys, then 64 of values, 2 D bytes each, in granules of 16 bytes.  Granule g of
// row x is at g ^ f(x), such that the 16-byte reads of 16 key rows, and the transposing reads of four
// value rows by 64 bytes, fall on different banks (256 bytes are all of them).
template <int D, bool FP8>
struct Layout {
    static constexpr int ROW = 2 * D, HALF = TILE * ROW, STAGE = 2 * HALF;
    static constexpr int G = ROW / 16;                       // granules of a row
    __device__ static uint32_t fk(uint32_t x) { return D == 128 ? x & 15 : (x >> 1) & 7; }
    __device__ static uint32_t fv(uint32_t x) { return D == 128 ? 4 * (x & 3) : 4 * ((x >> 1) & 1); }
    // e4m3: codes as they are in memory, in a ring; two tiles of bf16, the one in use and the next.
    static constexpr int CODES_WAVE = 8 * 2 * D;             // a wave's eight rows of keys, then of values
    static constexpr int CODES = WAVES * CODES_WAVE;
    // Scales: a wave's 8 + 8 floats (and as they come, repeated), for twice as many tiles, as they are
    // read when the codes' place is filled again.
    static constexpr int SCALES = WAVES * 256;
    static constexpr int SCALES_AT = STAGES * CODES;
    static constexpr int TILES_AT = FP8 ? SCALES_AT + 2 * STAGES * SCALES : 0;
    static constexpr int BUFFERS = FP8 ? 2 : STAGES;
    static constexpr int PAGES_AT = TILES_AT + BUFFERS * STAGE;
    static constexpr int FLAG_AT = PAGES_AT + PAGE_SLOTS * 4;
    static constexpr int BYTES = FLAG_AT + 16;
    static constexpr int SUMS_WAVE = D / 32 * 16 * 256 + 512;   // a wave's output sums, references and sums
    static_assert(4 * SUMS_WAVE <= PAGES_AT && BYTES <= 163840, "LDS");
    static constexpr int LOADS = FP8 ? (D == 128 ? 3 : 2) : (D == 128 ? 4 : 2);   // of a wave for a tile
    static constexpr uint32_t AHEAD = FP8 ? 4 : 3;           // step t asks for tile t + AHEAD
};

template <int D, bool FP8, bool PAGE8>
__global__ void __launch_bounds__(64 * WAVES) kv_attention_mfma(Params P)
{
    using Y = Layout<D, FP8>;
    constexpr int KS = D / 16, DB = D / 32;
    __shared__ __attribute__((aligned(1024))) char smem[Y::BYTES];
    uint32_t* const ids = reinterpret_cast<uint32_t*>(smem + Y::PAGES_AT);
    uint32_t* const flag = reinterpret_cast<uint32_t*>(smem + Y::FLAG_AT);
    const KvAttentionArgs& a = P.a;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = uniform(threadIdx.x >> 6);
    const uint32_t half = lane >> 5, col = lane & 31;

    Schedule sched(P, lane);
    // Neighbouring shares go to one XCD (block i runs on XCD i % 8): items of one key head then read
    // the same rows through one L2.
    const uint32_t per = (sched.groups + 7) / 8, w = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    const bool idle = (blockIdx.x >> 3) >= per || w >= sched.groups || sched.total == 0;
    Request r{};
    Item it{}, stop{};
    uint32_t tile = 0, stop_tile = 0;
    stop.b = a.L.batch;
    if (!idle) {
        if (w + 1 < sched.groups)
            stop = sched.cut(w + 1, r, stop_tile);
        if (w == 0) {
            // the first request that has tokens
            it.b = 0xFFFFFFFFu;
            it.kh = a.KH - 1;
            r = Request{};
            it = sched.next(r, it);
        } else {
            it = sched.cut(w, r, tile);
        }
    }
    r = uniform(r);
    it = uniform(it);
    stop = uniform(stop);
    tile = uniform(tile);
    stop_tile = uniform(stop_tile);
    // What the join needs: whether this share begins inside an item, and which.
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0)
            P.cuts[kKvGroups].tile = sched.total ? sched.groups : 0;
        KvCut cut{};
        if (!idle && it.b < a.L.batch)
            cut = KvCut{it.b, it.kh, it.m, tile, r.t0, it.m * r.R, min(r.R, r.rows - it.m * r.R), 0};
        if (!idle)
            P.cuts[w] = cut;
    }
    if (idle)
        return;
    if (threadIdx.x == 0)
        *flag = 0xFFFFFFFFu;
    uint32_t sequence = 0;                   // tiles this workgroup has had

    const uint32_t lds0 = lds_addr(smem);
    // Lane-constant offsets of the operand reads.
    uint32_t k_off[KS], v_off[DB];
    {
        const uint32_t k0 = col * Y::ROW + ((half ^ Y::fk(col)) * 16);
#pragma unroll
        for (int s = 0; s < KS; ++s)
            k_off[s] = k0 ^ (s * 32);
        // lane c of a 16-lane group addresses row c / 4 of four, and 8 bytes of 16 columns
        const uint32_t c16 = lane & 15, row = 4 * half + (c16 >> 2);
        const uint32_t v0 = row * Y::ROW + (((2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1)) ^ Y::fv(row)) * 16) + (c16 & 1) * 8;
#pragma unroll
        for (int d = 0; d < DB; ++d)
            v_off[d] = Y::HALF + (v0 ^ (d * 64));
    }
    const float c = fabsf(a.scale) * kLog2e;   // a negative scale turns the queries' signs; 0 is not taken
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    const float slack = kSlack / c;
    const uint32_t st_token = (uint32_t)a.L.stride_token;   // PAGE8: 8 rows below 2^31 bytes

    auto process = [&](auto narrow, uint32_t tile0, uint32_t tile1) __attribute__((always_inline)) {
        constexpr bool N = decltype(narrow)::value;
        constexpr int KB = N ? 1 : 2;        // blocks of 32 positions of a wave
        const uint32_t group = N ? wave & 3 : wave, kb0 = N ? wave >> 2 : 0;
        const uint32_t row0 = it.m * (N ? NARROW : WIDE) + group * 32;
        const bool live = row0 < r.rows;
        const uint32_t row = min(row0 + col, r.rows - 1), tok = row / P.G, g = row - tok * P.G;
        const uint32_t pos = r.cached + tok;
        // positions seen: low .. low + count - 1, and those below sunk
        const uint32_t hi = min(pos + 1, a.capacity);
        const uint32_t low = a.window && pos + 1 > a.window ? min(pos + 1 - a.window, hi) : 0;
        const uint32_t count = hi - low, sunk = min(a.sinks, low);
        const uint32_t len = r.len;
        // of all rows of the wave, and of the item
        const uint32_t w_hi0 = uniform(hi), w_low0 = uniform(low), w_sunk0 = uniform(sunk);
        const uint32_t w_hi1 = (uint32_t)__builtin_amdgcn_readlane((int)hi, 31);
        const uint32_t w_low1 = (uint32_t)__builtin_amdgcn_readlane((int)low, 31);
        const uint32_t b_tok0 = it.m * (N ? NARROW : WIDE) / P.G;
        const uint32_t b_tok1 = (min(r.rows, (it.m + 1) * (N ? NARROW : WIDE)) - 1) / P.G;
        const uint32_t b_hi0 = min(r.cached + b_tok0 + 1, a.capacity);
        auto low_of = [&](uint32_t tk) __attribute__((always_inline)) {
            const uint32_t p = r.cached + tk;
            return a.window && p + 1 > a.window ? p + 1 - a.window : 0u;
        };
        const uint32_t b_low1 = low_of(b_tok1), b_sunk0 = min(a.sinks, low_of(b_tok0));

        bf16x8 q[KS];
        {
            const char* src = a.q + (int64_t)(r.t0 + tok) * a.q_st + (int64_t)(it.kh * P.G + g) * Y::ROW + half * 16;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                q[s] = as_bf16x8(ld16(src + s * 32) ^ flip);
        }

        const uint32_t n_tiles = tile1 - tile0;
        auto tile_start = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t j = tile0 + t;
            return (j < it.ns ? j : it.lo + (j - it.ns)) * TILE;
        };
        // Page ids of tiles id0 .. id0 + hold - 1 of this item, P.ids each.
        const uint32_t hold = PAGE_SLOTS / P.ids;
        uint32_t id0 = 0;
        auto page_of = [&](uint32_t p) __attribute__((always_inline)) {
            return PAGE8 ? __umulhi(p, P.ps_magic) >> P.ps_shift : p / a.L.page_size;
        };
        auto fetch_ids = [&](uint32_t t0) __attribute__((always_inline)) {
            lds_barrier();
            id0 = t0;
            for (uint32_t k = threadIdx.x; k < hold * P.ids; k += 64 * WAVES) {
                const uint32_t s = k / P.ids, e = k - s * P.ids;
                if (t0 + s < n_tiles) {
                    const uint32_t lp = min(page_of(tile_start(t0 + s)) + e, a.L.max_pages - 1);
                    ids[k] = min(a.L.page_table[(size_t)it.b * a.L.max_pages + lp], a.L.num_pages - 1);
                }
            }
            lds_barrier();
        };
        fetch_ids(0);

        const int64_t head_bytes = (int64_t)it.kh * (FP8 ? D : 2 * D);
        const int64_t scale_bytes = (int64_t)(it.kh * D / 128) * 4;
        // Loads of tile t: this wave fetches rows 8 wave .. 8 wave + 7 of keys and values; those past the
        // end repeat the last one.
        auto issue = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t start = tile_start(t), slot = t & (STAGES - 1);
            const uint32_t* my_ids = ids + (t - id0) * P.ids;
            if constexpr (PAGE8) {
                // eight rows from a multiple of 8 on are in one page
                uint32_t p0 = start + wave * 8;
                p0 = p0 < len ? p0 : (len - 1) & ~7u;
                const uint32_t lp = page_of(p0), in_page = p0 - lp * a.L.page_size, last = len - 1 - p0;
                const uint32_t id = uniform(my_ids[lp - page_of(start)]);
                const char* src = a.L.base + (int64_t)id * a.L.stride_page + (int64_t)in_page * a.L.stride_token + head_bytes;
                if constexpr (!FP8 && D == 128) {
                    const uint32_t dst = lds0 + slot * Y::STAGE + wave * 2048;
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        const uint32_t x = 4 * i + (lane >> 4);
                        const uint32_t off = min(x, last) * st_token;
                        load_lds16(src, off + (((lane & 15) ^ Y::fk(wave * 8 + x)) * 16), dst + i * 1024);
                        load_lds16(src + a.L.stride_kv, off + (((lane & 15) ^ Y::fv(x)) * 16), dst + Y::HALF + i * 1024);
                    }
                } else if constexpr (!FP8) {
                    const uint32_t dst = lds0 + slot * Y::STAGE + wave * 1024, x = lane >> 3;
                    const uint32_t off = min(x, last) * st_token;
                    load_lds16(src, off + (((lane & 7) ^ Y::fk(wave * 8 + x)) * 16), dst);
                    load_lds16(src + a.L.stride_kv, off + (((lane & 7) ^ Y::fv(x)) * 16), dst + Y::HALF);
                } else {
                    const uint32_t dst = lds0 + slot * Y::CODES + wave * Y::CODES_WAVE;
                    if constexpr (D == 128) {
                        const uint32_t off = min((uint32_t)lane >> 3, last) * st_token + (lane & 7) * 16;
                        load_lds16(src, off, dst);
                        load_lds16(src + a.L.stride_kv, off, dst + 1024);
                    } else {
                        const uint32_t off = min(col >> 2, last) * st_token + (lane & 3) * 16;
                        asm_gld16_lds(src + (half ? a.L.stride_kv : 0) + off, dst);
                    }
                    const char* sc = a.Ls.base + (int64_t)id * a.Ls.stride_page +
                                     (int64_t)(in_page + min((uint32_t)lane & 7, last)) * a.Ls.stride_token + scale_bytes +
                                     ((lane & 8) ? a.Ls.stride_kv : 0);
                    load_lds4(sc, lds0 + Y::SCALES_AT + (t & (2 * STAGES - 1)) * Y::SCALES + wave * 256);
                }
            } else {
                const uint32_t first = page_of(start);
                auto at = [&](const PagedLayer& L, uint32_t x) __attribute__((always_inline)) {
                    const uint32_t p = min(start + wave * 8 + x, len - 1), lp = page_of(p);
                    return L.base + (int64_t)my_ids[lp - first] * L.stride_page +
                           (int64_t)(p - lp * L.page_size) * L.stride_token;
                };
                if constexpr (!FP8) {
                    constexpr uint32_t LR = D == 128 ? 16 : 8;   // lanes of a row
#pragma unroll
                    for (uint32_t i = 0; i < (D == 128 ? 2 : 1); ++i) {
                        const uint32_t x = 64 / LR * i + lane / LR, dst = lds0 + slot * Y::STAGE + wave * 8 * Y::ROW + i * 1024;
                        const char* src = at(a.L, x) + head_bytes;
                        asm_gld16_lds(src + (((lane & (LR - 1)) ^ Y::fk(wave * 8 + x)) * 16), dst);
                        asm_gld16_lds(src + a.L.stride_kv + (((lane & (LR - 1)) ^ Y::fv(x)) * 16), dst + Y::HALF);
                    }
                } else {
                    const uint32_t dst = lds0 + slot * Y::CODES + wave * Y::CODES_WAVE;
                    if constexpr (D == 128) {
                        const char* src = at(a.L, lane >> 3) + head_bytes + (lane & 7) * 16;
                        asm_gld16_lds(src, dst);
                        asm_gld16_lds(src + a.L.stride_kv, dst + 1024);
                    } else {
                        asm_gld16_lds(at(a.L, col >> 2) + head_bytes + (half ? a.L.stride_kv : 0) + (lane & 3) * 16, dst);
                    }
                    load_lds4(at(a.Ls, lane & 7) + scale_bytes + ((lane & 8) ? a.Ls.stride_kv : 0),
                              lds0 + Y::SCALES_AT + (t & (2 * STAGES - 1)) * Y::SCALES + wave * 256);
                }
            }
        };
        // e4m3: this wave's rows of tile t from codes to bf16.
        auto convert = [&](uint32_t t) __attribute__((always_inline)) {
            const char* src = smem + (t & (STAGES - 1)) * Y::CODES + wave * Y::CODES_WAVE + lane * 16;
            char* dst = smem + Y::TILES_AT + (t & 1) * Y::STAGE;
            auto put = [&](u32x4 x, char* to, uint32_t rr, uint32_t gr, uint32_t f) __attribute__((always_inline)) {
                const u32x2 c0 = bf16_of_codes(x[0]), c1 = bf16_of_codes(x[1]), c2 = bf16_of_codes(x[2]), c3 = bf16_of_codes(x[3]);
                lds_st16(to + rr * Y::ROW + ((gr ^ f) * 16), u32x4{c0[0], c0[1], c1[0], c1[1]});
                lds_st16(to + rr * Y::ROW + (((gr + 1) ^ f) * 16), u32x4{c2[0], c2[1], c3[0], c3[1]});
            };
            if constexpr (D == 128) {
                const u32x4 k = lds_ld16(src), v = lds_ld16(src + 1024);
                const uint32_t rr = wave * 8 + (lane >> 3), gr = 2 * (lane & 7);
                put(k, dst, rr, gr, Y::fk(rr));
                put(v, dst + Y::HALF, rr, gr, Y::fv(rr));
            } else {
                const u32x4 x = lds_ld16(src);
                const uint32_t rr = wave * 8 + (col >> 2), gr = 2 * (lane & 3);
                put(x, dst + (half ? Y::HALF : 0), rr, gr, half ? Y::fv(rr) : Y::fk(rr));
            }
        };
        // e4m3: scales (keys 0, values 1) of rows 8 i + 4 half .. + 3 of tile t.
        auto scales_of = [&](uint32_t t, uint32_t side, uint32_t i) __attribute__((always_inline)) {
            return *reinterpret_cast<const f32x4*>(smem + Y::SCALES_AT + (t & (2 * STAGES - 1)) * Y::SCALES + i * 256 +
                                                   side * 32 + half * 16);
        };

        for (uint32_t t = 0; t < Y::AHEAD && t < n_tiles; ++t)
            issue(t);
        if constexpr (FP8) {
            wait_tiles<Y::LOADS>(min(n_tiles - 1, 3u));
            convert(0);
        }

        f32x16 o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                o[d][e] = 0.0f;
        float mref = kNothing, l = 0.0f;

        for (uint32_t t = 0; t < n_tiles; ++t) {
            // Tile t is there (e4m3: this wave's codes of tile t + 1 are), for every wave, and the one before
            // is no longer read.
            if constexpr (FP8)
                wait_tiles<Y::LOADS>(n_tiles - 1 > t + 1 ? min(n_tiles - 2 - t, 2u) : 0u);
            else
                wait_tiles<Y::LOADS>(min(n_tiles - 1 - t, 2u));
            lds_barrier();
            const uint32_t ask = t + Y::AHEAD;
            if (ask < n_tiles) {
                if (ask >= id0 + hold)
                    fetch_ids(ask);
                issue(ask);
            }
            const uint32_t start = tile_start(t);
            const char* tl = smem + Y::TILES_AT + (t & (Y::BUFFERS - 1)) * Y::STAGE;
            if constexpr (FP8)
                if (t + 1 < n_tiles)
                    convert(t + 1);

            // Rows that some do not see may hold anything: a weight of 0 would turn their infinities and
            // NaN into NaN.  Where a tile has such rows, every wave looks at its eight of them.
            bool dirty = false;
            ++sequence;
            if (start + TILE > b_hi0 || (start < b_low1 && start + TILE > b_sunk0)) {
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 8 * Y::ROW / 1024; ++i) {
                    const u32x4 x = lds_ld16(tl + Y::HALF + wave * 8 * Y::ROW + i * 1024 + lane * 16);
                    bad |= nonfinite2(x[0]) || nonfinite2(x[1]) || nonfinite2(x[2]) || nonfinite2(x[3]);
                }
                if (__any(bad) && lane == 0)
                    *flag = sequence;
                lds_barrier();
                dirty = uniform(*flag) == sequence;
            }
            // No row of this wave sees any of it?
            const uint32_t my0 = start + kb0 * 32, my1 = my0 + KB * 32;
            if (!live || my0 >= w_hi1 || (my1 <= w_low0 && my0 >= min(a.sinks, w_low1)))
                continue;

            f32x16 s[KB];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    s[b][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        as_bf16x8(lds_ld16(tl + k_off[k] + (kb0 + b) * 32 * Y::ROW)), q[k], s[b], 0, 0, 0);
            }
            if constexpr (FP8) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 f = scales_of(t, 0, (kb0 + b) * 4 + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[b][4 * i + e] *= f[e];
                    }
            }
            // element 4 i + e of block b is position my0 + 32 b + 8 i + 4 half + e
            auto seen = [&](int b, int e) __attribute__((always_inline)) {
                const uint32_t p = my0 + 32 * b + 8 * (e / 4) + 4 * half + e % 4;
                return p - low < count || p < sunk;
            };
            const bool masked = my1 > w_hi0 || (my0 < w_low1 && my1 > w_sunk0);
            if (masked) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        s[b][e] = seen(b, e) ? s[b][e] : -INFINITY;
            }
            float top;
            {
                float x[4] = {s[0][0], s[0][1], s[0][2], s[0][3]};
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = b ? 0 : 4; e < 16; ++e)
                        x[e & 3] = __builtin_elementwise_maximum(x[e & 3], s[b][e]);
                const f32x2 h = halves(__builtin_elementwise_maximum(__builtin_elementwise_maximum(x[0], x[1]),
                                                                     __builtin_elementwise_maximum(x[2], x[3])));
                top = __builtin_elementwise_maximum(h[0], h[1]);
            }
            if (__any(top > mref + slack)) {
                const float now = fmaxf(mref, top);
                const float f = __builtin_amdgcn_exp2f((mref - now) * c);
                mref = now;
                l *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[d][e] *= f;
            }
            const float base = mref * c;
            float part[4] = {};
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    s[b][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], c, -base));
                    part[e & 3] += s[b][e];
                }
            l += (part[0] + part[1]) + (part[2] + part[3]);
            if constexpr (FP8) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 f = scales_of(t, 1, (kb0 + b) * 4 + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[b][4 * i + e] *= f[e];
                    }
                if (masked) {   // (0 times an infinite scale)
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            s[b][e] = seen(b, e) ? s[b][e] : 0.0f;
                }
            }
            auto weights = [&](int b, int st) __attribute__((always_inline)) {
                const f32x16& x = s[b];
                return as_bf16x8(u32x4{pack_bf16x2(x[8 * st], x[8 * st + 1]), pack_bf16x2(x[8 * st + 2], x[8 * st + 3]),
                                       pack_bf16x2(x[8 * st + 4], x[8 * st + 5]), pack_bf16x2(x[8 * st + 6], x[8 * st + 7])});
            };
            auto values = [&](int b, int st, int d) __attribute__((always_inline)) {
                const char* at = tl + v_off[d] + ((kb0 + b) * 32 + st * 16) * Y::ROW;
                return join8(lds_tr16(at), lds_tr16(at + 8 * Y::ROW));
            };
            if (!dirty) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const bf16x8 p = weights(b, st);
#pragma unroll
                        for (int d = 0; d < DB; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values(b, st, d), p, o[d], 0, 0, 0);
                    }
            } else {
                // With what is not finite left out; then that, one position at a time, for the rows that see it.
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const bf16x8 p = weights(b, st);
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            u32x4 v = __builtin_bit_cast(u32x4, values(b, st, d));
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                v[k] &= (v[k] & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : ~0u;
                                v[k] &= (v[k] & 0x7F800000u) == 0x7F800000u ? 0x0000FFFFu : ~0u;
                            }
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(v), p, o[d], 0, 0, 0);
                        }
                    }
#pragma unroll 1
                for (uint32_t k = 0; k < 32u * KB; ++k) {
                    const uint32_t p = my0 + k;
                    const bool sees = p - low < count || p < sunk;
                    // position k is element 16 (k / 32) + (k % 32) / 8 * 4 + k % 4 of half (k / 4) % 2
                    const uint32_t e0 = (k >> 5) * 16 + ((k >> 3) & 3) * 4 + (k & 3);
                    float x = 0.0f;
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            x = e0 == (uint32_t)(16 * b + e) ? s[b][e] : x;
                    const f32x2 h = halves(x);
                    x = (k >> 2) & 1 ? h[1] : h[0];
                    const uint32_t vr = kb0 * 32 + k;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // columns 32 d + 8 i + 4 half .. + 3
                            const uint32_t gr = 4 * d + i;
                            const u32x2 v = *reinterpret_cast<const u32x2*>(tl + Y::HALF + vr * Y::ROW +
                                                                            ((gr ^ Y::fv(vr)) * 16) + half * 8);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float y = e & 1 ? bf16_hi(v[e / 2]) : bf16_lo(v[e / 2]);
                                if (sees && !(fabsf(y) < INFINITY))
                                    o[d][4 * i + e] += x * y;
                            }
                        }
                }
            }
        }

        // The row's sum, over both halves; with two groups of waves, over both of them.
        {
            const f32x2 h = halves(l);
            l = h[0] + h[1];
        }
        bool mine = live;
        if constexpr (N) {
            lds_barrier();                   // the tiles are no longer read
            float* sums = reinterpret_cast<float*>(smem + group * Y::SUMS_WAVE);
            if (kb0 == 1 && live) {
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<f32x4*>(sums + ((d * 4 + i) * 64 + lane) * 4) =
                            f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
                sums[DB * 1024 + lane] = mref;
                sums[DB * 1024 + 64 + lane] = l;
            }
            lds_barrier();
            mine = live && kb0 == 0;
            if (mine) {
                const float m1 = sums[DB * 1024 + lane], l1 = sums[DB * 1024 + 64 + lane];
                const float now = fmaxf(mref, m1);
                const float f0 = __builtin_amdgcn_exp2f((mref - now) * c), f1 = __builtin_amdgcn_exp2f((m1 - now) * c);
                mref = now;
                l = l * f0 + l1 * f1;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 x = *reinterpret_cast<const f32x4*>(sums + ((d * 4 + i) * 64 + lane) * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[d][4 * i + e] = o[d][4 * i + e] * f0 + x[e] * f1;
                    }
            }
        }
        if (mine) {
            if (tile0 == 0 && tile1 == it.nt) {
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                const bool valid = row0 + col < r.rows;
                const int64_t head = (int64_t)(r.t0 + tok) * a.H + it.kh * P.G + g;
                uint16_t* out = static_cast<uint16_t*>(a.out) + head * D + 8 * half;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        // eight columns per lane: the halves exchange four
                        const uint32_t x0 = pack_bf16x2(o[d][i] * inv, o[d][i + 1] * inv);
                        const uint32_t x1 = pack_bf16x2(o[d][i + 2] * inv, o[d][i + 3] * inv);
                        const uint32_t y0 = pack_bf16x2(o[d][i + 4] * inv, o[d][i + 5] * inv);
                        const uint32_t y1 = pack_bf16x2(o[d][i + 6] * inv, o[d][i + 7] * inv);
                        const auto u = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
                        const auto v = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
                        if (valid)
                            st16(out + d * 32 + 2 * i, u32x4{u[0], v[0], u[1], v[1]});
                    }
                if (a.lse && valid && half == 0)
                    a.lse[head] = l == 0.0f ? -INFINITY : mref * fabsf(a.scale) + __logf(l);
            } else {
                // A share's sums as they are, in lane order.
                float* piece = a.ws + (size_t)(2 * w + (tile0 == 0)) * P.piece + group * (32 * (D + 2));
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<f32x4*>(piece + ((d * 4 + i) * 64 + lane) * 4) =
                            f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
                if (half == 0) {
                    piece[32 * D + col] = mref;
                    piece[32 * D + 32 + col] = l;
                }
            }
        }
    };

    // From this share's cut to the next one's: equal where the share is empty.
    while (it.b < a.L.batch) {
        const bool last = it.b == stop.b && it.kh == stop.kh && it.m == stop.m;
        const uint32_t end = last ? stop_tile : it.nt;
        if (tile < end) {
            if (r.R == (uint32_t)NARROW)
                process(std::true_type{}, tile, end);
            else
                process(std::false_type{}, tile, end);
        }
        if (last)
            break;
        tile = 0;
        it = sched.next(r, it);
        it = uniform(it);
        r = uniform(r);
    }
}

// ---------------------------------------------------------------------------
// the join
// ---------------------------------------------------------------------------
// Block (cut w, 32 rows) with w the first cut inside an item: the sums that the shares around the item's
// cuts left, each times its exp(reference - the largest one), in the order of the shares.  Four groups of
// waves take every fourth piece.
template <int D>
__global__ void __launch_bounds__(1024) kv_attention_join(Params P)
{
    constexpr int DB = D / 32, Q = DB;       // a thread has Q quads of the row group's sums
    const uint32_t w = blockIdx.x, group = blockIdx.y;
    const uint32_t groups = P.cuts[kKvGroups].tile;
    if (w == 0 || w >= groups)
        return;
    const KvCut cut = P.cuts[w];
    if (cut.tile == 0 || group * 32 >= cut.rows)
        return;
    const KvCut prev = P.cuts[w - 1];
    auto same = [&](const KvCut& x) { return x.tile != 0 && x.b == cut.b && x.kh == cut.kh && x.m == cut.m; };
    if (same(prev))
        return;
    __shared__ uint32_t last;
    __shared__ bool empty[kKvGroups];        // shares that end where they begin leave nothing
    __shared__ float top[4][64], all[4][64];
    __shared__ f32x4 part[3][Q][256];
    if (threadIdx.x == 0)
        last = groups - 1;
    __syncthreads();
    const uint32_t mine = w + threadIdx.x;   // at most kKvGroups shares
    if (mine < groups) {
        const KvCut x = P.cuts[mine], y = mine + 1 < groups ? P.cuts[mine + 1] : KvCut{};
        if (mine > w && !same(x))
            atomicMin(&last, mine - 1);
        empty[threadIdx.x] = same(y) && x.tile == y.tile;
    }
    __syncthreads();
    const uint32_t pieces = last - w + 2;    // the share before w begins the item

    const KvAttentionArgs& a = P.a;
    const float c = fabsf(a.scale) * kLog2e;
    const uint32_t tid = threadIdx.x & 255, set = threadIdx.x >> 8, lane = tid & 63, col = lane & 31;
    auto piece = [&](uint32_t k) {
        return a.ws + (size_t)(k == 0 ? 2 * (w - 1) + 1 : 2 * (w + k - 1)) * P.piece + group * (32 * (D + 2));
    };
    float mx = kNothing;
    for (uint32_t k = set; k < pieces; k += 4)
        if (k == 0 || !empty[k - 1])
            mx = fmaxf(mx, piece(k)[32 * D + col]);
    if (tid < 64)
        top[set][lane] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(top[0][lane], top[1][lane]), fmaxf(top[2][lane], top[3][lane]));
    float l = 0.0f;
    f32x4 sum[Q] = {};
    constexpr int U = 2;
    for (uint32_t k0 = set; k0 < pieces; k0 += 4 * U) {
        f32x4 v[U][Q];
        float m[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float* p = piece(min(k0 + 4 * u, pieces - 1));
            m[u] = p[32 * D + col];
            s[u] = p[32 * D + 32 + col];
#pragma unroll
            for (int j = 0; j < Q; ++j)
                v[u][j] = *reinterpret_cast<const f32x4*>(p + (j * 256 + tid) * 4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + 4 * u < pieces && (k0 + 4 * u == 0 || !empty[k0 + 4 * u - 1])) {
                const float f = __builtin_amdgcn_exp2f((m[u] - mx) * c);
                l += s[u] * f;
#pragma unroll
                for (int j = 0; j < Q; ++j)
                    sum[j] += v[u][j] * f;
            }
    }
    if (tid < 64)
        all[set][lane] = l;
    if (set > 0)
#pragma unroll
        for (int j = 0; j < Q; ++j)
            part[set - 1][j][tid] = sum[j];
    __syncthreads();
    if (set > 0)
        return;
    l = (all[0][lane] + all[1][lane]) + (all[2][lane] + all[3][lane]);
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const uint32_t row = cut.row0 + group * 32 + col;
    if (group * 32 + col >= cut.rows)
        return;
    const uint32_t tok = row / P.G, g = row - tok * P.G;
    const int64_t head = (int64_t)(cut.t0 + tok) * a.H + cut.kh * P.G + g;
    uint16_t* out = static_cast<uint16_t*>(a.out) + head * D;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        // quad j * 4 + tid / 64 of the lane: columns 32 j + 8 (tid / 64) + 4 (lane / 32) .. + 3
        const f32x4 x = ((sum[j] + part[0][j][tid]) + (part[1][j][tid] + part[2][j][tid])) * inv;
        *reinterpret_cast<u32x2*>(out + 32 * j + 8 * (tid >> 6) + 4 * (lane >> 5)) =
            u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    }
    if (a.lse && tid < 32)
        a.lse[head] = l == 0.0f ? -INFINITY : mx * fabsf(a.scale) + __logf(l);
}

}  // namespace

bool kv_attention_mfma_fits(const KvAttentionArgs& a, KvKind kind)
{
    // (the kernel's scale is in units of log2, and divides)
    return kind != KV_F32 && (a.D == 64 || a.D == 128) && std::isnormal(a.scale * kLog2e) &&
           // items are numbered in 32 bits, and their work together in 64
           (uint64_t)a.L.batch * a.KH < (uint64_t(1) << 24);
}

hipError_t launch_kv_attention_mfma(const KvAttentionArgs& a, KvKind kind, hipStream_t s)
{
    Params P{};
    P.a = a;
    P.G = (uint32_t)(a.H / a.KH);
    const uint32_t ps = a.L.page_size;
    P.ids = std::min((62 + ps) / ps, 65u) + 1;
    const bool page8 = ps % 8 == 0 && a.L.stride_token < (int64_t(1) << 27);
    if (page8) {
        // ps >= 8, positions below 2^31: with 2^(s-1) < ps <= 2^s, ceil(2^(31+s) / ps) fits 32 bits
        // and mulhi(p, that) >> (s - 1) is the quotient.
        uint32_t sh = 3;
        while ((uint64_t(1) << sh) < ps)
            ++sh;
        P.ps_magic = (uint32_t)(((uint64_t(1) << (31 + sh)) + ps - 1) / ps);
        P.ps_shift = sh - 1;
    }
    const uint32_t row_groups = kv_attention_row_groups(a.T, P.G);
    P.piece = row_groups * 32 * (a.D + 2);
    P.cuts = reinterpret_cast<KvCut*>(a.ws + (size_t)2 * kKvGroups * P.piece);
    const bool fp8 = kind == KV_E4M3;
    log_launch(fp8 ? "kv_attention_mfma<e4m3>" : "kv_attention_mfma<bf16>", kKvGroups, 64 * WAVES,
               "T=%d H=%d KH=%d D=%d page_size=%u", a.T, a.H, a.KH, a.D, ps);
    auto pick = [&](auto d, auto cache) {
        constexpr int D = decltype(d)::value;
        constexpr bool e = decltype(cache)::value;
        return page8 ? kv_attention_mfma<D, e, true> : kv_attention_mfma<D, e, false>;
    };
    const std::integral_constant<int, 64> d64;
    const std::integral_constant<int, 128> d128;
    const std::true_type yes;
    const std::false_type no;
    auto* kernel = a.D == 64 ? (fp8 ? pick(d64, yes) : pick(d64, no)) : (fp8 ? pick(d128, yes) : pick(d128, no));
    hipLaunchKernelGGL(kernel, dim3(kKvGroups), dim3(64 * WAVES), 0, s, P);
    if (hipError_t e = hipGetLastError())
        return e;
    log_launch("kv_attention_join", kKvGroups * row_groups, 1024, "T=%d H=%d", a.T, a.H);
    hipLaunchKernelGGL(a.D == 64 ? kv_attention_join<64> : kv_attention_join<128>, dim3(kKvGroups, row_groups), dim3(1024),
                       0, s, P);
    return hipGetLastError();
}

}  // namespace mla
