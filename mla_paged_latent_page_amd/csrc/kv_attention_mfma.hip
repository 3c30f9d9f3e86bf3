// Attention over a paged K/V cache on the matrix cores: heads of 64 or 128 columns, bf16 or e4m3 cache (see
// kv_attention.hip for the operator and the general form).
//
// The query heads that share a key head are rows of one product: row r of a request is token r / G, head r % G.  A
// wave holds 32 rows and takes 32 cached positions at a time: scores S^T = K Q^T, weights P = exp(S - reference),
// O^T += V^T P^T (products of 32x32x16).  Transposed like this a lane has one query row throughout: its maximum, sum
// and rescaling need no exchange but one swap of the wave's halves, and P goes from the score layout into the next
// product's operand as it is.  The reference is the running maximum, let lag by up to 2^8 (the weights stay below
// 2^8 in binary32), so the sums are rescaled only now and then.  Weights are rounded to bf16 for the product (2^-8
// of each at most, which the output's own rounding may cost too), their sum is not.
//
// A workgroup is eight waves, two per SIMD, and takes tiles of 64 positions.  Requests of more than 128 rows have
// items of 256 rows, 32 to a wave, which takes both blocks of 32 positions of a tile; the others have one item of
// up to 128, whose tiles two waves to 32 rows share, on different SIMDs.  (Short items throughout: prompt chunks
// 0.68 against 0.54 ms, each row of the cache is read and taken from LDS twice as often; long ones throughout: long
// e4m3 contexts with 20 rows an item 0.42 against 0.33 ms, all products in one wave.)
//
// A step t does the products of the sums of tile t - 1 and of the scores of tile t + 1, which do not wait for the
// softmax of tile t between them: a matrix instruction takes 32 cycles of its pipe, and five or six vector
// instructions fit beside one, in an order laid down by hand with fences (prompt chunks 0.62 to 0.56 ms).  Operands
// come from LDS four products ahead, across the step's one barrier too.  Tiles are loaded into LDS rings four steps
// ahead (bf16) without passing registers, in parts spread over the products.  e4m3 codes go there six steps ahead,
// each wave converts its eighth of a tile to bf16 (exactly) into a second ring, and the scales multiply scores
// (keys) and weights (values, behind their sum); they are read two products before their use, without which every
// group of four waits for LDS (long contexts 0.38 against 0.335 ms, windows 0.82 against 0.74).
//
// Steps whose tiles all rows see whole and whose loads are all whole ("plain" ones) skip masks and bounds. Values
// that are not finite in a tile that some row does not see whole (0 times them would be NaN) are cleared in LDS and
// added for the rows that see them.
//
// Work: every workgroup takes an equal share of the estimated work of all items, in an order that gives
// neighbouring shares one XCD's L2; shares that end inside an item leave their sums, maximum and sum in the
// workspace in binary32, and kv_attention_join adds them up in a fixed order.
//
// Measured (MI355X; 8 key heads of 128 columns): 5 prompt chunks of 1,000 to 4,096 tokens x 32 heads behind 1 to
// 8,000 cached rows, bf16, 0.54 to 0.56 ms = 808 to 846 TFLOP/s, where an 8192^3 library product reaches 1255.  The
// products alone would take 0.43 ms in this form; the rest is what lies between items (setup, first loads, results:
// 8 us each) and the join.  64 single tokens x 64 heads over 1,000 to 32,000 rows, bf16: 0.49 ms, 5.3 TB/s, where a
// large copy reaches 5.1.  6 requests x 40 heads over 60 to 131 thousand rows, e4m3: 0.335 ms, 3.4 TB/s: with at
// most 20 rows an item, two waves do all products, and the chain of their step bounds it (the loads and conversions
// alone take 0.25 ms).  Windows of 2,048 over e4m3, 64 heads: 0.74 to 0.75 ms = 688 to 698 TFLOP/s, bound by the
// issue of conversions, scalings and the softmax beside the products.  On e4m3 every store of converted values has a bank
// conflict: 256 cycles of LDS per tile.
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

#include "kv.hpp"

namespace mla {
namespace {

constexpr int WAVES = 8;
constexpr int TILE = 64;                     // positions of a step
constexpr int WIDE = 256, NARROW = 128;      // rows of an item
constexpr int STAGES = 4;
// Page ids that a wave holds in LDS, where the page size is no multiple of 8 or token rows are 2^24 bytes or more apart.
constexpr int PAGE_SLOTS = 128;
// An item counts as so many positions more than it has: what its start and end cost.  256, 384, 512: prompt chunks
// 0.578, 0.552, 0.551 ms, single tokens 0.497, 0.501, 0.504, long e4m3 contexts 0.447, 0.423, 0.445: all of heads of
// 128 columns; those of 64 take the same figure, unmeasured.
constexpr uint32_t OVER = 384;
// Positions of the smallest share: 128 against 256 takes four requests of at most 1,000 rows from 25.5 to 22 us, 64
// no further.
constexpr uint32_t LEAST = 128;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;               // the reference maximum may lag by 2^8
constexpr float kNothing = -1e30f;           // the reference of a row that has seen nothing

typedef short v4i16 __attribute__((ext_vector_type(4)));

// f(0), f(1), ..., f(N - 1) with constant arguments.
template <class F, int... I>
__device__ __attribute__((always_inline)) inline void each(F&& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __attribute__((always_inline)) inline void each(F&& f)
{
    each(f, std::make_integer_sequence<int, N>{});
}

// The order of a step: NV products of weighted sums, then KB blocks of KS products of scores, and between
// them the softmax of 16 KB elements.  The maximum is found beside the first TOP products; then the elements are
// weighed, those of the first block beside the sums, the others beside the first block of scores; added
// up one product later; and packed, in groups of 8, when their group's old weights have been used (DB
// products each).
template <int NV, int KS, int KB, int DB, bool FP8>
struct Order {
    static constexpr int HALF = NV >= 16 ? 2 : 1;   // e4m3, two blocks: products beside a block's maximum
    static constexpr int TOP = FP8 && KB == 2 ? 2 * HALF + 1 : NV >= 16 ? 4 : 2, E = 16 * KB, LAST = NV + KS - 2;
    static constexpr int weighed(int i)      // elements weighed before product i
    {
        return i <= TOP ? 0 : i <= NV ? 16 * (i - TOP) / (NV - TOP) : i >= LAST ? E : 16 + (E - 16) * (i - NV) / (LAST - NV);
    }
    static constexpr int added(int i) { return i == 0 ? 0 : i == NV ? 16 : weighed(i - 1); }   // and added
    static constexpr int packed(int g)       // the product that group g is packed behind
    {
        for (int i = 0; i < NV + KS * KB; ++i)
            if (added(i + 1) >= 8 * (g + 1) && i >= DB * (g + 1) - 1)
                return i;
        return -1;
    }
};

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
        const uint64_t done = work_before(r, m), cost = work_before(r, m + 1) - done;
        off -= done;
        Item it = item_at(P, r, kh, m);
        tile = 0;
        if (off > OVER)
            tile = min((uint32_t)((double)(off - OVER) * (double)it.nt / (double)(cost - OVER)), it.nt);
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
    return Item{uniform(i.b), uniform(i.kh), uniform(i.m), uniform(i.nt), uniform(i.ns), uniform(i.lo)};
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

// lds_barrier() with the last operand reads (READS, of two instructions each; or, among them, reads of the next
// tile's scales) still in flight: what they read is not written in the step that begins here.
constexpr int READS = 4;                     // products that an operand is read ahead
__device__ inline void step_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(%0)\n\ts_barrier" ::"n"(2 * READS) : "memory");
}

// This wave's LDS operations are done (step_barrier() counts on reads behind them).
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int N>
__device__ inline void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The same for a number that is not constant, up to N.
template <int N>
__device__ inline void wait_some(uint32_t left)
{
    if constexpr (N > 0) {
        if (left < N) {
            wait_some<N - 1>(left);
            return;
        }
    }
    wait_loads<N>();
}

// The lane's number, worked out where it is needed.
__device__ inline uint32_t lane_again()
{
    uint32_t x;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
    return x;
}

// 16 bytes per lane from a uniform base and a lane offset into LDS at lds + 16 * lane (see asm_ld16_lds).
__device__ inline void load_lds16(const char* base, uint32_t voff, uint32_t lds)
{
    base = reinterpret_cast<const char*>(uniform(reinterpret_cast<uint64_t>(base)));
    lds = uniform(lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory", "m0");
}
// 4 bytes per lane of the first sixteen (all lanes are on).
__device__ inline void load_lds4(const void* src, uint32_t lds)
{
    lds = uniform(lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 exec, 0xffff\n\tglobal_load_lds_dword %1, off\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(src)
                 : "memory", "m0");
}

// Four e4m3 codes as bf16 (every code's value is one).
__device__ inline u32x2 bf16_of_codes(uint32_t x)
{
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true))};
}

// Whether a code is NaN (0x7F, 0xFF), and 0 in its place.
__device__ inline bool nan4(uint32_t x) { return (((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }
__device__ inline uint32_t zero_nan4(uint32_t x)
{
    const uint32_t bad = (((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
    return x & ~(bad * 0xFFu);
}

// Whether one of two bf16 is not finite, and 0 in its place.
__device__ inline uint32_t finite2(uint32_t x)
{
    x &= (x & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : ~0u;
    return x & ((x & 0x7F800000u) == 0x7F800000u ? 0x0000FFFFu : ~0u);
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
    static constexpr int ROW = 2 * D, HALF = TILE * ROW;     // HALF: the keys, or the values, of a tile
    static constexpr int G = ROW / 16;                       // granules of a row
    __device__ static uint32_t fk(uint32_t x) { return D == 128 ? x & 15 : (x >> 1) & 7; }
    __device__ static uint32_t fv(uint32_t x) { return D == 128 ? 4 * (x & 3) : 4 * ((x >> 1) & 1); }
    // e4m3: codes as they are in memory, in a ring; two tiles of bf16, the one in use and the next.
    static constexpr int CODES_WAVE = 8 * 2 * D;             // a wave's eight rows of keys, then of values
    static constexpr int CODES = WAVES * CODES_WAVE;
    // Scales: a wave's 8 + 8 floats, for twice as many tiles, as they are read when the codes' place is
    // filled again.
    static constexpr int SCALES_WAVE = 64, SCALES = WAVES * SCALES_WAVE;
    static constexpr int SCALES_AT = STAGES * CODES;
    static constexpr int KEYS = FP8 ? 2 : 4, VALUES = FP8 ? 3 : 5;   // tiles of bf16 keys, and of values
    static constexpr int ONES_AT = FP8 ? SCALES_AT + 2 * STAGES * SCALES : 0;
    static constexpr int KEYS_AT = FP8 ? ONES_AT + SCALES : 0;
    static constexpr int VALUES_AT = KEYS_AT + KEYS * HALF;
    static constexpr int PAGES_AT = VALUES_AT + VALUES * HALF;
    __device__ static uint32_t keys_at(int x) { return KEYS_AT + ((uint32_t)x & (KEYS - 1)) * HALF; }
    __device__ static uint32_t values_at(int x) { return VALUES_AT + (uint32_t)(x + VALUES) % VALUES * HALF; }
    static constexpr int FLAG_AT = PAGES_AT + WAVES * PAGE_SLOTS * 4;
    static constexpr int BYTES = FLAG_AT + 16;
    static constexpr int SUMS_WAVE = D / 32 * 16 * 256 + 512;   // a wave's output sums, references and sums
    static_assert(4 * SUMS_WAVE <= PAGES_AT && BYTES <= 163840, "LDS");
    // A wave's loads of a tile: its keys (and scales), its values.
    static constexpr int KLOADS = FP8 ? (D == 128 ? 2 : 1) : (D == 128 ? 2 : 1), VLOADS = D == 128 && !FP8 ? 2 : 1;
    static constexpr int LEAD = FP8 ? 6 : 4;                 // turn i asks for the keys of tile i + LEAD, the values of the one before
};

template <int D, bool FP8, bool PAGE8>
__global__ void __launch_bounds__(64 * WAVES) kv_attention_mfma(Params P)
{
    using Y = Layout<D, FP8>;
    constexpr int KS = D / 16, DB = D / 32;
    __shared__ __attribute__((aligned(1024))) char smem[Y::BYTES];
    uint32_t* const flags = reinterpret_cast<uint32_t*>(smem + Y::FLAG_AT);   // of the last four tiles
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
    if (threadIdx.x < 4)
        flags[threadIdx.x] = 0xFFFFFFFFu;
    if (FP8 && threadIdx.x < Y::SCALES / 4)
        reinterpret_cast<float*>(smem + Y::ONES_AT)[threadIdx.x] = 1.0f;
    uint32_t sequence = 0;                   // tiles this workgroup has had

    const uint32_t lds0 = lds_addr(smem);
    // Lane-constant offsets of the operand reads: of the first columns; those of others differ in single bits.
    const uint32_t k0 = col * Y::ROW + ((half ^ Y::fk(col)) * 16);
    uint32_t v0;
    {
        // lane c of a 16-lane group addresses row c / 4 of four, and 8 bytes of 16 columns
        const uint32_t c16 = lane & 15, row = 4 * half + (c16 >> 2);
        v0 = row * Y::ROW + (((2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1)) ^ Y::fv(row)) * 16) + (c16 & 1) * 8;
    }
    const float c = fabsf(a.scale) * kLog2e;   // a negative scale turns the queries' signs; 0 is not taken
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    const float slack = kSlack / c;
    const uint32_t st_token = (uint32_t)a.L.stride_token;   // PAGE8: below 2^24

    auto process = [&](auto narrow, uint32_t tile0, uint32_t tile1) __attribute__((always_inline)) {
        constexpr bool N = decltype(narrow)::value;
        constexpr int KB = N ? 1 : 2;        // blocks of 32 positions of a wave
        const uint32_t group = N ? wave >> 1 : wave, kb0 = N ? wave & 1 : 0;
        const uint32_t row0 = it.m * (N ? NARROW : WIDE) + group * 32;
        const bool live = row0 < r.rows;
        const uint32_t my_row = min(row0 + col, r.rows - 1), my_tok = my_row / P.G;
        const uint32_t pos = r.cached + my_tok;
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
            const uint32_t head = it.kh * P.G + my_row - my_tok * P.G;
            const char* src = a.q + (int64_t)(r.t0 + my_tok) * a.q_st + (int64_t)head * Y::ROW + half * 16;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                q[s] = as_bf16x8(ld16(src + s * 32) ^ flip);
        }

        const uint32_t n = tile1 - tile0;
        auto tile_start = [&](uint32_t x) __attribute__((always_inline)) {
            const uint32_t j = tile0 + x;
            return (j < it.ns ? j : it.lo + (j - it.ns)) * TILE;
        };
        auto page_of = [&](uint32_t p) __attribute__((always_inline)) {
            return PAGE8 ? __umulhi(p, P.ps_magic) >> P.ps_shift : p / a.L.page_size;
        };
        auto page_id = [&](uint32_t lp) __attribute__((always_inline)) {
            const uint32_t id = a.L.page_table[(size_t)it.b * a.L.max_pages + min(lp, a.L.max_pages - 1)];
            return min(id, a.L.num_pages - 1);
        };
        // This wave fetches rows 8 wave .. 8 wave + 7 of every tile; rows past the end repeat the last one.
        // PAGE8: they are in one page, and lane x holds where, for tile id0 + x: the offset in the layer, with the
        // last of the eight rows to read in its lowest bits (and the offset of the scales).  Else the wave's part of
        // LDS holds P.ids page ids for each of `hold` tiles.
        auto first_row = [&](uint32_t x) __attribute__((always_inline)) {
            const uint32_t p = tile_start(x) + wave * 8;
            return p < len ? p : (PAGE8 ? (len - 1) & ~7u : len - 1);
        };
        uint32_t* const my_ids = reinterpret_cast<uint32_t*>(smem + Y::PAGES_AT) + wave * PAGE_SLOTS;
        const uint32_t hold = PAGE8 ? 64 : PAGE_SLOTS / P.ids;
        uint32_t id0 = 0;
        uint64_t at_reg = 0, scale_reg = 0;
        auto fetch_ids = [&](uint32_t x0) __attribute__((always_inline)) {
            id0 = x0;
            if constexpr (PAGE8) {
                const uint32_t p0 = first_row(min(x0 + lane, n - 1)), lp = page_of(p0);
                const uint32_t id = page_id(lp), in_page = p0 - lp * a.L.page_size;
                at_reg = (uint64_t)((int64_t)id * a.L.stride_page + (int64_t)in_page * a.L.stride_token) | min(len - 1 - p0, 7u);
                if constexpr (FP8)
                    scale_reg = (uint64_t)((int64_t)id * a.Ls.stride_page + (int64_t)in_page * a.Ls.stride_token);
            } else {
                for (uint32_t k = lane; k < hold * P.ids; k += 64) {
                    const uint32_t s = k / P.ids, e = k - s * P.ids;
                    my_ids[k] = page_id(page_of(first_row(min(x0 + s, n - 1))) + e);
                }
            }
        };

        const int64_t head_bytes = (int64_t)it.kh * (FP8 ? D : 2 * D);
        const int64_t scale_bytes = (int64_t)(it.kh * D / 128) * 4;
        // Turn i asks for the keys of tile i + LEAD and for the values of the tile before.  What the keys'
        // addresses were made of is kept for the values' turn.
        constexpr int ROWSETS = !FP8 && D == 128 ? 2 : 1;
        struct Source {
            const char* src;                 // PAGE8: of the eight rows, uniform
            uint32_t last;
            const char* row[ROWSETS];        // else of the lane's rows
        };
        Source now{a.L.base, 0, {}}, one = now;   // of this turn's keys and its values
        bool ask_keys = false, ask_vals = false;   // what the turn's loads are, and where they go
        uint32_t k_dst = 0, v_dst = 0, s_dst = 0;
        [[maybe_unused]] const char* scale_src = nullptr;
        auto prepare = [&](int i, auto all) __attribute__((always_inline)) {
            constexpr bool ALL = decltype(all)::value;   // there are keys and values to ask for, of known pages
            const int kt = i + Y::LEAD, vt = kt - 1;
            const bool keys = ALL || kt < (int)n, vals = ALL || (vt >= 0 && vt < (int)n);
            [[maybe_unused]] constexpr uint32_t LR = Y::G;    // bf16: lanes of a row
            one = now;
            ask_keys = keys;
            ask_vals = vals;
            k_dst = uniform(lds0 + (FP8 ? (uint32_t)(i & (STAGES - 1)) * Y::CODES + wave * Y::CODES_WAVE
                                                       : Y::keys_at(kt) + wave * 8 * Y::ROW));
            v_dst = uniform(FP8 ? k_dst + Y::CODES_WAVE / 2 : lds0 + Y::values_at(vt) + wave * 8 * Y::ROW);
            if (keys) {
                if (!ALL && (uint32_t)kt >= id0 + hold)
                    fetch_ids((uint32_t)kt);
                [[maybe_unused]] const char* scale_at = nullptr;
                if constexpr (PAGE8) {
                    auto held = [&](uint64_t v) __attribute__((always_inline)) {
                        const int x = (int)((uint32_t)kt - id0);
                        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, x) |
                               (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), x) << 32;
                    };
                    const uint64_t at = held(at_reg);
                    now.last = (uint32_t)at & 7;
                    now.src = a.L.base + (int64_t)(at - now.last) + head_bytes;
                    if constexpr (FP8)
                        scale_at = a.Ls.base + (int64_t)held(scale_reg) +
                                   (int64_t)min((uint32_t)lane & 7, now.last) * a.Ls.stride_token;
                } else {
                    const uint32_t* ids = my_ids + ((uint32_t)kt - id0) * P.ids;
                    const uint32_t first = page_of(first_row((uint32_t)kt)), start = tile_start((uint32_t)kt) + wave * 8;
                    auto at = [&](const PagedLayer& L, uint32_t x) __attribute__((always_inline)) {
                        const uint32_t p = min(start + x, len - 1), lp = page_of(p);
                        return L.base + (int64_t)ids[lp - first] * L.stride_page +
                               (int64_t)(p - lp * L.page_size) * L.stride_token;
                    };
#pragma unroll
                    for (uint32_t k = 0; k < ROWSETS; ++k)
                        now.row[k] = at(a.L, FP8 ? (D == 128 ? lane >> 3 : col >> 2) : 64 / LR * k + lane / LR) + head_bytes;
                    if constexpr (FP8)
                        scale_at = at(a.Ls, lane & 7);
                }
                if constexpr (FP8) {
                    scale_src = scale_at + scale_bytes + ((lane & 8) ? a.Ls.stride_kv : 0);
                    s_dst = uniform(lds0 + Y::SCALES_AT + (uint32_t)(kt & (2 * STAGES - 1)) * Y::SCALES +
                                    wave * Y::SCALES_WAVE);
                }
            }
        };
        // The turn's loads in PARTS parts: one after the other they would wait for one another (64 bytes per clock
        // and CU), so that they are issued between products.
        constexpr int PARTS = FP8 ? (D == 128 ? 3 : 2) : 2 * ROWSETS;
        auto load_part = [&](int part) __attribute__((always_inline)) {
            constexpr uint32_t LR = Y::G;    // bf16: lanes of a row
            if constexpr (FP8) {
                if (part == 0) {
                    if (ask_keys)
                        load_lds4(scale_src, s_dst);
                    return;
                }
            }
            if constexpr (FP8 && D == 64) {
                // Half the lanes fetch keys, the others values (or keys again: not read).
                if (ask_keys || ask_vals) {
                    const bool v = half && ask_vals;
                    const char* src;
                    if constexpr (PAGE8)
                        src = (v ? one.src : now.src) + __umul24(min(col >> 2, v ? one.last : now.last), st_token);
                    else
                        src = v ? one.row[0] : now.row[0];
                    asm_gld16_lds(src + (v ? a.L.stride_kv : 0) + (lane & 3) * 16, uniform(k_dst));
                }
            } else {
                auto load = [&](const Source& from, int64_t plus, uint32_t dst, uint32_t k, auto values) __attribute__((always_inline)) {
                    const uint32_t x = FP8 ? lane >> 3 : 64 / LR * k + lane / LR;
                    const uint32_t g = FP8 ? lane & 7
                                           : (lane & (LR - 1)) ^ (decltype(values)::value ? Y::fv(x) : Y::fk(wave * 8 + x));
                    if constexpr (PAGE8)
                        load_lds16(from.src + plus, __umul24(min(x, from.last), st_token) + g * 16, dst + k * 1024);
                    else
                        asm_gld16_lds(from.row[k] + plus + g * 16, uniform(dst + k * 1024));
                };
                const int p = FP8 ? part - 1 : part;
                if (p < ROWSETS) {
                    if (ask_keys)
                        load(now, 0, k_dst, p, std::false_type{});
                } else if (ask_vals) {
                    load(one, a.L.stride_kv, v_dst, p - ROWSETS, std::true_type{});
                }
            }
        };
        auto load_all = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
                load_part(k);
        };
        auto issue = [&](int i) __attribute__((always_inline)) {
            prepare(i, std::false_type{});
            load_all();
        };
        // Loads that a turn has asked for.
        auto asked = [&](int i) __attribute__((always_inline)) {
            const int kt = i + Y::LEAD, vt = kt - 1;
            if (FP8 && D == 64)              // the scales; keys and values together
                return (kt < (int)n ? 1u : 0u) + (kt < (int)n || (vt >= 0 && vt < (int)n) ? 1u : 0u);
            return (kt < (int)n ? (uint32_t)Y::KLOADS : 0u) + (vt >= 0 && vt < (int)n ? (uint32_t)Y::VLOADS : 0u);
        };
        // Waits until turn i - M is done, turns up to i - 1 having been issued.
        auto wait_turns = [&](int i, auto turns) __attribute__((always_inline)) {
            constexpr int M = decltype(turns)::value, ALL = (M - 1) * (Y::KLOADS + Y::VLOADS);
            if (i - 1 + Y::LEAD < (int)n && i - M + 1 + Y::LEAD >= 1) {
                wait_loads<ALL>();
                return;
            }
            uint32_t left = 0;
#pragma unroll
            for (int k = 1; k < M; ++k)
                left += asked(i - k);
            wait_some<ALL>(left);
        };
        // Whether some row of the item does not see all of a tile.  Such rows of values may hold anything, and a
        // weight of 0 would turn infinities and NaN into NaN: each wave looks at its eight rows, puts zeros in
        // their place and raises the tile's flag.  The rows that do see them get them behind the product.
        auto ragged = [&](uint32_t start) __attribute__((always_inline)) {
            return start + TILE > b_hi0 || (start < b_low1 && start + TILE > b_sunk0);
        };
        auto raise = [&](uint32_t x) __attribute__((always_inline)) {
            if (lane == 0)
                flags[x & 3] = sequence + x;
        };
        // bf16: the loads that step x needs (keys of tile x + 1, values of tile x) are done.
        auto ready = [&](int x) __attribute__((always_inline)) {
            if constexpr (!FP8) {
                wait_turns(x, std::integral_constant<int, 3>{});
                if (x >= 0 && x < (int)n && ragged(tile_start((uint32_t)x))) {
                    char* mine = smem + Y::values_at(x) + wave * 8 * Y::ROW + lane * 16;
#pragma unroll
                    for (int i = 0; i < 8 * Y::ROW / 1024; ++i) {
                        u32x4 v = lds_ld16(mine + i * 1024);
                        if (__any(nonfinite2(v[0]) || nonfinite2(v[1]) || nonfinite2(v[2]) || nonfinite2(v[3]))) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = finite2(v[k]);
                            lds_st16(mine + i * 1024, v);
                            raise((uint32_t)x);
                        }
                    }
                    wait_lds();
                }
            }
        };
        // e4m3: this wave's rows from codes to bf16, as turn i - 4 loaded them: keys of tile i + 2, values of tile
        // i + 1.  In three parts, to go between products.  (A lane's two stores are neighbouring granules, so eight
        // lanes write every other one: each store takes its banks twice, 8 of the 16 cycles of each.)
        [[maybe_unused]] u32x4 codes[2] = {};
        auto convert = [&](int i, bool all, int part) __attribute__((always_inline)) {
            const bool keys = all || i + 2 < (int)n, vals = all || (i + 1 >= 0 && i + 1 < (int)n);
            auto put = [&](u32x4 x, char* to, uint32_t rr, uint32_t gr, uint32_t f) __attribute__((always_inline)) {
                const u32x2 c0 = bf16_of_codes(x[0]), c1 = bf16_of_codes(x[1]), c2 = bf16_of_codes(x[2]), c3 = bf16_of_codes(x[3]);
                lds_st16(to + rr * Y::ROW + ((gr ^ f) * 16), u32x4{c0[0], c0[1], c1[0], c1[1]});
                lds_st16(to + rr * Y::ROW + (((gr + 1) ^ f) * 16), u32x4{c2[0], c2[1], c3[0], c3[1]});
            };
            if (part == 0) {
                if (all)
                    wait_loads<3 * (Y::KLOADS + Y::VLOADS)>();
                else
                    wait_turns(i, std::integral_constant<int, 4>{});
                const char* src = smem + (i & (STAGES - 1)) * Y::CODES + wave * Y::CODES_WAVE + lane * 16;
                codes[0] = lds_ld16(src);
                if constexpr (D == 128)
                    codes[1] = lds_ld16(src + 1024);
                return;
            }
            if (part == 1) {
                // Values, and scales of values, that are not finite in a tile that some row does not see whole.
                if (all || !vals || !ragged(tile_start((uint32_t)i + 1)))
                    return;
                u32x4& x = codes[D == 128 ? 1 : 0];
                const bool values = D == 128 || half;
                bool bad = false;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    bad |= values && nan4(x[k]);
                float* sv = reinterpret_cast<float*>(smem + Y::SCALES_AT + ((i + 1) & (2 * STAGES - 1)) * Y::SCALES +
                                                     wave * Y::SCALES_WAVE) + 8 + (lane & 7);
                const bool bad_scale = !(fabsf(*sv) < INFINITY);
                if (__any(bad || bad_scale)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = values ? zero_nan4(x[k]) : x[k];
                    if (bad_scale)
                        *sv = 0.0f;
                    raise((uint32_t)i + 1);
                }
                return;
            }
            char* k_to = smem + Y::keys_at(i);
            char* v_to = smem + Y::values_at(i + 1);
            if constexpr (D == 128) {
                const uint32_t rr = wave * 8 + (lane >> 3), gr = 2 * (lane & 7);
                if (part == 2 && keys)
                    put(codes[0], k_to, rr, gr, Y::fk(rr));
                if (part == 3 && vals)
                    put(codes[1], v_to, rr, gr, Y::fv(rr));
            } else {
                const uint32_t rr = wave * 8 + (col >> 2), gr = 2 * (lane & 3);
                if (part == 2 && (half ? vals : keys))
                    put(codes[0], half ? v_to : k_to, rr, gr, half ? Y::fv(rr) : Y::fk(rr));
            }
        };
        auto convert_all = [&](int i) __attribute__((always_inline)) {
            if constexpr (FP8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    convert(i, false, k);
        };
        // Steps plain0 .. plain1 - 1 are plain ones: all rows see all of the tiles t - 1 to t + 1, behind the first
        // positions, and the turn's tiles are whole and their pages' ids at hand.
        uint32_t plain0 = 0, plain1 = 0;
        auto find_plain = [&](uint32_t t) __attribute__((always_inline)) {
            // tiles x0 .. x1 - 1 are not ragged, and behind the first positions (or there are none)
            const uint32_t sunk_tiles = it.ns > tile0 ? it.ns - tile0 : 0;
            const uint32_t low_tile = (b_low1 + TILE - 1) / TILE, x_low = it.ns + (low_tile > it.lo ? low_tile - it.lo : 0);
            const uint32_t x0 = max(sunk_tiles, x_low > tile0 ? x_low - tile0 : 0);
            const uint32_t hi_tile = it.ns + (b_hi0 / TILE > it.lo ? b_hi0 / TILE - it.lo : 0);
            const uint32_t x1 = hi_tile > tile0 ? min(hi_tile - tile0, n) : 0;
            const uint32_t whole_tile = it.ns + (len / TILE > it.lo ? len / TILE - it.lo : 0);
            const uint32_t whole = whole_tile > tile0 ? min(whole_tile - tile0, n) : 0;
            const uint32_t most = min(whole, id0 + hold), ahead = Y::LEAD + 1;
            plain0 = max(max(x0 + 1, sunk_tiles + 1), t);
            plain1 = min(x1 > 0 ? x1 - 1 : 0, most > ahead ? most - ahead : 0);
        };
        auto prepare_turn = [&](int i, bool plain) __attribute__((always_inline)) {
            if (plain) {
                prepare(i, std::true_type{});
            } else {
                const uint32_t had = id0;
                prepare(i, std::false_type{});
                if (id0 != had)
                    find_plain((uint32_t)i);
            }
        };
        // Turn i, behind the barrier of step i.
        auto turn = [&](int i) __attribute__((always_inline)) {
            convert_all(i);
            prepare_turn(i, false);
            load_all();
        };
        // e4m3: scales (keys 0, values 1) of rows 8 i + 4 half .. + 3 of tile x.
        auto scales_at = [&](uint32_t x) __attribute__((always_inline)) {
            return Y::SCALES_AT + (x & (2 * STAGES - 1)) * Y::SCALES;
        };
        auto scales_of = [&](uint32_t at, uint32_t side, uint32_t i) __attribute__((always_inline)) {
            return *reinterpret_cast<const f32x4*>(smem + at + i * Y::SCALES_WAVE + side * 32 + half * 16);
        };

        lds_barrier();                       // the LDS of the item before is no longer read
        fetch_ids(0);
        find_plain(1);
        if constexpr (FP8) {
            for (int i = -Y::LEAD; i < -2; ++i)
                issue(i);
            turn(-2);
        } else {
            for (int i = -Y::LEAD; i < -1; ++i)
                issue(i);
        }

        f32x16 o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                o[d][e] = 0.0f;
        float mref = kNothing, l = 0.0f;
        f32x16 s[KB];                        // scores of tile t, then its weights
        [[maybe_unused]] f32x4 ks[4] = {};   // e4m3: scales of keys
        bf16x8 w8[KB][2];                    // weights of tile t - 1, then of tile t, as operands
#pragma unroll
        for (int b = 0; b < KB; ++b)
            w8[b][0] = w8[b][1] = as_bf16x8(u32x4{0u, 0u, 0u, 0u});

        // Does some row of this wave see some of tile x?
        auto sees_some = [&](uint32_t x) __attribute__((always_inline)) {
            const uint32_t my0 = tile_start(x) + kb0 * 32, my1 = my0 + KB * 32;
            return live && my0 < w_hi1 && !(my1 <= w_low0 && my0 >= min(a.sinks, w_low1));
        };
        // Scores of the first tile.  Operands are read READS products ahead, which the fences keep the compiler to.
        auto scores = [&](uint32_t x) __attribute__((always_inline)) {
            const uint32_t kt = Y::keys_at((int)x) + kb0 * 32 * Y::ROW + k0;
            constexpr int NP = KS * KB;
            bf16x8 k8[READS];
            auto operand = [&](int i) __attribute__((always_inline)) {
                return as_bf16x8(lds_ld16(smem + (kt ^ (i / KB * 32)) + i % KB * 32 * Y::ROW));
            };
#pragma unroll
            for (int i = 0; i < READS && i < NP; ++i)
                k8[i] = operand(i);
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    s[b][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                s[i % KB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8[i % READS], q[i / KB], s[i % KB], 0, 0, 0);
                if (i + READS < NP)
                    k8[i % READS] = operand(i + READS);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // Element 4 i + e of block b of a tile's scores is position 32 (kb0 + b) + 8 i + 4 half + e of it.
        // e4m3: the scales of the keys.
        auto scale_keys = [&](uint32_t x, int b0, int b1) __attribute__((always_inline)) {
            if constexpr (FP8) {
#pragma unroll
                for (int b = b0; b < b1; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 f = scales_of(scales_at(x), 0, (kb0 + b) * 4 + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[b][4 * i + e] *= f[e];
                    }
            }
        };
        // What rows do not see.
        auto mask = [&](uint32_t x, bool visible) __attribute__((always_inline)) {
            const uint32_t my0 = tile_start(x) + kb0 * 32, my1 = my0 + KB * 32;
            if (!visible || my1 > w_hi0 || (my0 < w_low1 && my1 > w_sunk0)) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint32_t p = my0 + 32 * b + 8 * (e / 4) + 4 * half + e % 4;
                        s[b][e] = visible && (p - low < count || p < sunk) ? s[b][e] : -INFINITY;
                    }
            }
        };
        bf16x8 x8[READS];                    // operands of the next products
        auto read_first = [&](int x) __attribute__((always_inline)) {
            const uint32_t vt = Y::values_at(x) + kb0 * 32 * Y::ROW + v0;
#pragma unroll
            for (int i = 0; i < READS; ++i) {
                const char* at = smem + (vt ^ (i % DB * 64)) + i / DB * 16 * Y::ROW;
                x8[i] = join8(lds_tr16(at), lds_tr16(at + 8 * Y::ROW));
            }
        };
        // The weighted sums of the last tile.
        auto last_sums = [&]() __attribute__((always_inline)) {
            const uint32_t vt = Y::values_at((int)n - 1) + kb0 * 32 * Y::ROW + v0;
            constexpr int NP = DB * 2 * KB;
            auto operand = [&](int i) __attribute__((always_inline)) {
                const char* at = smem + (vt ^ (i % DB * 64)) + i / DB * 16 * Y::ROW;
                return join8(lds_tr16(at), lds_tr16(at + 8 * Y::ROW));
            };
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                o[i % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x8[i % READS], w8[i / (2 * DB)][i / DB % 2], o[i % DB], 0, 0, 0);
                if (i + READS < NP)
                    x8[i % READS] = operand(i + READS);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // What was not finite in the values of tile x, from the pool, one position at a time, for the rows that
        // see it.  (Its weights are still the operands'.)
        auto add_nonfinite = [&](uint32_t x) __attribute__((always_inline)) {
            const uint32_t my0 = tile_start(x) + kb0 * 32;
#pragma unroll 1
            for (uint32_t k = 0; k < 32u * KB; ++k) {
                const uint32_t p = my0 + k;
                if (p >= len)
                    break;
                const bool sees = p - low < count || p < sunk;
                // position k is element 16 (k / 32) + (k % 32) / 8 * 4 + k % 4 of half (k / 4) % 2
                const uint32_t e0 = (k >> 5) * 16 + ((k >> 3) & 3) * 4 + (k & 3);
                uint32_t pair = 0;
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pair = e0 / 2 == (uint32_t)(8 * b + e) ? __builtin_bit_cast(u32x4, w8[b][e / 4])[e % 4] : pair;
                const f32x2 h = halves(e0 & 1 ? bf16_hi(pair) : bf16_lo(pair));
                const float w = (k >> 2) & 1 ? h[1] : h[0];
                const char* v = a.L.base + token_offset(a.L, it.b, p) + a.L.stride_kv + head_bytes + half * (FP8 ? 4 : 8);
                bool whole = false;          // e4m3: a scale that is not finite makes all columns NaN
                if constexpr (FP8)
                    whole = !(fabsf(*reinterpret_cast<const float*>(a.Ls.base + token_offset(a.Ls, it.b, p) + a.Ls.stride_kv +
                                                                    scale_bytes)) < INFINITY);
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // columns 32 d + 8 i + 4 half .. + 3
                        u32x2 y;
                        if constexpr (FP8)
                            y = bf16_of_codes(*reinterpret_cast<const uint32_t*>(v + 32 * d + 8 * i));
                        else
                            y = *reinterpret_cast<const u32x2*>(v + 64 * d + 16 * i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float z = whole ? NAN : e & 1 ? bf16_hi(y[e / 2]) : bf16_lo(y[e / 2]);
                            if (sees && !(fabsf(z) < INFINITY))
                                o[d][4 * i + e] += w * z;
                        }
                    }
            }
        };

        // The products of a step, of 32 cycles each, with the softmax between them, five or six other
        // instructions to a product.  The scores' first block is free, and taken by the next tile's, once its weights
        // are operands.
        auto whole_step = [&](uint32_t t, bool plain) __attribute__((always_inline)) {
            const uint32_t vt = Y::values_at((int)t - 1) + kb0 * 32 * Y::ROW + v0;
            const uint32_t vn = Y::values_at((int)t) + kb0 * 32 * Y::ROW + v0;
            const uint32_t kt = Y::keys_at((int)t + 1) + kb0 * 32 * Y::ROW + k0;
            constexpr int NV = DB * 2 * KB, NP = NV + KS * KB;
            [[maybe_unused]] const uint32_t ks_at = plain ? scales_at(t) : (uint32_t)Y::ONES_AT, vs_at = scales_at(t);
            auto operand = [&](int i) __attribute__((always_inline)) {
                if (i < NV || i >= NP) {     // (behind the last: the next step's first)
                    const int k = i < NV ? i : i - NP;
                    const char* at = smem + ((i < NV ? vt : vn) ^ (k % DB * 64)) + k / DB * 16 * Y::ROW;
                    return join8(lds_tr16(at), lds_tr16(at + 8 * Y::ROW));
                }
                const int j = i - NV;        // block by block
                return as_bf16x8(lds_ld16(smem + (kt ^ (j % KS * 32)) + j / KS * 32 * Y::ROW));
            };
            float y[4], base = 0.0f, f = 1.0f, part[4] = {};
            bool some = false;
            // e4m3: scales are read two products before their use.
            f32x4 vs[4 * KB];
            [[maybe_unused]] auto read_keys = [&](uint32_t at, int g) __attribute__((always_inline)) {
                ks[g % 4] = scales_of(at, 0, kb0 * 4 + g);
            };
            [[maybe_unused]] auto scale = [&](int g) __attribute__((always_inline)) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[g / 4][g % 4 * 4 + k] *= ks[g % 4][k];
            };
            auto read_values = [&](int e0, int e1) __attribute__((always_inline)) {
                if constexpr (FP8)
#pragma unroll
                    for (int e = (e0 + 3) / 4 * 4; e < e1; e += 4)
                        vs[e / 4] = scales_of(vs_at, 1, kb0 * 4 + e / 4);
            };
            auto greatest = [&](int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
                for (int e = e0; e < e1; ++e)
                    y[e & 3] = e < 4 ? s[0][e] : __builtin_elementwise_maximum(y[e & 3], s[e / 16][e % 16]);
            };
            auto reference = [&]() __attribute__((always_inline)) {
                const f32x2 h = halves(__builtin_elementwise_maximum(__builtin_elementwise_maximum(y[0], y[1]),
                                                                     __builtin_elementwise_maximum(y[2], y[3])));
                const float top = __builtin_elementwise_maximum(h[0], h[1]);
                const bool more = top > mref + slack;
                some = __any(more);
                const float next = more ? top : mref;
                f = __builtin_amdgcn_exp2f((mref - next) * c);
                mref = next;
                l *= f;
                base = -next * c;
            };
            auto weigh = [&](int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
                for (int e = e0; e < e1; ++e)
                    s[e / 16][e % 16] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 16][e % 16], c, base));
            };
            auto add = [&](int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
                for (int e = e0; e < e1; ++e) {
                    part[e & 3] += s[e / 16][e % 16];
                    if constexpr (FP8)
                        s[e / 16][e % 16] *= vs[e / 4][e % 4];
                }
                if (e1 > e0)
                    asm volatile("" : "+v"(part[0]), "+v"(part[1]), "+v"(part[2]), "+v"(part[3]));
            };
            auto pack = [&](int g) __attribute__((always_inline)) {
                const f32x16& z = s[g / 2];
                const int k = g % 2 * 8;
                u32x4 x = {pack_bf16x2(z[k], z[k + 1]), pack_bf16x2(z[k + 2], z[k + 3]), pack_bf16x2(z[k + 4], z[k + 5]),
                           pack_bf16x2(z[k + 6], z[k + 7])};
                asm volatile("" : "+v"(x));   // (here: the compiler would move it all behind the branch below)
                w8[g / 2][g % 2] = as_bf16x8(x);
            };
            using Z = Order<NV, KS, KB, DB, FP8>;
            each<NP>([&](auto step) __attribute__((always_inline)) {
                constexpr int i = decltype(step)::value;
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (i < NV) {
                    o[i % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x8[i % READS], w8[i / (2 * DB)][i / DB % 2], o[i % DB], 0,
                                                                        0, 0);
                } else {
                    constexpr int j = i - NV, b = j / KS;
                    if constexpr (j % KS == 0)
                        s[b] = f32x16{};     // (its weights are operands)
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x8[i % READS], q[j % KS], s[b], 0, 0, 0);
                }
                x8[(i + READS) % NP % READS] = operand(i + READS);
                if constexpr (FP8 && KB == 2) {
                    // The second block's scores are scaled here, the first one's behind its products.
                    constexpr int H = Z::HALF, PER = 4 / H, END = NV + KS, BY = 8 / KS;
                    if constexpr (i < H)
                        each<PER>([&](auto g) { read_keys(ks_at, 4 + i * PER + decltype(g)::value); });
                    else if constexpr (i < 2 * H)
                        each<PER>([&](auto g) { scale(4 + (i - H) * PER + decltype(g)::value); });
                    if constexpr (i >= END && i < END + KS / 2)
                        each<BY>([&](auto g) { read_keys(scales_at(t + 1), (i - END) * BY + decltype(g)::value); });
                    else if constexpr (i >= END + KS / 2)
                        each<BY>([&](auto g) { scale((i - END - KS / 2) * BY + decltype(g)::value); });
                } else if constexpr (FP8) {
                    if constexpr (i == 0)
                        each<4>([&](auto g) { scale(decltype(g)::value); });
                    if constexpr (i >= NP - 4)
                        read_keys(scales_at(t + 1), i - NP + 4);
                }
                read_values(i + 2 > NP ? Z::E : Z::weighed(i + 1), i + 2 > NP ? Z::E : Z::weighed(i + 2));
                if constexpr (i < Z::TOP - 1) {
                    greatest(Z::E * i / (Z::TOP - 1) / 4 * 4, Z::E * (i + 1) / (Z::TOP - 1) / 4 * 4);
                }
                if constexpr (i == Z::TOP - 1)
                    reference();
                weigh(Z::weighed(i), Z::weighed(i + 1));
                add(Z::added(i), Z::added(i + 1));
                each<2 * KB>([&](auto g) __attribute__((always_inline)) {
                    if constexpr (Z::packed(decltype(g)::value) == i)
                        pack(g);
                });
                // the turn: e4m3's conversion and the loads, one by one
                if constexpr (FP8) {
                    constexpr int AT[4] = {NP / 8, NP / 8 + 1, NP / 8 + 2, NP / 8 + 3};
                    static_assert(AT[D == 128 ? 3 : 2] < NP - READS, "the writes are older than the last reads");
                    each<4>([&](auto k) __attribute__((always_inline)) {
                        if constexpr (AT[decltype(k)::value] == i)
                            convert((int)t, plain, decltype(k)::value);
                    });
                }
                constexpr int FROM = FP8 ? NP / 8 + 4 : 1, EVERY = (NP - FROM) / PARTS;
                if constexpr (i == FROM - 1)
                    prepare_turn((int)t, plain);
                if constexpr (N) {           // (bound by memory: early)
                    if constexpr (i == FROM)
                        load_all();
                } else if constexpr (i >= FROM && (i - FROM) % EVERY == 0 && (i - FROM) / EVERY < PARTS) {
                    load_part((i - FROM) / EVERY);
                }
            });
            __builtin_amdgcn_sched_barrier(0);
            l += (part[0] + part[1]) + (part[2] + part[3]);
            if (some) {
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[d][e] *= f;
            }
        };

        // Step t: the sums of tile t - 1, the softmax of tile t, the scores of tile t + 1.  (Before the first tile
        // there are zeros; behind the last one, scores that nothing reads.)
        {
            char* mine = smem + Y::values_at(-1) + wave * 8 * Y::ROW + lane * 16;
#pragma unroll
            for (int i = 0; i < 8 * Y::ROW / 1024; ++i)
                lds_st16(mine + i * 1024, u32x4{0u, 0u, 0u, 0u});
        }
        ready(-1);
        lds_barrier();
        turn(-1);
        wait_lds();                          // (a wave that sees nothing of the first tile reads nothing before the barrier)
        bool weighed = false, visible = sees_some(0);   // tiles t - 1 and t
        if (visible) {
            scores(0);
            scale_keys(0, 0, KB - 1);
        }
#pragma unroll
        for (int i = 0; i < READS; ++i)
            x8[i] = as_bf16x8(u32x4{0u, 0u, 0u, 0u});
        bool read = true;                    // x8 holds the first operands of the values of tile t - 1
        for (uint32_t t = 0; t < n; ++t) {
            const bool plain = t >= plain0 && t < plain1;
            if (plain && !FP8)
                wait_loads<2 * (Y::KLOADS + Y::VLOADS)>();
            else
                ready((int)t);
            step_barrier();
            const bool next = plain ? live : t + 1 < n && sees_some(t + 1);
            if (weighed || visible || next) {
                if (!plain) {
                    scale_keys(t, KB - 1, KB);
                    if constexpr (FP8 && KB == 1)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ks[k] = f32x4{1.0f, 1.0f, 1.0f, 1.0f};
                    mask(t, visible);
                    // the operands of tile t - 1 are gone behind this, so what it lacks is added first
                    if (weighed && ragged(tile_start(t - 1)) && uniform(flags[(t - 1) & 3]) == sequence + t - 1)
                        add_nonfinite(t - 1);
                    if (!read)
                        read_first((int)t - 1);
                }
                whole_step(t, plain);
                read = true;
            } else {
                turn((int)t);
                wait_lds();
                read = false;
            }
            weighed = visible;
            visible = next;
        }
        ready((int)n);
        lds_barrier();
        if (weighed) {
            if (ragged(tile_start(n - 1)) && uniform(flags[(n - 1) & 3]) == sequence + n - 1)
                add_nonfinite(n - 1);
            last_sums();
        }
        sequence += n;

        // (Worked out again: they would hold registers through all of the steps.)
        const uint32_t ln = lane_again(), half = ln >> 5, col = ln & 31, lane = ln;
        const uint32_t row = min(row0 + col, r.rows - 1), tok = row / P.G, g = row - tok * P.G;

        // The row's sum, over both halves; with two groups of waves, over both of them.
        {
            const f32x2 h = halves(l);
            l = h[0] + h[1];
        }
        bool mine = live;
        if constexpr (N) {
            lds_barrier();                   // the tiles are no longer read by the others
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
// cuts left, each times its exp(reference - the largest one), in the order of the shares.  SETS groups of four
// waves take every SETS-th piece.
template <int D, int SETS>
__global__ void __launch_bounds__(256 * SETS) kv_attention_join(Params P)
{
    constexpr int Q = D / 32;                // a thread has Q quads of the row group's sums
    const uint32_t w = blockIdx.x + 1, group = blockIdx.y;
    const uint32_t groups = P.cuts[kKvGroups].tile;
    const KvCut cut = P.cuts[w], prev = P.cuts[w - 1];
    if (w >= groups || cut.tile == 0 || group * 32 >= cut.rows)
        return;
    auto same = [&](const KvCut& x) { return x.tile != 0 && x.b == cut.b && x.kh == cut.kh && x.m == cut.m; };
    if (same(prev))
        return;
    __shared__ uint32_t last;
    __shared__ bool empty[kKvGroups];        // shares that end where they begin leave nothing
    __shared__ float top[SETS][64], all[SETS][64];
    __shared__ f32x4 part[SETS > 1 ? SETS - 1 : 1][Q][256];
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
    float mx = kNothing, l = 0.0f;
    f32x4 sum[Q] = {};
    constexpr int U = 2;
    for (uint32_t k0 = set; k0 < pieces; k0 += SETS * U) {
        f32x4 v[U][Q];
        float m[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = k0 + SETS * u;
            const float* p = piece(min(k, pieces - 1));
            const bool on = k < pieces && (k == 0 || !empty[k - 1]);
            m[u] = p[32 * D + col];
            s[u] = p[32 * D + 32 + col];
#pragma unroll
            for (int j = 0; j < Q; ++j)
                v[u][j] = *reinterpret_cast<const f32x4*>(p + (j * 256 + tid) * 4);
            m[u] = on ? m[u] : kNothing;
            s[u] = on ? s[u] : 0.0f;
#pragma unroll
            for (int j = 0; j < Q; ++j)
                v[u][j] = on ? v[u][j] : f32x4{};
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float now = fmaxf(mx, m[u]);
            const float f0 = __builtin_amdgcn_exp2f((mx - now) * c), f1 = __builtin_amdgcn_exp2f((m[u] - now) * c);
            mx = now;
            l = l * f0 + s[u] * f1;
#pragma unroll
            for (int j = 0; j < Q; ++j)
                sum[j] = sum[j] * f0 + v[u][j] * f1;
        }
    }
    if constexpr (SETS > 1) {
        if (tid < 64) {
            top[set][lane] = mx;
            all[set][lane] = l;
        }
        if (set > 0)
#pragma unroll
            for (int j = 0; j < Q; ++j)
                part[set - 1][j][tid] = sum[j];
        __syncthreads();
        if (set > 0)
            return;
#pragma unroll
        for (int k = 1; k < SETS; ++k) {
            const float m1 = top[k][lane], now = fmaxf(mx, m1);
            const float f0 = __builtin_amdgcn_exp2f((mx - now) * c), f1 = __builtin_amdgcn_exp2f((m1 - now) * c);
            mx = now;
            l = l * f0 + all[k][lane] * f1;
#pragma unroll
            for (int j = 0; j < Q; ++j)
                sum[j] = sum[j] * f0 + part[k - 1][j][tid] * f1;
        }
    }
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
        const f32x4 x = sum[j] * inv;
        *reinterpret_cast<u32x2*>(out + 32 * j + 8 * (tid >> 6) + 4 * (lane >> 5)) =
            u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    }
    if (a.lse && tid < 32)
        a.lse[head] = l == 0.0f ? -INFINITY : mx * fabsf(a.scale) + __logf(l);
}

}  // namespace

bool kv_attention_mfma_fits(const KvAttentionArgs& a, KvKind kind)
{
    // The kernel's references are scores before scaling.  With a scale below 2^-64 these could lie below kNothing, and
    // with one above 2^26 kNothing times it could be infinite.
    const float c = std::fabs(a.scale) * kLog2e;
    return kind != KV_F32 && (a.D == 64 || a.D == 128) && c >= 0x1p-64f && c <= 0x1p26f &&
           // items are numbered in 32 bits, and their work together in 64
           (uint64_t)a.L.batch * a.KH < (uint64_t(1) << 24);
}

hipError_t launch_kv_attention_mfma(const KvAttentionArgs& a, KvKind kind, hipStream_t s)
{
    Params P{};
    P.a = a;
    P.G = (uint32_t)(a.H / a.KH);
    const uint32_t ps = a.L.page_size;
    P.ids = (6 + ps) / ps + 1;               // pages that eight positions can lie in
    const bool page8 = ps % 8 == 0 && a.L.stride_token < (int64_t(1) << 24);
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
    // Fewer items than 64: they have more than four pieces each.  Four groups of waves against one: one token of 8 heads on
    // a key head behind 131,071 rows (256 pieces) 69 against 118 us, of 32 on 8 behind 32,767 43 against 49; prompt
    // chunks (2 or 3 pieces) 551 against 536.
    const bool many = ((int64_t)a.L.batch + (int64_t)a.T * P.G / WIDE) * a.KH < 64;
    log_launch("kv_attention_join", (kKvGroups - 1) * row_groups, many ? 1024 : 256, "T=%d H=%d", a.T, a.H);
    hipLaunchKernelGGL(a.D == 64 ? (many ? kv_attention_join<64, 4> : kv_attention_join<64, 1>)
                                 : (many ? kv_attention_join<128, 4> : kv_attention_join<128, 1>),
                       dim3(kKvGroups - 1, row_groups), dim3(many ? 1024 : 256), 0, s, P);
    return hipGetLastError();
}

}  // namespace mla
