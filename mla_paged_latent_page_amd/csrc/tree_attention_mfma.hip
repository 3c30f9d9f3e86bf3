// Tree attention on the matrix cores: rows of 576 columns (512 latent + 64 rope), bf16 or
// e4m3 cache (see tree_attention.hip for the operator and the general form).
//
// A wave holds 32 query rows (tokens x heads) and takes 32 cache rows at a time: scores
// S^T = K Q^T (36 products of 32x32x16), weights P = exp(S - reference), O^T += V^T P^T (32
// products), V being the first 512 columns of K.  Transposed like this a lane has one query row
// throughout: its maximum, sum and rescaling need no exchange but one swap of the wave's halves,
// and P goes from the score layout into the next product's operand as it is.  The 32 x 512
// output sums are the wave's 256 accumulation registers, so there is one wave per SIMD, and
// everything else has the 256 ordinary ones: the scores of tile t + 1 are computed while the weights
// of tile t are, the loads of tile t + 3 go into a four-stage LDS ring in between.  They do not
// quite suffice: 74 to 102 values per variant are spilled (284 to 368 bytes a lane), most of them
// before the first step and around the join of two pairs.  Inside the steps, sixteen are reloaded
// for each tile that has to be masked (the bits of its rows; every reload also waits for the loads
// in flight), and constants that come back in the first step put a wait into all of them.  The
// reference is the running maximum, let lag by up to 2^8 (the weights stay below 2^8 in binary32),
// so the sums are rescaled only now and then.  Weights are rounded to bf16 for the product, their
// sum is not.
//
// Work: every workgroup takes an equal share of all tiles of all requests (one workgroup per
// CU); shares that end inside an item leave their sums, maximum and sum in the workspace in
// binary32, and tree_attention_join adds them up in a fixed order.  Requests with few query rows
// take narrower items, whose cache rows two pairs of waves share (Shape).
//
// Measured (MI355X; kernel trace, mean of 25 calls with their range, main kernel + join; then the
// calls back to back):
//   12 requests of 17-33 tokens x 128 heads, 1300-6000 rows, bf16: 272 (243-292) + 26 us; 260 us, 897
//     TFLOP/s.  Bound by the matrix cores (53 % busy) and by what a single wave per SIMD can issue
//     between their instructions, at the clock the power limit leaves.
//   64 requests of one token x 128 heads, 256-4096 rows, bf16: 52 (51-66) + 12 us; 70 us with rows from
//     memory.  Bound by memory: 140 MB read and 66 MB written by the main kernel, 39 MB read by the join.
//     About 90 MB of it are partial results, written and read again; fewer, larger shares side by side
//     would leave fewer.
//   5 requests of 5-8 tokens x 16 heads, 78-94 thousand rows, e4m3: 181 (172-190) + 11 us; 163 us.  Bound
//     by instruction issue: each wave converts every tile's codes to bf16 (272 conversions next to
//     68 products); 80-128 of an item's 128 rows hold queries.
//   4 requests of one token x 16 heads, 100-600 rows, bf16: 15 + 6 us, a chain of loads
//     (offsets, page ids, rows) and two launches.
//   Page sizes that are no multiple of 8 look up a page id per lane in every step, which waits for the
//     loads in flight: 100 against 64 tokens, the cases above with bf16 / e4m3 rows: trees 269 against
//     268 / 345 against 322 us, 64 requests 67 against 63 / 81 against 74, long contexts 190 against
//     164 / 209 against 164.
//   A chain is multiplied in full, hidden tiles included, and every tile of its own tokens is masked: a
//     prompt chunk of 2048 tokens x 128 heads 2.3 ms (bf16) and 1.9 ms (e4m3), behind 4096 rows 4.0 and
//     4.2 ms.
// An e4m3 product with the queries split into two e4m3 parts would need no conversion, but the
// matrix cores align the 64 terms of such a product to about 13 bits below the largest (probed:
// errors of 1.5e-4 of the sum of magnitudes), so it is not used.
#include <algorithm>
#include <cmath>
#include <utility>

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
// e4m3: a tile stays in codes, 4 blocks of 32 rows x 128 codes and one of 32 x 64, with its
// scales behind the four stages; then the query fragments for which the conversion leaves no
// registers.
constexpr int STAGE8 = TILE * D;
constexpr int SCALES_WAVE = 256;             // 5 blocks x 8 rows, floats
constexpr int SCALES = WAVES * SCALES_WAVE;
constexpr int SCALES_AT = STAGES * STAGE8;
constexpr int QUERY_AT = SCALES_AT + STAGES * SCALES;
constexpr int QUERY_KEPT = 26;               // fragments in registers; the others are in LDS
constexpr int QUERY_WAVE = (D / 16 - QUERY_KEPT) * 1024;
constexpr int JOIN_WAVE = 8 * 16 * 256 + 256; // a wave's half of the output sums, maxima and sums (SPLIT 2)
constexpr int SMEM8 = std::max(QUERY_AT + WAVES * QUERY_WAVE, WAVES * JOIN_WAVE);
constexpr int FLAG_BYTES = 16;               // behind all of it: whether clear_nonfinite found something
static_assert(SMEM8 + FLAG_BYTES <= 163840 && STAGES * STAGE + FLAG_BYTES <= 163840, "LDS");
constexpr int PIECE_WAVE = 32 * (K + 2);     // floats of one wave's partial result: 32 rows, maximum, sum
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.0f;               // the reference maximum may lag by 2^8

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

// What the join needs of the cut a workgroup starts at; every workgroup leaves one.
struct Cut {
    uint32_t w, w0, w1;                      // this cut, and the first and last one inside its item
    uint32_t row0, rows;                     // first query row of the item, rows it has (0: no split item)
    uint32_t pad[3];
};
static_assert(sizeof(Cut) == kAttnCutBytes, "workspace");

struct MfmaParams {
    TreeAttentionArgs a;
    uint32_t ps_magic, ps_shift;             // p / page_size = mulhi(p, magic) >> shift for p < 2^31
    uint32_t piece;                          // floats of a partial result slot
    Cut* cuts;                               // [kAttnGroups]
    uint32_t twins;                          // SPLIT 2: workgroups that share an item's rows
    uint32_t groups;                         // of 32 rows in an item: 4, or 2
    int min_tiles;                           // least steps of a workgroup's share
};

__device__ inline uint64_t uniform(uint64_t v)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
           ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32);
}
__device__ inline uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// How a workgroup's four waves share an item.  SPLIT 1: 128 query rows, 32 per wave, every wave
// reads all tiles.  SPLIT 2: 64 query rows, two pairs of waves; a step takes two tiles, one per
// pair, and the pairs' results are joined at the end; with twins, an item has 128 rows and two
// workgroups of one XCD take 64 each, at the same time from the same cache rows.  An item counts as COST units before its
// steps' one each: fetching its queries, filling the ring and writing its results takes about as
// long as that many steps.
template <int SPLIT>
struct Shape {
    static constexpr uint32_t ROWS = kAttnRows / SPLIT;   // query rows of a workgroup
    static constexpr uint32_t STEP = TILE * SPLIT;        // cache rows of a step
    static constexpr uint32_t COST = 8;
};

// Rows of a request and its share of the work: nm items.
struct Request {
    uint32_t b, t0, n, cached, len, nm, nu;  // nu = COST + steps
    uint32_t base;                           // units of all requests before it
};

template <int SPLIT>
__device__ inline Request request_at(const TreeAttentionArgs& a, uint32_t twins, uint32_t b)
{
    Request r{};
    const uint32_t end = min(a.iro[a.L.batch], (uint32_t)a.T);
    r.b = b;
    r.t0 = min(a.iro[b], end);
    const uint32_t t1 = min(a.iro[b + 1], end);
    r.n = t1 > r.t0 ? t1 - r.t0 : 0;
    r.cached = min(a.cache_len[b], a.capacity);
    r.len = min(r.cached + r.n, a.capacity);
    const uint32_t rows = Shape<SPLIT>::ROWS * twins;
    r.nm = (r.n * (uint32_t)a.H + rows - 1) / rows;   // n * H below 2^31 / D
    r.nu = (r.len + Shape<SPLIT>::STEP - 1) / Shape<SPLIT>::STEP + Shape<SPLIT>::COST;
    return r;
}

// A wave-uniform request, in scalar registers.
__device__ inline Request uniform(Request r)
{
    return Request{uniform(r.b), uniform(r.t0), uniform(r.n), uniform(r.cached), uniform(r.len), uniform(r.nm),
                   uniform(r.nu), uniform(r.base)};
}

// Sum over the lanes up to and including this one: within rows of 16 lanes, then a row's last
// lane into the next row, and lane 31 into the upper half.
__device__ inline uint32_t wave_inclusive(uint32_t v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return v;
}

// The schedule: all units (of all items of all requests, in that order) in equal shares.  A
// cut that falls within `snap` tiles of an item's first or last one is moved there: the item
// is then not split for so little.  Every wave works it out for itself; the requests of the last 64
// looked at stay in its lanes.  The host has checked that the units of ascending offsets number
// below 2^31; offsets that decrease can name a token in many requests, so nothing is done for them.
template <int SPLIT>
struct Schedule {
    static constexpr uint32_t COST = Shape<SPLIT>::COST;
    const TreeAttentionArgs& a;
    uint32_t twins;
    int lane;
    uint32_t total, groups, share, rest, snap;
    uint32_t first;                          // first request in the lanes
    uint32_t before;                         // units before it
    Request mine;
    uint32_t scan;                           // units up to and including mine, from `before`

    __device__ void load(uint32_t b0, uint32_t tiles_before)
    {
        first = b0;
        before = tiles_before;
        mine = Request{};
        if (b0 + lane < a.L.batch)
            mine = request_at<SPLIT>(a, twins, b0 + lane);
        scan = wave_inclusive(mine.nm * mine.nu);
    }
    // Some offset among those of the 64 requests from b0 on is above the next one.
    __device__ bool decreasing(uint32_t b0) const
    {
        return __ballot(b0 + lane < a.L.batch && a.iro[b0 + lane] > a.iro[b0 + lane + 1]) != 0;
    }
    __device__ uint32_t loaded() const { return (uint32_t)__builtin_amdgcn_readlane((int)scan, 63); }

    __device__ Schedule(const MfmaParams& P, int l) : a(P.a), twins(SPLIT == 1 ? 1 : P.twins), lane(l)
    {
        load(0, 0);
        total = loaded();
        bool bad = decreasing(0);
        for (uint32_t b0 = 64; b0 < a.L.batch; b0 += 64) {
            load(b0, total);
            total += loaded();
            bad |= decreasing(b0);
        }
        if (bad)
            total = 0;
        if (a.L.batch > 64)
            load(0, 0);
        const uint32_t want = (total + P.min_tiles - 1) / P.min_tiles, most = kAttnGroups / twins;
        groups = want < 1 ? 1u : want > most ? most : want;
        share = groups == kAttnGroups ? total / kAttnGroups : total / groups;
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
        r.nu = get(mine.nu);
        r.base = uniform(before + get(scan) - r.nm * r.nu);
        return r;
    }
    // Cut w, and the request it lies in.
    __device__ uint32_t cut(uint32_t w, Request& r)
    {
        const uint32_t x = raw(w);
        r = find(x);
        const uint32_t lo = r.base + (x - r.base) / r.nu * r.nu;
        return x - lo <= COST + snap ? lo : lo + r.nu - x <= snap ? lo + r.nu : x;
    }
};

typedef int v2i32 __attribute__((ext_vector_type(2)));
__device__ inline u32x2 lds_tr8(const char* p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                         (__attribute__((address_space(3))) v2i32*)(__attribute__((address_space(3))) void*)p));
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

// N loads of 16 bytes per lane into LDS, load j from 128 j bytes past the lane's address to
// lds + j * BLOCK_BYTES + 16 * lane (the instruction's offset moves both), by the lanes of the
// masks lo and hi; from a uniform base and a 32-bit lane offset, or from a lane address.  One
// piece of assembly, as the masks are the whole wave's.  A wait state lies between a write of m0 and a load.
#define MLA_LOAD(addr, offset) "global_load_lds_dwordx4 " addr " offset:" offset "\n\t"
#define MLA_NEXT "s_add_u32 m0, m0, 3968\n\ts_nop 0\n\t"
#define MLA_LOADS(N, addr)                                                                                        \
    if constexpr (J == 0 && N == 3)                                                                               \
        asm volatile(MLA_ON MLA_LOAD(addr, "0") MLA_NEXT MLA_LOAD(addr, "128") MLA_NEXT MLA_LOAD(addr, "256")     \
                     MLA_OFF MLA_ARGS);                                                                           \
    else if constexpr (J == 3 && N == 3)                                                                          \
        asm volatile(MLA_ON MLA_LOAD(addr, "384") MLA_NEXT MLA_LOAD(addr, "512") MLA_NEXT MLA_LOAD(addr, "640")   \
                     MLA_OFF MLA_ARGS);                                                                           \
    else if constexpr (J == 6 && N == 3)                                                                          \
        asm volatile(MLA_ON MLA_LOAD(addr, "768") MLA_NEXT MLA_LOAD(addr, "896") MLA_NEXT MLA_LOAD(addr, "1024")  \
                     MLA_OFF MLA_ARGS);                                                                           \
    else if constexpr (J == 0 && N == 2)                                                                          \
        asm volatile(MLA_ON MLA_LOAD(addr, "0") MLA_NEXT MLA_LOAD(addr, "128") MLA_OFF MLA_ARGS);                 \
    else if constexpr (J == 2 && N == 2)                                                                          \
        asm volatile(MLA_ON MLA_LOAD(addr, "256") MLA_NEXT MLA_LOAD(addr, "384") MLA_OFF MLA_ARGS);               \
    else                                                                                                          \
        asm volatile(MLA_ON MLA_LOAD(addr, "0") MLA_OFF MLA_ARGS)
#define MLA_ON "s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %3\n\t"
#define MLA_OFF "s_mov_b64 exec, -1"

template <int J, int N>
__device__ inline void load_lds(const char* base, uint32_t voff, uint32_t lds, uint32_t lo, uint32_t hi)
{
    lds += J * (BLOCK_BYTES - 128);
#define MLA_ARGS : : "s"(lds), "v"(voff), "s"(lo), "s"(hi), "s"(base) : "memory", "m0", "scc"
    MLA_LOADS(N, "%1, %4");
#undef MLA_ARGS
}
template <int J, int N>
__device__ inline void load_lds(const char* src, uint32_t lds, uint32_t lo, uint32_t hi)
{
    lds += J * (BLOCK_BYTES - 128);
#define MLA_ARGS : : "s"(lds), "v"(src), "s"(lo), "s"(hi) : "memory", "m0", "scc"
    MLA_LOADS(N, "%1, off");
#undef MLA_ARGS
}
#undef MLA_OFF
#undef MLA_ON
#undef MLA_LOADS
#undef MLA_NEXT
#undef MLA_LOAD
static_assert(BLOCK_BYTES - 128 == 3968, "the step of m0 in the loads");

// 4 bytes per lane.
__device__ inline void load_lds4(const char* base, uint32_t voff, uint32_t lds, uint32_t lo, uint32_t hi)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %4\n\t"
                 "global_load_lds_dword %1, %2\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(voff), "s"(base), "s"(lo), "s"(hi)
                 : "memory", "m0");
}
__device__ inline void load_lds4(const char* src, uint32_t lds, uint32_t lo, uint32_t hi)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %3\n\t"
                 "global_load_lds_dword %1, off\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(src), "s"(lo), "s"(hi)
                 : "memory", "m0");
}

// The lane's number, worked out where it is needed (it and what is derived from it would
// otherwise hold registers through the whole kernel).
__device__ inline uint32_t lane_again()
{
    uint32_t x;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
    return x;
}

template <int N>
__device__ inline void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One product with its sums in ordinary registers: the output sums take all 256 accumulation
// registers, and the compiler would put these there too.  It does not see that this is a matrix
// instruction, so the last one of a chain waits for its result before anything can read it (12
// wait states after 8 passes; back-to-back products into the same registers need none), and no
// operand may come from a vector instruction in the two states before.  Nor must it move the
// sums inside a chain: tests/test_matrix_waits.py reads the generated code for both.
__device__ inline void mfma_first(f32x16& acc, bf16x8 x, bf16x8 y)
{
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(acc) : "v"(x), "v"(y));
}
__device__ inline void mfma_next(f32x16& acc, bf16x8 x, bf16x8 y)
{
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(acc) : "v"(x), "v"(y));
}
template <bool IN_PLACE>   // else into other registers, where the result stays
__device__ inline f32x16 mfma_last(f32x16& acc, bf16x8 x, bf16x8 y)
{
    if constexpr (IN_PLACE) {
        asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0\n\ts_nop 13" : "+v"(acc) : "v"(x), "v"(y));
        return acc;
    } else {
        f32x16 out;
        asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %3\n\ts_nop 13" : "=&v"(out) : "v"(x), "v"(y), "v"(acc));
        return out;
    }
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

// Eight e4m3 codes as bf16 (every code's value is one).
__device__ inline bf16x8 bf16_of_codes(u32x2 v)
{
    auto two = [](uint32_t x, auto high) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, decltype(high)::value));
    };
    const std::false_type lo;
    const std::true_type hi;
    return as_bf16x8(u32x4{two(v[0], lo), two(v[0], hi), two(v[1], lo), two(v[1], hi)});
}

__device__ inline bool nonfinite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// The result of one lane pair's row, feature blocks FIRST .. FIRST + N - 1: the final output,
// eight features per 16-byte store, or a share's sums, maximum and sum as they are, in lane order.
template <int FIRST, int N>
__device__ __attribute__((always_inline)) inline void store_result(const TreeAttentionArgs& a, const f32x16 (&o)[16],
                                                                   float mref, float l, uint32_t qrow, bool valid,
                                                                   bool whole, float* piece, int lane)
{
    const int half = lane >> 5, col = lane & 31;
    if (whole) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)qrow * K + 8 * half;
#pragma unroll
        for (int fb = FIRST; fb < FIRST + N; ++fb)
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                uint32_t x0 = pack_bf16x2(o[fb][i] * inv, o[fb][i + 1] * inv);
                uint32_t x1 = pack_bf16x2(o[fb][i + 2] * inv, o[fb][i + 3] * inv);
                uint32_t y0 = pack_bf16x2(o[fb][i + 4] * inv, o[fb][i + 5] * inv);
                uint32_t y1 = pack_bf16x2(o[fb][i + 6] * inv, o[fb][i + 7] * inv);
                const auto u = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
                const auto v = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
                if (valid)
                    st16(out + fb * 32 + 2 * i, u32x4{u[0], v[0], u[1], v[1]});
                __builtin_amdgcn_sched_barrier(0);
            }
        if (FIRST == 0 && a.lse && valid && half == 0)
            a.lse[qrow] = l == 0.0f ? -INFINITY : mref * kLn2 + __logf(l);
    } else {
#pragma unroll
        for (int fb = FIRST; fb < FIRST + N; ++fb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                *reinterpret_cast<f32x4*>(piece + ((fb * 4 + i) * 64 + lane) * 4) =
                    f32x4{o[fb][4 * i], o[fb][4 * i + 1], o[fb][4 * i + 2], o[fb][4 * i + 3]};
                __builtin_amdgcn_sched_barrier(0);
            }
        if (FIRST == 0 && half == 0) {
            piece[32 * K + col] = mref;
            piece[32 * K + 32 + col] = l;
        }
    }
}

template <bool PAGE8, bool FP8, int SPLIT>
__global__ void __launch_bounds__(64 * WAVES, 1) tree_attention_mfma(MfmaParams P)
{
    constexpr int FLAG_AT = FP8 ? SMEM8 : STAGES * STAGE;
    __shared__ __attribute__((aligned(1024))) char smem[FLAG_AT + FLAG_BYTES];
    uint32_t* const cleared = reinterpret_cast<uint32_t*>(smem + FLAG_AT);
    constexpr int LOADS = FP8 ? 6 : BLOCKS;   // LDS loads of 8 rows
    constexpr uint32_t ROWS = Shape<SPLIT>::ROWS, STEP = Shape<SPLIT>::STEP, COST = Shape<SPLIT>::COST;
    const TreeAttentionArgs& a = P.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    // The wave's 32 query rows, and its tile of each step.
    const uint32_t qwave = SPLIT == 1 ? wave : wave & 1, pair = SPLIT == 1 ? 0 : wave >> 1;

    Schedule<SPLIT> sched(P, lane);
    const uint32_t twins = sched.twins, twin = twins == 1 ? 0 : blockIdx.x >> 3 & 1;
    // Neighbouring shares go to one XCD (block i runs on XCD i % 8): items of one request
    // then read the same rows through one L2.
    const uint32_t per = (sched.groups + 7) / 8, at = twins == 1 ? blockIdx.x >> 3 : blockIdx.x >> 4;
    const uint32_t w = (blockIdx.x & 7) * per + at;
    const bool idle = at >= per || w >= sched.groups || sched.total == 0;
    Request r{};
    uint32_t stop = sched.total, u = 0;
    Cut rec{};
    if (!idle) {
        if (w + 1 < sched.groups)
            stop = uniform(sched.cut(w + 1, r));
        u = uniform(sched.cut(w, r));
        if (u == sched.raw(w)) {
            const uint32_t m = (u - r.base) / r.nu, lo = r.base + m * r.nu;
            if (u != lo)   // (an end of an item may be a cut, within `snap` of it)
                rec = Cut{w, sched.first_cut_past(lo + COST + sched.snap),
                          sched.first_cut_past(lo + r.nu - sched.snap - 1) - 1,
                          r.t0 * (uint32_t)a.H + m * ROWS * twins, r.n * (uint32_t)a.H - m * ROWS * twins, {}};
        }
    }
    if (threadIdx.x == 0 && twin == 0)
        P.cuts[at * 8 + (blockIdx.x & 7)] = rec;
    if (idle)
        return;

    // Lane-constant offsets.  A tile is stored in blocks of 32 rows x 128 bytes (64 bf16 columns
    // or 128 codes); the 16-byte granule g of row x sits at g ^ f(x), f(x) a permutation of bits
    // 1 to 3 of x.  (Two rows fill the 256 bytes of all banks.)  bf16: 16 rows of the 16-byte
    // reads, and 4 rows x 64 bytes of the transposing reads, fall on different banks.  e4m3:
    // 8 rows x 32 bytes of the transposing reads do; the 8-byte reads of all 32 rows touch each
    // bank twice.  In the last 64 codes of a row granule g sits at g ^ (x / 4) % 4.
    auto f = [](uint32_t x) {
        return FP8 ? (x >> 1 & 1) << 2 | (x >> 3 & 1) << 1 | (x >> 2 & 1) : (x >> 1 & 1) << 2 | (x >> 2 & 1) << 1 | (x >> 3 & 1);
    };
    const uint32_t fk = f(col);
    // Score operands: granules 2 s + half of a block; bf16: s = 0 .. 3, e4m3: 0 (others by
    // exclusive or), of a whole block and of the last half one.
    uint32_t k_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        k_off[s] = !FP8    ? col * 128 + (((2 * s + half) ^ fk) * 16)
                   : s == 0 ? col * 128 + ((half ^ fk) * 16)
                            : col * 64 + ((half ^ (col >> 2 & 3)) * 16);
    // Transposing reads.  bf16: lane c of a 16-lane group addresses row c / 4 and 8 bytes of its
    // columns; e4m3: row c / 2 of the eight (rows 0 .. 3 and 8 .. 11, + 4 half) and 8 codes.
    [[maybe_unused]] uint32_t v_off[2][2];   // bf16: [feature block parity][rows vrow or vrow + 8]
    if constexpr (!FP8) {
        const uint32_t c16 = lane & 15, vrow = 4 * half + (c16 >> 2);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v_off[s][h] = (vrow + 8 * h) * 128 + (c16 & 1) * 8 +
                              (((uint32_t)(4 * s + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1)) ^ f(vrow + 8 * h)) * 16);
    }
    auto v_off8 = [&]() __attribute__((always_inline)) {
        const uint32_t ln = lane_again(), c16 = ln & 15, vrow = 4 * (ln >> 5) + (c16 >> 1 & 3) + 8 * (c16 >> 3);
        return vrow * 128 + (c16 & 1) * 8 + (((ln >> 4 & 1) ^ f(vrow)) * 16);
    };
    const uint32_t lds0 = lds_addr(smem);
    // Stage of the wave's tile of step t (the steps of an item counted from 0).
    auto stage_no = [=](uint32_t t) __attribute__((always_inline)) {
        return SPLIT == 1 ? t & (STAGES - 1) : (t & 1) * 2 + pair;
    };
    auto stage_of = [=](uint32_t t) __attribute__((always_inline)) { return stage_no(t) * (FP8 ? STAGE8 : STAGE); };
    const float c = fabsf(a.scale) * kLog2e;   // a negative scale turns the queries' signs; 0 is not taken
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;

    while (u < stop) {
        while (u >= r.base + r.nm * r.nu) {
            const uint32_t next = r.base + r.nm * r.nu;
            r = request_at<SPLIT>(a, twins, r.b + 1);
            r.base = next;
            r = uniform(r);
        }
        const uint32_t m = uniform((u - r.base) / r.nu);
        const uint32_t item = r.base + m * r.nu;
        const uint32_t tile0 = u - item < COST ? 0 : u - item - COST;
        u = min(stop, item + r.nu);
        const uint32_t tile1 = u - item - COST;
        const uint32_t n_tiles = tile1 - tile0;
        const uint32_t len = r.len, cached = r.cached;
        const uint32_t table_row = r.b * a.L.max_pages;   // checked on the host: below 2^32

        const uint32_t rows = r.n * (uint32_t)a.H;                 // below 2^31 / D
        const uint32_t block0 = (m * twins + twin) * ROWS, row = block0 + qwave * 32 + col;
        if (SPLIT == 2 && block0 >= rows)
            continue;   // no rows for this twin
        const bool live = uniform(block0 + qwave * 32) < rows;
        const bool valid = row < rows;
        const uint32_t qrow = r.t0 * (uint32_t)a.H + min(row, rows - 1);
        const uint32_t tok = min(row, rows - 1) / (uint32_t)a.H;   // token of the request

        // SPLIT 2: the join of the item before is done with LDS, the queries' part included.
        if (SPLIT == 2)
            lds_barrier();
        // Query fragments: lane holds features 16 s + 8 half .. + 7 of its row; e4m3: 8 (s % 2) .. + 7
        // of granule s / 2 * 2 + half, as one 16-byte read of codes serves two products.
        constexpr int KEPT = FP8 ? QUERY_KEPT : D / 16;
        bf16x8 q[KEPT];
        char* my_q = FP8 ? smem + QUERY_AT + wave * QUERY_WAVE + lane * 16 : nullptr;
        {
            const char* src = static_cast<const char*>(a.q) + (int64_t)qrow * (D * 2) + half * (FP8 ? 32 : 16);
            auto at = [](int s) { return FP8 ? (s >> 1) * 64 + (s & 1) * 16 : s * 32; };
#pragma unroll
            for (int s = 0; s < KEPT; ++s)
                q[s] = as_bf16x8(ld16(src + at(s)));
            if (flip)
#pragma unroll
                for (int s = 0; s < KEPT; ++s)
                    q[s] = as_bf16x8(__builtin_bit_cast(u32x4, q[s]) ^ flip);
            if constexpr (FP8) {
#pragma unroll
                for (int s = KEPT; s < D / 16; ++s)
                    lds_st16(my_q + (s - KEPT) * 1024, ld16(src + at(s)) ^ flip);
            }
        }
        // The stages of the item before are no longer read (and no load into them is in flight:
        // the last step waited for all of them, and those behind the last tile are switched off).
        if (SPLIT == 1)
            lds_barrier();
        if (threadIdx.x == 0)
            *cleared = 0;   // (every wave has read the last item's; there is a barrier before it is set)

        // Loads of one tile: this wave fetches rows 8 i .. 8 i + 7 for its one or two bands i,
        // lane l granule l % 8 of every block of row l / 8.  Rows past the end repeat the last one.
        // The page id of a tile's rows (PAGE8: 8 rows starting at a multiple of 8 are in one page)
        // is asked for one tile early, when no LDS read is outstanding: a scalar load makes every
        // wait for LDS reads wait for all of them.
        [[maybe_unused]] uint32_t next_id[SPLIT] = {};
        [[maybe_unused]] const uint32_t* next_entry[SPLIT] = {};
        auto band = [&](int i) __attribute__((always_inline)) { return SPLIT * qwave + i; };
        auto tile_start = [&](uint32_t t) __attribute__((always_inline)) { return (tile0 + t) * STEP + pair * TILE; };
        auto group_start = [&](uint32_t t, int i) __attribute__((always_inline)) {
            const uint32_t p0 = tile_start(t) + band(i) * 8;
            return p0 < len ? p0 : (len - 1) & ~7u;
        };
        auto entry_of = [&](uint32_t t, int i) __attribute__((always_inline)) {
            const uint32_t lp = __umulhi(group_start(t, i), P.ps_magic) >> P.ps_shift;
            return a.L.page_table + table_row + min(lp, a.L.max_pages - 1);
        };
        auto id_at = [&](const uint32_t* entry) __attribute__((always_inline)) {
            return *(const __attribute__((address_space(4))) uint32_t*)(uint64_t)entry;
        };

        // Where the loads of a tile come from and go to; then its loads one by one: spread over
        // a step they never wait for one another (64 bytes per clock and CU).
        const char* src_base = nullptr;     // PAGE8: uniform; else the lane's address
        const char* scale_src = nullptr;
        uint32_t src_off = 0, src_off4 = 0, scale_off = 0, dst = 0, scale_dst = 0, src_on = 0;
        [[maybe_unused]] const char* src_base4 = nullptr;
        uint32_t last_tile = n_tiles;
        asm("" : "+s"(last_tile));   // the switch below stays scalar arithmetic
        auto locate = [&](uint32_t t, int i) __attribute__((always_inline)) {
            src_on = (uint32_t)((int32_t)(t - last_tile) >> 31);   // all ones while t < n_tiles
            dst = lds0 + stage_of(t) + band(i) * 1024;
            const uint32_t ln = lane_again();
            const uint32_t load_off = ((ln & 7) ^ f(band(i) * 8 + (ln >> 3))) * 16;
            [[maybe_unused]] const uint32_t load_off4 = 512 + ((ln ^ (2 * band(i) + (ln >> 4))) & 3) * 16;
            if constexpr (PAGE8) {
                const uint32_t pg = group_start(t, i);
                const uint32_t slot = pg - (__umulhi(pg, P.ps_magic) >> P.ps_shift) * a.L.page_size;
                const uint32_t id = min(next_id[i], a.L.num_pages - 1);
                src_base = a.L.base + (int64_t)id * a.L.stride_page + (int64_t)slot * a.L.stride_token;
                const uint32_t last = len - 1 - pg;
                src_off = min(ln >> 3, last) * (uint32_t)a.L.stride_token + load_off;
                if constexpr (FP8) {
                    src_off4 = min(ln >> 2, last) * (uint32_t)a.L.stride_token + load_off4;
                    scale_src = a.Ls.base + (int64_t)id * a.Ls.stride_page + (int64_t)slot * a.Ls.stride_token;
                    scale_off = min(ln & 7, last) * (uint32_t)a.Ls.stride_token + (ln >> 3) * 4;
                }
            } else {
                auto at = [&](const PagedLayer& L, uint32_t row) __attribute__((always_inline)) {
                    const uint32_t p = min(tile_start(t) + band(i) * 8 + row, len - 1);
                    const uint32_t lp = p / L.page_size;
                    const uint32_t id = min(L.page_table[table_row + min(lp, L.max_pages - 1)], L.num_pages - 1);
                    return L.base + (int64_t)id * L.stride_page + (int64_t)(p - lp * L.page_size) * L.stride_token;
                };
                src_base = at(a.L, ln >> 3) + load_off;
                if constexpr (FP8) {
                    src_base4 = at(a.L, (ln >> 2) & 7) + load_off4;
                    scale_src = at(a.Ls, ln & 7) + (ln >> 3) * 4;
                }
            }
            if constexpr (FP8)
                scale_dst = lds0 + SCALES_AT + stage_no(t) * SCALES + band(i) * SCALES_WAVE;
        };
        // Its loads in GROUPS groups.
        auto load = [&](auto group, int i) __attribute__((always_inline)) {
            constexpr int g = group;
            if constexpr (FP8 && g == 2) {
                // Lanes 0 .. 31: the last 64 codes of row l / 4; then lane l: scale of block l / 8 of row l % 8.
                const uint32_t to = dst - band(i) * 512 + 4 * BLOCK_BYTES;
                if constexpr (PAGE8) {
                    load_lds<0, 1>(src_base, src_off4, to, src_on, 0);
                    load_lds4(scale_src, scale_off, scale_dst, src_on, src_on & 0xFFu);
                } else {
                    load_lds<0, 1>(src_base4, to, src_on, 0);
                    load_lds4(scale_src, scale_dst, src_on, src_on & 0xFFu);
                }
            } else {
                constexpr int n = FP8 ? 2 : 3;
                if constexpr (PAGE8)
                    load_lds<g * n, n>(src_base, src_off, dst, src_on, src_on);
                else
                    load_lds<g * n, n>(src_base, dst, src_on, src_on);
            }
        };
        constexpr int GROUPS = 3;
        auto issue = [&](uint32_t t) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < SPLIT; ++i) {
                locate(t, i);
                each<GROUPS>([&](auto group) __attribute__((always_inline)) { load(group, i); });
            }
        };
        // e4m3: scales of block b of the rows 8 i + 4 half .. + 3 of a tile.
        auto scales_at = [&](uint32_t t) __attribute__((always_inline)) {
            return SCALES_AT + stage_no(t) * SCALES + (lane_again() >> 5) * 16;
        };
        auto scales_of = [&](uint32_t at, int b, int i) __attribute__((always_inline)) {
            return *reinterpret_cast<const f32x4*>(smem + at + i * SCALES_WAVE + b * 32);
        };

        // Steps loaded ahead of the first; then step t loads step t + AHEAD.
        constexpr int FIRST = SPLIT == 1 ? 3 : 2, AHEAD = SPLIT == 1 ? 3 : 1;
        {
            constexpr int IDS = AHEAD + 1;
            uint32_t ids[IDS][SPLIT] = {};
            if constexpr (PAGE8)
#pragma unroll
                for (int t = 0; t < IDS; ++t)
#pragma unroll
                    for (int i = 0; i < SPLIT; ++i)
                        ids[t][i] = id_at(entry_of(t, i));
#pragma unroll
            for (int t = 0; t < IDS; ++t) {
#pragma unroll
                for (int i = 0; i < SPLIT; ++i)
                    next_id[i] = ids[t][i];
                if (t < FIRST)
                    issue(t);
            }
        }
        auto locate_next = [&](uint32_t t) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < SPLIT; ++i)
                next_entry[i] = entry_of(t + AHEAD + 1, i);
        };
        // Ids for the loads of the next step, once `next_entry` has their places.
        auto next_ids = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < SPLIT; ++i)
                next_id[i] = id_at(next_entry[i]);
        };

        // Drafted rows may be hidden from some tokens and hold anything: a weight of 0 would turn
        // their infinities and NaN into NaN, so those become 0 here, between the scores and the
        // weighted sums of step t, and `cleared` is set.  (A token that sees such a row has a NaN
        // weight for it, but one of 0 where its score is -infinity: restored at the end.)
        auto clear_nonfinite = [&](uint32_t t) __attribute__((always_inline)) {
            if ((tile0 + t + 1) * STEP <= cached || !(r.n > 1 || a.mask))
                return;
            if (SPLIT == 2)
                lds_barrier();   // the scores are done
            const uint32_t p0 = tile_start(t);
            for (int i = 0; i < SPLIT; ++i) {
                char* mine = smem + stage_of(t) + band(i) * 1024 + lane * 16;
                if (p0 + band(i) * 8 + (lane >> 3) >= cached)
                    for (int j = 0; j < K / (FP8 ? 128 : 64); ++j) {
                        const u32x4 was = lds_ld16(mine + j * BLOCK_BYTES);
                        u32x4 v = was;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (FP8) {   // bytes of 0x7F or 0xFF
                                const uint32_t nan = ((v[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                v[e] &= ~((nan >> 7) * 0xFFu);
                            } else {
                                v[e] = nonfinite16(v[e]) ? v[e] & 0xFFFF0000u : v[e];
                                v[e] = nonfinite16(v[e] >> 16) ? v[e] & 0xFFFFu : v[e];
                            }
                        }
                        if (((was[0] ^ v[0]) | (was[1] ^ v[1]) | (was[2] ^ v[2]) | (was[3] ^ v[3])) != 0) {
                            lds_st16(mine + j * BLOCK_BYTES, v);
                            *cleared = 1;
                        }
                    }
                if (FP8 && lane < 40 && p0 + band(i) * 8 + (lane & 7) >= cached) {
                    float* sc = reinterpret_cast<float*>(smem + SCALES_AT + stage_no(t) * SCALES + band(i) * SCALES_WAVE) + lane;
                    if (!(fabsf(*sc) < INFINITY)) {
                        *sc = 0.0f;
                        *cleared = 1;
                    }
                }
            }
            lds_barrier();
        };

        // Start of step t.  SPLIT 1: tile t + 1 is there for every wave and every wave is done with
        // tile t - 1, whose stage takes tile t + 3.  SPLIT 2: the tiles of step t are there, and
        // those of step t + 1 take the place of those of step t - 1 (step 0: they are on their way).
        auto enter = [&](uint32_t t) __attribute__((always_inline)) {
            if (SPLIT == 1 ? t + 2 < n_tiles : t == 0 && n_tiles > 1)
                wait_loads<SPLIT * LOADS>();
            else
                wait_loads<0>();
            lds_barrier();
            if (SPLIT == 1)
                clear_nonfinite(t);
        };
        // Bits of the tile's rows that this lane's token sees.
        auto seen_rows = [&](uint32_t p0) __attribute__((always_inline)) {
            if (SPLIT == 2 && p0 >= len)
                return 0u;
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

        f32x16 o[16];   // cleared while the first tiles are on their way
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            o[i] = f32x16{0.f};
            asm volatile("" : "+a"(o[i]));
        }
        if constexpr (SPLIT == 1) {
            if (n_tiles > 2)
                wait_loads<2 * LOADS>();
            else if (n_tiles > 1)
                wait_loads<LOADS>();
            else
                wait_loads<0>();
            lds_barrier();
        }
        if (!live) {
            // No query rows for this wave: it only loads.
            for (uint32_t t = 0; t < n_tiles; ++t) {
                enter(t);
                if (SPLIT == 1 || t > 0)
                    issue(t + AHEAD);
                if (SPLIT == 2)
                    clear_nonfinite(t);
                if constexpr (PAGE8) {
                    locate_next(t);
                    next_ids();
                }
            }
            if constexpr (SPLIT == 2) {   // as the waves that join their results
                lds_barrier();
                lds_barrier();
            }
            continue;
        }

        float mref = -INFINITY, l = 0.0f;

        // Scores of tile t: lane (col, half) gets rows 8 (i / 4) + 4 half + i % 4 for its query.
        // Fragments are read KD products ahead; `between(k)` is other work during product k.
        // e4m3: codes become bf16 on the way to the matrix cores; each block
        // of 128 columns has sums of its own, times the block's scale of each row.
        constexpr int KN = D / 16, KD = FP8 ? 4 : 8, VN = 2 * (K / 32), VD = 8;   // e4m3: KD reads, two products each
        using Frag = std::conditional_t<FP8, u32x2, bf16x8>;
        using KFrag = std::conditional_t<FP8, u32x4, bf16x8>;
        auto scores = [&](uint32_t t, auto between) __attribute__((always_inline)) {
            const char* st = smem + stage_of(t);
            // Exclusive or of the granule after the sum with the stage: it is not worth keeping.
            [[maybe_unused]] const uint32_t at8[2] = {stage_of(t) + k_off[0], stage_of(t) + k_off[1]};
            auto frag = [&](int k) __attribute__((always_inline)) -> KFrag {
                if constexpr (FP8)
                    return lds_ld16(smem + (at8[k >> 4] ^ ((k < 16 ? k & 3 : k & 1) * 32)) + (k >> 2) * BLOCK_BYTES);
                else
                    return as_bf16x8(lds_ld16(st + k_off[k & 3] + (k >> 2) * BLOCK_BYTES));
            };
            auto query = [&](int k) __attribute__((always_inline)) { return as_bf16x8(lds_ld16(my_q + (k - KEPT) * 1024)); };
            const uint32_t scale_row = FP8 ? scales_at(t) : 0;
            f32x16 acc, part;
            KFrag kf[KD];
            bf16x8 qx[2];
            f32x4 bs[4];
#pragma unroll
            for (int k = 0; k < KD; ++k)
                kf[k] = frag(k);
            [[maybe_unused]] auto converted = [&](int k) __attribute__((always_inline)) {
                if constexpr (FP8) {
                    const u32x4 two = kf[(k >> 1) % KD];
                    return bf16_of_codes(k & 1 ? u32x2{two[2], two[3]} : u32x2{two[0], two[1]});
                } else {
                    return bf16x8{};
                }
            };
            [[maybe_unused]] bf16x8 xn = converted(0);
            between(std::integral_constant<int, -1>{});
            __builtin_amdgcn_sched_barrier(0);
            each<KN>([&](auto index) __attribute__((always_inline)) {
                constexpr int k = index;
                constexpr int blk = FP8 ? k >> 3 : 0, at = FP8 ? k & 7 : k;
                constexpr bool end = k == KN - 1 || (FP8 && at == 7);
                f32x16& sum = blk == 0 ? acc : part;
                // (the next product's codes are converted first: its operands are never just written)
                bf16x8 x;
                if constexpr (FP8) {
                    x = xn;
                    if constexpr (k + 1 < KN)
                        xn = converted(k + 1);
                    __builtin_amdgcn_sched_barrier(0);
                } else {
                    x = kf[k % KD];
                }
                bf16x8 y;
                if constexpr (k < KEPT)
                    y = q[k];
                else
                    y = qx[k % 2];
                if (at == 0)
                    mfma_first(sum, x, y);
                else if (end)
                    sum = mfma_last<FP8>(sum, x, y);
                else
                    mfma_next(sum, x, y);
                if constexpr (FP8 && (k & 1) == 0 && (k >> 1) + KD < KN / 2)
                    kf[(k >> 1) % KD] = frag((k >> 1) + KD);
                if constexpr (!FP8 && k + KD < KN)
                    kf[k % KD] = frag(k + KD);
                if constexpr (FP8 && k + 2 >= KEPT && k + 2 < KN)
                    qx[k % 2] = query(k + 2);
                if constexpr (FP8) {
                    if (at == (blk == 4 ? 1 : 4)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bs[i] = scales_of(scale_row, blk, i);
                    }
                }
                between(index);
                if constexpr (FP8 && end) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[i] = blk == 0 ? acc[i] * bs[i >> 2][i & 3] : acc[i] + part[i] * bs[i >> 2][i & 3];
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            return acc;
        };
        // Scores of the tile at hand, their maximum (in units of log2, as mref), and whether the
        // reference lags too far behind it anywhere.
        f32x16 s;
        float mx;
        uint64_t lagging;
        // Masks the scores of tile t if they have to be, and moves the reference if it lags.
        auto settle = [&](uint32_t t) __attribute__((always_inline)) {
            const uint32_t p0 = tile_start(t);
            if (p0 + TILE > cached) {
                const uint32_t seen = seen_rows(p0);
                mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[i] = (seen >> (8 * (i >> 2) + 4 * half + (i & 3))) & 1 ? s[i] : -INFINITY;
                    mx = fmaxf(mx, s[i]);
                }
                mx = fmaxf(mx, swap32(mx)) * c;
                lagging = __ballot(mx > mref + kSlack);
            }
            if (lagging) {
                const float next = fmaxf(mref, mx);
                const float keep = next == mref ? 1.0f : __builtin_amdgcn_exp2f(mref - next);
                mref = next;
                l *= keep;
                if (t > 0) {   // the first tile finds no sums
                    asm volatile("s_nop 15");   // the last products' sums are in their registers
#pragma unroll
                    for (int i = 0; i < 16; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            scale_sum(o[i], e, keep);
                }
            }
        };
        auto maximum = [&]() __attribute__((always_inline)) {
            mx = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i)
                mx = fmaxf(mx, s[i]);
            mx = fmaxf(mx, swap32(mx)) * c;
            lagging = __ballot(mx > mref + kSlack);
        };
        if constexpr (SPLIT == 1) {
            s = scores(0, [](auto) {});
            maximum();
            settle(0);
        }

        for (uint32_t t = 0; t < n_tiles; ++t) {
            enter(t);
            if constexpr (SPLIT == 2) {
                // The loads of step t + 1 are spread over the products.
                s = scores(t, [&](auto index) __attribute__((always_inline)) {
                    constexpr int k = index, i = k / 16, g = k % 16 / 4;
                    if constexpr (k >= 0 && k % 16 == 0 && i < SPLIT) {
                        locate(t + 1, i);
                        src_on &= (uint32_t)((int32_t)(0u - t) >> 31);   // step 0: they are on their way
                    }
                    if constexpr (k >= 0 && k % 4 == 3 && i < SPLIT && g < GROUPS)
                        load(std::integral_constant<int, g>{}, i);
                });
                maximum();
                settle(t);
                clear_nonfinite(t);
            }
            const char* st = smem + stage_of(t);
            const uint32_t v_at = FP8 ? stage_of(t) + v_off8() : 0;
            auto vfrag = [&](int v) __attribute__((always_inline)) -> Frag {
                const int fb = v >> 1, ks = v & 1;
                if constexpr (FP8) {
                    return lds_tr8(smem + (v_at ^ ((2 * fb & 7) * 16)) + (fb >> 2) * BLOCK_BYTES + ks * 2048);
                } else {
                    const v4i16 lo = lds_tr16(st + v_off[fb & 1][0] + (fb >> 1) * BLOCK_BYTES + ks * 2048);
                    const v4i16 hi = lds_tr16(st + v_off[fb & 1][1] + (fb >> 1) * BLOCK_BYTES + ks * 2048);
                    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
            };
            const float ref = mref == -INFINITY ? 0.0f : mref;
            // The scores of the next tile, and the weights of this one while the matrix cores
            // run.  (The last step computes scores that nobody uses, from whatever the stage holds.)
            uint32_t pk[8];
            float sum = 0.0f;
            [[maybe_unused]] float e[16];
            Frag vf[VD];
            auto weights = [&](int k) __attribute__((always_inline)) {
                const float e0 = __builtin_amdgcn_exp2f(fmaf(s[2 * k], c, -ref));
                const float e1 = __builtin_amdgcn_exp2f(fmaf(s[2 * k + 1], c, -ref));
                sum += e0 + e1;
                if constexpr (FP8) {
                    e[2 * k] = e0;
                    e[2 * k + 1] = e1;
                } else {
                    pk[k] = pack_bf16x2(e0, e1);
                }
            };
            if constexpr (SPLIT == 1) {
                const f32x16 next_s = scores(t + 1, [&](auto index) __attribute__((always_inline)) {
                    constexpr int k = index;
                    if constexpr (k < 0) {
                        weights(0);
                        weights(1);
                    } else if constexpr (FP8 ? k < 6 : k % 3 == 0 && k / 3 < 6) {
                        weights(2 + (FP8 ? k : k / 3));
                    }
                    if constexpr (k == 4)
                        locate(t + AHEAD, 0);
                    if constexpr (k >= KN - VD)
                        vf[k - (KN - VD)] = vfrag(k - (KN - VD));
                });
                s = next_s;
            } else {
#pragma unroll
                for (int v = 0; v < VD; ++v)
                    vf[v] = vfrag(v);
                each<8>([&](auto k) __attribute__((always_inline)) { weights(k); });
            }
            l += sum;
            // e4m3: the weights times the scales of one block of 128 features at a time, rounded
            // to bf16 once.
            bf16x8 pf[2];
            [[maybe_unused]] f32x4 ps[2];
            auto block_weights = [&](int i) __attribute__((always_inline)) {   // of four rows
                pk[2 * i] = pack_bf16x2(e[4 * i] * ps[i & 1][0], e[4 * i + 1] * ps[i & 1][1]);
                pk[2 * i + 1] = pack_bf16x2(e[4 * i + 2] * ps[i & 1][2], e[4 * i + 3] * ps[i & 1][3]);
            };
            const uint32_t scale_row = FP8 ? scales_at(t) : 0;
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ps[i & 1] = scales_of(scale_row, 0, i);
                    block_weights(i);
                }
            }
            [[maybe_unused]] bf16x8 vn;
            if constexpr (FP8) {
                vn = bf16_of_codes(vf[0]);
                vf[0] = vfrag(VD);
            }
            each<VN>([&](auto index) __attribute__((always_inline)) {
                constexpr int v = index;
                if constexpr (v == 0 || (FP8 && (v & 7) == 0)) {
                    pf[0] = as_bf16x8(u32x4{pk[0], pk[1], pk[2], pk[3]});
                    pf[1] = as_bf16x8(u32x4{pk[4], pk[5], pk[6], pk[7]});
                }
                if constexpr (FP8) {
                    const bf16x8 x = vn;
                    if constexpr (v + 1 < VN)
                        vn = bf16_of_codes(vf[(v + 1) % VD]);
                    __builtin_amdgcn_sched_barrier(0);
                    o[v >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, pf[v & 1], o[v >> 1], 0, 0, 0);
                    if constexpr (v + 1 + VD < VN)
                        vf[(v + 1) % VD] = vfrag(v + 1 + VD);
                } else {
                    o[v >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[v % VD], pf[v & 1], o[v >> 1], 0, 0, 0);
                    if constexpr (v + VD < VN)
                        vf[v % VD] = vfrag(v + VD);
                }
                if constexpr (SPLIT == 1) {
                    if constexpr (v % 8 == 3 && v / 8 < GROUPS)
                        load(std::integral_constant<int, v / 8>{}, 0);
                    if constexpr (v >= 4 && v < 20 && v % 2 == 0)
                        mx = v == 4 ? fmaxf(s[0], s[1]) : fmaxf(fmaxf(mx, s[v - 4]), s[v - 3]);
                    if constexpr (v == 20)
                        mx = fmaxf(mx, swap32(mx)) * c;
                    if constexpr (v == 22)
                        lagging = __ballot(mx > mref + kSlack);
                }
                if constexpr (PAGE8 && v == 24)
                    locate_next(t);
                if constexpr (FP8) {
                    // The next block's weights, a quarter at a time.
                    constexpr int b = (v >> 3) + 1, at = v & 7;
                    if constexpr (b < 4 && at >= 3 && at < 7)
                        block_weights(at - 3);
                    if constexpr (b < 4 && at >= 1 && at < 5)
                        ps[(at - 1) & 1] = scales_of(scale_row, b, at - 1);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (PAGE8)
                next_ids();
            if (SPLIT == 1 && t + 1 < n_tiles)
                settle(t + 1);
        }

        l += swap32(l);
        const bool whole = tile0 == 0 && tile1 + COST == r.nu;
        float* piece = a.ws + (size_t)(2 * w + (tile0 == 0 ? 1 : 0)) * P.piece +
                       (size_t)(SPLIT == 1 ? qwave : twin * 2 + qwave) * PIECE_WAVE;
        if constexpr (SPLIT == 1) {
            store_result<0, 16>(a, o, mref, l, qrow, valid, whole, piece, lane);
        } else {
            // The two waves of the same rows join their results: each hands the other half of its
            // sums through LDS, and keeps the half it stores.
            static_assert(WAVES * JOIN_WAVE <= sizeof(smem), "LDS");
            auto join = [&](auto first) __attribute__((always_inline)) {
                constexpr int keep = first, give = 8 - keep;
                char* mine = smem + wave * JOIN_WAVE;
                const char* other = smem + (wave ^ 2) * JOIN_WAVE;
                lds_barrier();   // the stages are no longer read
                each<32>([&](auto index) __attribute__((always_inline)) {
                    constexpr int q = index, fb = give + q / 4, i = q % 4;
                    *reinterpret_cast<f32x4*>(mine + (q * 64 + lane) * 16) =
                        f32x4{o[fb][4 * i], o[fb][4 * i + 1], o[fb][4 * i + 2], o[fb][4 * i + 3]};
                    __builtin_amdgcn_sched_barrier(0);
                });
                reinterpret_cast<float*>(mine + 8 * 16 * 256)[lane] = half ? l : mref;
                lds_barrier();
                const float* ml = reinterpret_cast<const float*>(other + 8 * 16 * 256);
                const float m2 = ml[col], l2 = ml[32 + col];
                const float next = fmaxf(mref, m2);
                const float at = next == -INFINITY ? 0.0f : next;
                const float f1 = __builtin_amdgcn_exp2f(mref - at), f2 = __builtin_amdgcn_exp2f(m2 - at);
                l = l * f1 + l2 * f2;
                mref = next;
                each<32>([&](auto index) __attribute__((always_inline)) {
                    constexpr int q = index, fb = keep + q / 4, i = q % 4;
                    const f32x4 y = *reinterpret_cast<const f32x4*>(other + (q * 64 + lane) * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[fb][4 * i + e] = o[fb][4 * i + e] * f1 + y[e] * f2;
                    if constexpr (q % 4 == 3)
                        __builtin_amdgcn_sched_barrier(0);
                });
                store_result<keep, 8>(a, o, mref, l, qrow, valid, whole, piece, lane);
            };
            if (pair == 0)
                join(std::integral_constant<int, 0>{});
            else
                join(std::integral_constant<int, 8>{});
        }
        // What clear_nonfinite took from the tokens that see it: 0 times infinity (or NaN) is NaN in
        // the columns where a row they see is not finite.  Written over the features that the wave
        // stored: only a broken row comes here, and the wave has no registers to spare before.
        if (tile1 * STEP > cached && (r.n > 1 || a.mask) && uniform(*cleared)) {
            wait_loads<0>();   // (stores too: other lanes stored some of these values)
            const uint32_t ln = lane_again();
            const uint32_t mine = block0 + qwave * 32 + (ln & 31), there = min(mine, rows - 1);
            const uint32_t token = there / (uint32_t)a.H, column = 4 * (ln >> 5);
            uint16_t* out = static_cast<uint16_t*>(a.out) + ((int64_t)r.t0 * a.H + there) * K + column;
#pragma unroll 1
            for (uint32_t p = max(tile0 * STEP, cached); p < min(tile1 * STEP, len); ++p) {
                const uint32_t j = p - cached;
                const bool sees = a.mask ? j < 64u * (uint32_t)a.words &&
                                               (a.mask[(int64_t)(r.t0 + token) * a.words + (j >> 6)] >> (j & 63)) & 1
                                         : j <= token;
                if (!sees || mine >= rows)
                    continue;
                const char* row_p = a.L.base + token_offset(a.L, r.b, p) + column * (FP8 ? 1 : 2);
#pragma unroll 1
                for (uint32_t q = pair * 32; q < pair * 32 + 64 / SPLIT; ++q) {   // features 8 q + column .. + 3
                    uint32_t broken;   // a bit for each
                    if constexpr (FP8) {
                        const uint32_t x = *reinterpret_cast<const uint32_t*>(row_p + q * 8);
                        const float* scale = reinterpret_cast<const float*>(a.Ls.base + token_offset(a.Ls, r.b, p)) + (q >> 4);
                        broken = 0;
                        for (int e = 0; e < 4; ++e)
                            broken |= (uint32_t)((x >> (8 * e) & 0x7F) == 0x7F) << e;
                        broken = fabsf(*scale) < INFINITY ? broken : 15;
                    } else {
                        const u32x2 x = *reinterpret_cast<const u32x2*>(row_p + q * 16);
                        broken = nonfinite16(x[0]) | nonfinite16(x[0] >> 16) << 1 | nonfinite16(x[1]) << 2 |
                                 nonfinite16(x[1] >> 16) << 3;
                    }
                    for (int e = 0; e < 4; ++e)
                        if (broken >> e & 1) {
                            if (whole)
                                out[q * 8 + e] = 0x7FC0;
                            else
                                piece[(q * 64 + ln) * 4 + e] = NAN;
                        }
                }
            }
        }
    }
}

// Joins the pieces of split items.  Block (i, g): rows 32 g .. of the item that cut record i
// lies in, if any; the blocks of all cuts inside one item share its 64 quads of features (in
// the lane order of the accumulators).  With many pieces the waves of a block share the pieces,
// else the quads: pieces of two shares each are read by 4 waves at once either way.
__global__ void __launch_bounds__(256) tree_attention_join(MfmaParams P)
{
    __shared__ float factor[kAttnGroups][32];    // per piece and row: its maximum, then its weight
    __shared__ float top[8][32];
    __shared__ f32x4 part[3][2][64];
    const TreeAttentionArgs& a = P.a;
    const uint32_t g = blockIdx.x & (P.groups - 1);
    const auto* words = (const __attribute__((address_space(4))) uint32_t*)(uint64_t)(P.cuts + blockIdx.x / P.groups);
    const Cut rec{words[0], words[1], words[2], words[3], words[4], {}};
    if (rec.rows <= g * 32)
        return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const uint32_t w0 = rec.w0, w1 = rec.w1;
    const bool valid = g * 32 + col < rec.rows;
    const int64_t qrow = rec.row0 + g * 32 + (valid ? col : 0);
    const uint32_t share = rec.w - w0, shares = w1 - w0 + 1;
    const uint32_t pieces = shares + 1;          // at most kAttnGroups
    // Piece 0 is the end of share w0 - 1, piece k the start of share w0 + k - 1.
    const float* first = a.ws + (size_t)(2 * (w0 - 1) + 1) * P.piece + (size_t)g * PIECE_WAVE;
    const float* rest = a.ws + (size_t)(2 * w0) * P.piece + (size_t)g * PIECE_WAVE;
    auto piece = [&](uint32_t k) __attribute__((always_inline)) {
        return k == 0 ? first : rest + (size_t)(k - 1) * 2 * P.piece;
    };
    auto finish = [&](uint32_t quad, f32x4 v) __attribute__((always_inline)) {
        if (valid && quad < 64)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + qrow * K + (quad >> 2) * 32 + (quad & 3) * 8 +
                                      half * 4) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
    auto finish_lse = [&](float mx, float l) __attribute__((always_inline)) {
        if (a.lse && share == 0 && threadIdx.x < 32 && valid)
            a.lse[qrow] = l == 0.0f ? -INFINITY : mx * kLn2 + __logf(l);
    };

    constexpr uint32_t FEW = 8;
    if (pieces <= FEW) {
        float f[FEW], s[FEW];
        float mx = -INFINITY;
#pragma unroll
        for (uint32_t k = 0; k < FEW; ++k) {
            const float* src = piece(min(k, pieces - 1)) + 32 * K + col;
            f[k] = k < pieces ? src[0] : -INFINITY;
            s[k] = src[32];
        }
#pragma unroll
        for (uint32_t k = 0; k < FEW; ++k)
            mx = fmaxf(mx, f[k]);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        float l = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < FEW; ++k) {
            f[k] = k < pieces ? __builtin_amdgcn_exp2f(f[k] - ref) : 0.0f;
            l += k < pieces ? s[k] * f[k] : 0.0f;
        }
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        finish_lse(mx, l);
        constexpr int Q = 4;
        const uint32_t step = shares * WAVES;
        for (uint32_t q0 = share * WAVES + wave; q0 < 64; q0 += step * Q) {
            f32x4 sum[Q];
#pragma unroll
            for (int j = 0; j < Q; ++j)
                sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t k = 0; k < FEW; k += 2) {
                if (k < pieces) {
                    f32x4 v[2][Q];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < Q; ++j)
                            v[i][j] = *reinterpret_cast<const f32x4*>(piece(min(k + i, pieces - 1)) +
                                                                      (min(q0 + step * j, 63u) * 64 + lane) * 4);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (k + i < pieces)
#pragma unroll
                            for (int j = 0; j < Q; ++j)
                                sum[j] += v[i][j] * f[k + i];
                }
            }
#pragma unroll
            for (int j = 0; j < Q; ++j)
                finish(q0 + step * j, sum[j] * inv);
        }
        return;
    }

    // Weights of the pieces: thread (p, x) takes row x of pieces p, p + 8, ...
    const uint32_t p = threadIdx.x >> 5, x = threadIdx.x & 31;
    float mx = -INFINITY;
    for (uint32_t k0 = p; k0 < pieces; k0 += 32) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = piece(min(k0 + 8 * i, pieces - 1))[32 * K + x];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k0 + 8 * i < pieces) {
                factor[k0 + 8 * i][x] = v[i];
                mx = fmaxf(mx, v[i]);
            }
    }
    top[p][x] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mx = fmaxf(mx, top[i][x]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    for (uint32_t k0 = p; k0 < pieces; k0 += 32) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = piece(min(k0 + 8 * i, pieces - 1))[32 * K + 32 + x];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k0 + 8 * i < pieces) {
                const float f = __builtin_amdgcn_exp2f(factor[k0 + 8 * i][x] - ref);
                factor[k0 + 8 * i][x] = f;
                l += v[i] * f;
            }
    }
    __syncthreads();
    top[p][x] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        l += top[i][col];
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    finish_lse(mx, l);   // thread x < 32 holds row x of both

    // Quads share, share + shares, ...: two at a time, the wave's pieces four at a time.
    constexpr int Q = 2, U = 4;
    for (uint32_t q0 = share; q0 < 64; q0 += shares * Q) {
        f32x4 sum[Q] = {};
        for (uint32_t k0 = wave; k0 < pieces; k0 += WAVES * U) {
            f32x4 v[U][Q];
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < Q; ++j)
                    v[i][j] = *reinterpret_cast<const f32x4*>(piece(min(k0 + WAVES * i, pieces - 1)) +
                                                              (min(q0 + shares * j, 63u) * 64 + lane) * 4);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (k0 + WAVES * i < pieces) {
                    const float f = factor[k0 + WAVES * i][col];
#pragma unroll
                    for (int j = 0; j < Q; ++j)
                        sum[j] += v[i][j] * f;
                }
        }
        if (wave > 0)
#pragma unroll
            for (int j = 0; j < Q; ++j)
                part[wave - 1][j][lane] = sum[j];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int j = 0; j < Q; ++j)
                finish(q0 + shares * j, ((sum[j] + part[0][j][lane]) + (part[1][j][lane] + part[2][j][lane])) * inv);
        __syncthreads();
    }
}

}  // namespace

bool tree_attention_mfma_fits(const TreeAttentionArgs& a, AttnKind kind)
{
    // (the kernel's scale is in units of log2)
    return (kind == ATTN_BF16 || kind == ATTN_E4M3) && a.scale != 0.0f && std::isfinite(a.scale * kLog2e) && a.D == D &&
           a.K == K && a.L.stride_token < (int64_t(1) << 28) &&
           (kind == ATTN_BF16 || a.Ls.stride_token < (int64_t(1) << 28)) &&
           (uint64_t)a.L.batch * a.L.max_pages < (uint64_t(1) << 32) &&
           // items (at most one partly filled per request) times units
           ((uint64_t)a.T * a.H / Shape<2>::ROWS + std::min<uint64_t>(a.L.batch, a.T)) * (a.capacity / TILE + 1 + Shape<1>::COST) <
               (uint64_t(1) << 31);
}

hipError_t launch_tree_attention_mfma(const TreeAttentionArgs& a, AttnKind kind, hipStream_t s)
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
    // Two pairs of waves where an average request fills no more than half of a wide item, and two
    // such workgroups side by side where it fills no more than one: they leave partial results of
    // half as many shares.  Wide / two pairs, us: 16 requests x 16 heads x 3-4 tokens, 20-40 thousand
    // rows: e4m3 187 / 136, bf16 151 / 147; 64 x 16 heads, 256-4096 rows: e4m3 64 / 50, bf16 54 / 43.
    // Wide / two workgroups: 64 x 128 heads, 256-4096 rows: e4m3 80 / 75, bf16 70 / 62; 2 x 128 heads,
    // 60-120 thousand rows: e4m3 101 / 89, bf16 90 / 75; 16 x 16 heads x 8 tokens, 20-40 thousand rows:
    // e4m3 235 / 235, bf16 188 / 193, and x 5-6 tokens, bf16 165 / 181 (their loads run
    // only one step ahead).
    const int64_t query_rows = (int64_t)a.T * a.H;
    const bool split = query_rows <= (int64_t)kAttnRows * a.L.batch;
    const bool twins = split && query_rows > (int64_t)Shape<2>::ROWS * a.L.batch;
    P.twins = twins ? 2 : 1;
    P.groups = split && !twins ? 2 : 4;
    const int64_t waves = (std::min<int64_t>(query_rows, (int64_t)P.groups * 32) + 31) / 32;
    P.piece = (uint32_t)(waves * PIECE_WAVE);
    P.min_tiles = split ? 2 : 4;   // steps: 4 tiles either way
    P.cuts = reinterpret_cast<Cut*>(a.ws + (size_t)2 * kAttnGroups * P.piece);
    const bool fp8 = kind == ATTN_E4M3, page8 = ps % 8 == 0;
    log_launch(fp8 ? "tree_attention_mfma<e4m3>" : "tree_attention_mfma<bf16>", kAttnGroups, 64 * WAVES,
               "T=%d H=%d page_size=%u rows=%u", a.T, a.H, ps, P.groups * 32);
    auto pick = [&](auto page, auto cache) {
        constexpr bool p = decltype(page)::value, e = decltype(cache)::value;
        return split ? tree_attention_mfma<p, e, 2> : tree_attention_mfma<p, e, 1>;
    };
    const std::true_type yes;
    const std::false_type no;
    auto* kernel = fp8 ? (page8 ? pick(yes, yes) : pick(no, yes)) : (page8 ? pick(yes, no) : pick(no, no));
    hipLaunchKernelGGL(kernel, dim3(kAttnGroups), dim3(64 * WAVES), 0, s, P);
    if (hipError_t e = hipGetLastError())
        return e;
    // One block per cut and 32 rows of an item.
    const unsigned join_blocks = kAttnGroups / P.twins * P.groups;
    log_launch("tree_attention_join", join_blocks, 256, "T=%d H=%d", a.T, a.H);
    hipLaunchKernelGGL(tree_attention_join, dim3(join_blocks), dim3(256), 0, s, P);
    return hipGetLastError();
}

}  // namespace mla
