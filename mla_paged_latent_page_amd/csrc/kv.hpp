// Launchers of the paged K/V cache's operators: writes, reads and attention.
// api_kv.hip validates arguments and calls exactly one of these.
#pragma once

#include "launch.hpp"

namespace mla {

struct KvWriteArgs {
    const char* k;                    // [T][HD] bf16 rows, k_st / v_st bytes apart
    const char* v;
    int64_t k_st, v_st;
    const uint32_t* iro;              // [batch + 1]
    const uint32_t* cache_len;        // [batch]
    const uint32_t* pos;              // [T] freqs row of each token, or null: the position written to
    const float* freqs;               // [max_seq][R]
    PagedLayer L;
    PagedLayer Ls;                    // e4m3: the scale pool
    int T, HD, D, R, max_seq;         // R: rotated columns, the last of every head
};

struct KvGatherArgs {
    const uint32_t* bro;              // buffer_row_offsets [batch + 1]
    const uint32_t* co;               // cache_offsets [>= batch]
    PagedLayer L;
    PagedLayer Ls;                    // e4m3: the scale pool
    char* k;                          // [M][HD]
    char* v;
    int M, HD;
};

struct KvAttentionArgs {
    const char* q;                    // [T][H][D], q_st bytes between tokens
    int64_t q_st;
    const uint32_t* iro;              // [batch + 1]
    const uint32_t* cache_len;        // [batch]
    void* out;                        // [T][H][D]
    float* lse;                       // [T][H] or null
    float* ws;                        // partial results
    PagedLayer L;
    PagedLayer Ls;                    // e4m3: the scale pool
    float scale;
    int T, H, KH, D;
    uint32_t window, sinks;           // window 0: none
    uint32_t capacity;                // max_pages * page_size: positions a request can have
};

enum KvKind { KV_F32, KV_BF16, KV_E4M3 };

// Partial results of the split attention: every workgroup leaves at most two (the item its share begins
// in and the one it ends in), of 32 rows of output sums, references and sums per row group.
constexpr int kKvGroups = 256;        // workgroups, one per CU
struct KvCut {                        // where a workgroup's share begins: tile 0 is the item's start
    uint32_t b, kh, m, tile;
    uint32_t t0, row0, rows, pad;     // the request's first token, the item's rows
};
// Groups of 32 rows (tokens x query heads of a key head) that an item of a call can have: up to 8.
inline uint32_t kv_attention_row_groups(int64_t T, int64_t G)
{
    return (uint32_t)((T * G < 256 ? T * G : 256) + 31) / 32;
}

hipError_t launch_kv_write(const KvWriteArgs& a, bool fp8, bool half, hipStream_t s);
hipError_t launch_kv_gather(const KvGatherArgs& a, KvKind kind, hipStream_t s);
// Matrix-core form (heads of 64 and 128 columns), and whether it takes a call.
bool kv_attention_mfma_fits(const KvAttentionArgs& a, KvKind kind);
hipError_t launch_kv_attention_mfma(const KvAttentionArgs& a, KvKind kind, hipStream_t s);
hipError_t launch_kv_attention(const KvAttentionArgs& a, KvKind kind, hipStream_t s);

}  // namespace mla
