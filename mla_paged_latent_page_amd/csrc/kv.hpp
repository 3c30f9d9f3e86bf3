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

hipError_t launch_kv_write(const KvWriteArgs& a, bool fp8, bool half, hipStream_t s);
hipError_t launch_kv_gather(const KvGatherArgs& a, KvKind kind, hipStream_t s);
hipError_t launch_kv_attention(const KvAttentionArgs& a, KvKind kind, hipStream_t s);

}  // namespace mla
