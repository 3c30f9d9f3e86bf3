// Launchers of the speculative-decoding step: rotary positions, tree attention
// over the latent cache, and page upkeep.  api_step.hip validates arguments and
// calls exactly one of these.
#pragma once

#include "launch.hpp"

namespace mla {

constexpr int kMaxRopePairs = 256;

struct RopeFreqsArgs {
    double quarters[kMaxRopePairs];   // quarter turns per position of each pair
    float* out;                       // [rows][2 * pairs]
    double amplitude;
    int first, rows, pairs;
};

struct RopeQArgs {
    const char* q;
    char* out;
    int64_t q_st, q_sh, o_st, o_sh;   // byte strides of tokens and heads
    const uint32_t* pos;
    const float* freqs;               // [max_seq][R]
    int T, H, nope_bytes, R, max_seq;
    bool copy;                        // nope columns are copied (not in place)
};

struct LatentWriteAtArgs : LatentWriteArgs {
    const uint32_t* pos;              // [T] freqs row of each token
    int half;                         // rope pairs (j, j + R/2) instead of (2j, 2j + 1)
};

struct TreeAttentionArgs {
    const void* q;                    // [T][H][D]
    const uint32_t* iro;              // [batch + 1]
    const uint32_t* cache_len;        // [batch]
    const uint64_t* mask;             // [T][words], or null: causal chain
    void* out;                        // [T][H][K]
    float* lse;                       // [T][H] or null
    float* ws;                        // partial results
    PagedLayer L;
    PagedLayer Ls;                    // e4m3: the scale pool
    float scale;
    int T, H, K, D, words;
    uint32_t capacity;                // max_pages * page_size: positions a request can have
};

// Partial results of the split attention: every workgroup leaves at most two
// (the item its share begins in and the one it ends in).
constexpr int kAttnGroups = 256;      // workgroups, one per CU: the whole LDS and register file
constexpr int kAttnRows = 128;        // query rows (tokens x heads) of an item
constexpr int kAttnCutBytes = 32;     // and a record of the cut it starts at

enum AttnKind { ATTN_F32, ATTN_BF16, ATTN_E4M3 };

struct PageArgs {
    char* pool;
    float* scales;                    // null: none
    uint32_t* page_table;
    uint32_t* cache_len;
    int64_t sp, sl, sk, st;           // byte strides: page, layer, kv, token
    int64_t ssp, ssl, ssk, sst;       // scale pool, floats
    uint32_t num_pages, page_size, max_pages, batch, layers, kvs;
    int granules;                     // 16-byte pieces of a token row
    int nblk;                         // scales of a token row
    const uint32_t* a;                // src / parents / requests / accepted
    const uint32_t* b;                // dst / children / - / accepted_offsets
    const uint32_t* c;                // - / new_pages
    uint32_t* refs;
    uint32_t* free_list;
    uint32_t* free_count;
    int count;
};

hipError_t launch_rope_freqs(const RopeFreqsArgs& a, hipStream_t s);
hipError_t launch_rope_q(const RopeQArgs& a, bool f32, bool half, hipStream_t s);
hipError_t launch_latent_write_at(const LatentWriteAtArgs& a, hipStream_t s);
hipError_t launch_latent_write_fp8_at(const LatentWriteAtArgs& a, hipStream_t s);
// Matrix-core form (576-column rows, K = 512), and whether it takes a call.
bool tree_attention_mfma_fits(const TreeAttentionArgs& a, AttnKind kind);
hipError_t launch_tree_attention_mfma(const TreeAttentionArgs& a, AttnKind kind, hipStream_t s);
hipError_t launch_tree_attention(const TreeAttentionArgs& a, AttnKind kind, hipStream_t s);
hipError_t launch_copy_pages(const PageArgs& a, hipStream_t s);
hipError_t launch_fork(const PageArgs& a, hipStream_t s);
hipError_t launch_free(const PageArgs& a, hipStream_t s);
hipError_t launch_compact(const PageArgs& a, hipStream_t s);

}  // namespace mla
