/*
 * mla_paged.h -- C ABI of the MI355X (gfx950) paged MLA latent-K library.
 *
 * Three operations, after the MAX kernel API pages (and the two steps of the
 * first one as calls of their own: mla_gather_latent_paged, mla_latent_matmul):
 *
 *   mla_decompress_k_paged      page "generic_flare_mla_decompress_k_cache_ragged_paged"
 *                               (summary; Args buffer_row_offsets_1d, cache_offsets_1d,
 *                               buffer_length, weight, kv_collection, layer_idx,
 *                               k_latent_buffer, k_buffer, context)
 *   mla_decompress_k_paged_fp8  the same operation with the fp8 block-scaled weight of
 *                               page "mla_prefill_decode_graph_fp8" (Parameters fp8_dtype,
 *                               fp8_scale_dtype, m/n/k_scale_granularity; Args w_k, w_k_scale)
 *   kv_matmul_paged             page "kv_matmul_ragged_paged" (summary; Args hidden_state,
 *                               input_row_offsets, weight, kv_collection, layer_idx, ctx)
 *
 * Conventions for every call:
 *   - Pointers marked [device] are HIP device pointers; [host] pointers are read
 *     during the call only.  The caller allocates and frees every buffer and keeps
 *     it valid until the work queued on `stream` has finished.
 *   - Matrices are row-major with the innermost dimension contiguous.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue work:
 *     they never synchronise, never allocate device memory and keep no state
 *     between calls.  They are safe to call from several host threads.
 *   - Errors are returned synchronously, before anything is enqueued, in this
 *     order: host pointers and shapes (MLA_ERR_NULL_POINTER, MLA_ERR_INVALID_SHAPE,
 *     MLA_ERR_INVALID_DTYPE, MLA_ERR_MISALIGNED, MLA_ERR_OUT_OF_RANGE,
 *     MLA_ERR_WORKSPACE), then the current device (MLA_ERR_UNSUPPORTED_DEVICE unless
 *     it is a gfx950), then the launch (MLA_ERR_HIP; mla_last_hip_error() gives the
 *     hipError_t).  A call with no rows to process returns MLA_OK after the host
 *     checks and enqueues nothing.
 *   - With MLA_PAGED_LOG set in the environment (to anything but "0"; read once
 *     per process) every kernel launch prints one line to stderr naming the
 *     kernel, its grid and block sizes and its shapes.
 *   - Index contents in device memory (offsets, positions, page ids) are the caller's
 *     contract and are not validated on the host.  Read paths clamp every page
 *     id, page index and row to the buffers they were given, so a bad index
 *     yields unspecified values in the output rows it affects but never an
 *     access outside the pool, the weight or the outputs.  Write paths
 *     (kv_matmul_paged, mla_write_latent_paged(_fp8)(_at)) store nothing for a token
 *     whose position lies past its request's page table or whose page id lies
 *     past the pool; every other byte of the pool keeps its value.
 *   - Shapes whose 256-row tiles would need byte offsets of 2^31 or more (a
 *     row of 2^22 bf16 elements in an output, a weight or the cache) return
 *     MLA_ERR_INVALID_SHAPE.
 */
#ifndef MLA_PAGED_H
#define MLA_PAGED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_PAGED_ABI_VERSION 1

typedef enum {
    MLA_OK = 0,
    MLA_ERR_NULL_POINTER = 1,
    MLA_ERR_INVALID_SHAPE = 2,
    MLA_ERR_INVALID_DTYPE = 3,
    MLA_ERR_MISALIGNED = 4,
    MLA_ERR_OUT_OF_RANGE = 5,
    MLA_ERR_WORKSPACE = 6,
    MLA_ERR_UNSUPPORTED_DEVICE = 7,
    MLA_ERR_HIP = 8
} mla_status_t;

typedef enum {
    MLA_DTYPE_F32 = 0,       /* IEEE binary32 */
    MLA_DTYPE_BF16 = 1,      /* bfloat16 */
    MLA_DTYPE_F8E4M3FN = 2   /* OCP OFP8 E4M3 (finite, max 448) */
} mla_dtype_t;

/*
 * A paged KV cache collection (the `kv_collection` + `layer_idx` of the pages):
 * one pool holds every layer.  Element (page, layer, kv, slot, i) of the pool is at
 *   blocks + page*stride_page + layer*stride_layer + kv*stride_kv + slot*stride_token + i
 * (strides in elements), where i < num_heads*head_dim indexes one token's row.
 * Token position p of request b lives in physical page page_table[b][p / page_size]
 * at slot p % page_size.
 */
typedef struct {
    void* blocks;                   /* [device] pool base; 16-byte aligned */
    int32_t dtype;                  /* mla_dtype_t of the pool: F32 or BF16 (F8E4M3FN with
                                       scales, mla_decompress_k_paged_fp8_cache only) */
    uint32_t num_layers;
    uint32_t num_pages;
    uint32_t page_size;             /* tokens per page, >= 1 */
    uint32_t num_kv;                /* 1 = MLA latent cache, 2 = K then V */
    uint32_t num_heads;             /* heads per token row */
    uint32_t head_dim;              /* elements per head */
    int64_t stride_page;            /* elements */
    int64_t stride_layer;
    int64_t stride_kv;
    int64_t stride_token;           /* token rows are contiguous: row = num_heads*head_dim */
    const uint32_t* page_table;     /* [device] [batch_size][max_pages_per_seq] page ids */
    uint32_t batch_size;            /* requests in the batch */
    uint32_t max_pages_per_seq;
    const uint32_t* cache_lengths;  /* [device] [batch_size] tokens already cached
                                       (read by kv_matmul_paged: where appends start;
                                       may be NULL for the decompress calls) */
} mla_paged_cache_t;

/* [host] Fill the four strides for a contiguous pool laid out
 * [page][layer][kv][slot][head][dim].  Returns MLA_ERR_NULL_POINTER or MLA_OK. */
mla_status_t mla_paged_cache_default_strides(mla_paged_cache_t* cache);

/*
 * The scales of an fp8 (F8E4M3FN) pool (the collection's scale_dtype_ = fp32 and
 * quantization_granularity_ of page "generic_flare_mla_decompress_k_cache_ragged_paged",
 * signature): every token row of num_heads*head_dim codes has
 * nblk = ceil(num_heads*head_dim / granularity) fp32 scales; scale j multiplies the
 * codes of columns [j*granularity, (j+1)*granularity).  The scales of (page, layer,
 * kv, slot) start at
 *   scales + page*stride_page + layer*stride_layer + kv*stride_kv + slot*stride_token
 * (strides in floats) and are contiguous.  The same page table addresses both pools.
 */
typedef struct {
    const float* scales;            /* [device] scale pool; 4-byte aligned */
    uint32_t granularity;           /* columns per scale; supported: 128 */
    int64_t stride_page;            /* floats */
    int64_t stride_layer;
    int64_t stride_kv;
    int64_t stride_token;           /* >= nblk */
} mla_cache_scales_t;

/*
 * Gather each request's latent rows from the paged cache, then up-project them
 * (page "generic_flare_mla_decompress_k_cache_ragged_paged", summary and Args;
 * weight shape from page "mla_prefill_decode_graph_fp8", Args w_k).
 *
 *   For request b < cache->batch_size and i < rows_b = buffer_row_offsets[b+1] -
 *   buffer_row_offsets[b], with r = buffer_row_offsets[b] + i and
 *   p = cache_offsets[b] + i:
 *     k_latent_buffer[r][0:D_c] = cache row of token p of request b in layer layer_idx
 *                                 (a bit copy; D_c = num_heads*head_dim)
 *     k_buffer[r][n]            = sum_{k<K} k_latent_buffer[r][k] * weight[n][k]
 *   accumulated in fp32 and rounded to the cache dtype (round to nearest even).
 *
 * buffer_row_offsets  [device] uint32 [batch_size+1], [0] = 0, nondecreasing
 * cache_offsets       [device] uint32 [>= batch_size]; a [batch_size+1] array is accepted
 *                     (the last entry is not read)
 * buffer_length       [host] M = buffer_row_offsets[batch_size], the rows to produce;
 *                     the grid is sized from it, rows >= M are never written
 * weight              [device] [N][K] in the cache dtype (F32 or BF16), 16-byte aligned
 * N, K                N = num_heads*qk_nope_head_dim, K = kv_lora_rank; 1 <= K <= D_c.
 *                     BF16: K % 64 == 0 and N % 64 == 0.  F32: K % 4 == 0 and N % 4 == 0.
 * cache               [host] num_kv == 1; D_c*elem_size and stride_token*elem_size
 *                     multiples of 16 bytes
 * k_latent_buffer     [device] [>= M][D_c] cache dtype, written
 * k_buffer            [device] [>= M][N] cache dtype, written
 */
mla_status_t mla_decompress_k_paged(const uint32_t* buffer_row_offsets,
                                    const uint32_t* cache_offsets,
                                    int32_t buffer_length,
                                    const void* weight, int32_t N, int32_t K,
                                    const mla_paged_cache_t* cache, uint32_t layer_idx,
                                    void* k_latent_buffer, void* k_buffer,
                                    void* stream);

/*
 * The first step of mla_decompress_k_paged on its own: the paged gather
 * (page "generic_flare_mla_decompress_k_cache_ragged_paged", Args
 * buffer_row_offsets_1d, cache_offsets_1d, k_latent_buffer).
 *
 *   k_latent_buffer[r][0:D_c] = cache row of token cache_offsets[b] + i of request b
 *   (r = buffer_row_offsets[b] + i), a bit copy.
 *
 * Arguments as in mla_decompress_k_paged; the cache dtype is F32 or BF16.
 */
mla_status_t mla_gather_latent_paged(const uint32_t* buffer_row_offsets,
                                     const uint32_t* cache_offsets,
                                     int32_t buffer_length,
                                     const mla_paged_cache_t* cache, uint32_t layer_idx,
                                     void* k_latent_buffer, void* stream);

/*
 * The second step of mla_decompress_k_paged on its own: the up-projection of
 * rows already gathered (page "generic_flare_mla_decompress_k_cache_ragged_paged",
 * Args weight, k_buffer; shape from page "mla_prefill_decode_graph_fp8", Args w_k).
 *
 *   k_buffer[r][n] = sum_{k<K} k_latent_buffer[r * ld_latent + k] * weight[n][k],
 *   fp32 accumulation, rounded to `dtype` (round to nearest even).
 *
 * k_latent_buffer  [device] [buffer_length][ld_latent] in `dtype`; columns >= K are not read
 * ld_latent        row stride in elements, K <= ld_latent <= 2^20, ld_latent*elem % 16 == 0
 * weight           [device] [N][K] in `dtype`
 * dtype            MLA_DTYPE_BF16 (K % 64 == 0, N % 64 == 0) or MLA_DTYPE_F32 (K, N % 4 == 0)
 * k_buffer         [device] [>= buffer_length][N] in `dtype`, written
 * All pointers 16-byte aligned.
 */
mla_status_t mla_latent_matmul(const void* k_latent_buffer, int64_t ld_latent, int32_t buffer_length,
                               const void* weight, int32_t N, int32_t K, int32_t dtype,
                               void* k_buffer, void* stream);

/*
 * Bytes of device workspace mla_decompress_k_paged_fp8 needs for buffer_length rows
 * (the activation codes and scales of the on-the-fly quantisation).  0 on bad
 * arguments.
 */
size_t mla_decompress_k_paged_fp8_workspace_size(int32_t buffer_length, int32_t K, int32_t k_gran);

/*
 * The fp8 block-scaled form of mla_decompress_k_paged (page
 * "mla_prefill_decode_graph_fp8": Parameters fp8_dtype, fp8_scale_dtype,
 * m/n/k_scale_granularity; Args w_k, w_k_scale).
 *
 *   The gather is as in mla_decompress_k_paged (cache dtype BF16).  Each gathered
 *   row is quantised per block of k_gran columns (m_gran = 1): amax = max|x|,
 *   s_a = amax / 448, codes = e4m3fn(x * (448 / amax)) (binary32 quotients, round
 *   to nearest even; an all-zero block takes s_a = 1).  Then
 *     k_buffer[r][n] = bf16( sum_kb s_a[r][kb] * weight_scale[n / n_gran][kb]
 *                                  * sum_{k in block kb} codes[r][k] * weight[n][k] )
 *   with fp32 accumulation.
 *
 * weight_e4m3      [device] [N][K] e4m3fn codes, 16-byte aligned
 * weight_scale     [device] float [N / n_gran][K / k_gran] multipliers (W ~= s * codes)
 * m_gran, n_gran, k_gran  granularities along M, N, K; supported: 1, 128, 128
 * N, K             N % 128 == 0, K % 128 == 0, K <= D_c
 * workspace        [device] >= mla_decompress_k_paged_fp8_workspace_size(M, K, k_gran)
 *                  bytes, 256-byte aligned; its contents on return are the activation
 *                  codes [M][K] followed (at offset align256(M*K)) by the scales
 *                  float [M][K / k_gran]
 * other arguments  as in mla_decompress_k_paged; k_latent_buffer and k_buffer are BF16
 *
 * The workspace argument is an addition to the page's signature: the codes and
 * scales go through device memory between the quantising gather and the product
 * (the product reads codes, half the bytes of the bf16 rows, in a loop bound by
 * its operand loads).  Callers that cannot pass one use
 * mla_decompress_k_paged_fp8_noalloc.
 */
mla_status_t mla_decompress_k_paged_fp8(const uint32_t* buffer_row_offsets,
                                        const uint32_t* cache_offsets,
                                        int32_t buffer_length,
                                        const void* weight_e4m3, const float* weight_scale,
                                        int32_t N, int32_t K,
                                        int32_t m_gran, int32_t n_gran, int32_t k_gran,
                                        const mla_paged_cache_t* cache, uint32_t layer_idx,
                                        void* k_latent_buffer, void* k_buffer,
                                        void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * Fused K and V decompression: one gather, two up-projections of the gathered
 * rows (page "mla_prefill_decode_graph_fp8", Args w_k and w_uv: w_uv projects the
 * latent values to V, shape [num_heads][v_head_dim][kv_latent_dim], i.e. an
 * [N_v][K] matrix with N_v = num_heads*v_head_dim; the gather and the product
 * are those of page "generic_flare_mla_decompress_k_cache_ragged_paged").
 *
 *   k_latent_buffer and k_buffer exactly as mla_decompress_k_paged(..., w_k, N_k, ...)
 *   v_buffer[r][n] = sum_{k<K} k_latent_buffer[r][k] * w_v[n][k]   (n < N_v),
 *   fp32 accumulation, rounded to the cache dtype (round to nearest even).
 *
 * Every element of k_buffer and v_buffer equals, bit for bit, what
 * mla_decompress_k_paged returns with w_k or w_v alone.  Each latent row is read
 * once from the cache; with BF16, K % 128 == 0 and N_k % 256 == 0 both products
 * run in a single launch that reads each tile of gathered rows for both.
 *
 * w_v        [device] [N_v][K] in the cache dtype, 16-byte aligned
 * N_v        BF16: N_v % 64 == 0; F32: N_v % 4 == 0
 * v_buffer   [device] [>= M][N_v] cache dtype, written
 * Other arguments, errors and validation order as in mla_decompress_k_paged
 * (w_k, N_k play the roles of weight, N).
 */
mla_status_t mla_decompress_kv_paged(const uint32_t* buffer_row_offsets,
                                     const uint32_t* cache_offsets,
                                     int32_t buffer_length,
                                     const void* w_k, int32_t N_k,
                                     const void* w_v, int32_t N_v, int32_t K,
                                     const mla_paged_cache_t* cache, uint32_t layer_idx,
                                     void* k_latent_buffer, void* k_buffer, void* v_buffer,
                                     void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc):
 * mla_decompress_k_paged_fp8 without the workspace argument.  The activation
 * codes and scales go to a fixed array of MLA_FP8_NOALLOC_SCRATCH_BYTES in
 * device memory that the library holds on each GPU it runs on until the
 * process ends; nothing is allocated per call.
 *
 *   Same arguments, arithmetic and results as mla_decompress_k_paged_fp8 (the
 *   same kernels run).  Calls whose workspace would exceed the array
 *   (mla_decompress_k_paged_fp8_workspace_size(M, K, k_gran) >
 *   MLA_FP8_NOALLOC_SCRATCH_BYTES: more than 65536 rows at K = 512) return
 *   MLA_ERR_WORKSPACE before anything is enqueued.
 *   Every call on one GPU shares that GPU's array: calls that overlap on one
 *   GPU (other streams, other host threads) race on it and must be ordered by
 *   the caller.  Nothing in the array has to start at zero: each call writes
 *   every code and scale it reads.
 *   The first call on a device looks up the array's address there
 *   (MLA_ERR_HIP if that fails).
 */
#define MLA_FP8_NOALLOC_SCRATCH_BYTES (33u << 20)   /* the workspace of 65536 rows at K = 512 */
mla_status_t mla_decompress_k_paged_fp8_noalloc(const uint32_t* buffer_row_offsets,
                                                const uint32_t* cache_offsets, int32_t buffer_length,
                                                const void* weight_e4m3, const float* weight_scale,
                                                int32_t N, int32_t K, int32_t m_gran, int32_t n_gran,
                                                int32_t k_gran, const mla_paged_cache_t* cache,
                                                uint32_t layer_idx, void* k_latent_buffer, void* k_buffer,
                                                void* stream);

/*
 * The fp8 block-scaled form of mla_decompress_kv_paged (page
 * "mla_prefill_decode_graph_fp8": Args w_k, w_k_scale, w_uv, w_uv_scale; the
 * quantisation of the gathered rows as in mla_decompress_k_paged_fp8, done once
 * for both products, which run in a single launch).
 *
 *   v_buffer[r][n] = bf16( sum_kb s_a[r][kb] * w_v_scale[n / n_gran][kb]
 *                                * sum_{k in block kb} codes[r][k] * w_v[n][k] )
 *
 * w_v_e4m3   [device] [N_v][K] e4m3fn codes, 16-byte aligned; N_v % 128 == 0
 * w_v_scale  [device] float [N_v / n_gran][K / k_gran]
 * v_buffer   [device] [>= M][N_v] bf16, written
 * Other arguments (workspace included), errors and validation order as in
 * mla_decompress_k_paged_fp8.
 */
mla_status_t mla_decompress_kv_paged_fp8(const uint32_t* buffer_row_offsets,
                                         const uint32_t* cache_offsets,
                                         int32_t buffer_length,
                                         const void* w_k_e4m3, const float* w_k_scale, int32_t N_k,
                                         const void* w_v_e4m3, const float* w_v_scale, int32_t N_v,
                                         int32_t K, int32_t m_gran, int32_t n_gran, int32_t k_gran,
                                         const mla_paged_cache_t* cache, uint32_t layer_idx,
                                         void* k_latent_buffer, void* k_buffer, void* v_buffer,
                                         void* workspace, size_t workspace_bytes,
                                         void* stream);

/*
 * The decompress call on an fp8 paged cache (page
 * "generic_flare_mla_decompress_k_cache_ragged_paged", summary and Args, with a
 * collection whose scale_dtype_ / quantization_granularity_ are fp32 / 128; the
 * weight and its block scales as page "mla_prefill_decode_graph_fp8", Args w_k,
 * w_k_scale, granularities 1 x 128 x 128).
 *
 *   For request b, i < rows_b, r = buffer_row_offsets[b] + i, p = cache_offsets[b] + i:
 *     k_latent_buffer[r][0:D_c]  = e4m3 codes of token p of request b (a bit copy)
 *     k_latent_scales[r][0:nblk] = that token's fp32 scales (a bit copy)
 *     k_buffer[r][n] = bf16( sum_kb k_latent_scales[r][kb] * weight_scale[n/128][kb]
 *                              * sum_{k in block kb} k_latent_buffer[r][k] * weight[n][k] )
 *   over the K/128 blocks of the first K columns, fp32 accumulation, round to
 *   nearest even.  The cache is already quantised: no quantisation step, no workspace.
 *
 * weight_e4m3      [device] [N][K] e4m3fn codes, 16-byte aligned
 * weight_scale     [device] float [N/128][K/128], 4-byte aligned
 * N, K             N % 128 == 0, K % 128 == 0, K <= D_c
 * cache            [host] dtype F8E4M3FN, num_kv == 1, D_c % 16 == 0, byte strides
 *                  multiples of 16
 * cache_scales     [host] granularity 128, stride_token >= nblk = ceil(D_c / 128)
 * k_latent_buffer  [device] uint8 [>= M][D_c], 16-byte aligned, written
 * k_latent_scales  [device] float [>= M][nblk], 4-byte aligned, written
 * k_buffer         [device] bf16 [>= M][N], 16-byte aligned, written
 * M * D_c < 2^31.  Other arguments, errors and validation order as in
 * mla_decompress_k_paged.
 */
mla_status_t mla_decompress_k_paged_fp8_cache(const uint32_t* buffer_row_offsets,
                                              const uint32_t* cache_offsets,
                                              int32_t buffer_length,
                                              const void* weight_e4m3, const float* weight_scale,
                                              int32_t N, int32_t K,
                                              const mla_paged_cache_t* cache,
                                              const mla_cache_scales_t* cache_scales,
                                              uint32_t layer_idx,
                                              void* k_latent_buffer, float* k_latent_scales,
                                              void* k_buffer, void* stream);

/*
 * K and V decompression from an e4m3 cache in one call (the fused form of
 * mla_decompress_kv_paged_fp8 on the cache of mla_decompress_k_paged_fp8_cache;
 * page "mla_prefill_decode_graph_fp8", Args w_k, w_k_scale, w_uv, w_uv_scale):
 * one gather of codes and scales, then
 *   k_buffer[r][n] as mla_decompress_k_paged_fp8_cache with w_k_e4m3 / w_k_scale (N_k columns)
 *   v_buffer[r][n] the same with w_v_e4m3 / w_v_scale (N_v columns)
 * in one product launch over both projections' column tiles.
 *
 * w_v_e4m3         [device] [N_v][K] e4m3fn codes, 16-byte aligned; N_v % 128 == 0
 * w_v_scale        [device] float [N_v/128][K/128], 4-byte aligned
 * v_buffer         [device] bf16 [>= M][N_v], 16-byte aligned, written
 * Other arguments, errors and validation order as in mla_decompress_k_paged_fp8_cache.
 */
mla_status_t mla_decompress_kv_paged_fp8_cache(const uint32_t* buffer_row_offsets,
                                               const uint32_t* cache_offsets, int32_t buffer_length,
                                               const void* w_k_e4m3, const float* w_k_scale, int32_t N_k,
                                               const void* w_v_e4m3, const float* w_v_scale, int32_t N_v,
                                               int32_t K, const mla_paged_cache_t* cache,
                                               const mla_cache_scales_t* cache_scales, uint32_t layer_idx,
                                               void* k_latent_buffer, float* k_latent_scales,
                                               void* k_buffer, void* v_buffer, void* stream);

/*
 * Query absorption for decode (page "mla_prefill_decode_graph_fp8", Args q
 * [tot_seq_len, num_heads, qk_nope_head_dim + qk_rope_head_dim] and w_uk
 * [num_heads, kv_latent_dim, qk_nope_head_dim], the weight that projects the
 * non-rope part of each query head to the KV latent space), bf16:
 *
 *   q_latent[t][h][c] = bf16( sum_{d < d_nope} q[t][h][d] * w_uk[h][c][d] ),  c < kv_latent_dim
 *   q_latent[t][h][kv_latent_dim + i] = q[t][h][d_nope + i],  i < d_rope   (copy_rope = 1 only)
 *
 * fp32 accumulation, round to nearest even.  With copy_rope = 1 an absorbed head
 * has the layout of an MLA cache row (latent, then rope).
 *
 * q             [device] bf16 [total_tokens][num_heads][d_nope + d_rope], 16-byte aligned
 * d_nope        128 (the supported qk_nope_head_dim); d_rope % 8 == 0
 * w_uk          [device] bf16 [num_heads][kv_latent_dim][d_nope], 16-byte aligned
 * kv_latent_dim % 128 == 0
 * copy_rope     0 or 1
 * q_latent      [device] bf16 [total_tokens][num_heads][kv_latent_dim + (copy_rope ? d_rope : 0)],
 *               16-byte aligned, written
 * (total_tokens + 128) * num_heads * (d_nope + d_rope) * 2 < 2^31.
 * Errors and validation order as for the other calls (pointers, shapes,
 * alignment, device).
 */
mla_status_t mla_absorb_q(const void* q, int32_t total_tokens, int32_t num_heads, int32_t d_nope,
                          int32_t d_rope, const void* w_uk, int32_t kv_latent_dim, int32_t copy_rope,
                          void* q_latent, void* stream);

/*
 * The fp8 form of mla_absorb_q (page "mla_prefill_decode_graph_fp8": w_uk in
 * fp8_dtype with w_uk_scale, Parameters m/n/k_scale_granularity).  The non-rope
 * part of each query head is quantised per 1 x 128 block as in
 * mla_decompress_k_paged_fp8 (s_q = amax / 448, codes = e4m3fn(x * (448 / amax)),
 * binary32 quotients, round to nearest even; an all-zero block takes s_q = 1):
 *
 *   q_latent[t][h][c] = bf16( s_q[t][h] * w_uk_scale[h][c / 128][0]
 *                             * sum_{d < 128} codes[t][h][d] * w_uk_e4m3[h][c][d] )
 *
 * with fp32 accumulation; the rope part as in mla_absorb_q.
 *
 * w_uk_e4m3     [device] e4m3fn codes [num_heads][kv_latent_dim][d_nope], 16-byte aligned
 * w_uk_scale    [device] float [num_heads][kv_latent_dim / 128][d_nope / 128], 4-byte aligned
 * m_gran, n_gran, k_gran  supported: 1, 128, 128
 * Other arguments, limits and errors as in mla_absorb_q.
 */
mla_status_t mla_absorb_q_fp8(const void* q, int32_t total_tokens, int32_t num_heads, int32_t d_nope,
                              int32_t d_rope, const void* w_uk_e4m3, const float* w_uk_scale,
                              int32_t kv_latent_dim, int32_t m_gran, int32_t n_gran, int32_t k_gran,
                              int32_t copy_rope, void* q_latent, void* stream);

/*
 * The latent write path: new tokens' latent rows, normalised and rotated, into
 * the MLA cache pages this library's decompress calls read (page
 * "mla_prefill_decode_graph_fp8", Args kv_input_fn (the latent values,
 * [tot_seq_len, cache_head_dim] with cache_head_dim = kv_lora_rank +
 * qk_rope_head_dim), kv_norm_gamma [kv_lora_rank], epsilon, freqs_cis
 * [max_seq_len, qk_rope_head_dim], input_row_offsets, kv_collection, layer_idx).
 *
 *   Token t of request b (input_row_offsets[b] <= t < input_row_offsets[b+1]) is
 *   written at position p = cache_lengths[b] + (t - input_row_offsets[b]):
 *     row[k]       = bf16( gamma[k] * x[k] / sqrt(mean_{k<K} x[k]^2 + epsilon) ),  k < K
 *     row[K+2j]    = bf16( x[K+2j] * c - x[K+2j+1] * s )
 *     row[K+2j+1]  = bf16( x[K+2j] * s + x[K+2j+1] * c ),  (c, s) = freqs_cis[p][2j], [2j+1]
 *   with x = kv_input[t], fp32 arithmetic, round to nearest even; stored as the
 *   cache row of (page_table[b][p / page_size], slot p % page_size) in layer
 *   layer_idx.  Other cache bytes are not touched; cache_lengths is not updated.
 *
 * kv_input         [device] bf16 [total_tokens][D_c], D_c = num_heads*head_dim = K + R
 * input_row_offsets [device] uint32 [batch_size+1], [0] = 0, nondecreasing
 * total_tokens     [host] input_row_offsets[batch_size]
 * kv_norm_gamma    [device] float [K], 16-byte aligned
 * epsilon          >= 0
 * freqs_cis        [device] float [max_seq_len][R], (cos, sin) of each rope pair;
 *                  may be NULL when R == 0; positions must be < max_seq_len
 * K                kv_lora_rank: K % 8 == 0, K <= 512; R = D_c - K: R % 8 == 0, R <= 512
 * cache            [host] num_kv == 1, BF16, cache_lengths set; pages are WRITTEN
 * Errors and validation order as for the other calls (pointers, shapes, dtype,
 * alignment, ranges, device).
 */
mla_status_t mla_write_latent_paged(const void* kv_input, const uint32_t* input_row_offsets,
                                    int32_t total_tokens, const float* kv_norm_gamma, float epsilon,
                                    const float* freqs_cis, int32_t max_seq_len, int32_t K,
                                    const mla_paged_cache_t* cache, uint32_t layer_idx, void* stream);

/*
 * The latent write path into an e4m3 cache (page "mla_prefill_decode_graph_fp8",
 * Args kv_input_fn, kv_norm_gamma, epsilon, freqs_cis, input_row_offsets,
 * kv_collection, layer_idx; the collection's scale_dtype_ fp32 and
 * quantization_granularity_ 128 of page
 * "generic_flare_mla_decompress_k_cache_ragged_paged"): the rows of
 * mla_write_latent_paged, computed the same way in fp32, then quantised per
 * block of 128 columns of the row:
 *   y = the fp32 row values (RMS-normalised latent part, rotated rope part)
 *   amax_j = max |y| over block j, s_j = amax_j / 448 (1 for an all-zero block)
 *   codes = e4m3fn(y * (448 / amax_j)), round to nearest even; s_j into the scale pool
 * at the token's (page, slot) in layer layer_idx, codes into the e4m3 pool.
 * mla_decompress_k_paged_fp8_cache reads what this writes.
 *
 * cache            [host] num_kv == 1, dtype F8E4M3FN, D_c % 16 == 0, cache_lengths set;
 *                  pages are WRITTEN
 * cache_scales     [host] granularity 128, stride_token >= ceil(D_c / 128); WRITTEN
 * K                kv_lora_rank: K % 128 == 0, K <= 512; R = D_c - K: R % 8 == 0, R <= 512
 * Other arguments, errors and validation order as in mla_write_latent_paged.
 */
mla_status_t mla_write_latent_paged_fp8(const void* kv_input, const uint32_t* input_row_offsets,
                                        int32_t total_tokens, const float* kv_norm_gamma, float epsilon,
                                        const float* freqs_cis, int32_t max_seq_len, int32_t K,
                                        const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales,
                                        uint32_t layer_idx, void* stream);

/*
 * Project hidden states and write them into the paged K/V cache (page
 * "kv_matmul_ragged_paged", summary and Args).
 *
 *   out[t][n] = sum_k hidden_state[t][k] * weight[k][n], fp32 accumulation.
 *   Token t of request b (input_row_offsets[b] <= t < input_row_offsets[b+1]) is
 *   appended at position p = cache_lengths[b] + (t - input_row_offsets[b]):
 *     K row of (page_table[b][p / page_size], slot p % page_size) = bf16(out[t][0 : HD])
 *     V row of the same slot                                        = bf16(out[t][HD : 2HD])
 *   with HD = num_heads*head_dim.  No other cache element is written, and
 *   cache_lengths is not updated (that bookkeeping is the cache owner's).
 *
 * hidden_state       [device] bf16 [total_tokens][hidden_dim], 16-byte aligned
 * input_row_offsets  [device] uint32 [batch_size+1], [0] = 0, nondecreasing,
 *                    [batch_size] = total_tokens
 * total_tokens       [host] T >= 0
 * hidden_dim         [host] % 64 == 0
 * weight             [device] bf16 [hidden_dim][2*HD], 16-byte aligned
 * cache              [host] BF16, num_kv == 2, HD % 64 == 0, cache_lengths non-NULL;
 *                    pages are written in place
 */
mla_status_t kv_matmul_paged(const void* hidden_state, const uint32_t* input_row_offsets,
                             int32_t total_tokens, int32_t hidden_dim,
                             const void* weight,
                             const mla_paged_cache_t* cache, uint32_t layer_idx,
                             void* stream);

/*
 * Debug check of the index arrays of a call (the preconditions the pages leave to
 * the caller: offsets start at 0 and never decrease, every position a request
 * touches lies inside its page-table row and maps to a page id < num_pages).
 * Copies the arrays to the host and synchronises `stream`; meant for debugging,
 * not for the hot path.
 *
 * row_offsets    [device] uint32 [batch_size+1] (buffer_row_offsets or input_row_offsets)
 * cache_offsets  [device] uint32 [>= batch_size]: positions read start there
 *                (decompress calls), and when cache->cache_lengths is non-NULL they
 *                must also end at or before cache_lengths[b].  NULL: positions
 *                written start at cache_lengths[b] (kv_matmul_paged).
 * rows           [host] must equal row_offsets[batch_size]
 * bad_request    [host] optional; receives the first failing request (-1 if none)
 * Returns MLA_OK, MLA_ERR_INVALID_SHAPE (offsets), MLA_ERR_OUT_OF_RANGE (positions
 * or page ids), MLA_ERR_NULL_POINTER, MLA_ERR_UNSUPPORTED_DEVICE or MLA_ERR_HIP.
 */
mla_status_t mla_check_indices(const uint32_t* row_offsets, const uint32_t* cache_offsets,
                               int32_t rows, const mla_paged_cache_t* cache, int64_t* bad_request,
                               void* stream);

/*
 * Rotary positions.  A freqs_cis table row p holds, for rope pair j, (cos, sin) of the
 * pair's angle at position p in columns 2j and 2j+1, whatever the layout of the columns
 * that are rotated:
 *   MLA_ROPE_INTERLEAVED  pair j is columns (2j, 2j+1) of the rope part
 *   MLA_ROPE_HALF         pair j is columns (j, j + d_rope/2)
 *   (x0, x1) -> (x0*c - x1*s, x0*s + x1*c)
 */
typedef enum {
    MLA_ROPE_INTERLEAVED = 0,
    MLA_ROPE_HALF = 1
} mla_rope_layout_t;

/* How a table's frequencies f_j = theta^(-2j/d_rope) are scaled for contexts longer
 * than the original ones. */
typedef enum {
    MLA_ROPE_SCALING_NONE = 0,
    MLA_ROPE_SCALING_LINEAR = 1,     /* f_j / factor: positions interpolated */
    MLA_ROPE_SCALING_BY_PARTS = 2    /* f_j / factor where a pair turns fewer than beta_slow
                                        times in original_max_position positions, f_j where
                                        more than beta_fast times, mixed linearly in j between */
} mla_rope_scaling_t;

typedef struct {
    double theta;                    /* > 0, and > 1 with BY_PARTS */
    double factor;                   /* > 0 (LINEAR, BY_PARTS) */
    double beta_fast;                /* BY_PARTS: > 0 */
    double beta_slow;                /* BY_PARTS: > 0 */
    double amplitude;                /* every cos and sin is multiplied by it */
    int32_t scaling;                 /* mla_rope_scaling_t */
    int32_t original_max_position;   /* BY_PARTS: > 0 */
} mla_rope_params_t;

/*
 * Fill rows of a freqs_cis table (the freqs_cis argument of the latent write and of
 * mla_rope_q; page "mla_prefill_decode_graph_fp8", Args freqs_cis):
 *
 *   freqs_cis[i][2j]   = float(amplitude * cos((first_position + i) * g_j))
 *   freqs_cis[i][2j+1] = float(amplitude * sin((first_position + i) * g_j))
 *   g_j = f_j                                          (NONE),  f_j = theta^(-2j/d_rope)
 *   g_j = f_j / factor                                 (LINEAR)
 *   g_j = f_j / factor * r_j + f_j * (1 - r_j)         (BY_PARTS)
 *     r_j  = clamp((j - low) / max(high - low, 0.001), 0, 1)
 *     low  = max(floor(pair(beta_fast)), 0),  high = min(ceil(pair(beta_slow)), d_rope - 1)
 *     pair(b) = d_rope * ln(original_max_position / (2 pi b)) / (2 ln theta)
 *   (the by-parts interpolation published as YaRN, Peng et al. 2023).
 *
 * All of it is in binary64, up to the one rounding to float.
 *
 * params          [host]
 * first_position  >= 0; first_position + rows <= 2^31
 * d_rope          even, 2 <= d_rope <= 512
 * freqs_cis       [device] float [rows][d_rope], 8-byte aligned, written
 * Parameters that are not finite or out of the ranges above, and frequencies that reach
 * angles of 2^50 quarter turns within the rows: MLA_ERR_INVALID_SHAPE.
 */
mla_status_t mla_rope_freqs(const mla_rope_params_t* params, int32_t first_position, int32_t rows,
                            int32_t d_rope, float* freqs_cis, void* stream);

/*
 * Rotate the rope part of every query head at its token's position (page
 * "mla_prefill_decode_graph_fp8", Args q [tot_seq_len, num_heads, qk_nope_head_dim +
 * qk_rope_head_dim], freqs_cis): the step before mla_absorb_q, which carries the rope
 * columns over as they are.
 *
 *   q_out[t][h][0:d_nope]  = q[t][h][0:d_nope]
 *   q_out[t][h][d_nope:]   = q[t][h][d_nope:] rotated with freqs_cis[positions[t]]
 *   binary32 arithmetic, rounded to `dtype` (round to nearest even).
 *
 * positions are given, not derived from the cache: a drafted token's position is its
 * depth in the tree, not the slot its row is stored in.  A position past the table takes
 * the table's last row.
 *
 * q, q_out        [device] rows of d_nope + d_rope contiguous elements at
 *                 t * stride_token + h * stride_head (elements, one pair of strides each),
 *                 16-byte aligned, strides and d_nope multiples of 16 bytes.  q_out == q
 *                 with the same strides rotates in place and touches the rope columns only;
 *                 any other overlap, also of q_out's rows with one another, is not allowed.
 * total_tokens    [host] T >= 0;  num_heads >= 1;  T * num_heads * (d_nope + d_rope) < 2^40
 * d_nope          0 <= d_nope <= 4096
 * d_rope          8 <= d_rope <= 512; % 8 == 0, and % 16 == 0 with MLA_ROPE_HALF
 * dtype           MLA_DTYPE_BF16 or MLA_DTYPE_F32
 * positions       [device] uint32 [total_tokens]
 * freqs_cis       [device] float [max_seq_len][d_rope], 16-byte aligned
 */
mla_status_t mla_rope_q(const void* q, int64_t q_stride_token, int64_t q_stride_head, int32_t total_tokens,
                        int32_t num_heads, int32_t d_nope, int32_t d_rope, int32_t dtype,
                        const uint32_t* positions, const float* freqs_cis, int32_t max_seq_len, int32_t layout,
                        void* q_out, int64_t out_stride_token, int64_t out_stride_head, void* stream);

/*
 * mla_write_latent_paged and mla_write_latent_paged_fp8 with the rope position of each
 * token given and either layout of the rope columns: the writes of drafted tokens, whose
 * slots follow one another (token t of request b still goes to position cache_lengths[b] +
 * (t - input_row_offsets[b])) while their rope positions are their depths in the tree.
 *
 * positions       [device] uint32 [total_tokens]: the freqs_cis row of each token; past the
 *                 table: its last row
 * rope_layout     mla_rope_layout_t; MLA_ROPE_HALF needs R % 16 == 0
 * Other arguments, results, errors and validation order as in the calls without _at.
 */
mla_status_t mla_write_latent_paged_at(const void* kv_input, const uint32_t* input_row_offsets,
                                       int32_t total_tokens, const uint32_t* positions,
                                       const float* kv_norm_gamma, float epsilon, const float* freqs_cis,
                                       int32_t max_seq_len, int32_t K, int32_t rope_layout,
                                       const mla_paged_cache_t* cache, uint32_t layer_idx, void* stream);
mla_status_t mla_write_latent_paged_fp8_at(const void* kv_input, const uint32_t* input_row_offsets,
                                           int32_t total_tokens, const uint32_t* positions,
                                           const float* kv_norm_gamma, float epsilon, const float* freqs_cis,
                                           int32_t max_seq_len, int32_t K, int32_t rope_layout,
                                           const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales,
                                           uint32_t layer_idx, void* stream);

/*
 * Attention of absorbed queries over the paged latent cache, for trees of drafted tokens
 * (a decode step is the tree of one token, a chunk of a prompt the chain): the consumer of
 * mla_absorb_q's q_latent and of the rows the latent write stored.
 *
 *   Request b has cached = cache_lengths[b] rows and n = input_row_offsets[b+1] -
 *   input_row_offsets[b] drafted ones behind them, at positions cached + j.  Token i of
 *   its n tokens (t = input_row_offsets[b] + i) sees every cached row, and drafted row j
 *   if bit j % 64 of tree_mask[t][j / 64] is set (tree_mask NULL: if j <= i).
 *     s_p             = scale * sum_c q_latent[t][h][c] * row_p[c]        (c < D_c, p seen)
 *     out_latent[t][h][k] = sum_p exp(s_p) * row_p[k] / sum_p exp(s_p)    (k < K)
 *     lse[t][h]       = ln sum_p exp(s_p)
 *   A token that sees no row gets zeros and an lse of -infinity.  Scores, the running
 *   maximum and sum, and the output sums are binary32; the weights exp(s_p - max) are
 *   rounded to bf16 for the product with the rows on bf16 and e4m3 caches.  out_latent is
 *   rounded once (round to nearest even).  Scores are to stay below 2^30 in magnitude, where
 *   binary32 still tells them apart by less than 2^7.
 *
 * What a row that a token does not see holds (NaN and infinities included) does not change
 * that token's output; neither does anything behind a request's last drafted row.
 * Of the rows it does see, a score of NaN or +infinity makes the token's whole output and
 * lse NaN; a score of -infinity is a weight of 0, which makes NaN of the output columns in
 * which that row is not finite, and of no other.
 *
 * q_latent        [device] [total_tokens][num_heads][D_c], D_c the cache's row width; bf16
 *                 with a BF16 cache, float with an F32 cache
 * input_row_offsets [device] uint32 [batch_size+1], [0] = 0, nondecreasing; rows of q_latent
 *                 at or past input_row_offsets[batch_size] are neither read nor written to.
 *                 Where they do decrease the outputs are unspecified.
 * total_tokens    [host] T >= input_row_offsets[batch_size]
 * num_heads       query heads, >= 1; T * num_heads * D_c < 2^31
 * tree_mask       [device] uint64 [total_tokens][mask_words], 8-byte aligned, or NULL.
 *                 Bits at or past n are ignored; drafted rows at or past 64 * mask_words are
 *                 not seen.
 * mask_words      >= 1 with a mask, 0 without; T * mask_words < 2^31
 * scale           finite
 * K               latent columns: K % 8 == 0, K <= 512; R = D_c - K: R % 8 == 0, R <= 512
 * cache           [host] num_kv == 1, BF16 or F32, cache_lengths set.  Positions past the page
 *                 table (max_pages_per_seq * page_size) are not seen; that product < 2^31.
 * out_latent      [device] [total_tokens][num_heads][K] in q_latent's dtype, 16-byte aligned, written
 * lse             [device] float [total_tokens][num_heads], 4-byte aligned, written; or NULL
 * workspace       [device] >= mla_tree_attention_workspace_size(T, num_heads, K) bytes,
 *                 256-byte aligned: partial results of requests that several workgroups
 *                 share.  Nothing in it has to start at zero.  Calls that may overlap (other
 *                 streams, captured graphs replayed side by side) need workspaces of their own.
 * Rows of 576 columns with K = 512 on BF16 or e4m3 caches run on the matrix cores; other
 * shapes and F32 run 4 or 16 waves per token and head, which read each row for it alone.
 */
size_t mla_tree_attention_workspace_size(int32_t total_tokens, int32_t num_heads, int32_t K);
mla_status_t mla_tree_attention_paged(const void* q_latent, const uint32_t* input_row_offsets,
                                      int32_t total_tokens, int32_t num_heads, const uint64_t* tree_mask,
                                      int32_t mask_words, float scale, int32_t K, const mla_paged_cache_t* cache,
                                      uint32_t layer_idx, void* out_latent, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * mla_tree_attention_paged on an e4m3 cache: row_p[c] = code * scale of its block of 128
 * columns.  The codes go into the products as they are (bf16 holds every e4m3 value); the
 * scales multiply the scores' block sums and the weights, in binary32 (an infinite scale
 * thus makes a block's sum infinite, and its 128 columns NaN for the tokens that see the row).
 * Shapes off the matrix cores multiply the codes by the scales first.
 *
 * q_latent, out_latent  bf16
 * cache           dtype F8E4M3FN, D_c % 16 == 0
 * cache_scales    [host] granularity 128, stride_token >= ceil(D_c / 128)
 * Other arguments, limits and errors as in mla_tree_attention_paged.
 */
mla_status_t mla_tree_attention_paged_fp8_cache(const void* q_latent, const uint32_t* input_row_offsets,
                                                int32_t total_tokens, int32_t num_heads,
                                                const uint64_t* tree_mask, int32_t mask_words, float scale,
                                                int32_t K, const mla_paged_cache_t* cache,
                                                const mla_cache_scales_t* cache_scales, uint32_t layer_idx,
                                                void* out_latent, float* lse, void* workspace,
                                                size_t workspace_bytes, void* stream);

/*
 * Page upkeep: copying, forking, compacting and freeing pages of a paged cache, all layers
 * and kv halves at once.  The four calls take any cache this library knows (BF16, F32, or
 * F8E4M3FN with cache_scales; cache_scales is NULL for the others); all copies are bit
 * copies, of the scales too.  Which page is free is the cache owner's bookkeeping: page ids
 * are handed in, and freed ones handed back in a list.  Counts are at most 2^30.
 *
 * mla_copy_pages: page dst_pages[i] becomes a copy of page src_pages[i], i < count.
 *   No destination may be the source of another pair or appear twice.  Pairs with an id
 *   past the pool are skipped.
 * src_pages, dst_pages  [device] uint32 [count]
 */
mla_status_t mla_copy_pages(const uint32_t* src_pages, const uint32_t* dst_pages, int32_t count,
                            const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales,
                            void* stream);

/*
 * Fork requests: request children[i] becomes a copy of request parents[i] (rows of the
 * page table), i < count, sharing its whole pages.
 *
 *   With L = cache_lengths[parent], full = L / page_size, part = L % page_size:
 *     page_table[child][0:full] = page_table[parent][0:full], ref_counts of those pages + 1
 *     if part > 0:  page_table[child][full] = new_pages[i], ref_counts[new_pages[i]] = 1,
 *                   and the first `part` token rows of it, in every layer, are copied
 *     cache_lengths[child] = L
 *   Entries of the child's table row past these keep their values; with part == 0
 *   new_pages[i] is not used and stays the caller's.  What the child held before must have
 *   been freed.
 *
 * No child may be a parent in the same call, and no child or new page may appear twice.
 * Pairs whose parent or child lies past the batch or that are equal, and pairs that need a
 * new page and are given one past the pool, are skipped.  A length past the page table is
 * taken as the table's.
 *
 * parents, children, new_pages  [device] uint32 [count]
 * ref_counts      [device] uint32 [num_pages], updated: requests that hold each page
 * cache           pages, page_table and cache_lengths are WRITTEN
 */
mla_status_t mla_fork_paged(const uint32_t* parents, const uint32_t* children, const uint32_t* new_pages,
                            int32_t count, uint32_t* ref_counts, const mla_paged_cache_t* cache,
                            const mla_cache_scales_t* cache_scales, void* stream);

/*
 * Free requests: every page that requests[i], i < count, holds (the first
 * ceil(cache_lengths / page_size) entries of its table row) loses one reference; its
 * entries become 0xFFFFFFFF and its length 0.  Pages left without references are appended
 * to free_list at free_count[0], in ascending order of their ids, and free_count[0] grows
 * by their number.
 *
 * A request that is listed twice is freed once; ids past the batch and entries past the
 * pool are skipped; a page whose count is already 0 is left alone.  Entries that do not fit
 * into the list (num_pages entries) are not stored, and free_count stops at num_pages.
 *
 * requests        [device] uint32 [count], count <= 65536
 * ref_counts      [device] uint32 [num_pages], updated; counts below 2^31
 * free_list       [device] uint32 [num_pages], entries from free_count[0] on are written
 * free_count      [device] uint32 [1], updated
 * cache           num_pages < 2^31; page_table and cache_lengths are WRITTEN; blocks may be NULL
 */
mla_status_t mla_free_paged(const uint32_t* requests, int32_t count, uint32_t* ref_counts, uint32_t* free_list,
                            uint32_t* free_count, const mla_paged_cache_t* cache, void* stream);

/*
 * Move the rows of accepted drafted tokens together behind the cached ones: with c =
 * accepted_offsets[b+1] - accepted_offsets[b] and a = accepted + accepted_offsets[b],
 *   row at position cache_lengths[b] + i = row at position cache_lengths[b] + a[i],  i < c
 * in every layer and kv half.  a[0] < a[1] < ... are positions in the request's drafted
 * tokens (so a[i] >= i); rows of tokens that are not accepted are left as they are unless
 * an accepted one takes their place.  cache_lengths is not updated.  Rows whose source or
 * destination has no slot (past the page table, page id past the pool) are skipped.
 * A page that is written must be the request's alone.
 *
 * accepted          [device] uint32 [total_accepted]
 * accepted_offsets  [device] uint32 [batch_size+1], [0] = 0, nondecreasing
 * total_accepted    [host] accepted_offsets[batch_size]
 * cache             cache_lengths set; pages are WRITTEN
 */
mla_status_t mla_compact_paged(const uint32_t* accepted, const uint32_t* accepted_offsets, int32_t total_accepted,
                               const mla_paged_cache_t* cache, const mla_cache_scales_t* cache_scales,
                               void* stream);

/* Static text for a status code. */
const char* mla_status_string(mla_status_t status);

/* hipError_t of the last MLA_ERR_HIP returned on this host thread (0 if none). */
int32_t mla_last_hip_error(void);

/* MLA_PAGED_ABI_VERSION of the loaded library. */
int32_t mla_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PAGED_H */
