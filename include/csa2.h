/*
 * csa2.h -- C ABI of the CSA2 sparse-attention hot path over an FP4 global
 * KV cache, for NVIDIA GB300 (sm_103a).
 *
 * The operation follows the CSA2 layer of "DeepSeek-V4.1-Flash: Pushing the
 * Limits of KV Cache Compression" (technical report, sections 2.3, 2.3.1,
 * 2.3.2 and 2.4.4), with the sizes given in the mer.dev notes on the same
 * report (section 1 setup, section 2 byte layout, section 4):
 *   - lightning-indexer score of every visible entry,
 *       s[j] = sum_h w[h] * ReLU(q_h . k_j)   (32 heads x 128, MXFP4 q and k)
 *   - optional hierarchical candidate pool (top 2,048 blocks of 8 positions
 *     by block-max score) that restricts later Reindex layers;
 *   - Top-512 selection;
 *   - 64-head, head-dim-512 attention in which the selected 512-channel
 *     latents (E2M1 + one E4M3 scale per 16 channels) serve as both K and V,
 *     in one softmax with the 128-row FP8 sliding window of the layer.
 *
 * Conventions shared by every entry point
 *   - Every pointer is a caller-owned DEVICE pointer unless stated otherwise.
 *     No entry point allocates device memory. Scratch space is sized by the
 *     matching *_workspace_size function and passed in by the caller.
 *   - Every call is asynchronous and ordered on `stream` (a cudaStream_t;
 *     NULL is the legacy default stream). A return of CSA2_OK means the work
 *     was enqueued; errors found by the kernels themselves (an index out of
 *     range, a bounded wait that ran out) are recorded in a sticky device
 *     word that csa2_get_last_error() reads and clears.
 *   - Host-side argument checks return a negative status and enqueue nothing.
 *   - bf16 arrays are passed as `const void*` holding IEEE bfloat16 values.
 *   - Packed FP4: element 2i of a row is the low nibble of byte i, element
 *     2i+1 the high nibble.
 *   - Cache planes are struct-of-arrays, one plane per field, sequences
 *     `cap` entries apart:
 *         ik_data  [B][cap][64]  E2M1 indexer key       (64 B / entry)
 *         ik_scale [B][cap][4]   E8M0, one per 32       ( 4 B / entry)
 *         kv_data  [B][cap][256] E2M1 main-KV latent    (256 B / entry)
 *         kv_scale [B][cap][32]  E4M3, one per 16       ( 32 B / entry)
 *     which is 68 + 288 = 356 bytes per entry as in the notes' section 2.
 *     `cap` must be a multiple of CSA2_CAP_ALIGN and plane base pointers
 *     16-byte aligned; entries at positions >= n_visible[b] may hold any
 *     bytes and are never selected.
 *   - Rounding of the encoders: round-to-nearest-even, saturating at the
 *     largest finite value; inputs must be finite.
 */
#ifndef CSA2_H
#define CSA2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/** A cudaStream_t. */
typedef struct CUstream_st* csa2_stream_t;

/* status codes */
#define CSA2_OK 0
#define CSA2_ERR_INVALID_ARG (-1)      /* null pointer, negative size, bad value   */
#define CSA2_ERR_UNSUPPORTED_SHAPE (-2) /* a size outside what the kernels support  */
#define CSA2_ERR_ALIGNMENT (-3)        /* pointer or capacity not aligned          */
#define CSA2_ERR_CUDA (-4)             /* a CUDA runtime call or launch failed     */
#define CSA2_ERR_TIMEOUT (-5)          /* a bounded device-side wait ran out       */
#define CSA2_ERR_WORKSPACE (-6)        /* workspace too small or misaligned        */
#define CSA2_ERR_DEVICE (-7)           /* a kernel rejected an input (e.g. index)  */
#define CSA2_ERR_SCRATCH_LIMIT (-8)    /* problem needs more than the static scratch */

/* sizes fixed by the method (notes section 1 setup) */
#define CSA2_IDX_HEADS 32
#define CSA2_IDX_DIM 128
#define CSA2_HEADS 64
#define CSA2_HEAD_DIM 512
#define CSA2_TOPK 512
#define CSA2_SWA 128
#define CSA2_POOL_BLOCK 8
#define CSA2_POOL_BLOCKS 2048
#define CSA2_CAP_ALIGN 128
#define CSA2_MAX_TOPK 4096

/** Library version, major*10000 + minor*100 + patch. */
int csa2_version(void);

/** A static string naming a status code. */
const char* csa2_status_string(int status);

/**
 * Waits for `stream`, then reads and clears the sticky device error words of
 * all kernels. *device_status receives CSA2_OK or the first negative status a
 * kernel recorded. Returns CSA2_ERR_CUDA if the synchronisation failed.
 */
int csa2_get_last_error(csa2_stream_t stream, int* device_status);

/* ======================================================================== */
/* FP4 / FP8 codecs                                                          */
/* ======================================================================== */

/**
 * MXFP4 quantisation (report section 2.4.4: OCP-standard MXFP4 for indexer
 * queries and keys; notes section 2: one E8M0 scale per 32 elements).
 * x [rows][cols] bf16 -> data [rows][cols/2] packed E2M1, e8m0 [rows][cols/32].
 * Per 32-element block: X = floor(log2(amax)) - 2 clamped to [-127, 127]
 * (X = -127 for an all-zero block), scale byte X + 127, element
 * RNE_E2M1(x * 2^-X) saturating at +-6. cols must be a positive multiple of
 * 32. Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA.
 */
int csa2_quant_mxfp4(const void* x_bf16, int64_t rows, int32_t cols,
                     uint8_t* data, uint8_t* e8m0, csa2_stream_t stream);

/** Inverse of csa2_quant_mxfp4: out [rows][cols] fp32 = e2m1 * 2^(e - 127). */
int csa2_dequant_mxfp4(const uint8_t* data, const uint8_t* e8m0, int64_t rows,
                       int32_t cols, float* out, csa2_stream_t stream);

/**
 * Main-KV packing (report section 2.4.4: E2M1 with one E4M3 scale per 16
 * channels, NVFP4 without its second-level global scale).
 * x [n][512] bf16 -> kv_data [n][256], kv_scale [n][32].
 * Per 16-channel block: s = RNE_E4M3(amax / 6) with the quotient in IEEE
 * fp32; element RNE_E2M1(x / s) in fp32 saturating at +-6; s == 0 gives an
 * all-zero block. Errors: INVALID_ARG, CUDA.
 */
int csa2_pack_kv_fp4(const void* x_bf16, int64_t n, uint8_t* kv_data,
                     uint8_t* kv_scale, csa2_stream_t stream);

/** Inverse of csa2_pack_kv_fp4: out [n][512] bf16 = e2m1 * e4m3 (exact). */
int csa2_unpack_kv_fp4(const uint8_t* kv_data, const uint8_t* kv_scale,
                       int64_t n, void* out_bf16, csa2_stream_t stream);

/**
 * SWA KV in FP8 (report section 2.4.4, last paragraph: SWA KV stays FP8).
 * x [n] bf16 -> out [n] E4M3 bytes, RNE saturating at +-448, no scale.
 */
int csa2_pack_fp8_e4m3(const void* x_bf16, int64_t n, uint8_t* out,
                       csa2_stream_t stream);

/** Inverse of csa2_pack_fp8_e4m3: out [n] bf16 (exact). */
int csa2_unpack_fp8_e4m3(const uint8_t* in, int64_t n, void* out_bf16,
                         csa2_stream_t stream);

/**
 * Fused KV append (report section 2.4.4: the main-KV latent is quantised
 * after RoPE into E2M1 with one E4M3 scale per 16 channels, no global scale;
 * the indexer key into OCP MXFP4): T new entries per sequence, written at
 * positions n_visible[b] .. n_visible[b] + T - 1 of its planes.
 *   kv_bf16 [B][T][512] bf16 (the RoPE'd latents, 16-byte aligned),
 *   ik_bf16 [B][T][128] bf16 (the indexer keys, 16-byte aligned);
 *   kv planes [B][cap][256] / [B][cap][32] (kv_data 8-byte aligned),
 *   ik planes [B][cap][64] / [B][cap][4] (ik_data 16-byte aligned);
 *   n_visible [B] int32; n_visible_out [B] int32 (nullable) receives
 *   n_visible + T. It may be n_visible itself (advanced in place).
 * The bytes written equal csa2_pack_kv_fp4 and csa2_quant_mxfp4 of the same
 * rows. A sequence whose T entries do not fit below cap gets none of them and
 * keeps its count; csa2_get_last_error then reports DEVICE.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE (cap above 2^31-1), ALIGNMENT, CUDA.
 */
int csa2_kv_append(const void* kv_bf16, const void* ik_bf16, int32_t B,
                   int32_t T, uint8_t* kv_data, uint8_t* kv_scale,
                   uint8_t* ik_data, uint8_t* ik_scale, int64_t cap,
                   const int32_t* n_visible, int32_t* n_visible_out,
                   csa2_stream_t stream);

/**
 * Sequence compressor of the encoder's Full layers (the paperglide summary of
 * DeepSeek-V4, "Compressed Sparse Attention": every m tokens merge into one
 * compressed entry; the notes' section 4.1: CSA2 blocks do not overlap and
 * the merge is softmax-weighted). For entry e (tokens em .. em+m-1) and
 * channel c:  w_a = softmax_a( Z[em+a][c] + bias[a][c] ),
 *             entry[e][c] = sum_a w_a * C[em+a][c]   (fp32),
 * rounded to bf16 and packed as the main-KV latent (E2M1 + E4M3/16, the bytes
 * csa2_pack_kv_fp4 writes for that bf16 row).
 *   c_bf16, z_bf16 [n_tokens][512] bf16 (16-byte aligned), bias [m][512]
 *   fp32 (16-byte aligned); n_tokens a multiple of m. Entries 0 .. n_tokens/m - 1 of kv_data
 *   [..][256] (8-byte aligned) and kv_scale [..][32] are written (offset the
 *   plane pointers to append); out_bf16 [n_tokens/m][512] (nullable, 16-byte
 *   aligned) receives the bf16 entries.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE (n_tokens % m), ALIGNMENT, CUDA.
 */
int csa2_compress_kv(const void* c_bf16, const void* z_bf16, const float* bias,
                     int64_t n_tokens, int32_t m, uint8_t* kv_data,
                     uint8_t* kv_scale, void* out_bf16, csa2_stream_t stream);

/* ======================================================================== */
/* Lightning indexer, pool and Top-K                                         */
/* ======================================================================== */

/**
 * Indexer scores (report sections 2.3 and 2.3.2; notes section 4.1 and 4.4:
 * 32 x 128 multiply-adds per query-entry pair).
 *   s[b][i] = sum_h w[b][h] * ReLU( sum_c qhat[b][h][c] * khat[b][p][c] )
 * with p = i (positions == NULL) or p = positions[b][i] (a Reindex layer
 * scoring its candidate pool). qhat, khat are the MXFP4 values.
 *   q_data [B][32][64], q_e8m0 [B][32][4]  (from csa2_quant_mxfp4)
 *   w [B][32] fp32 head weights
 *   ik planes with capacity `cap`, n_visible [B] int32 (0 <= n_visible <= cap)
 *   positions [B][n_pos] int32 or NULL
 *   scores [B][n_pos] fp32 out; -inf where p < 0 or p >= n_visible[b].
 * Errors: INVALID_ARG, ALIGNMENT (cap or plane pointers), CUDA.
 */
int csa2_index_score(const uint8_t* q_data, const uint8_t* q_e8m0,
                     const float* w, int32_t B, const uint8_t* ik_data,
                     const uint8_t* ik_scale, int64_t cap,
                     const int32_t* n_visible, const int32_t* positions,
                     int64_t n_pos, float* scores, csa2_stream_t stream);

/**
 * The same scores as csa2_index_score with positions == NULL, with another
 * schedule. csa2_index_score gives each CTA a fixed range of a sequence's
 * 128-entry tiles. Here, after one fixed pipeline depth, the CTAs of a
 * sequence claim tiles two at a time from a counter, so CTAs with a larger
 * share of the memory bandwidth take more (csa2_index_topk schedules its scan
 * this way, with counters in its workspace).
 *   tile_counters [2 * B] int32, device, 8-byte aligned, owned by the caller:
 *   all zero before the first call; every call that completes leaves them
 *   zero again. Calls that may run at the same time need their own buffers.
 *   Other arguments as csa2_index_score (n_pos <= cap).
 * Errors: INVALID_ARG (also a NULL tile_counters), ALIGNMENT, CUDA.
 */
int csa2_index_score_claimed(const uint8_t* q_data, const uint8_t* q_e8m0,
                             const float* w, int32_t B, const uint8_t* ik_data,
                             const uint8_t* ik_scale, int64_t cap,
                             const int32_t* n_visible, int64_t n_pos,
                             float* scores, int32_t* tile_counters,
                             csa2_stream_t stream);

/**
 * Bytes of workspace csa2_topk needs for B rows of n scores and a given k.
 */
size_t csa2_topk_workspace_size(int32_t B, int64_t n, int32_t k);

/**
 * Top-K per row (report section 2.3: the indexer selects the Top-K entries
 * for each query; K = 512 in the notes' setup).
 *   scores [B][n] fp32; an element is a candidate when its score is neither
 *   NaN nor -inf, its column is < n_valid[b] (n_valid may be NULL) and its
 *   position is >= 0. position = positions[b][i] (or i when NULL).
 *   idx [B][k] int32 out: the positions of the k largest candidates, ties
 *   broken by smaller position, written in ascending position order and
 *   padded with -1 at the end when fewer than k candidates exist.
 * 1 <= k <= CSA2_MAX_TOPK. The result is deterministic.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, WORKSPACE, CUDA.
 */
int csa2_topk(const float* scores, int32_t B, int64_t n,
              const int32_t* n_valid, const int32_t* positions, int32_t k,
              int32_t* idx, void* workspace, size_t workspace_bytes,
              csa2_stream_t stream);

/**
 * Top-K that allocates nothing and takes no workspace: the same selection as
 * csa2_topk (same arguments, same result), with its scratch held in a fixed
 * device buffer of CSA2_TOPK_STATIC_SCRATCH_BYTES that lives inside this
 * library. The report has no counterpart of this entry point; it exists for
 * callers that may not allocate device memory at all -- for example a plugin
 * whose host engine owns every device allocation and hands it only input and
 * output buffers, or a serving loop that must not pay cudaMalloc's implicit
 * device synchronisation on its request path.
 *   - Every GPU that loads the library holds the buffer until the process
 *     exits.
 *   - The first call on a device looks up the buffer's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture. The address is kept for the life of the
 *     process: it is not valid after cudaDeviceReset, so a caller that resets
 *     a device must not call this entry point on it again.
 *   - All calls share the one buffer and it keeps the last call's contents;
 *     the call clears what must start at zero. Calls that overlap on the GPU
 *     (different streams, or different host threads) race on the buffer:
 *     order them on one stream.
 *   - Returns CSA2_ERR_SCRATCH_LIMIT when csa2_topk_workspace_size(B, n, k)
 *     exceeds CSA2_TOPK_STATIC_SCRATCH_BYTES (32 MiB: at k = 512, up to 61
 *     rows of 65,536 scores fit), and otherwise the errors of csa2_topk.
 */
#define CSA2_TOPK_STATIC_SCRATCH_BYTES (32u << 20)
int csa2_topk_static(const float* scores, int32_t B, int64_t n,
                     const int32_t* n_valid, const int32_t* positions,
                     int32_t k, int32_t* idx, csa2_stream_t stream);

/** Bytes of workspace csa2_block_pool needs. */
size_t csa2_block_pool_workspace_size(int32_t B, int64_t n, int32_t block,
                                      int32_t n_blocks);

/**
 * Hierarchical candidate pool (report section 2.3.2 and Figure 5: each block
 * takes the maximum index score among its positions; the best blocks form
 * the pool, e.g. 2,048 blocks of 8 = 16,384 positions).
 *   scores [B][n] fp32 from the Full layer's scan; block b covers positions
 *   [block*b, block*b + block) within [0, n_visible[b]).
 *   pool [B][n_blocks * block] int32 out: the positions of the n_blocks
 *   blocks with the largest block maxima (ties: smaller block id), blocks in
 *   ascending order, -1 past n_visible and in unused slots.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, WORKSPACE, CUDA.
 */
int csa2_block_pool(const float* scores, int32_t B, int64_t n,
                    const int32_t* n_visible, int32_t block, int32_t n_blocks,
                    int32_t* pool, void* workspace, size_t workspace_bytes,
                    csa2_stream_t stream);

/**
 * Block maxima (report section 2.3.2: a block's score is the maximum index
 * score among its positions).
 *   bmax[b][j] = max of the non-NaN scores[b][block*j .. block*j+block) within
 *   [0, n_visible[b]) (n_visible may be NULL: all n), -inf for none.
 *   bmax [B][ceil(n / block)] fp32 out. Errors: INVALID_ARG, CUDA.
 */
int csa2_block_max(const float* scores, int32_t B, int64_t n,
                   const int32_t* n_visible, int32_t block, float* bmax,
                   csa2_stream_t stream);

/* ======================================================================== */
/* Context sharding: the exchange steps of a step split across ranks          */
/* ======================================================================== */
/* A rank owns the contiguous entries [lo, hi) of every sequence (its planes
 * hold them at local positions 0 .. hi-lo-1). Exact because a global Top-K
 * winner is in its own range's local Top-K (report section 2.3: Top-K over
 * all entries; section 2.3.2: the best blocks likewise), and attention over
 * disjoint row sets merges by log-sum-exp (section 2.3: one softmax over the
 * selected and SWA rows). A candidate is an 8-byte pair {fp32 score, int32
 * global position}; -1 marks an empty slot (its score is -inf). */

/**
 * Candidates of a local Top-K: cand[b][j] = {scores[b][c], pos(c) + offset}
 * for c = idx[b][j], pos(c) = positions[b][c] (positions non-NULL) or c;
 * {-inf, -1} where c < 0, c >= n or pos(c) < 0.
 *   scores [B][n] fp32, positions [B][n] int32 or NULL, idx [B][k] int32
 *   columns (from csa2_topk without positions), cand [B][k] pairs out
 *   (8-byte aligned). Errors: INVALID_ARG, UNSUPPORTED_SHAPE (a position
 *   above 2^31-1), ALIGNMENT, CUDA.
 */
int csa2_topk_candidates(const float* scores, int32_t B, int64_t n,
                         const int32_t* positions, const int32_t* idx,
                         int32_t k, int64_t offset, void* cand,
                         csa2_stream_t stream);

/** Bytes of workspace csa2_topk_merge needs. */
size_t csa2_topk_merge_workspace_size(int32_t R, int32_t B, int32_t k,
                                      int32_t k_out);

/**
 * Merge of R ranks' candidates: idx[b] = the global positions of the k_out
 * best candidates of row b over all ranks, as csa2_topk orders and pads them
 * (ascending position, -1 at the end).
 *   cand [R][B][k] pairs (each rank's csa2_topk_candidates, gathered in rank
 *   order), idx [B][k_out] int32 out, 1 <= k_out <= CSA2_MAX_TOPK.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, WORKSPACE, CUDA.
 */
int csa2_topk_merge(const void* cand, int32_t R, int32_t B, int32_t k,
                    int32_t k_out, int32_t* idx, void* workspace,
                    size_t workspace_bytes, csa2_stream_t stream);

/**
 * local_idx[b][j] = idx[b][j] - lo when lo <= idx[b][j] < hi, else -1: the
 * merged global positions that fall into this rank's range, as local ones
 * (the attention's idx).
 *   idx, local_idx [B][k] int32. Errors: INVALID_ARG, CUDA.
 */
int csa2_shard_positions(const int32_t* idx, int32_t B, int32_t k,
                         int64_t lo, int64_t hi, int32_t* local_idx,
                         csa2_stream_t stream);

/**
 * The merged pool restricted to this rank: for the global block ids
 * blocks[b][j] (-1 = unused), pool[b][j*block + r] = p - lo for the position
 * p = blocks[b][j]*block + r when lo <= p < hi and p - lo < n_visible[b]
 * (n_visible local, may be NULL), else -1.
 *   blocks [B][n_blocks] int32, pool [B][n_blocks*block] int32 out.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA.
 */
int csa2_shard_pool(const int32_t* blocks, int32_t B, int32_t n_blocks,
                    int32_t block, int64_t lo, int64_t hi,
                    const int32_t* n_visible, int32_t* pool,
                    csa2_stream_t stream);

/**
 * Merges R partial attention outputs of disjoint row sets in rank order
 * 0..R-1: out = sum_r exp(lse_r - L) / S * o_r with L = max_r lse_r,
 * S = sum_r exp(lse_r - L); lse_out = L + log S. A set with lse = -inf (no
 * rows) contributes nothing; a query-head with no rows at all gets 0, -inf.
 *   parts [R][n_q][64][512] fp32 (each rank's out_f32, 16-byte aligned),
 *   lses [R][n_q][64] fp32 (each rank's lse), out_bf16 [n_q][64][512] out
 *   (8-byte aligned), out_f32 (nullable, 16-byte aligned) and lse_out
 *   [n_q][64] (nullable). Errors: INVALID_ARG, ALIGNMENT, CUDA.
 */
int csa2_attn_merge(const float* parts, const float* lses, int32_t R,
                    int32_t n_q, void* out_bf16, float* out_f32,
                    float* lse_out, csa2_stream_t stream);

/** Bytes of workspace csa2_index_topk needs (pool_blocks 0 = no pool). */
size_t csa2_index_topk_workspace_size(int32_t B, int64_t n_pos, int32_t k,
                                      int32_t pool_blocks);

/**
 * Fused indexer scan + Top-K (+ pool): the Full-layer and Reindex-layer
 * index path of report section 2.3.1 in one call. Arguments as in
 * csa2_index_score and csa2_topk; if pool != NULL and pool_blocks > 0 the
 * call also builds the block pool [B][pool_blocks * CSA2_POOL_BLOCK] from the
 * same scores (only meaningful when positions == NULL).
 * Errors: as csa2_index_score and csa2_topk.
 */
int csa2_index_topk(const uint8_t* q_data, const uint8_t* q_e8m0,
                    const float* w, int32_t B, const uint8_t* ik_data,
                    const uint8_t* ik_scale, int64_t cap,
                    const int32_t* n_visible, const int32_t* positions,
                    int64_t n_pos, int32_t k, int32_t* idx,
                    int32_t pool_blocks, int32_t* pool, void* workspace,
                    size_t workspace_bytes, csa2_stream_t stream);

/**
 * csa2_index_topk with the indexer q given in bf16: the scan quantises it to
 * MXFP4 in its prologue with the same block encoder as csa2_quant_mxfp4 (same
 * bytes, so the same scores and indices), saving that kernel and its launch.
 *   q_bf16 [B][32][128] bf16 (16-byte aligned); the rest as csa2_index_topk.
 */
int csa2_index_topk_bf16(const void* q_bf16, const float* w, int32_t B,
                         const uint8_t* ik_data, const uint8_t* ik_scale,
                         int64_t cap, const int32_t* n_visible,
                         const int32_t* positions, int64_t n_pos, int32_t k,
                         int32_t* idx, int32_t pool_blocks, int32_t* pool,
                         void* workspace, size_t workspace_bytes,
                         csa2_stream_t stream);

/**
 * Prefill indexer scores with causal masking (report section 2.3; the
 * encoder-side prefill indexer cost in notes section 4.4 item 4).
 * T queries at positions p0 .. p0+T-1 of one sequence; query t sees entries
 * 0 .. p0+t (itself included).
 *   q_data [T][32][64] (16-byte aligned), q_e8m0 [T][32][4], w [T][32]
 *   ik planes of the sequence with n_entries >= p0 + T entries (ik_data
 *     16-byte aligned, ik_scale 4-byte aligned; no padding rows needed)
 *   scores [T][n_entries] fp32 out, -inf beyond each query's prefix.
 * Runs on the tensor cores: blocks of 32 queries against 128-entry key
 * tiles (block-scaled MXF4 products), a fp32 ReLU-weighted epilogue.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_SHAPE (T*32 or n_entries above
 * 2^31-1), CUDA; a bounded device wait that runs out is reported by
 * csa2_get_last_error as TIMEOUT.
 */
int csa2_prefill_index_score(const uint8_t* q_data, const uint8_t* q_e8m0,
                             const float* w, int32_t T,
                             const uint8_t* ik_data, const uint8_t* ik_scale,
                             int64_t n_entries, int64_t p0, float* scores,
                             csa2_stream_t stream);

/**
 * Prefill indexer scores over compressed entries (notes section 4.4 item 4:
 * the encoder's Full layers score each query against the visible compressed
 * entries, about 3,072 N^2 multiply-adds at m = 2): as
 * csa2_prefill_index_score with p0 the token position of query 0 and m tokens
 * per entry; query t sees the complete entries j < floor((p0 + t + 1) / m).
 * m = 1 is csa2_prefill_index_score. Requires floor((p0 + T) / m) <= n_entries.
 * Errors: as csa2_prefill_index_score.
 */
int csa2_prefill_index_score_compressed(const uint8_t* q_data,
                                        const uint8_t* q_e8m0, const float* w,
                                        int32_t T, const uint8_t* ik_data,
                                        const uint8_t* ik_scale,
                                        int64_t n_entries, int64_t p0,
                                        int32_t m, float* scores,
                                        csa2_stream_t stream);

/* ======================================================================== */
/* Sparse attention                                                          */
/* ======================================================================== */

/** Bytes of workspace the attention entry points need for n_queries
 *  (query-layers in decode, queries in prefill). */
size_t csa2_sparse_attn_workspace_size(int32_t n_queries, int32_t k,
                                       int32_t n_swa);

/** Kernel launches one attention call makes for n_queries on the current
 *  device (one per batch of up to 256 queries); 0 for invalid sizes. */
int csa2_sparse_attn_kernel_launches(int32_t n_queries, int32_t k,
                                     int32_t n_swa);

/**
 * Sparse decode attention (report section 2.3: each query attends to the
 * selected entries together with the layer-local SWA KV; section 2.3.1:
 * Reuse layers use the Top-K of the preceding indexing layer with their own
 * query and SWA KV; notes section 1: 64 heads of dim 512, the 512-dim latent
 * shared as K and V).
 *   q [B][L][64][512] bf16: the L layers of sequence b share idx[b]
 *     (L = 1 for one layer, 4 for 1 Full + 3 Reuse).
 *   kv planes with capacity cap; n_visible [B]; idx [B][k] int32 positions
 *     (-1 entries are skipped; a position >= n_visible[b] is a device error).
 *   swa [B][L][n_swa][512] E4M3 bytes (0 <= n_swa <= 512).
 *   S = sm_scale * q . row over the k selected rows and the n_swa SWA rows,
 *   one softmax, out = P . rows.
 *   out [B][L][64][512] bf16; out_f32 (nullable) the same before the bf16
 *   rounding; lse (nullable) [B][L][64] natural-log sum of exp(S), -inf for
 *   a query with no rows (its output is 0).
 *   k <= CSA2_MAX_TOPK, n_swa <= 512. q, swa and out_f32 16-byte aligned,
 *   out 8-byte aligned, the planes 16-byte aligned as in the conventions above.
 *   q and the swa rows are read before this call waits for the kernel just
 *   before it on the stream (the indices and n_visible are read after): they
 *   must not be written by that kernel when it is one of this library's
 *   attention or merge kernels (which let their successor start early); the
 *   packers, csa2_rope and anything launched without programmatic dependence
 *   are safe.
 *   Precision: rows and q enter the tensor cores as fp16 (exact: the row
 *   values have at most 6 significant bits, q is scaled by a power of two per
 *   head), P as fp16 (relative rounding 2^-11), fp32 accumulation.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, WORKSPACE, CUDA.
 */
int csa2_sparse_attn_decode(const void* q_bf16, int32_t B, int32_t L,
                            const uint8_t* kv_data, const uint8_t* kv_scale,
                            int64_t cap, const int32_t* n_visible,
                            const int32_t* idx, int32_t k, const uint8_t* swa,
                            int32_t n_swa, float sm_scale, void* out_bf16,
                            float* out_f32, float* lse, void* workspace,
                            size_t workspace_bytes, csa2_stream_t stream);

/**
 * Fused Reuse-layer decode attention (report section 2.3.1: the Reuse layers
 * of a sequence attend to the selection of its Full layer, each with its own
 * query and SWA KV; notes section 4.2: they share that selection): the same
 * arguments, results and limits as csa2_sparse_attn_decode, computed with one
 * cluster of CTAs per sequence in which every 128-row tile of selected
 * entries is gathered and dequantised once per pair of layers (once for all
 * L when L is odd) instead of once per layer. The partials of one layer are
 * the same as csa2_sparse_attn_decode's and are merged in the same order, so
 * the outputs are bit-identical to that call's.
 * When to use it: the per-layer call spreads the layers over more CTAs and
 * is faster at small batches; this call does less gather and dequantisation
 * work and is faster once the per-layer call fills the device several times
 * over (measured on GB300 at k = 512, 128 SWA rows: L = 2, B = 64: 81 vs
 * 91 us; L = 4 only at parity from B = 64).
 * Errors: those of csa2_sparse_attn_decode, and UNSUPPORTED_SHAPE when one
 * cluster (at most 8 CTAs) cannot hold the merge of the L x 64 (layer, head)
 * rows: L > 8, or k and n_swa so large that the tiles' (max, sum) pairs do
 * not fit its table ((ceil(k/128) + ceil(n_swa/128)) * ceil(64 L / C) > 576
 * for the cluster size C = min(8, the sequence's work items)).
 */
int csa2_sparse_attn_reuse(const void* q_bf16, int32_t B, int32_t L,
                           const uint8_t* kv_data, const uint8_t* kv_scale,
                           int64_t cap, const int32_t* n_visible,
                           const int32_t* idx, int32_t k, const uint8_t* swa,
                           int32_t n_swa, float sm_scale, void* out_bf16,
                           float* out_f32, float* lse, void* workspace,
                           size_t workspace_bytes, csa2_stream_t stream);

/**
 * Sparse prefill attention: T queries of one sequence, each with its own
 * Top-K and its own causal SWA window.
 *   q [T][64][512] bf16; kv planes of the sequence with n_entries entries;
 *   idx [T][k]; swa [T + n_swa - 1][512] E4M3 where query t uses rows
 *   t .. t + n_swa - 1 (the last one is the query's own position).
 *   out/out_f32/lse as in csa2_sparse_attn_decode with [T] leading.
 * Errors: as csa2_sparse_attn_decode.
 */
int csa2_sparse_attn_prefill(const void* q_bf16, int32_t T,
                             const uint8_t* kv_data, const uint8_t* kv_scale,
                             int64_t n_entries, const int32_t* idx, int32_t k,
                             const uint8_t* swa, int32_t n_swa, float sm_scale,
                             void* out_bf16, float* out_f32, float* lse,
                             void* workspace, size_t workspace_bytes,
                             csa2_stream_t stream);

/**
 * Sparse prefill attention with the Bounded-Replay SWA mask (notes section 6:
 * after the SWA cache of a prefix was evicted, only the last n_win tokens are
 * replayed and the sliding window is cut at the replay start s, so the query
 * at position i sees SWA positions [max(s, i - W + 1), i]).
 *   As csa2_sparse_attn_prefill, with replay_row >= 0 the first row of the swa
 *   array inside the replay segment: query t uses rows
 *   max(t, replay_row) .. t + n_swa - 1. With swa row r holding position
 *   p0 - (n_swa - 1) + r, replay_row = s - p0 + n_swa - 1 (0: no truncation).
 * Errors: as csa2_sparse_attn_decode.
 */
int csa2_sparse_attn_prefill_replay(const void* q_bf16, int32_t T,
                                    const uint8_t* kv_data,
                                    const uint8_t* kv_scale, int64_t n_entries,
                                    const int32_t* idx, int32_t k,
                                    const uint8_t* swa, int32_t n_swa,
                                    int32_t replay_row, float sm_scale,
                                    void* out_bf16, float* out_f32, float* lse,
                                    void* workspace, size_t workspace_bytes,
                                    csa2_stream_t stream);

/* ======================================================================== */
/* The cache in pages                                                        */
/* ======================================================================== */
/* Entries of many sequences in one pool of pages. The planes are
 *     kv_data [n_pages][page_size][256], kv_scale [n_pages][page_size][32],
 *     ik_data [n_pages][page_size][64],  ik_scale [n_pages][page_size][4],
 * an entry being laid out as in the planes of the conventions above. Entry e of
 * sequence b is row e % page_size of page page_table[b][e / page_size].
 *   - page_size is a power of two, at least CSA2_MIN_PAGE. A pool holds at most
 *     2^31 - 1 entries. Plane base pointers are 16-byte aligned; a pool without
 *     pages needs none.
 *   - page_table [B][max_pages] int32. Only the table's first
 *     ceil(n / page_size) places of a sequence with n entries are read; the
 *     others may hold anything. A page outside [0, n_pages) that is needed is
 *     not followed: the entry point says what happens to its entries, and
 *     csa2_get_last_error then reports DEVICE. Sequences may share pages that
 *     are only read.
 *   - cu [B+1] int32, rising, gives each sequence its run of token rows:
 *     sequence b has rows cu[b] .. cu[b+1]-1. NULL: n_tokens / B rows each (B
 *     must divide n_tokens). Rows before cu[0] and from cu[B] on belong to
 *     no sequence: they are neither read nor written. A sequence whose run is
 *     not within 0 .. n_tokens is passed over and reported as DEVICE.
 *   - Position rotation: a row x of d channels at position p has its last
 *     rope_dim channels turned, pair i by the angle whose cosine and sine are
 *     rope[p][i][0] and rope[p][i][1] (fp32, [n_rope][rope_dim/2][2],
 *     16-byte aligned):
 *         (u, v) -> (u cos - v sin, u sin + v cos).
 *     Pair i is channels (2i, 2i+1) of the turned part when `interleaved` is
 *     not 0, else channels (i, i + rope_dim/2). rope_dim is a multiple of 32.
 *     A turned value is held in fp32, rounded once. */

#define CSA2_MIN_PAGE 16
#define CSA2_MAX_ROPE_DIM 128

/**
 * Position rotation of [n_tokens][heads][dim] bf16 rows (queries, indexer
 * queries, or with `inverse` attention outputs turned back: the latent is key
 * and value at once, so an output carries its entries' rotation). The turned
 * channels are rounded to bf16, the others copied. (Report section 2.4.4: the
 * main-KV latent has RoPE and non-RoPE channels.)
 *   positions [n_tokens] int32, NULL: row t is at position t. A token whose
 *   position is not within 0 .. n_rope-1 keeps its output as it was and is
 *   reported as DEVICE.
 *   x_bf16, out_bf16 16-byte aligned; out may be x (not overlap it otherwise).
 *   dim is a multiple of 8, at least rope_dim; rope_dim 32 .. CSA2_MAX_ROPE_DIM.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CUDA.
 */
int csa2_rope(const void* x_bf16, int64_t n_tokens, int32_t heads, int32_t dim,
              const float* rope, int64_t n_rope, int32_t rope_dim,
              const int32_t* positions, int32_t interleaved, int32_t inverse,
              void* out_bf16, csa2_stream_t stream);

/**
 * KV append into pages: csa2_kv_append for ragged batches, with the position
 * rotation applied on the way (report section 2.4.4: the latent is quantised
 * after RoPE, with one format for RoPE and non-RoPE channels). Token t of
 * sequence b becomes its entry n_visible[b] + t.
 *   kv_bf16 [n_tokens][512], ik_bf16 [n_tokens][128] (16-byte aligned): the
 *   last rope_dim channels of each are turned at the token's position, then
 *   encoded as csa2_pack_kv_fp4 and csa2_quant_mxfp4 encode (from the fp32
 *   values: no rounding to bf16 in between). rope_dim 0 or rope NULL: rows are
 *   taken as they are, and the bytes equal csa2_kv_append's.
 *   positions [n_tokens] int32, NULL: a token's position is its entry's index.
 *   n_visible [B] int32; n_visible_out [B] int32 (nullable) receives n_visible
 *   plus the sequence's new tokens; it may be n_visible itself.
 * A sequence whose tokens do not fit below max_pages * page_size (or whose
 * count is negative) gets none of them and keeps its count. An entry whose page
 * is outside the pool or whose position is outside the table is not written
 * (the count still advances). Both are reported as DEVICE. Pages written by one
 * call must not be shared between its sequences.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CUDA.
 */
int csa2_paged_kv_append(const void* kv_bf16, const void* ik_bf16,
                         int32_t n_tokens, const int32_t* cu_tokens, int32_t B,
                         const float* rope, int64_t n_rope, int32_t rope_dim,
                         const int32_t* positions, int32_t interleaved,
                         uint8_t* kv_data, uint8_t* kv_scale, uint8_t* ik_data,
                         uint8_t* ik_scale, int64_t n_pages, int32_t page_size,
                         const int32_t* page_table, int32_t max_pages,
                         const int32_t* n_visible, int32_t* n_visible_out,
                         csa2_stream_t stream);

/**
 * csa2_index_score over pages: s[b][i] for entries i = 0 .. n_pos-1 of every
 * sequence, -inf from n_visible[b] on and for entries of a page outside the
 * pool (reported as DEVICE). n_pos <= max_pages * page_size.
 *   tile_counters: NULL, or [2 * B] int32 as in csa2_index_score_claimed (the
 *   CTAs of a sequence then claim its tiles; all zero before the first call,
 *   left zero by every call, one buffer per call that may run at the same time;
 *   a negative counter is reported as DEVICE and the scores of that sequence are
 *   not complete).
 * The scores feed csa2_topk and csa2_block_pool (with n_visible) as usual.
 * Errors: as csa2_index_score.
 */
int csa2_paged_index_score(const uint8_t* q_data, const uint8_t* q_e8m0,
                           const float* w, int32_t B, const uint8_t* ik_data,
                           const uint8_t* ik_scale, int64_t n_pages,
                           int32_t page_size, const int32_t* page_table,
                           int32_t max_pages, const int32_t* n_visible,
                           int64_t n_pos, float* scores,
                           int32_t* tile_counters, csa2_stream_t stream);

/** Bytes of workspace csa2_paged_sparse_attn_decode needs. */
size_t csa2_paged_sparse_attn_workspace_size(int32_t B, int32_t L, int32_t k,
                                             int32_t n_swa);

/**
 * csa2_sparse_attn_decode over pages: idx holds entries of the sequences
 * (from csa2_topk over csa2_paged_index_score); the results are those of that
 * call on flat planes of the same entries. An entry >= n_visible[b], or of a
 * page outside the pool, is skipped and reported as DEVICE.
 * Errors: as csa2_sparse_attn_decode.
 */
int csa2_paged_sparse_attn_decode(const void* q_bf16, int32_t B, int32_t L,
                                  const uint8_t* kv_data,
                                  const uint8_t* kv_scale, int64_t n_pages,
                                  int32_t page_size, const int32_t* page_table,
                                  int32_t max_pages, const int32_t* n_visible,
                                  const int32_t* idx, int32_t k,
                                  const uint8_t* swa, int32_t n_swa,
                                  float sm_scale, void* out_bf16,
                                  float* out_f32, float* lse, void* workspace,
                                  size_t workspace_bytes, csa2_stream_t stream);

/** Bytes of workspace csa2_paged_attn needs on the current device: the same for
 *  every n_tokens > 0 and B > 0, two parts of 128 KiB per SM and their lists
 *  (38 MiB on 152 SMs), 0 otherwise. One buffer serves calls of any size, one
 *  after another. */
size_t csa2_paged_attn_workspace_size(int32_t n_tokens, int32_t B);

/**
 * Dense attention over the paged FP4 cache: every query token attends to all
 * the entries that it sees (report section 2.3 with every entry selected; a
 * context no longer than the Top-K, or a layer without an index).
 *   q [n_tokens][64][512] bf16; sequence b's tokens are rows cu_q[b] ..
 *   cu_q[b+1]-1 (T of them). causal != 0: its token t sees entries
 *   0 .. n_visible[b] - T + t (the sequence's last T entries are the tokens'
 *   own; a token before entry 0 sees nothing). causal == 0: every token sees
 *   entries 0 .. n_visible[b]-1.
 *   S = sm_scale * q . row over those entries' latents (one latent for all 64
 *   heads), softmax, out = P . rows.
 *   out_bf16, out_f32 (nullable), lse (nullable, [n_tokens][64]) as in
 *   csa2_sparse_attn_decode: a token that sees nothing gets 0 and -inf. To
 *   join the sliding window, merge with csa2_attn_merge.
 *   Entries of a page outside the pool are left out of the softmax, a sequence
 *   whose n_visible is negative or above max_pages * page_size is passed over
 *   (its rows stay as they were); both are reported as DEVICE.
 *   q, out_bf16 and out_f32 16-byte aligned. q is finite.
 *   Precision: as csa2_sparse_attn_decode (rows and q exact in fp16, P in fp16).
 *   Results do not depend on the schedule but for the last bits: the entries of
 *   a token may be summed in parts whose bounds follow from the batch and the
 *   device. The same call gives the same bits.
 *   workspace: csa2_paged_attn_workspace_size bytes, 256-byte aligned, its
 *   contents need not be kept; calls that may run at the same time (graphs
 *   among them) need one each.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, WORKSPACE, CUDA; a
 * bounded device wait that runs out is reported by csa2_get_last_error as
 * TIMEOUT.
 */
int csa2_paged_attn(const void* q_bf16, int32_t n_tokens, const int32_t* cu_q,
                    int32_t B, const uint8_t* kv_data, const uint8_t* kv_scale,
                    int64_t n_pages, int32_t page_size,
                    const int32_t* page_table, int32_t max_pages,
                    const int32_t* n_visible, int32_t causal, float sm_scale,
                    void* out_bf16, float* out_f32, float* lse, void* workspace,
                    size_t workspace_bytes, csa2_stream_t stream);

/* ======================================================================== */
/* Products with 4-bit weights                                               */
/* ======================================================================== */

/* A matrix W [n_out][n_in] of packed weights: E2M1 codes [n_out][n_in/2] and scales
 *     CSA2_FP4_E8M0  one E8M0 per 32 inputs [n_out][n_in/32] (csa2_quant_mxfp4),
 *     CSA2_FP4_E4M3  one E4M3 per 16 inputs [n_out][n_in/16], not negative, not NaN
 *                    (csa2_pack_kv_fp4 over the matrix as rows of 512).
 * n_in is a multiple of 32, at most 2^30. */
#define CSA2_FP4_E8M0 0
#define CSA2_FP4_E4M3 1

/** Bytes of the laid-out form of an n_out x n_in matrix (rows rounded up to 128,
 *  inputs to 256); 0 for sizes or a format that are refused. */
size_t csa2_fp4_weights_size(int32_t n_out, int32_t n_in, int32_t format);

/**
 * Lays packed weights out for csa2_fp4_linear, once for a matrix: blocks of 128
 * rows x 256 inputs as the tensor cores read them, codes and scales unchanged.
 *   data, weights 16-byte aligned; weights has csa2_fp4_weights_size bytes, all of
 *   them written; it must not overlap data or scale.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CUDA.
 */
int csa2_fp4_weights(const uint8_t* data, const uint8_t* scale, int32_t n_out,
                     int32_t n_in, int32_t format, uint8_t* weights,
                     csa2_stream_t stream);

/** Bytes of workspace csa2_fp4_linear needs: the same for every n_out, and no fewer
 * for more tokens (one for the most does for all). */
size_t csa2_fp4_linear_workspace_size(int32_t n_tokens, int32_t n_in,
                                      int32_t format);

/**
 * out[t][n] = scale * sum_k x[t][k] * W[n][k]: the projections around the cache
 * (report section 2.3: latents, indexer keys and queries; notes section 4.4: FP4
 * weights), from one token, a matrix-vector product, to a prompt.
 *   x [n_tokens][n_in] bf16; weights from csa2_fp4_weights with the same n_out, n_in
 *   and format; out_bf16 and out_f32 [n_tokens][n_out], at least one of them
 *   (rounded from the same fp32 value).
 *   Precision: up to 64 tokens, a token's blocks of 32 (E8M0) or 16 (E4M3) channels
 *   enter as sums of eight E2M1 vectors: exact for channels within 2^-14 of their block's
 *   largest, off by at most 2^-22 of the largest otherwise (with E4M3 scales, or 2^-39 of
 *   the token's largest; with either, or 2^-121). More tokens enter as they are. The
 *   weights are exact, products too, sums are in fp32. A token with an infinity or a NaN
 *   has infinities or NaN in all its outputs; other tokens do not notice it. The same call
 *   gives the same bits; a token's result may differ in the last fp32 bits with the number
 *   of tokens.
 *   x, weights 16-byte aligned; the outputs must not overlap anything that is read.
 *   Whatever came before on the stream may have written x and weights.
 *   workspace: csa2_fp4_linear_workspace_size bytes, 256-byte aligned, contents
 *   need not be kept; calls that may run at the same time need one each.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, WORKSPACE, CUDA; a bounded device
 * wait that runs out is reported by csa2_get_last_error as TIMEOUT (the outputs then hold
 * anything).
 */
int csa2_fp4_linear(const void* x_bf16, int32_t n_tokens,
                    const uint8_t* weights, int32_t n_out, int32_t n_in,
                    int32_t format, float scale, void* out_bf16, float* out_f32,
                    void* workspace, size_t workspace_bytes,
                    csa2_stream_t stream);

/* ======================================================================== */
/* Beam search                                                               */
/* ======================================================================== */

#define CSA2_MAX_BEAMS 64
#define CSA2_MAX_BEAM_K 64

/** Bytes of workspace csa2_beam_select needs. */
size_t csa2_beam_select_workspace_size(int32_t B, int32_t W, int32_t V,
                                       int32_t k);

/**
 * Beam search's selection: for each of B sequences with W beams the k best of the
 * W * V candidates (w, v) by
 *     scores[b][w] + x[b][w][v] - log sum_u exp(x[b][w][u]),
 * falling, ties to the lowest w * V + v (W = 1: the k likeliest tokens of each row).
 *   logits: row b * W + w begins at element (b * W + w) * ld, ld >= V; bf16, or fp32
 *   with logits_f32 = 1. A logit of -inf is no candidate. A row whose logits are all
 *   -inf takes no part, nor does one whose score is not finite (a beam that is not in
 *   use); a row that holds a NaN or +inf takes none either and is reported as DEVICE.
 *   (A beam that has ended stands by itself with 0 for its end token and -inf for the
 *   others.)
 *   scores [B][W] fp32, NULL: 0. out_scores [B][k] fp32; out_parents [B][k] int32, the
 *   row b * W + w (what csa2_paged_reorder takes); out_tokens [B][k] int32. Behind the
 *   last candidate: -inf, -1, -1. lse (nullable) [B][W] fp32: the rows' log sums (NaN
 *   for one that holds a NaN or +inf).
 *   Sums are held in fp32, scores as sums of two fp32 values (48 bits) until they are
 *   written: candidates of one row are in exact order, those of different rows in that of
 *   their scores with log sums good to (V / 1024 + 160) 2^-23, 3.4e-5 for V = 128,000. (Rows
 *   that are alike tie exactly where they lie alike in memory: ld * the type's size a
 *   multiple of 16.) The result is deterministic.
 *   1 <= k <= CSA2_MAX_BEAM_K, 1 <= W <= CSA2_MAX_BEAMS, B * W < 2^23.
 *   workspace: csa2_beam_select_workspace_size bytes, 256-byte aligned; calls that may
 *   run at the same time need one each.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, WORKSPACE, CUDA.
 */
int csa2_beam_select(const void* logits, int32_t logits_f32, int32_t B,
                     int32_t W, int32_t V, int64_t ld, const float* scores,
                     int32_t k, float* out_scores, int32_t* out_parents,
                     int32_t* out_tokens, float* lse, void* workspace,
                     size_t workspace_bytes, csa2_stream_t stream);

/**
 * Reordering of paged sequences after a selection (or forking them): row r of the new
 * batch takes over the entries of row parents[r] of the old one. Full pages are
 * shared. The partly filled last page, which the next append writes, goes to the
 * lowest r with that parent; every other row gets its entries copied into page
 * fresh_pages[r].
 *   parents [R] int32, 0 .. rows_in-1; -1: row r is empty (its count is 0).
 *   fresh_pages [R] int32: looked at only where a copy is needed (page_table_out then
 *   holds it); those pages must be in use by nothing else, each given to one row.
 *   kv_data, kv_scale, ik_data, ik_scale: planes [layers][n_pages][page_size][..] of the
 *   pool, the layers' caches sharing one table; either pair may be NULL.
 *   page_table [rows_in][max_pages], n_visible [rows_in]; page_table_out [R][max_pages],
 *   n_visible_out [R], which must not overlap them. Only the first
 *   ceil(n / page_size) places of a row of page_table_out are written.
 *   A parent that is neither -1 nor a row, or whose count is negative or above
 *   max_pages * page_size, leaves row r's place and count as they were; a copy whose
 *   page or source is outside the pool leaves -1 in the table. Both are reported as
 *   DEVICE.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CUDA.
 */
int csa2_paged_reorder(const int32_t* parents, const int32_t* fresh_pages,
                       int32_t R, uint8_t* kv_data, uint8_t* kv_scale,
                       uint8_t* ik_data, uint8_t* ik_scale, int32_t layers,
                       int64_t n_pages, int32_t page_size,
                       const int32_t* page_table, int32_t rows_in,
                       int32_t max_pages, const int32_t* n_visible,
                       int32_t* page_table_out, int32_t* n_visible_out,
                       csa2_stream_t stream);

/**
 * dst[r] = src[parents[r]] for rows of row_bytes bytes: any other state of a sequence,
 * such as its layers' sliding windows [L][n_swa][512].
 *   src [rows_in][row_bytes], dst [R][row_bytes], 16-byte aligned, not overlapping;
 *   row_bytes a multiple of 16. parents[r] = -1 leaves row r as it was; another value
 *   that is no row too, and is reported as DEVICE.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CUDA.
 */
int csa2_reorder_rows(const void* src, int64_t rows_in, int64_t row_bytes,
                      const int32_t* parents, int32_t R, void* dst,
                      csa2_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_H */
