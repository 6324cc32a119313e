/*
 * dsa_indexer.h -- C ABI of the GB300 (sm_103a) DSA indexer library.
 *
 * The DeepSeek-Sparse-Attention indexer that GLM5's glm_moe_dsa layers run
 * scores every causal query/key pair and keeps each query's best keys
 * (GLM5 TensorCast adaptation design, section "DSA Indexer 融合语义算子";
 * cost buckets 6-10 of section "性能模型设计"):
 *
 *     x[t,h,s]   = sq[t,h] * sk[s] * sum_d q[t,h,d] * k[s,d]      (sq = sk = 1 for bf16)
 *     score[t,s] = sum_h w[t,h] * max(x[t,h,s], 0)                 for keys s <= pos(t)
 *     topk[t,:]  = the min(topk_limit, pos(t)+1) keys of highest score, ties to the
 *                  lower key index, then -1 up to k_out
 *
 * and GLM-5.2 IndexShare (same page, section "GLM-5.2 IndexShare"): a layer
 * typed "shared" runs no indexer and forwards the top-k of the nearest earlier
 * "full" layer unchanged.
 *
 * Conventions for every entry point:
 *  - Pointers named q, k, k_cache, w, scales, scores, topk, cu_q_lens,
 *    seq_lens, block_tables and workspace are DEVICE pointers, owned by the
 *    caller; the library keeps none of them after returning and allocates no
 *    device memory per call.  Held for the process lifetime once first used on a
 *    device: the fixed scratch array of dsa_indexer_static, the streams and events
 *    of dsa_indexer_dense_host, and the streams and events of dsa_indexer_prepare.
 *    Pointers named
 *    types / src / full_args / topk_out are host.
 *  - All work is enqueued on `stream` (NULL = legacy default stream) and is
 *    asynchronous; nothing synchronises except dsa_check_device_status.
 *  - Host-side validation happens before any launch; a failing call launches
 *    nothing and returns the status.
 *  - Device-side checks (a page id outside [0, num_pages), a key position that
 *    the block table does not cover, a bounded wait that gave up) never trap:
 *    the kernel records a bit in a library-owned device status word and skips
 *    the access; dsa_check_device_status reports and clears it.
 *  - Tensors are dense row-major with the strides implied by their shapes
 *    (only scores takes an explicit leading dimension).
 *  - Every device pointer must be 16-byte aligned; row pitches of q/k
 *    (D * element size) are then multiples of 16 bytes for the supported D.
 */
#ifndef DSA_INDEXER_H
#define DSA_INDEXER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* dsa_stream_t; /* the same handle as cudaStream_t */

typedef enum {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, bad indexer_types, ... */
    DSA_ERR_UNSUPPORTED = 2,      /* valid but not implemented: D, H, dtype mix, k_out */
    DSA_ERR_CUDA = 3,             /* a CUDA runtime/driver call or launch failed */
    DSA_ERR_DEVICE_CHECK = 4,     /* a kernel found a bad page id / uncovered key */
    DSA_ERR_TIMEOUT = 5,          /* a bounded device wait gave up */
    DSA_ERR_WORKSPACE = 6         /* workspace missing or smaller than required */
} dsa_status;

typedef enum { DSA_BF16 = 0, DSA_FP8_E4M3 = 1, DSA_FP4_E2M1 = 2 /* quantised latent cache only */ } dsa_dtype;

typedef enum { DSA_LAYER_FULL = 0, DSA_LAYER_SHARED = 1 } dsa_layer_type;

/* Output order of a top-k row.  Both are unique for a given score row.
 *  DSA_ORDER_SCORE: by (score desc, key index asc) -- torch.topk's sorted order with
 *                   deterministic ties (GLM5 LoRA blog, section 1, on tie order).
 *  DSA_ORDER_INDEX: the same set of keys in ascending key index.             */
typedef enum { DSA_ORDER_SCORE = 0, DSA_ORDER_INDEX = 1 } dsa_topk_order;

/* Largest k_out / topk_limit the top-k kernels accept. */
#define DSA_MAX_TOPK 4096

/* Human-readable name of a status code (static storage; never NULL). */
const char* dsa_status_string(int status);

/* Library version string (static storage). */
const char* dsa_version(void);

/* Width of a top-k row: min(topk_limit, active_seq_len), never negative
 * (GLM5 TensorCast adaptation design, "DSA Indexer 融合语义算子": the op returns
 * (batch, seq_len, min(topk_limit, active_seq_len))). */
int dsa_topk_width(int topk_limit, int64_t active_seq_len);

/*
 * dsa_indexer_scores -- dense scoring of one sequence (cost buckets 6 and 7:
 * q-k index score MMA; head weight multiply, head reduce, FP8 relu / q-scale /
 * k-scale shaping).
 *
 *   q        [T, H, D]  q_dtype        query rows, query t at position q_pos0 + t
 *   q_scale  [T, H]     fp32 > 0       FP8 q only (NULL for bf16 q)
 *   k        [S, D]     k_dtype        keys 0..S-1
 *   k_scale  [S]        fp32 > 0       FP8 k only (NULL for bf16 k)
 *   w        [T, H]     fp32           per-head weights (any sign)
 *   scores   [T, ld_scores] fp32       out: scores[t, s] for s <= min(q_pos0 + t, S - 1);
 *                                      entries with s > q_pos0 + t are NOT written
 *
 * Supported: (q_dtype, k_dtype) in {(BF16, BF16), (FP8, FP8)}; D in {64, 128} for
 * bf16, D = 128 for FP8; H in {4, 8, 16, 32, 64, 128}; ld_scores >= S and a
 * multiple of 4; q_pos0 >= 0.  T == 0 or S == 0 is a no-op.
 * Inputs must be finite; scales must be finite and > 0 (the library applies the
 * q scale to w and the k scale after the head sum, which commutes with ReLU
 * only for positive scales).
 */
dsa_status dsa_indexer_scores(const void* q, int q_dtype, const float* q_scale,
                              const void* k, int k_dtype, const float* k_scale,
                              const float* w, int T, int S, int H, int D, int q_pos0,
                              float* scores, int64_t ld_scores, dsa_stream_t stream);

/*
 * dsa_indexer_topk -- per-row top-k of dense scores (cost bucket 8, top-k selection).
 *
 *   scores [T, ld_scores] fp32   row t has n_t = max(0, min(q_pos0 + t + 1, S)) visible
 *                                entries scores[t, 0..n_t-1]; nothing else is read
 *   topk   [T, k_out] int32      out: min(topk_limit, n_t) key indices, then -1
 *
 * topk_limit >= 1, 1 <= k_out <= DSA_MAX_TOPK, topk_limit <= DSA_MAX_TOPK unless
 * no row is longer than DSA_MAX_TOPK; order is a dsa_topk_order.  Ties between equal
 * scores go to the lower key index; -0.0 and +0.0 are equal.  NaN scores are
 * outside the contract.  Needs no workspace.
 */
dsa_status dsa_indexer_topk(const float* scores, int64_t ld_scores, int T, int S, int q_pos0,
                            int topk_limit, int k_out, int order, int32_t* topk,
                            dsa_stream_t stream);

/*
 * Fused indexer over a paged key cache for a varlen batch: prefill, chunked
 * prefill and decode (op inputs indexer_cache, block_tables, seq_lens of section
 * "DSA Indexer 融合语义算子"; key and scale cache read bytes, buckets 9 and 10).
 *
 * Sequence b owns query rows cu_q_lens[b] .. cu_q_lens[b+1]-1; its i-th query
 * sits at position pos = seq_lens[b] - q_len_b + i and sees keys 0..pos.  Key s
 * of sequence b is k_cache[block_tables[b * max_pages_per_seq + s / page_size]]
 * [s % page_size].  Returned indices are logical key positions in the sequence.
 */
typedef struct {
    int q_dtype;                 /* dsa_dtype of q                                   */
    int k_dtype;                 /* dsa_dtype of k_cache                             */
    int B;                       /* sequences                                        */
    int total_q;                 /* cu_q_lens[B] (host copy; rows of q, w, topk)     */
    int H, D;                    /* indexer heads, head dim                          */
    int page_size;               /* tokens per page: 16, 32, 64 or 128               */
    int num_pages;               /* pages in k_cache                                 */
    int max_pages_per_seq;       /* columns of block_tables                          */
    int max_seq_len;             /* host upper bound of seq_lens[b]                  */
    const void* q;               /* [total_q, H, D]                                  */
    const float* q_scale;        /* [total_q, H] fp32 (FP8 q) or NULL                */
    const float* w;              /* [total_q, H] fp32                                */
    const int32_t* cu_q_lens;    /* [B + 1], cu_q_lens[0] = 0, non-decreasing        */
    const int32_t* seq_lens;     /* [B], q_len_b <= seq_lens[b] <= max_seq_len       */
    const int32_t* block_tables; /* [B, max_pages_per_seq]                           */
    void* k_cache;               /* [num_pages, page_size, D] (written when k_new)   */
    float* k_scale_cache;        /* [num_pages, page_size] fp32 (FP8 k) or NULL      */
    int topk_limit;              /* index_topk / topk_limit                          */
    int k_out;                   /* columns of topk, >= 1                            */
    int order;                   /* dsa_topk_order                                   */
    int32_t* topk;               /* out [total_q, k_out]                             */
    void* workspace;             /* device scratch, >= dsa_indexer_workspace_size    */
    size_t workspace_bytes;
    const void* k_new;           /* NULL, or [total_q, D] bf16: this step's new keys, */
                                 /* appended to the cache before scoring             */
    const int64_t* slot_mapping; /* [total_q] with k_new: cache slot of each new key */
} dsa_indexer_args;

/* Bytes of device workspace dsa_indexer needs for these sizes (pointers may be NULL). */
dsa_status dsa_indexer_workspace_size(const dsa_indexer_args* args, size_t* bytes);

/* Run the fused indexer.  Same dtype / H / D support as dsa_indexer_scores, plus
 * BF16 q against an FP8-e4m3 cache (GLM5 TensorCast adaptation design, background
 * item 5: the indexer cache takes the FP8 dtype when attention is quantised).  That
 * mix is taken on decode batches (total_q <= B) with D = 128 and k_scale_cache set
 * (q_scale is ignored): each bf16 query row x is first rewritten as s x = hi + lo,
 * two e4m3 rows with a power-of-two scale s (largest |s x| in [128, 256)), exact for
 * every element within ~2^9 of the row's largest |x| and within 2^-17 of that largest
 * value otherwise; the keys then meet both rows in FP8 MMAs whose two halves are added
 * before the ReLU, and w is divided by s.  The two e4m3 NaN codes are not accepted in
 * the cache.  On a prefill batch the mix returns DSA_ERR_UNSUPPORTED.  The workspace
 * (which also holds the rewritten queries) must not be used by another call that
 * overlaps on the GPU. */
dsa_status dsa_indexer(const dsa_indexer_args* args, dsa_stream_t stream);

/*
 * dsa_indexer_cache_append -- write this step's new indexer keys into the paged cache
 * (GLM5 TensorCast adaptation design, "DSA Indexer 融合语义算子": the op's indexer cache
 * is a mutable argument written through slot_mapping; its FP8 path writes the key
 * cache and the scale cache after an activation quantisation, cost buckets 9 and 10).
 *
 *   k_new [n, D] bf16 device rows; slot_mapping [n] int64, slot = page * page_size + row
 *   (negative: skip the token); k_cache [num_pages, page_size, D] of cache_dtype;
 *   k_scale_cache [num_pages, page_size] fp32 (e4m3 cache only).
 *   bf16 cache (D = 64 or 128): the row is copied.  e4m3 cache (D = 128): scale =
 *   amax / 448 (fp32; 1 for an all-zero row), each element the e4m3 value nearest to
 *   k / scale (ties to even, saturating at +-448), the scale stored beside the row.
 * A slot past the cache is skipped and reported through dsa_check_device_status.
 * The same append runs first inside dsa_indexer when dsa_indexer_args.k_new is set.
 */
dsa_status dsa_indexer_cache_append(const void* k_new, int n, int D, const int64_t* slot_mapping,
                                    void* k_cache, int cache_dtype, float* k_scale_cache, int page_size,
                                    int num_pages, dsa_stream_t stream);

/*
 * dsa_indexer_prepare -- the indexer front-end: this step's q, k and head weights from
 * the layer's activations (GLM5 TensorCast adaptation design, "DSA Indexer 融合语义算子":
 * the op's inputs hidden_states, qa_normed, RoPE cos / sin, wq_b, wk, weights_proj,
 * k_norm weight, indexer cache, slot_mapping; performance-model buckets 1-5, 9, 10).
 *
 *   q  = RoPE(qa_normed @ wq_b^T), one row of D per head          [T, H, D]
 *   k  = RoPE(layer_norm(hidden @ wk^T) * k_norm_weight + bias)    [T, D]
 *   w  = hidden @ weights_proj^T                                   [T, H] fp32 -> w_out
 * e4m3 cache: q and k are then rotated by the Walsh-Hadamard transform (Sylvester order,
 * times D^-1/2) and quantised per row: scale = amax / 448 (1 for an all-zero row), codes
 * the e4m3 value nearest to x / scale; q -> q_out (e4m3) and q_scale_out [T, H]; k and
 * its scale -> the cache slot.  bf16 cache: q -> q_out (bf16), k -> the cache slot (bf16).
 * The outputs feed dsa_indexer (q, q_scale, w; the cache now holds this step's keys).
 *
 * Readings (the page gives no formulas): projection weights are [out, in] row-major
 * (x @ W^T); k_norm is a layer norm with the biased variance and eps k_norm_eps, times
 * the weight, plus k_norm_bias when not NULL; RoPE turns pair i of the first rope_dim
 * values -- (i, i + rope_dim/2), or (2i, 2i+1) when rope_interleaved -- by the angle with
 * cosine rope_cos[t, i] and sine rope_sin[t, i]: (a, b) -> (a cos - b sin, a sin + b cos).
 *
 * All pointers are device memory, 16-byte aligned (slot_mapping 8-byte).  hidden
 * [T, hidden_dim] and qa_normed [T, q_rank] bf16; wq_b [H*D, q_rank], wk [D, hidden_dim],
 * weights_proj [H, hidden_dim] bf16; rope_cos / rope_sin [T, rope_dim/2] fp32;
 * k_norm_weight [D] fp32, k_norm_bias [D] fp32 or NULL.  D = 128; H a power of two up to
 * 128; rope_dim even, at most D, a multiple of 8 unless interleaved; hidden_dim and
 * q_rank multiples of 8.  The three projections run on the tensor cores as bf16
 * products with fp32 accumulation, in the library's kernels like everything else; with
 * 512 tokens or more and rope_dim 0, 64 or 128 the q projection finishes its rows
 * (RoPE, rotation, quantisation) in its own epilogue.  workspace:
 * dsa_indexer_prepare_workspace_size bytes of device memory (the fp32 partial sums of
 * the projections that are not finished in their epilogue), not shared with
 * overlapping work.  Slots past the cache are skipped and reported through
 * dsa_check_device_status; negative slots are skipped.
 */
typedef struct {
  int T, hidden_dim, q_rank, H, D, rope_dim, rope_interleaved;
  const void* hidden;
  const void* qa_normed;
  const float* rope_cos;
  const float* rope_sin;
  const void* wq_b;
  const void* wk;
  const void* weights_proj;
  const float* k_norm_weight;
  const float* k_norm_bias;
  float k_norm_eps;
  int cache_dtype;           /* DSA_BF16 or DSA_FP8_E4M3 */
  const int64_t* slot_mapping;
  void* k_cache;             /* [num_pages, page_size, D] */
  float* k_scale_cache;      /* [num_pages, page_size] (e4m3 cache) */
  int page_size, num_pages;
  void* q_out;               /* [T, H, D] bf16 or e4m3 */
  float* q_scale_out;        /* [T, H] (e4m3 cache) */
  float* w_out;              /* [T, H] */
  void* workspace;
  size_t workspace_bytes;
} dsa_indexer_prepare_args;

dsa_status dsa_indexer_prepare_workspace_size(const dsa_indexer_prepare_args* args, size_t* bytes);
dsa_status dsa_indexer_prepare(const dsa_indexer_prepare_args* args, dsa_stream_t stream);

/*
 * dsa_indexer_dense_host -- dsa_indexer_scores + dsa_indexer_topk of one sequence whose
 * inputs and output are in HOST memory, with the transfers overlapped with the kernels.
 * The pages describe the indexer on device tensors; this entry point exists for callers
 * that hold the step's inputs on the host (and is what an end-to-end measurement calls).
 *
 *   q_host [T, H, D], w_host [T, H], k_host [S, D] (+ q_scale_host [T, H], k_scale_host [S]
 *   for e4m3): row-major host arrays, pinned (cudaHostAlloc / cudaHostRegister) for the
 *   copies to overlap; pageable memory works but the copies then serialise.
 *   topk_host [T, k_out]: written with the same rows dsa_indexer_topk returns.
 *   chunk_rows: query rows per chunk (0 = max(512, T/16); raised so there are at most
 *   256 chunks).
 *   workspace: device memory of dsa_indexer_dense_host_workspace_size bytes, 256-byte
 *   aligned, owned by the caller and not shared with overlapping work.
 *
 * The query rows travel in chunks (last rows first) on a library-owned copy stream;
 * each chunk is scored and selected as soon as its rows land, alternately on `stream`
 * and on a library-owned compute stream so consecutive chunks' kernels overlap; another
 * library-owned stream copies the chunk's top-k rows back.  The call returns once everything is enqueued; `stream` waits
 * for the last copy, so synchronising it makes topk_host final.  Same element types, H,
 * D and errors as dsa_indexer_scores / dsa_indexer_topk; S = 0 is DSA_ERR_UNSUPPORTED.
 * Concurrent calls from several host threads on one device are serialised internally.
 */
dsa_status dsa_indexer_dense_host_workspace_size(int T, int S, int H, int D, int q_dtype, int k_out,
                                                 int chunk_rows, size_t* bytes);
dsa_status dsa_indexer_dense_host(const void* q_host, int q_dtype, const float* q_scale_host,
                                  const void* k_host, int k_dtype, const float* k_scale_host,
                                  const float* w_host, int T, int S, int H, int D, int q_pos0,
                                  int topk_limit, int k_out, int order, int chunk_rows,
                                  int32_t* topk_host, void* workspace, size_t workspace_bytes,
                                  dsa_stream_t stream);

/*
 * Key-sharded top-k (GLM5 LoRA blog, section 3.1, 训练侧: context parallelism; a top-k
 * taken per shard of a long sequence matches the full-sequence top-k only 68 % of the
 * time, gathering the shards' indexer results 99.97 %).  The exact form: every shard of
 * keys keeps its best min(k, visible) keys as (score, global index) candidates in
 * (score desc, index asc) order; the caller gathers the candidates of all shards (for
 * shards on several devices, one all-gather of [T, k_cand] indices and scores per
 * shard); dsa_indexer_merge_candidates keeps the best of their union under the same
 * order, which equals the top-k of the whole row.
 *
 * dsa_indexer_shard_candidates -- one shard's candidates.
 *   q, q_scale, w, H, D, dtypes   as dsa_indexer_scores; query t at position q_pos0 + t
 *   k_shard [S, D], k_scale [S]   the shard's keys: global key positions
 *                                 key_offset .. key_offset + S - 1 (query t sees global key
 *                                 g when g <= q_pos0 + t)
 *   k_cand                        candidates per row, 1..DSA_MAX_TOPK (use the top-k width)
 *   cand_idx [T, k_cand] int32    out: global key indices, then -1
 *   cand_scores [T, k_cand] fp32  out: their scores, then -inf
 *   workspace                     16-byte aligned device scratch of at least
 *                                 dsa_indexer_shard_candidates_workspace_size(T, S) bytes
 *                                 (the shard's fp32 score rows), caller-owned
 * q_pos0 >= 0, key_offset >= 0.  Same element types, H, D and errors as
 * dsa_indexer_scores; a missing or small workspace is DSA_ERR_WORKSPACE.
 */
dsa_status dsa_indexer_shard_candidates_workspace_size(int T, int S, size_t* bytes);
dsa_status dsa_indexer_shard_candidates(const void* q, int q_dtype, const float* q_scale, const void* k_shard,
                                        int k_dtype, const float* k_scale, const float* w, int T, int S, int H,
                                        int D, int q_pos0, int key_offset, int k_cand, int32_t* cand_idx,
                                        float* cand_scores, void* workspace, size_t workspace_bytes,
                                        dsa_stream_t stream);

/*
 * dsa_indexer_merge_candidates -- the top-k of the union of n_shards candidate lists.
 *   cand_scores [n_shards, T, k_cand] fp32, cand_idx [n_shards, T, k_cand] int32: list j
 *   of row t holds shard j's candidates as written by dsa_indexer_shard_candidates
 *   (valid entries first, in (score desc, index asc) order, then index -1); the shards'
 *   key ranges must not overlap.
 *   topk [T, k_out] int32 out: min(topk_limit, valid candidates) indices in `order`,
 *   then -1.
 * 1 <= n_shards <= 32, n_shards * k_cand <= 16384, 1 <= k_out <= DSA_MAX_TOPK.  Ties go
 * to the lower key index; -0.0 and +0.0 are equal.
 */
dsa_status dsa_indexer_merge_candidates(const float* cand_scores, const int32_t* cand_idx, int n_shards, int T,
                                        int k_cand, int topk_limit, int k_out, int order, int32_t* topk,
                                        dsa_stream_t stream);

/*
 * Sparse MLA over the indexer's top-k (GLM5 TensorCast adaptation design: the fused
 * indexer hands topk_indices / topk_limit to the multi-head latent attention backend,
 * whose attention length is capped by the top-k width -- "Sparse MLA 配置兼容", the
 * performance model's sparse prefill / decode length).  Absorbed multi-head latent
 * attention on the selected keys only: for query row t of sequence b and head h, over the
 * logical key positions s = topk[t, j] >= 0 (s < seq_lens[b]; others are skipped),
 *     logit = scale * (q_nope[t, h] . c_kv[s] + q_rope[t, h] . k_rope[s])
 *     out[t, h, :] = sum_s softmax_s(logit) * c_kv[s]            (fp32, latent space)
 * with c_kv[s] = cache_c[block_tables[b, s / page_size], s % page_size] and k_rope[s] the
 * same row of cache_r.  An empty selection gives zeros.  The value up-projection and the
 * output projection are the caller's.
 *   q_nope [total_q, H, kv_rank] bf16, q_rope [total_q, H, rope_dim] bf16
 *   cache_c [num_pages, page_size, kv_rank] bf16, cache_r [num_pages, page_size, rope_dim] bf16
 *   topk [total_q, topk_width] int32 (any order, -1 padding); out [total_q, H, kv_rank] fp32
 * kv_rank = 512 and rope_dim = 64; H = 16, 32 or a multiple of 64; scale > 0.  workspace:
 * dsa_sparse_mla_workspace_size bytes (the key splits' partial outputs), 16-byte aligned.
 * A selected position whose page is outside the cache is skipped and reported through
 * dsa_check_device_status.  Probabilities enter the P.V product rounded to bf16.
 */
typedef struct {
  int B, total_q, H, kv_rank, rope_dim, page_size, num_pages, max_pages_per_seq, topk_width;
  float scale;
  const void* q_nope;
  const void* q_rope;
  const void* cache_c;
  const void* cache_r;
  const int32_t* block_tables;
  const int32_t* cu_q_lens;
  const int32_t* seq_lens;
  const int32_t* topk;
  float* out;
  void* workspace;
  size_t workspace_bytes;
} dsa_sparse_mla_args;
dsa_status dsa_sparse_mla_workspace_size(const dsa_sparse_mla_args* args, size_t* bytes);
dsa_status dsa_sparse_mla(const dsa_sparse_mla_args* args, dsa_stream_t stream);

/*
 * A serving step for a batch whose requests begin with the same prompt: page plan, latent
 * cache append, shared-prefix attention.  They share the paged layout of the calls above
 * (block_tables, slot_mapping, cache_c / cache_r of dsa_sparse_mla), so the indexer and
 * dsa_sparse_mla run on the same tables and caches.
 */

/*
 * dsa_page_plan -- block tables, slot mapping, positions and query offsets of a step, from
 * the request lengths, in one launch.  Request b holds seq_lens[b] tokens after the step,
 * the last q_lens[b] of them new.  With c = seq_lens[b] - q_lens[b], P = page_size, row b
 * of block_tables holds before the call
 *     held(b) = max(ceil(c / P), num_prefix_pages)         pages
 * and after it have(b) = max(ceil(seq_lens[b] / P), num_prefix_pages):
 *     entry j < num_prefix_pages     prefix_pages[j]            (written in every row)
 *     entry j < held(b)              as it was
 *     entry j < have(b)              free_pages[first(b) + j - held(b)]
 *     the rest                       -1
 * first(b) = the new pages of requests 0 .. b-1: free pages are handed out in request order
 * from the front of free_pages, and used[0] = the new pages of all requests.  A request of
 * seq_lens[b] = 0 gets a row of -1 and takes nothing.
 *   cu_q_lens [B + 1]        0, q_lens[0], q_lens[0] + q_lens[1], ...
 *   positions [total_q]      of each new token in its sequence: seq_lens[b] - q_lens[b] + i
 *   slot_mapping [total_q]   page * P + row of that position (int64)
 * total_q is the outputs' length: at least the sum of q_lens; entries past the sum (a step
 * padded to a captured graph's size) are -1 in both.
 * Only whole pages of a shared prompt can be shared: a request writes its own pages, so a
 * partly filled last prompt page is each request's own, and c is num_prefix_pages * P at
 * least (new tokens before that would get slots of the shared pages).
 * Recorded in the device status word (DSA_ERR_DEVICE_CHECK), never out of bounds: a
 * free list that is too short (its entries and slots become -1; used[0] is still what the
 * step needs), a page id < 0, a length that is negative, exceeds the table, or q_lens[b] >
 * seq_lens[b] (taken as the nearest allowed value), and more new tokens than total_q (dropped).
 * All arrays are 4-byte aligned device memory (slot_mapping 8-byte); prefix_pages may be
 * NULL when num_prefix_pages is 0, free_pages when num_free is 0, slot_mapping and positions
 * when total_q is 0.
 */
typedef struct {
  int B, total_q, page_size, max_pages_per_seq, num_prefix_pages, num_free;
  const int32_t* q_lens;
  const int32_t* seq_lens;
  const int32_t* prefix_pages;
  const int32_t* free_pages;
  int32_t* block_tables;
  int32_t* cu_q_lens;
  int64_t* slot_mapping;
  int32_t* positions;
  int32_t* used;
} dsa_page_plan_args;
dsa_status dsa_page_plan(const dsa_page_plan_args* args, dsa_stream_t stream);

/*
 * dsa_mla_cache_append -- this step's latent rows into the paged cache that dsa_sparse_mla
 * and dsa_prefix_mla read:
 *     cache_c[slot] = bf16( norm_weight * c / sqrt(mean(c^2) + norm_eps) )   (c itself without norm_weight)
 *     cache_r[slot] = bf16( RoPE(r) )                                        (r itself without rope_cos)
 * in fp32, rounded once.  c_kv [n, 512] and k_rope [n, 64] are bf16 rows c_stride / r_stride
 * elements apart, so both may be views of one projection output [n, 576].  norm_weight [512]
 * fp32.  rope_cos, rope_sin [rope_rows, 32] fp32; token t uses row positions[t] (row t when
 * positions is NULL); pairs (i, i + 32), or (2i, 2i + 1) when rope_interleaved, turn as in
 * dsa_indexer_prepare.  slot_mapping [n] int64, negative: the token is skipped.  A slot past
 * the cache, or a position outside the tables, skips the token and is reported through
 * dsa_check_device_status.  Two tokens with one slot leave either's values there.
 * Pointers 16-byte aligned (slot_mapping 8, positions 4), strides multiples of 8 elements
 * (any when n = 1).
 */
typedef struct {
  int n, kv_rank, rope_dim, page_size, num_pages, rope_interleaved, rope_rows;
  float norm_eps;
  const void* c_kv;
  const void* k_rope;
  int64_t c_stride, r_stride;
  const int64_t* slot_mapping;
  const float* norm_weight;
  const float* rope_cos;
  const float* rope_sin;
  const int32_t* positions;
  void* cache_c;
  void* cache_r;
} dsa_mla_cache_append_args;
dsa_status dsa_mla_cache_append(const dsa_mla_cache_append_args* args, dsa_stream_t stream);

/*
 * dsa_prefix_mla -- absorbed multi-head latent attention for a batch whose sequences share
 * their first prefix_len tokens; the shared keys are scored for the queries of all requests
 * together.  Query row i of sequence b sits at position p = seq_lens[b] - q_len(b) + i and
 * sees the positions s <= p:
 *     logit = scale * (q_nope[t, h] . c_kv[s] + q_rope[t, h] . k_rope[s])
 *     out[t, h, :] = sum_s softmax_s(logit) * c_kv[s]     (bf16, latent space)
 *     lse[t, h]    = ln sum_s exp(logit)                  (fp32; optional)
 * where position s lies at page prefix_pages[s / page_size] when s < prefix_len and at page
 * block_tables[b, s / page_size] otherwise, row s % page_size of cache_c / cache_r.
 * prefix_len may end inside a page (that page of the request's own table then starts with
 * rows nobody reads) and may be 0; a sequence may be shorter than it.  A query that sees
 * nothing (p < 0) and the rows t >= cu_q_lens[B] (padding) give zeros and lse = -inf.
 *   q_nope [total_q, H, 512] bf16 and q_rope [total_q, H, 64] bf16 with the given element
 *   strides (multiples of 8, any in a dimension of size 1; the last dimension dense); cache_c, cache_r as in dsa_sparse_mla;
 *   block_tables [B, max_pages_per_seq]; out [total_q, H, 512] bf16 dense; lse [total_q, H].
 * kv_rank = 512, rope_dim = 64, 1 <= H <= 128, page_size 16, 32, 64 or 128, scale > 0; total_q * H,
 * num_pages * page_size and the keys that a query sees below 2^31 - 128 (a longer sequence is cut
 * there and reported like one that passes its table).
 * Cache rows that no query sees may hold anything, NaN included; rows that some query sees
 * must be finite.  A NaN in a query makes out and lse of its (t, h) NaN and no others.  A page
 * outside the cache, or a position past the table, is skipped and reported through
 * dsa_check_device_status.  Probabilities enter P.V rounded to
 * bf16; statistics and sums are fp32.  Results do not depend on the run (no atomics on data).
 * workspace: dsa_prefix_mla_workspace_size bytes, 16-byte aligned like the other pointers; some
 * 40 MB on a GB300 (two results of 128 rows for each pair of SMs), and where requests may share
 * tiles (H no multiple of 128, at most some 850 rows a request) 4 KB more for every row.
 */
typedef struct {
  int B, total_q, H, kv_rank, rope_dim, page_size, num_pages, max_pages_per_seq;
  int prefix_len, num_prefix_pages;
  float scale;
  const void* q_nope;
  const void* q_rope;
  int64_t qn_stride_t, qn_stride_h, qr_stride_t, qr_stride_h;
  const void* cache_c;
  const void* cache_r;
  const int32_t* prefix_pages;
  const int32_t* block_tables;
  const int32_t* cu_q_lens;
  const int32_t* seq_lens;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
} dsa_prefix_mla_args;
dsa_status dsa_prefix_mla_workspace_size(const dsa_prefix_mla_args* args, size_t* bytes);
dsa_status dsa_prefix_mla(const dsa_prefix_mla_args* args, dsa_stream_t stream);

/*
 * A latent cache in 8 or 4 bits: quantised as it is written, attended over as it is, read back as
 * bf16.  One array cache [num_pages, page_size, row] of bytes holds a token's 512 latent and 64
 * rotary values; block tables, slots and positions are those of the calls above.
 *   DSA_FP8_E4M3  656 bytes a row (bf16: 1152): 512 e4m3 codes, 64 bf16, one scale
 *   DSA_FP4_E2M1  416 bytes a row: 512 e2m1 codes, 64 bf16, 32 scales of blocks of 16
 * With c the latent row and a_max its largest magnitude:
 *   E = the smallest integer with a_max <= 448 * 2^E (432 * 2^E in 4 bits), in [-60, 60], 0 for zeros
 *   e4m3   code = the e4m3 value nearest to c / 2^E; it stands for 2^E * code
 *   e2m1   per block of 16: s = the smallest value of 4 significant bits, at least 2^-5, with
 *          6 * s >= the block's largest |c| / 2^E; code = the e2m1 value nearest to c / (2^E * s); it
 *          stands for 2^E * e4m3(code * s), the product rounded to e4m3
 * (nearest: ties to even; 2^-5 <= s <= 72).  The codes are those of c itself, not of a rounded c: with
 * a norm, of c to within 2^-40.  Every value that a row stands for is exact in bf16.  The rotary part is
 * held as bf16(r) / 2^E (exact for 2^-66 <= |r| < 2^67).  A mean over 512 normal values is off by
 * 2.7 % (e4m3) and 10 % (e2m1) of their size.
 * Rows are the library's own: dsa_mla_quant_append writes and dsa_mla_quant_read reads them.  A page
 * may be moved or copied as bytes.  Nothing in a row tells its format: a cache of another layout whose rows
 * have as many bytes is taken for one of these, and read wrongly.
 */

/* Bytes of a row of this format; 0 for one that there is not. */
int dsa_mla_quant_row_bytes(int format);

/*
 * dsa_mla_quant_append -- dsa_mla_cache_append into a quantised cache: c = norm_weight * c_kv /
 * sqrt(mean(c_kv^2) + norm_eps) (c_kv itself without norm_weight) and r = RoPE(k_rope) (k_rope itself
 * without rope_cos), written to row slot of the cache in `format`.  Arguments, slots and reports are
 * those of dsa_mla_cache_append; cache is 16-byte aligned.  Inputs of rows that are written must be
 * finite, the sum of squares of a row too (codes hold no infinity, and 4-bit ones no NaN: the largest code of the
 * block stands in its place, and nothing is reported).  Two rows for one slot: one of them, or a mixture.
 */
typedef struct {
  int format, n, kv_rank, rope_dim, page_size, num_pages, rope_interleaved, rope_rows;
  float norm_eps;
  const void* c_kv;
  const void* k_rope;
  int64_t c_stride, r_stride;
  const int64_t* slot_mapping;
  const float* norm_weight;
  const float* rope_cos;
  const float* rope_sin;
  const int32_t* positions;
  void* cache;
} dsa_mla_quant_append_args;
dsa_status dsa_mla_quant_append(const dsa_mla_quant_append_args* args, dsa_stream_t stream);

/*
 * dsa_mla_quant_read -- rows of a quantised cache as bf16: for request b and 0 <= i < cu_lens[b + 1] -
 * cu_lens[b], row t = cu_lens[b] + i of c_kv and k_rope gets what position starts[b] + i of the request
 * (i itself when starts is NULL) stands for, exactly.  The rows may be views of one [total, 576] array
 * (c_stride, r_stride elements apart, 512 and 64 or more, multiples of 8; any when total = 1).  total is the outputs'
 * length: rows before cu_lens[0] and from cu_lens[B] on are left as they were, rows past total are dropped.  A position whose
 * page is outside the cache, or that the table does not cover, leaves its row as it was and is
 * reported through dsa_check_device_status.  c_kv, k_rope and cache 16-byte aligned.
 * With pages of its own, the result is a bf16 cache that dsa_prefix_mla and dsa_sparse_mla take.
 */
typedef struct {
  int format, B, total, kv_rank, rope_dim, page_size, num_pages, max_pages_per_seq;
  const void* cache;
  const int32_t* block_tables;
  const int32_t* cu_lens;
  const int32_t* starts;
  void* c_kv;
  void* k_rope;
  int64_t c_stride, r_stride;
} dsa_mla_quant_read_args;
dsa_status dsa_mla_quant_read(const dsa_mla_quant_read_args* args, dsa_stream_t stream);

/*
 * dsa_quant_mla -- absorbed multi-head latent attention over a quantised cache, each query over its
 * selected keys or over all that it sees:
 *     logit = scale * (q_nope[t, h] . c[s] + q_rope[t, h] . r[s])
 *     out[t, h, :] = sum_s softmax_s(logit) * c[s]     (bf16, latent space)
 *     lse[t, h]    = ln sum_s exp(logit)               (fp32; optional)
 * with c, r what row s of the cache stands for.  topk_width > 0: over the positions s = topk[t, j] with
 * 0 <= s < seq_lens[b], others are skipped (any order; one that is named twice counts twice).
 * topk_width = 0: over all s <= p, p = seq_lens[b] - q_len(b) + i the position of the sequence's i-th
 * query; the cache is then read once for every query, so a prompt of many tokens is better served by
 * dsa_mla_quant_read and dsa_prefix_mla.  A query without keys and the rows t >= cu_q_lens[B]
 * (padding) give zeros and lse = -inf.
 *   q_nope [total_q, H, 512], q_rope [total_q, H, 64] bf16 with the given element strides (multiples of
 *   8, any in a dimension of size 1; the last dimension dense); out [total_q, H, 512] bf16 dense;
 *   lse [total_q, H]; topk [total_q, topk_width].
 * kv_rank = 512, rope_dim = 64, 1 <= H <= 128, scale > 0; total_q * H and num_pages * page_size below
 * 2^31 - 128; topk_width at most 2^31 - 256.  Rows of the cache that no query attends to may hold
 * anything; the others are finite, their 2^E within a factor of 2^100 for one query (rows of zeros count
 * as 2^-60), and the queries of rows that are not padding are finite (what is not makes its own query
 * and head NaN).  A page outside the cache is skipped and reported through dsa_check_device_status, as
 * are positions past the table.  Results do not depend on the run.  workspace:
 * dsa_quant_mla_workspace_size bytes (0: none is taken), 16-byte aligned like the other pointers.
 * Weights enter out to 2^-7 each.  Small ones, of which many may count together, are rounded up for some keys and down for
 * others: a key whose weight times its row's 2^E is below 2^-11 of the largest such product is off by up to 2^-17 of that,
 * and the mean of many that weigh alike by 2^-7 of itself and 2^-30 of that product.  Below 2^-30 of it a key adds nothing to
 * out (to lse all do); the product of a row of zeros, which adds nothing to out, counts with E = -60.
 */
typedef struct {
  int format, B, total_q, H, kv_rank, rope_dim, page_size, num_pages, max_pages_per_seq, topk_width;
  float scale;
  const void* q_nope;
  const void* q_rope;
  int64_t qn_stride_t, qn_stride_h, qr_stride_t, qr_stride_h;
  const void* cache;
  const int32_t* block_tables;
  const int32_t* cu_q_lens;
  const int32_t* seq_lens;
  const int32_t* topk;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
} dsa_quant_mla_args;
dsa_status dsa_quant_mla_workspace_size(const dsa_quant_mla_args* args, size_t* bytes);
dsa_status dsa_quant_mla(const dsa_quant_mla_args* args, dsa_stream_t stream);

/*
 * dsa_indexer_static -- dsa_indexer for callers that cannot allocate device memory.
 * The pages have no counterpart of this entry point; it exists for library users.
 *
 * Some callers cannot hand the library a workspace: plugin hosts that pass only the
 * input and output tensors, and serving loops that reserve nearly all device memory
 * up front and forbid allocation during a step (cudaMalloc / cudaFree may synchronise
 * the device and stall every stream).  This call runs the same kernels as dsa_indexer
 * with their scratch (work-list counters, work items, fp32 score rows) in one
 * library-owned device array of DSA_STATIC_WORKSPACE_BYTES, which every GPU that
 * loads this code holds until the process exits.  args->workspace and
 * args->workspace_bytes are ignored; every other field means what it means for
 * dsa_indexer, and the caller still provides every input and the topk output.
 *  - A problem whose dsa_indexer_workspace_size exceeds DSA_STATIC_WORKSPACE_BYTES
 *    returns DSA_ERR_WORKSPACE before anything is launched (use dsa_indexer with a
 *    caller workspace for it).
 *  - The array is placed on a device when the library's device code is loaded there,
 *    which under CUDA's default lazy module loading can be during the first call into
 *    the library on that device, and the first dsa_indexer_static call on a device
 *    looks up the array's device address with that device current.  So make one call
 *    into the library (this one, or any other) on each device before reserving most of
 *    its memory, and make the first dsa_indexer_static call there before any stream
 *    capture.  A failed lookup returns DSA_ERR_CUDA and is tried again by the next call.
 *  - All calls on a device share the array and it keeps the last call's contents; each
 *    call clears the part that must start at zero (the work-list counters).  Calls that
 *    overlap on the GPU (other streams, other host threads) race on the array: serialise them.
 *  - It calls no cudaMalloc, cudaFree or other allocating routine.
 */
#define DSA_STATIC_WORKSPACE_BYTES ((size_t)24 << 20)
dsa_status dsa_indexer_static(const dsa_indexer_args* args, dsa_stream_t stream);

/*
 * IndexShare source resolution (host only, GLM5 TensorCast adaptation design,
 * "GLM-5.2 IndexShare"): src[l] = l for a full layer, the nearest earlier full
 * layer for a shared layer.  types[l] is a dsa_layer_type.  An unknown type or a
 * shared layer with no earlier full layer returns DSA_ERR_INVALID_ARGUMENT and
 * leaves src unspecified.
 */
dsa_status dsa_resolve_indexer_sources(int L, const int32_t* types, int32_t* src);

/*
 * dsa_indexer_stack -- an IndexShare stack of L layers.
 *   full_args[l]  host pointer to the args of full layer l (its own cache, q, w and
 *                 output buffer); NULL for shared layers (they own no cache).
 *   topk_out[l]   host array of L device pointers, written by the call: a full layer's
 *                 entry is full_args[l]->topk, a shared layer's entry is its source
 *                 layer's buffer -- the same memory, forwarded unchanged, no launch.
 *   src_out       host [L] or NULL: the resolved source layers.
 * Every argument is validated before the first launch.
 */
dsa_status dsa_indexer_stack(int L, const int32_t* types, const dsa_indexer_args* const* full_args,
                             int32_t** topk_out, int32_t* src_out, dsa_stream_t stream);

/* Synchronise `stream`, then report and clear the device status word of the current
 * device: DSA_OK, DSA_ERR_DEVICE_CHECK or DSA_ERR_TIMEOUT (or DSA_ERR_CUDA). */
dsa_status dsa_check_device_status(dsa_stream_t stream);

/*
 * Clock sample (diagnostic, not part of the method): n_ctas one-thread blocks each write
 * {SM id, that SM's cycle counter (clock64), the global nanosecond timer} as three
 * uint64 to out[3 * i .. 3 * i + 2].  Two samples on a stream bracket an interval; per SM,
 * (cycles after - cycles before) / (ns after - ns before) is its average clock over it.
 *   out     device [3 * n_ctas] uint64, caller-owned
 *   n_ctas  >= 1 (a few per SM reach every SM)
 * Asynchronous on `stream`; DSA_ERR_INVALID_ARGUMENT for a null out or n_ctas < 1.
 */
dsa_status dsa_clock_sample(uint64_t* out, int n_ctas, dsa_stream_t stream);

/*
 * dsa_test_arm_score_timeout -- failure-path test hook; the pages have no counterpart.
 * Every wait inside the library's kernels is bounded: a wait that runs out records
 * DSA_ERR_TIMEOUT in the device status word and makes the kernel stop, wait (bounded)
 * for its own copies and tensor-core work in flight, free its tensor memory and
 * return, so the device stays usable.  This call arms the next score-kernel launch
 * made by the calling host thread (by any entry point) so that its MMA-issuing thread
 * first waits on an internal barrier that nothing ever completes, for at most
 * limit_ns nanoseconds; that launch then takes the path above and its outputs are
 * unspecified.  The arming is used up by that one launch; limit_ns = 0 disarms.
 * Returns DSA_OK.
 */
dsa_status dsa_test_arm_score_timeout(unsigned long long limit_ns);

/*
 * dsa_test_arm_prefix_mla_timeout -- the same for the attention kernel of dsa_prefix_mla,
 * which runs on pairs of CTAs: in the next dsa_prefix_mla launch of the calling host thread
 * one role (in the same CTA of every pair) waits on an internal barrier that nothing ever
 * completes, for about limit_ns (at most 1e9).  site:
 *   1 MMA issuer, before its block of keys number `at`; 2 copies of the keys for the logits,
 *   3 copies of the keys for the output, before the first; 4 query rows, before piece `at`
 *   (1 and up); 5 softmax, at its start; 10 .. 13 are 2 .. 5 in the odd CTAs.
 * DSA_ERR_INVALID_ARGUMENT for another site or limit; limit_ns = 0 disarms.
 */
dsa_status dsa_test_arm_prefix_mla_timeout(int site, unsigned at, unsigned long long limit_ns);

/*
 * dsa_test_arm_quant_mla_timeout -- the same for the attention kernel of dsa_quant_mla, in its CTAs of
 * even number.  site, each before its number `at` of a CTA:
 *   1 MMA issuer, block of 64 keys; 2, 3 either warp that copies rows, block; 4 the warp that looks
 *   them up, batch of 4 blocks; 5 one warp of the queries, query and 64 heads; 6 one warp that decodes
 *   4-bit rows, block; 7 one warp of the softmax, block; 9 .. 15 are 1 .. 7 in the CTAs of odd number.
 * A site that the call does not come to changes nothing.
 */
dsa_status dsa_test_arm_quant_mla_timeout(int site, unsigned at, unsigned long long limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* DSA_INDEXER_H */
