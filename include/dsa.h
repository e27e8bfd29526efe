/*
 * dsa.h — C ABI of libdsa.so, the GB300 (sm_103a) DSA hot path.
 *
 * DSA ("dynamic sparse attention") is the sparse-attention layer of a hybrid
 * MLA-based model.  A lightweight Lightning Indexer scores every historical
 * position of a query, keeps the Top-K positions, and Sparse Flash Attention
 * (SFA) attends over the MLA latent KV rows at just those positions
 * ("Day0 Inference Adaptation and Performance Optimization for New-Architecture
 * LLMs", §2.2 The Sparse Attention Path and §4.1 Indexer Fusion; "Day0 Inference
 * Adaptation and Performance Optimization for a New Architecture Domestic Large
 * Language Model on Ascend", §2 and §4).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Return value.  Every call returns a dsa_status code (0 = DSA_OK).  No C++
 *   exception crosses the ABI.  dsa_last_error() gives a message for the last
 *   failing call of the calling thread.
 * Pointers.  Every tensor pointer is caller-owned DEVICE memory (cudaMalloc or
 *   torch), 16-byte aligned.  The library never allocates, frees or retains
 *   them.  Tensors are dense, row-major, packed along tokens (no padding
 *   between sequences).
 * Streams.  `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *   stream).  Calls only enqueue work; argument checks are synchronous and a
 *   failing check launches nothing.
 * Workspace.  Every call takes a caller-owned device workspace of at least
 *   dsa_workspace_size() bytes.  Its first 16384 bytes are the status block.  Its
 *   first word is the device status word: kernels OR DSA_FLAG_* bits into it when
 *   they detect bad data (an index out of range, inconsistent cu_q/cu_k) or give
 *   up a bounded wait.  The word is sticky: clear it with dsa_clear_status() and
 *   read it with dsa_read_status().  The block's other words are counters through
 *   which the thread blocks of one kernel wait for each other; they must be zero
 *   before the workspace's first call (a zero-filled workspace, or
 *   dsa_clear_status()), and every call that completes without DSA_FLAG_TIMEOUT
 *   leaves them consistent.  After a call that set DSA_FLAG_TIMEOUT, call
 *   dsa_clear_status() before the next one.  The rest of the
 *   workspace is scratch owned by the call while it runs; calls sharing one
 *   workspace must be stream-ordered.  Its contents between calls are the
 *   caller's (a call never relies on earlier contents).
 * Sequences.  Query rows and key rows are packed: sequence b owns query rows
 *   cu_q[b] .. cu_q[b+1]-1 and key rows cu_k[b] .. cu_k[b+1]-1, with
 *   T_b = cu_q[b+1]-cu_q[b] <= L_b = cu_k[b+1]-cu_k[b].  The queries of a
 *   sequence are its last T_b tokens: query i of sequence b is at position
 *   pos = L_b - T_b + i and sees keys 0..pos of its own sequence (causal,
 *   inclusive; index computation is causal, "… New-Architecture LLMs" §6.2).
 *   Prefill has T_b = L_b (pos = i); decode has T_b = 1 (pos = L_b - 1).
 *   Positions written to / read from `idx` are local to the sequence.  The key-side
 *   tensors (k_idx, kv, k_scale) are either packed the same way or paged through a
 *   block table (dsa_problem.page_size, below).
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_ABI_VERSION 4

/* Return codes. */
enum dsa_status {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, bad size, inconsistent descriptor */
  DSA_ERR_UNSUPPORTED = 2,  /* a valid combination this build has no kernel for */
  DSA_ERR_CUDA = 3,         /* a CUDA runtime call or a launch failed */
  DSA_ERR_WORKSPACE = 4,    /* workspace missing or smaller than dsa_workspace_size() */
  DSA_ERR_TIMEOUT = 5       /* dsa_read_status saw DSA_FLAG_TIMEOUT */
};

/* Element types. */
enum dsa_dtype {
  DSA_F32 = 0,       /* IEEE binary32 */
  DSA_BF16 = 1,      /* bfloat16 */
  DSA_FP8_E4M3 = 2,  /* OCP FP8 E4M3 ("fn": no infinities), with fp32 scales */
  DSA_MXFP8_E4M3 = 3 /* MXFP8: E4M3 codes with one E8M0 scale (2^(e-127)) per 32 elements */
};

/* Device status flags (bits of the workspace status word). */
#define DSA_FLAG_BAD_INDEX 0x1u  /* SFA met an index outside [0, pos]; that entry was skipped */
#define DSA_FLAG_BAD_SEQS  0x2u  /* cu_q/cu_k inconsistent with the descriptor; rows were skipped */
#define DSA_FLAG_TIMEOUT   0x4u  /* a bounded on-device wait gave up; outputs are not valid */
#define DSA_FLAG_CHECK     0x8u  /* checked build only (libdsa_checked.so, -DDSA_CHECKED): an
                                  * internal invariant failed (a gather row outside the cache, a
                                  * tile coordinate or query row out of range, an output slot at
                                  * or past top_k); the access was clamped or skipped */
#define DSA_FLAG_NO_PAGES  0x10u /* dsa_reserve_pages: too few free pages; some rows got none */

/* Operations, for dsa_workspace_size(). */
enum dsa_op {
  DSA_OP_INDEXER_SCORES = 1,
  DSA_OP_TOPK = 2,
  DSA_OP_FUSED_INDEXER = 3,
  DSA_OP_SPARSE_MLA_ATTN = 4,
  DSA_OP_FUSED_FORWARD = 5,
  DSA_OP_PREFIX_MLA_ATTN = 6,
  DSA_OP_ATTN_WEIGHTS = 7,
  DSA_OP_EVICT = 8,
  DSA_OP_KV4_ROWS = 9,         /* dsa_write_kv4, dsa_read_kv4 */
  DSA_OP_SPARSE_MLA_ATTN4 = 10
};

/* Shape, types and sequence layout of one DSA problem. */
typedef struct dsa_problem {
  int32_t num_seqs;    /* B >= 1 */
  int32_t total_q;     /* ΣT_b >= 0: packed query rows */
  int32_t total_k;     /* ΣL_b >= 1: packed key rows */
  int32_t max_q_len;   /* max_b T_b (an upper bound is fine) */
  int32_t max_k_len;   /* max_b L_b (an upper bound is fine) */
  int32_t h_idx;       /* H_I: indexer heads */
  int32_t d_idx;       /* d_I: indexer head width */
  int32_t h;           /* H: MLA query heads (all share one latent row per key) */
  int32_t d_c;         /* latent width = value width */
  int32_t d_rope;      /* rope width; a latent row has D = d_c + d_rope columns */
  int32_t top_k;       /* k: positions kept per query */
  int32_t idx_dtype;   /* dsa_dtype of q_idx and k_idx (F32, BF16, FP8_E4M3, MXFP8_E4M3) */
  int32_t kv_dtype;    /* dsa_dtype of q and kv (F32 or BF16) */
  int32_t out_dtype;   /* dsa_dtype of out (F32 or BF16) */
  float sm_scale;      /* softmax scale; 0 selects 1/sqrt(D) */
  const int32_t* cu_q; /* device int32 [B+1], cu_q[0] = 0, cu_q[B] = total_q */
  const int32_t* cu_k; /* device int32 [B+1], cu_k[0] = 0, cu_k[B] = total_k */
  /* Paged key caches ("Day0 Inference Adaptation and Performance Optimization for
   * New-Architecture LLMs", §4.1: the fused indexer reads the paged K cache directly; "… on
   * Ascend", §4: the cache layout has to match the operators' addressing).  page_size = 0:
   * the caches are packed along tokens as described above (k_idx, kv and k_scale have
   * total_k rows, sequence b owning rows cu_k[b] .. cu_k[b+1]-1).  page_size > 0: the
   * caches hold num_pages pages of page_size rows each (num_pages * page_size rows), and
   * key position s of sequence b lives in cache row
   *   block_table[b * max_pages + s / page_size] * page_size + s % page_size;
   * cu_k then only gives the sequence lengths L_b = cu_k[b+1] - cu_k[b].  page_size must be
   * a power of two >= 16; max_pages * page_size >= max_k_len; num_pages * page_size < 2^31.  A block-table entry outside [0, num_pages) is reported with
   * DSA_FLAG_BAD_SEQS when the indexer reads it (those keys score 0) and with
   * DSA_FLAG_BAD_INDEX when attention meets one of its positions (the entry is skipped). */
  int32_t page_size;          /* 0 (contiguous) or the rows of a page */
  int32_t max_pages;          /* pages per block-table row */
  int32_t num_pages;          /* pages in the caches */
  const int32_t* block_table; /* device int32 [num_seqs][max_pages], or NULL if not paged */
} dsa_problem;

/* Limits of this build: 1 <= h_idx <= 128, d_idx in {16..256, multiple of 16},
 * 1 <= h <= 128, d_c in {16..1024, multiple of 16}, d_rope in {0..256, multiple
 * of 16}, 1 <= top_k <= 2048, max_k_len <= 2^30.  Outside them a call returns
 * DSA_ERR_UNSUPPORTED. */

/* Bytes of workspace `op` needs for problem `p` (always >= 16384). */
int dsa_workspace_size(const dsa_problem* p, int op, size_t* bytes);

/*
 * Lightning-Indexer relevance scores, materialised (for checking and
 * debugging; the fused calls below never write them to memory).
 *   scores[t, s] = Σ_j w[t,j] · ReLU(q_idx[t,j,:] · k_idx[s,:])   for s <= pos(t)
 *   scores[t, s] = -inf                                          for pos(t) < s < ld
 * ("… New-Architecture LLMs" §4.1: batched dot of the indexer query with the K
 * cache, then a weighted sum over heads; §2.2: each historical position gets a
 * relevance score.)
 * q_idx  [total_q, h_idx, d_idx] idx_dtype
 * k_idx  [total_k, d_idx]        idx_dtype
 * w      [total_q, h_idx]        f32 head weights
 * q_scale [total_q, h_idx] f32, k_scale [total_k] f32: dequantisation scales,
 *        required (and > 0) for FP8_E4M3, ignored (may be NULL) for F32/BF16:
 *        q = code·q_scale[t,j], k = code·k_scale[s].
 *        For MXFP8_E4M3 ("… New-Architecture LLMs" §5.1: index-side Q and K in
 *        MXFP8, one scale per 32 elements; d_idx a multiple of 32) the same two
 *        arguments point to E8M0 bytes instead: q_scale [total_q, h_idx, d_idx/32],
 *        k_scale [total_k, d_idx/32] (paged like k_idx), and
 *        q[t,j,c] = code·2^(q_scale[t,j,c/32] - 127), k[s,c] = code·2^(k_scale[s,c/32] - 127);
 *        byte 255 (NaN) is not allowed.
 * scores [total_q, ld] f32, ld >= max_k_len.
 */
int dsa_indexer_scores(const dsa_problem* p, const void* q_idx, const void* k_idx,
                       const float* w, const float* q_scale, const float* k_scale,
                       float* scores, int64_t ld, void* ws, size_t ws_bytes, void* stream);

/*
 * Causal Top-K of materialised scores (Top-K selection of the indexer,
 * "… New-Architecture LLMs" §4.1).  For each query row t, idx[t, 0..n-1]
 * (n = min(top_k, pos+1)) receives the positions of the n largest
 * scores[t, 0..pos], in ascending position order; among equal scores the
 * smaller positions are kept.  idx[t, n..top_k-1] = -1.
 * scores [total_q, ld] f32 (only columns 0..pos(t) are read)
 * idx    [total_q, top_k] int32
 * vals   [total_q, top_k] f32 or NULL: the selected scores (-inf in padding).
 */
int dsa_topk(const dsa_problem* p, const float* scores, int64_t ld, int32_t* idx, float* vals,
             void* ws, size_t ws_bytes, void* stream);

/*
 * The fused Lightning Indexer: scoring, head weighting and Top-K in one pass
 * over the K cache, writing only the selected positions ("… New-Architecture
 * LLMs" §4.1 fused_indexer(q_idx, k_cache, head_weights, top_k); "Optimizing
 * LLM Inference for New Architectures", §3: only the final Top-K indices leave
 * the operator).  Arguments and results are those of dsa_indexer_scores
 * followed by dsa_topk, except that the selected positions of a row may come
 * in any (deterministic) order: valid entries first, then -1 padding.
 */
int dsa_fused_indexer(const dsa_problem* p, const void* q_idx, const void* k_idx,
                      const float* w, const float* q_scale, const float* k_scale,
                      int32_t* idx, float* vals, void* ws, size_t ws_bytes, void* stream);

/*
 * Sparse Flash Attention over the MLA latent cache at the selected positions
 * ("… New-Architecture LLMs" §2.2 and §4.1: gather the selected KV rows and
 * attend over that subset; "… on Ascend" §4: SFA reads the KV cache at the
 * position set the indexer outputs).  For query row t and head h, over the
 * valid entries i of idx[t, :]:
 *   S_i = sm_scale · q[t,h,:] · kv[cu_k[b] + idx[t,i], :]        (all D columns)
 *   out[t,h,:] = Σ_i softmax(S)_i · kv[cu_k[b] + idx[t,i], 0:d_c]
 *   lse[t,h]   = log Σ_i exp(S_i)                                 (natural log)
 * q   [total_q, h, D] kv_dtype;  kv [total_k, D] kv_dtype (D = d_c + d_rope)
 * idx [total_q, top_k] int32: -1 entries are skipped; an entry outside
 *     [0, pos(t)] sets DSA_FLAG_BAD_INDEX and is skipped; order is free;
 *     a repeated entry counts as often as it appears.
 * out [total_q, h, d_c] out_dtype; lse [total_q, h] f32 or NULL.
 * A row with no valid entry gets out = 0 and lse = -inf.
 */
int dsa_sparse_mla_attn(const dsa_problem* p, const void* q, const void* kv, const int32_t* idx,
                        void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * The whole DSA layer: dsa_fused_indexer then dsa_sparse_mla_attn on the same
 * stream ("… on Ascend" §4: the fused indexer's selected positions feed SFA).
 * idx_out [total_q, top_k] int32 and vals_out [total_q, top_k] f32 are optional
 * (NULL: kept in the workspace only).
 */
int dsa_fused_forward(const dsa_problem* p, const void* q_idx, const void* k_idx,
                      const float* w, const float* q_scale, const float* k_scale,
                      const void* q, const void* kv, void* out, float* lse,
                      int32_t* idx_out, float* vals_out, void* ws, size_t ws_bytes,
                      void* stream);

/*
 * dsa_fused_indexer_static: dsa_fused_indexer for callers that cannot allocate
 * device memory.  The pages have no counterpart of this call; it exists for
 * code that runs inside a host framework owning all device memory (a fixed
 * budget or its own caching allocator, raw cudaMalloc forbidden) and for
 * latency-critical loops where cudaMalloc/cudaFree would synchronise the
 * device.  Such callers pass inputs and outputs but no workspace.
 *
 * Scratch is a static device array inside the library: a 16384-byte status block
 * plus room for 4,194,304 fp32 scores (16 MiB), held by every device that loads
 * the library until the process exits.  Problems with total_q * max_k_len above
 * 4,194,304 are rejected with DSA_ERR_UNSUPPORTED.  The call allocates nothing
 * (no cudaMalloc, cudaFree or allocating library routine).  Its first call on a
 * device looks up the array's address with that device current; make that first
 * call before any stream capture.  All calls on one device share the array:
 * calls that overlap on the GPU race, and the array keeps the last call's
 * contents.  Each call zeroes the status block first; if flags_out (device
 * memory, may be NULL) is given, the call's DSA_FLAG_* bits are copied there
 * at its end.  Other arguments and results are those of dsa_fused_indexer.
 */
int dsa_fused_indexer_static(const dsa_problem* p, const void* q_idx, const void* k_idx,
                             const float* w, const float* q_scale, const float* k_scale,
                             int32_t* idx, float* vals, uint32_t* flags_out, void* stream);

/*
 * The indexer prolog: Q quantisation and the head-weight projection, the two
 * input-preparation steps that share one stream ahead of the fused indexer
 * ("… New-Architecture LLMs" §4.2 Three-Stream Coordination for Indexer
 * Preprocessing: q_quant = quant(q_proj), w_proj = W_h @ x; "Optimizing LLM
 * Inference for New Architectures", §3), fused into one launch.  For token t:
 *   amax = max |q_proj[t, :, :]|,  scale = amax / 448 (fp32; 1 if amax = 0)
 *   q_codes[t, j, e] = E4M3(q_proj[t, j, e] / scale)  (fp32 division, round to
 *                      nearest even, saturated to ±448)
 *   q_scale[t, j]    = scale for every head j (one scale per token)
 *   w[t, j]          = Σ_c W_h[j, c] · x[t, c]   (fp32 accumulation)
 * These are the FP8 inputs (q_idx, q_scale, w) of dsa_fused_indexer.
 * q_proj  [total_q, h_idx, d_idx] bf16, d_idx a multiple of 8, or NULL (no
 *         quantisation; q_codes and q_scale are then ignored);
 * x       [total_q, d_model] bf16 and w_h [h_idx, d_model] bf16, d_model a
 *         positive multiple of 8, or both NULL (no projection; w ignored);
 * q_codes [total_q, h_idx, d_idx] uint8 (E4M3 codes), q_scale [total_q, h_idx]
 *         f32, w [total_q, h_idx] f32: outputs, caller-owned device memory.
 * q_proj, x, w_h and q_codes are 16-byte aligned; q_scale and w 4-byte.
 * One launch on `stream`, no workspace.  total_q = 0 launches nothing and
 * accepts NULL pointers.
 * DSA_ERR_INVALID_ARG for missing or misaligned pointers (or all inputs NULL),
 * DSA_ERR_UNSUPPORTED for sizes outside those limits.
 */
int dsa_indexer_prolog(int32_t total_q, int32_t h_idx, int32_t d_idx, int32_t d_model,
                       const void* q_proj, const void* x, const void* w_h, uint8_t* q_codes,
                       float* q_scale, float* w, void* stream);

/*
 * The residual's addition and the root-mean-square norm, with the output in the input's type,
 * in 8 bits with scales, or both ("… New-Architecture LLMs" §4.2: the indexer's preprocessing
 * normalises the K side; §5.1: the index side is quantised).  For each of `rows` rows of d
 * elements, in fp32:
 *   h = x + residual  (h = x without a residual; h_out is h rounded to dtype)
 *   y = h · rsqrt(Σ h² / d + eps) · weight  (from the unrounded h)
 *   quant = DSA_FP8_E4M3: scale[r] = max|y| / 448 (f32, formed as max|h · weight| · rsqrt(...) / 448; 1 where
 *     that is below the smallest normal number), codes = E4M3(y · r) (nearest even, saturated to ±448) with r the
 *     fp32 reciprocal of scale (E4M3(y / scale) differs, by one code, only where y / scale lies within a few fp32
 *     roundings of the middle between two codes): on rows of d_idx elements these are k_idx and k_scale of the FP8 indexer;
 *   quant = DSA_MXFP8_E4M3: scale[r, g] the E8M0 byte e + 127 of the smallest power of two with
 *     max|y| <= 448·2^e over the 32 elements of group g (127 for an all-zero group; byte 255
 *     is never written), codes = E4M3(y / 2^e): k_idx and k_scale of the MXFP8 indexer;
 *   quant = 0: no codes (codes and scale are ignored).
 * A row with a NaN or an infinity comes out as NaN where 0 · infinity or a NaN arises, like the formula; so does
 * Σ h² that overflows fp32 (|h| from about 2^64 / √d on) count as infinite: y is 0 there.
 * x [rows, d] and residual [rows, d] dtype (F32 or BF16), row strides ld_x, ld_res >= d elements;
 * weight [d] dtype; h_out [rows, d] dtype, required with residual (NULL without); y [rows, d]
 * dtype, required without quant (may be NULL with); codes [rows, d] bytes; scale [rows] f32 or
 * [rows, d/32] bytes.  h_out and y may be x or residual themselves where that one's row stride is
 * d; other overlaps of an output are refused.  Pointers need the alignment of their element; 16-byte aligned
 * rows are faster.  Any d in 1 .. 2^24 (MXFP8: a multiple of 32).
 * One launch, no workspace.  rows = 0 launches nothing and accepts NULL pointers.
 */
int dsa_add_rmsnorm(int64_t rows, int32_t d, int32_t dtype, int32_t quant, float eps,
                    const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                    const void* weight, void* h_out, void* y, uint8_t* codes, void* scale,
                    void* stream);

/*
 * Dense MLA attention for a batch that shares a prefix.  Every query attends over the prefix's
 * prefix_len latent rows and, causally, over its own sequence's (the cache rows p describes:
 * the sequence's tokens after the prefix).  For query row t at position pos of its sequence b
 * and head h, over the keys x = the prefix rows, then rows 0..pos of sequence b:
 *   S_x = sm_scale · q[t,h,:] · key_x   (all D columns)
 *   out[t,h,:] = Σ_x softmax(S)_x · key_x[0:d_c],   lse[t,h] = log Σ_x exp(S_x)
 * The prefix is attended by all rows together, 128 (token, head) rows at a time, not sequence by
 * sequence.  prefix_len = 0 gives dense causal attention over each sequence alone (what sparse
 * attention equals while a history has at most top_k positions).
 * q, kv, out, lse as in dsa_sparse_mla_attn; h_idx, d_idx, top_k and idx_dtype are not used
 * (top_k still has to be valid).
 * prefix_kv [prefix_len, D] kv_dtype, 16-byte aligned: the prefix's rows; or NULL with
 * prefix_table [ceil(prefix_len / page_size)] device int32 (4-byte aligned): its pages in the
 * paged cache kv.  Exactly one of the two where prefix_len > 0; prefix_table needs a paged p.
 * A key that a row does not see adds nothing to it, whatever it holds.  A visible key with an infinity or a NaN among its
 * value columns makes those columns of out NaN (0 times it, where its logit is -inf), or all of them.
 * A page outside the cache sets DSA_FLAG_BAD_INDEX; its keys are skipped.  A row without any key, or
 * whose logits are all -inf, gets out = 0 and lse = -inf (but for NaN columns as above).  Rows of a sequence whose cu_q/cu_k are inconsistent are flagged
 * (DSA_FLAG_BAD_SEQS) and left as they were.
 * prefix_len + max_k_len < 2^30.
 */
int dsa_prefix_mla_attn(const dsa_problem* p, int32_t prefix_len, const void* prefix_kv,
                        const int32_t* prefix_table, const void* q, const void* kv, void* out,
                        float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * The attention weight that cached positions received, accumulated (what dsa_evict goes by).
 * For every query row t of sequence b and every valid entry i of idx[t, :]:
 *   acc[b, idx[t,i]] += Σ_h exp(sm_scale · q[t,h,:]·kv[row of idx[t,i], :] − lse[t,h])
 * with idx and lse those of dsa_sparse_mla_attn on the same q and kv.  Entries that attention
 * skips add nothing (rows of a sequence whose cu_q/cu_k are inconsistent, or that has more than max_q_len
 * queries, set DSA_FLAG_BAD_SEQS; an entry outside [0, pos(t)] or on a page outside the cache sets
 * DSA_FLAG_BAD_INDEX); neither do heads whose lse is -inf; a repeated entry adds as often
 * as it appears.  The result does not depend on the order of the additions: the same call gives the
 * same bytes.  Where max_q_len > 1 the weights are added in 64-bit fixed point, each rounded to half a unit of
 * 2^-(62 - c), 2^c the first power of two from 2 · h · max_q_len on (128 heads x 4096 queries: 2^-42), and then once to acc.
 * That holds a position's sum as long as lse belongs to this idx (a query's weights then add up to
 * h over its entries).  With a smaller lse the sums mean nothing, may wrap around where an entry is repeated, and
 * weights above 2 · h are added in no fixed order.
 * q, kv, idx, lse as in dsa_sparse_mla_attn (lse required); acc [num_seqs, ld_acc] f32, ld_acc >=
 * max_k_len, added to in place (columns at or past a sequence's length stay as they are).
 */
int dsa_accumulate_attn_weights(const dsa_problem* p, const void* q, const void* kv,
                                const int32_t* idx, const float* lse, float* acc, int64_t ld_acc,
                                void* ws, size_t ws_bytes, void* stream);

/*
 * Eviction from the caches by accumulated attention weight.  Sequence b (L_b positions) keeps
 * n_b = min(L_b, budget): all where L_b <= budget; otherwise its first `sink` positions, its last
 * `recent` ones, and the budget - sink - recent with the largest acc between them (among equal
 * ones the smaller positions; every NaN counts as larger than any number).  Kept
 * positions keep their order and move to the caches' *_out tensors:
 *   kept[b, 0..n_b-1] = the kept positions, ascending; kept[b, n_b..budget-1] = -1
 *   cu_k_out[b] = Σ_{b' < b} n_b'                           (num_seqs + 1 entries)
 *   acc_out[b, i] = acc[b, kept[b, i]] for i < n_b, 0 for n_b <= i < budget (columns at or past
 *     budget stay as they were)
 *   kv_out, k_idx_out, k_scale_out: row of position i of sequence b in the destination =
 *     the source's row of position kept[b, i].
 * The destination is packed (sequence b at rows cu_k_out[b] ..; rows_out rows in all), or, with
 * table_out [num_seqs, max_pages_out] (device int32; p paged), paged with p's page_size over
 * num_pages_out pages (rows_out is then ignored).  Rows of the destination that
 * hold no kept position stay as they were.  A page outside either cache, or a packed row at or
 * past rows_out, sets DSA_FLAG_BAD_SEQS and the row is not moved.  A sequence whose cu_k is inconsistent keeps
 * nothing (DSA_FLAG_BAD_SEQS).
 * Each of kv (row: D of kv_dtype), k_idx (d_idx of idx_dtype) and k_scale (4 bytes for FP8, d_idx/32 for
 * MXFP8) comes with its *_out, or both are NULL (not moved).  Destination rows must not be rows
 * the call reads: a packed *_out that overlaps its source is refused; with pages, source and
 * destination may be one pool, in which the destination's pages must not be the sources'.
 * acc [num_seqs, ld_acc >= max_k_len] f32; acc_out [num_seqs, ld_acc_out >= budget] f32 or NULL, whose bytes from first to
 * last element and acc's do not overlap; cu_k_out not overlapping p's cu_k; 1 <= budget, 0 <= sink, 0 <= recent, sink + recent <= budget.
 */
int dsa_evict(const dsa_problem* p, const float* acc, int64_t ld_acc, int32_t budget, int32_t sink,
              int32_t recent, int32_t* kept, int32_t* cu_k_out, float* acc_out, int64_t ld_acc_out,
              const void* kv, void* kv_out, const void* k_idx, void* k_idx_out,
              const void* k_scale, void* k_scale_out, const int32_t* table_out,
              int32_t max_pages_out, int32_t num_pages_out, int64_t rows_out, void* ws,
              size_t ws_bytes, void* stream);

/*
 * Rotary positions with several axes (time, height, width, ...), on the rope columns of queries or
 * of keys ahead of their cache.  For token t, head h and pair i of d / 2, (u, v) the pair's columns:
 *   phi = positions[axis[i], t] * turn[i] * 2 pi / 2^64
 *   (u, v) -> (u cos phi - v sin phi, u sin phi + v cos phi);  inverse: with -phi
 * turn[i] is the turns of one position as a fixed-point fraction of 2^64 (a frequency of f radians a position:
 * f / (2 pi) * 2^64, modulo 2^64), so that angles of positions up to +-2^31 are exact modulo one turn
 * but for turn's own rounding; sine, cosine and products are fp32, rounded once to dtype.
 * interleaved: pair i is columns 2i and 2i + 1; otherwise i and i + d/2.
 * x, out: element (t, h, c) at t * x_token + h * x_head + c (strides in elements, >= 0), F32 or BF16,
 * aligned to their element (rows on 16-byte boundaries are faster); out may be x with the same strides,
 * and otherwise must not overlap it (tensors with the same strides that interleave without
 * sharing an element, as two column ranges of one tensor, may, whichever of tokens and heads is outside) nor the positions.
 * positions [axes][ld_pos] device int32, ld_pos >= tokens or 0 (all axes have the same ones); turn [d/2] and axis [d/2] HOST memory, read before
 * the call returns; axis[i] < axes <= 255.  d even, 2 .. 256.  One launch, no workspace; tokens = 0 launches nothing.
 */
int dsa_rotate_axes(int64_t tokens, int32_t heads, int32_t d, int32_t dtype, int32_t interleaved,
                    int32_t inverse, int32_t axes, const uint64_t* turn, const uint8_t* axis,
                    const int32_t* positions, int64_t ld_pos, const void* x, int64_t x_token,
                    int64_t x_head, void* out, int64_t out_token, int64_t out_head, void* stream);

/*
 * The latent cache in 4 bits.  A cache row of D = d_c + d_rope columns takes
 * dsa_kv4_row_bytes(d_c, d_rope) bytes (512 + 64: 416 instead of 1152), in this order:
 *   d_c / 2     codes: E2M1 (a sign; magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6), eight columns a
 *               little-endian 32-bit word: of eight, column 2k at bit 4k, column 2k + 1 at bit 16 + 4k
 *   2 * d_rope  the rope columns in bf16
 *   d_c / 16    scales, a byte for 16 columns: an fp16 number without its sign and its seven
 *               lowest bits (byte << 7; 0 .. 61440 in steps of at most 1/8, 0xf8 and above: NaN)
 *   zeros up to a multiple of 16 bytes
 * Column c < d_c is code[c] * scale[c / 16], which is a bf16 number exactly.  The cache is packed or
 * paged like kv: [cache rows][row bytes] uint8.
 */
int dsa_kv4_row_bytes(int32_t d_c, int32_t d_rope, int32_t* bytes);

/*
 * Write the new tokens' rows: query row t of p (the last T_b positions of its sequence b) goes to the
 * cache row of its position.  Over every 16 latent columns
 *   scale = max|x| / 6 to the nearest scale (ties to even, at most 61440),
 *   code  = x / scale to the nearest code (ties to even, at most 6 in magnitude; 0 where the scale is 0);
 * 16 columns with an infinity or a NaN among them become NaN (scale byte 0xff).  Rope columns are rounded to bf16.
 * latent [total_q, d_c] and k_rope [total_q, d_rope] kv_dtype, rows ld_latent >= d_c and ld_rope >= d_rope
 * elements apart, aligned to their element (16-byte aligned rows are faster); k_rope may be NULL
 * where d_rope = 0.  kv4 must not overlap them.  Rows of a sequence whose cu_q/cu_k are inconsistent, and rows on
 * a page outside the cache, set DSA_FLAG_BAD_SEQS and are not written.  Other rows stay as they were.
 */
int dsa_write_kv4(const dsa_problem* p, const void* latent, int64_t ld_latent, const void* k_rope,
                  int64_t ld_rope, void* kv4, void* ws, size_t ws_bytes, void* stream);

/*
 * Read every position's row back, packed: out [total_k, D] kv_dtype, row cu_k[b] + s = position s of
 * sequence b (what dense attention over the sequence, or over it as a shared prefix, takes).  Rows of a sequence
 * whose cu_k is inconsistent (DSA_FLAG_BAD_SEQS) or on a page outside the cache (DSA_FLAG_BAD_INDEX) are left as
 * they were.  out must not overlap kv4.
 */
int dsa_read_kv4(const dsa_problem* p, const void* kv4, void* out, void* ws, size_t ws_bytes,
                 void* stream);

/*
 * dsa_sparse_mla_attn over a 4-bit latent cache: the same sums with kv's rows decoded from kv4
 * [cache rows][row bytes].  q, idx, out and lse, skipped and repeated entries as there; a row without a valid entry,
 * or whose logits are all -inf, gets out = 0 and lse = -inf.  An entry that is skipped adds nothing, whatever its row holds.
 * Rows of a sequence whose cu_q/cu_k are inconsistent, or that has more than max_q_len queries, set DSA_FLAG_BAD_SEQS
 * and are left as they were.  out and lse must not overlap each other, q, kv4 or idx.
 * Rounding: fp32 throughout, but for bf16 queries over 512 + 64 columns (tensor cores).  There each probability is rounded to bf16 ahead
 * of its product with the values (the sum it is divided by is of unrounded ones), also where out_dtype is F32; and a query's
 * latent columns are held relative to the head's largest finite one, each off by at most 2^-39 of that: columns smaller than
 * 2^-29 of it lose bits, those smaller than 2^-39 count as 0.
 */
int dsa_sparse_mla_attn4(const dsa_problem* p, const void* q, const void* kv4, const int32_t* idx,
                         void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * Pages shared by rows of a block table.  table [rows, width] int32 (rows ld_table >= width apart) holds the pages of a
 * row in order, -1 behind them; refs [num_pages] int32 counts the table entries that hold a page.  A page
 * with refs <= 0 is free.  All results depend on the arguments alone: the lowest free pages are given out first.
 * page_size: a power of two >= 16; num_pages * page_size < 2^31, rows * width < 2^31.  All int32 arrays are device
 * memory, 4-byte aligned, and must not overlap.  caches: `num_caches` <= 8 device addresses (16-byte aligned) of
 * caches with num_pages * page_size rows of row_bytes[c] bytes each (both arrays HOST memory, read before the call returns).
 * An entry that names a row outside the table, positions beyond it or a page outside the pool is left out and sets
 * DSA_FLAG_BAD_INDEX.
 */

/* Bytes of workspace that the calls below need: with n entries at most, whatever their order (n = 0:
 * dsa_fork_pages and dsa_free_pages need 16384). */
int dsa_pages_workspace_size(int32_t rows, int32_t n, int32_t num_pages, size_t* bytes);

/*
 * Fork: for each entry i, row dst[i] gets the pages of row src[i]'s first lens[i] positions, shared
 * (refs + 1 each), and -1 behind them.  What row dst[i] held before is not given back (dsa_free_pages does that).  Where a row
 * is named by several dst the first entry counts; an entry whose src is some entry's dst is left out.
 * Neither row's cache rows are touched: dsa_reserve_pages makes a page of its own for the tokens that follow.
 */
int dsa_fork_pages(int32_t* table, int32_t rows, int32_t width, int64_t ld_table, int32_t* refs,
                   int32_t num_pages, int32_t page_size, int32_t n, const int32_t* src,
                   const int32_t* dst, const int32_t* lens, void* ws, size_t ws_bytes, void* stream);

/* Free: every page of the rows named has a holder less, and their entries become -1.  A row may be named twice. */
int dsa_free_pages(int32_t* table, int32_t rows, int32_t width, int64_t ld_table, int32_t* refs,
                   int32_t num_pages, int32_t n, const int32_t* row, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * Reserve: row[i], which holds lens[i] positions, gets pages of its own for positions lens[i] ..
 * new_lens[i] - 1.  New pages where it has none (or shares one there); and where its last held page is not
 * full, will be written to and has other holders, a new page with the held positions' rows copied in all
 * caches (their other rows stay as they were) - but if all the page's holders are entries of this call that
 * would copy it, the first of them keeps it.  Pages are given out entry by entry; an entry gets
 * all it needs or nothing (then DSA_FLAG_NO_PAGES is set, also for every later entry that needs pages).  An entry that was to
 * keep a page gets nothing where one of those that were to copy it gets nothing, as that one goes on holding the page: no page of
 * positions lens[i] .. held[i] - 1 has another holder after the call.
 * held[i] = new_lens[i], or lens[i] where the entry got nothing.  Of several entries of one row the first counts.  Which pages are free and
 * shared is as at the call's start.
 */
int dsa_reserve_pages(int32_t* table, int32_t rows, int32_t width, int64_t ld_table, int32_t* refs,
                      int32_t num_pages, int32_t page_size, int32_t n, const int32_t* row,
                      const int32_t* lens, const int32_t* new_lens, int32_t* held,
                      int32_t num_caches, void* const* caches, const int64_t* row_bytes, void* ws,
                      size_t ws_bytes, void* stream);

/*
 * Compact: the pages in use become pages 0 .. live - 1.  The k-th page in use at or behind `live` moves, in all
 * caches, to the k-th free page before it; table and refs follow.  moved[p] (num_pages) is where page p went (p itself
 * where it stayed, -1 for a free page), live[0] the number of pages in use.  Rows of pages at or behind live
 * keep their bytes.  Every holder has to be in the table: an entry of a free page becomes -1 (DSA_FLAG_BAD_INDEX).
 */
int dsa_compact_pages(int32_t* table, int32_t rows, int32_t width, int64_t ld_table, int32_t* refs,
                      int32_t num_pages, int32_t page_size, int32_t* moved, int32_t* live,
                      int32_t num_caches, void* const* caches, const int64_t* row_bytes, void* ws,
                      size_t ws_bytes, void* stream);

/* Zero the workspace status block (the status word and the kernels' counters; enqueued on
 * `stream`). */
int dsa_clear_status(void* ws, void* stream);

/* Self-test of the bounded-wait path every kernel's waits go through: one thread waits on an
 * mbarrier that nothing arrives at, gives up after limit_ns (0 < limit_ns <= 1e8) and ORs
 * DSA_FLAG_TIMEOUT into the status word of `ws` (enqueued on `stream`; no other effect: the
 * context stays usable).  DSA_ERR_WORKSPACE for a NULL or misaligned `ws`,
 * DSA_ERR_INVALID_ARG for a limit out of range. */
int dsa_selftest_wait_timeout(void* ws, uint64_t limit_ns, void* stream);

/* Synchronise `stream`, then copy the workspace status word into *flags.
 * Returns DSA_ERR_TIMEOUT if DSA_FLAG_TIMEOUT is set, DSA_OK otherwise. */
int dsa_read_status(const void* ws, void* stream, uint32_t* flags);

/* Message of a dsa_status code (static storage). */
const char* dsa_status_str(int status);

/* Message of the last failing call on this thread ("" if none). */
const char* dsa_last_error(void);

/* DSA_ABI_VERSION of the loaded library. */
int dsa_abi_version(void);

/*
 * Launch tracing.  Between dsa_trace_begin(capacity) and dsa_trace_end(), every
 * kernel the library launches is bracketed by a pair of CUDA events recorded on
 * its stream (at most `capacity` launches are kept).  dsa_trace_get() returns
 * the kernel name and the elapsed milliseconds of launch i (it waits for that
 * launch's end event).  dsa_trace_count() gives the number recorded.
 */
int dsa_trace_begin(int capacity);
int dsa_trace_end(void);
int dsa_trace_count(void);
int dsa_trace_get(int i, char* name, int name_len, float* ms);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H_ */
