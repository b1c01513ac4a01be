/*
 * dsa.h -- C ABI of the GB300 (sm_103a) DeepSeek Sparse Attention hot path.
 *
 * Conventions for every entry point:
 *  - Tensor arguments are caller-owned DEVICE pointers to contiguous row-major
 *    storage (innermost dimension last); host pointers are named *_host.
 *  - bf16 tensors are passed as dsa_bf16_t (the raw 16-bit pattern).
 *  - Calls are asynchronous on the caller's CUDA stream (NULL = legacy default
 *    stream); only dsa_packed_metadata and dsa_read_device_status synchronise.
 *  - The library never allocates device memory.  Scratch comes from the
 *    caller's `workspace` (at least dsa_*_workspace_size() bytes, 256-byte
 *    aligned); its first 4 bytes are the device error word (see
 *    dsa_read_device_status).
 *  - Every call returns a dsa_status_t; argument errors are detected on the
 *    host before anything is launched and leave all outputs untouched.
 *    dsa_last_error_message() describes the most recent failure of the calling
 *    thread.
 *
 * Pages cited (title, then section or API entry):
 *  [DSA-blog]  "Accelerating GLM-5.2 Long-Context Training with cuDNN Fused DSA
 *              Kernels and THD-Packed Context Parallelism using Megatron Bridge"
 *  [NoPE-PR]   SkyRL pull request 2388 (NoPE / unaligned top-k SparseMLA)
 *  [cudnn_dsa] NeMo AutoModel API: glm_moe_dsa.kernels.cudnn_dsa
 *  [Chunk-PR]  SkyRL pull request 2423 (query-chunked sparse attention)
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* dsa_stream_t; /* same type as cudaStream_t */
typedef uint16_t dsa_bf16_t;              /* bfloat16 bit pattern */

typedef enum {
  DSA_OK = 0,
  DSA_ERR_UNSUPPORTED = 1,      /* no CUDA device, or the device is not sm_103 */
  DSA_ERR_DTYPE = 2,            /* reserved: the ABI fixes every dtype */
  DSA_ERR_INVALID_ARGUMENT = 3, /* null pointer, bad shape, K or scale */
  DSA_ERR_WORKSPACE = 4,        /* workspace missing, too small or misaligned */
  DSA_ERR_CUDA = 5,             /* a CUDA runtime call or launch failed */
  DSA_ERR_DEVICE_INDEX = 6,     /* device saw an index outside [-1, T_k) (slot masked) */
  DSA_ERR_TIMEOUT = 7,          /* a bounded device-side wait gave up (CTA exited) */
  DSA_ERR_CAPACITY = 8          /* dsa_paged_slots: new tokens do not fit (no request got one) */
} dsa_status_t;

/* Text for a status code (static storage). */
const char* dsa_status_string(dsa_status_t status);
/* Message of the calling thread's most recent failed call ("" if none). */
const char* dsa_last_error_message(void);
/* ABI version: 2 (attention sink arguments of the sparse MLA calls). */
int32_t dsa_abi_version(void);

/*
 * dsa_packed_metadata -- THD packing metadata, no context parallelism.
 * Source: [cudnn_dsa] prepare_cudnn_dsa_packed_metadata and
 * CudnnDsaPackedMetadata (starts, causal_lengths, max_seqlen,
 * all_rows_nonempty): per query token t of sequence i,
 *   seq_start[t] = cu_seqlens[i],  causal_len[t] = t - cu_seqlens[i] + 1.
 *  cu_seqlens   device int32 [num_seqs + 1], cu[0] = 0, non-decreasing, cu[num_seqs] = total_tokens
 *  seq_start    device int32 [total_tokens] (out)
 *  causal_len   device int32 [total_tokens] (out)
 *  max_seqlen_host, all_rows_nonempty_host: host int32 scalars (out), may be NULL
 * Like the pages' routine it performs one device-to-host synchronisation (to
 * validate cu_seqlens and return max_seqlen).  Returns
 * DSA_ERR_INVALID_ARGUMENT if cu_seqlens is not a valid cover of [0, T).
 */
dsa_status_t dsa_packed_metadata(const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                                 int32_t* seq_start, int32_t* causal_len, int32_t* max_seqlen_host,
                                 int32_t* all_rows_nonempty_host, dsa_stream_t stream);

/*
 * dsa_packed_metadata_cp -- THD packing metadata for rank-local queries and
 * gathered global keys (context parallelism).
 * Source: [cudnn_dsa] prepare_cudnn_dsa_packed_metadata (query_indices,
 * cu_seqlens_padded, padding_mask; per-query global padded-storage starts and
 * real causal lengths) and cudnn_indexer_topk (rank-local index_q, gathered
 * global index_k).  With P = cu_seqlens_padded (or cu_seqlens when NULL) and
 * L_i = cu_seqlens[i+1] - cu_seqlens[i], local row r has global coordinate
 * g = query_indices[r] (r when NULL); when P[i] <= g < P[i+1]:
 *   seq_start[r] = P[i],  causal_len[r] = g - P[i] + 1 if g - P[i] < L_i and
 *   padding_mask[r] == 0, else 0 (a padding row);
 * a row outside every sequence's storage gets seq_start[r] = g, causal_len 0.
 *  cu_seqlens         device int32 [num_seqs + 1], from 0, non-decreasing (real tokens)
 *  cu_seqlens_padded  device int32 [num_seqs + 1] or NULL, from 0, non-decreasing,
 *                     P[i+1] - P[i] >= L_i, P[num_seqs] <= total_key_tokens
 *  query_indices      device int32 [T_q] or NULL (then row r is coordinate r and
 *                     T_q <= total_key_tokens), each in [0, total_key_tokens)
 *  padding_mask       device uint8 [T_q] or NULL; nonzero marks a padding row
 *  seq_start, causal_len  device int32 [T_q] (out)
 *  max_seqlen_host    host int32 (out) = max_i L_i, may be NULL
 *  all_rows_nonempty_host  host int32 (out) = 1 iff T_q > 0 and every
 *                     causal_len > 0, may be NULL
 * Performs one device-to-host synchronisation (to validate the inputs and
 * compute the host scalars) and returns DSA_ERR_INVALID_ARGUMENT when any rule
 * above is broken; the outputs are then untouched.  With no optional input it
 * equals dsa_packed_metadata.
 */
dsa_status_t dsa_packed_metadata_cp(const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, int32_t num_seqs,
                                    int32_t total_key_tokens, const int32_t* query_indices,
                                    const uint8_t* padding_mask, int32_t T_q, int32_t* seq_start,
                                    int32_t* causal_len, int32_t* max_seqlen_host, int32_t* all_rows_nonempty_host,
                                    dsa_stream_t stream);

/*
 * dsa_indexer_topk -- lightning-indexer score fused with per-query causal top-k.
 * Source: [DSA-blog] "How DSA works" (the indexer scores query-key relevance
 * and emits the top-k indices per query); [cudnn_dsa] cudnn_indexer_topk
 * (index_q [T, H_index, 128], index_k [T_k, 128], already-scaled head weights,
 * output int32 global indices, K in [1, 2048]); canonical output form from
 * cudnn_sparse_attention's topk_length (compact ascending prefix).
 *   score(t, s) = sum_h w[t,h] * max(0, <q_idx[t,h,:], k_idx[s,:]>),  s in [seq_start[t], t]
 * For each t the n = min(K, causal_len[t]) highest-scoring keys (ties to the
 * lower index) are written ascending to topk_idx[t, 0:n], then -1 up to K.
 * The [T, T_k] score matrix is never written to memory.
 *  q_idx        device bf16 [T, Hi, Di]; Hi in [1, 64], Di = 128
 *  k_idx        device bf16 [T_k, Di]
 *  head_weights device fp32 [T, Hi] (caller applies any scaling)
 *  seq_start    device int32 [T] from dsa_packed_metadata (window start; the
 *               window end is the token itself, so T_k >= T is required)
 *  topk_idx     device int32 [T, K] (out);  topk_len device int32 [T] (out) or NULL
 *  workspace    >= dsa_indexer_topk_workspace_size() bytes
 */
size_t dsa_indexer_topk_workspace_size(int32_t T, int32_t K);
dsa_status_t dsa_indexer_topk(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_idx, const float* head_weights,
                              const int32_t* seq_start, int32_t T, int32_t T_k, int32_t Hi, int32_t Di, int32_t K,
                              int32_t* topk_idx, int32_t* topk_len, void* workspace, size_t workspace_bytes,
                              dsa_stream_t stream);

/*
 * dsa_indexer_topk_cp -- the same kernel for rank-local query rows against the
 * gathered global keys (context parallelism).
 * Source: [cudnn_dsa] cudnn_indexer_topk (rank-local index_q [T_q, H_index,
 * 128], gathered global index_k [T_k, 128], query_indices / packed_metadata).
 * Row r's candidates are the keys [seq_start[r], seq_start[r] + causal_len[r]
 * - 1] (none when causal_len[r] = 0), clipped to [0, T_k); otherwise as
 * dsa_indexer_topk: n = min(K, window size) best keys, ascending, -1 suffix.
 *  q_idx        device bf16 [T_q, Hi, Di] (local rows)
 *  k_idx        device bf16 [T_k, Di] (global keys; no relation between T_k and T_q)
 *  head_weights device fp32 [T_q, Hi]
 *  seq_start, causal_len  device int32 [T_q] from dsa_packed_metadata_cp
 *  topk_idx, topk_len, workspace  as dsa_indexer_topk
 * Errors as dsa_indexer_topk (without the T_k >= T rule), plus
 * DSA_ERR_INVALID_ARGUMENT when causal_len is NULL and T_q > 0.
 */
dsa_status_t dsa_indexer_topk_cp(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_idx, const float* head_weights,
                                 const int32_t* seq_start, const int32_t* causal_len, int32_t T_q, int32_t T_k,
                                 int32_t Hi, int32_t Di, int32_t K, int32_t* topk_idx, int32_t* topk_len,
                                 void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_indexer_topk_with_scores -- diagnostic form of dsa_indexer_topk: the same
 * kernel code and the same results (topk_idx, topk_len), and in addition the
 * fp32 score of every key of the window of rows [score_row0, score_row0 +
 * score_rows), stored at scores[(t - score_row0) * T_k + key] (device fp32
 * [score_rows, T_k], caller-owned; entries outside a row's window are left
 * untouched).  These are exactly the values the selection ranked, so a test
 * can check the selection itself (order by score descending, ties to the
 * lower index) independently of fp32 rounding.  The pages have no
 * counterpart; this entry is for tests and diagnostics.  Errors as for
 * dsa_indexer_topk, plus DSA_ERR_INVALID_ARGUMENT unless 0 <= score_row0,
 * score_row0 + score_rows <= T and scores != NULL when score_rows > 0.
 */
dsa_status_t dsa_indexer_topk_with_scores(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_idx, const float* head_weights,
                                          const int32_t* seq_start, int32_t T, int32_t T_k, int32_t Hi, int32_t Di,
                                          int32_t K, int32_t* topk_idx, int32_t* topk_len, float* scores,
                                          int32_t score_row0, int32_t score_rows, void* workspace,
                                          size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_indexer_topk_scored -- dsa_indexer_topk (causal_len NULL) or
 * dsa_indexer_topk_cp (causal_len given) that also returns, slot for slot, the
 * fp32 score the selection ranked: topk_score[t, j] = score(t, topk_idx[t, j])
 * for j < topk_len[t], -inf after.  Same kernel and same topk_idx / topk_len as
 * those calls; the scores are the ones the kernel kept with each candidate.
 * Their consumer is dsa_indexer_kl, whose loss needs exactly these values
 * (the KL term of [DSA-blog] "How DSA works" compares the indexer's score
 * distribution over the selected slots with the attention's).
 *  topk_score   device fp32 [T, K] (out; required when T > 0)
 *  the rest     as dsa_indexer_topk / dsa_indexer_topk_cp
 * Errors as those calls, plus DSA_ERR_INVALID_ARGUMENT when topk_score is NULL.
 */
dsa_status_t dsa_indexer_topk_scored(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_idx, const float* head_weights,
                                     const int32_t* seq_start, const int32_t* causal_len, int32_t T, int32_t T_k,
                                     int32_t Hi, int32_t Di, int32_t K, int32_t* topk_idx, int32_t* topk_len,
                                     float* topk_score, void* workspace, size_t workspace_bytes,
                                     dsa_stream_t stream);

/*
 * dsa_indexer_kl -- the indexer's KL auxiliary loss over each row's selected
 * slots, and its gradient.
 * Source: [DSA-blog] "How DSA works" (the indexer emits an auxiliary KL loss
 * that aligns its score distribution with the main attention's; its graph is
 * independent of the main model's) and the training-results section (indexer
 * loss, sparse formulation, coefficient 0.001).  The pages print no formula;
 * reading taken, per row t over its valid slots J (as in the sparse MLA calls):
 *   I_j = score(t, topk_idx[t,j])  (the indexer score of dsa_indexer_topk)
 *   q_j = softmax_J(I),  p_j = attn_prob[t,j] / sum_J attn_prob[t,:]
 *   kl[t] = sum_{j: p_j > 0} p_j (log p_j - log q_j)
 * with g_j = coeff (q_j - p_j), s_hj = <q_idx[t,h], k_idx[idx_j]> and
 * m_hj = g_j w[t,h] [s_hj > 0]:
 *   dw[t,h] = sum_j g_j max(0, s_hj),  dq_idx[t,h,:] = sum_j m_hj k_idx[idx_j,:],
 *   dk_idx_accum[idx_j,:] += sum_h m_hj q_idx[t,h,:].
 * A row with no valid slot, or whose attn_prob sums to 0, gets kl = 0 and no
 * gradient.  The attention side is a constant (no gradient reaches it).
 *  q_idx, k_idx, head_weights  as dsa_indexer_topk (Hi in [1, 64], Di = 128)
 *  topk_idx     device int32 [T, K], K in [1, 4096];  topk_len device int32 [T] or NULL
 *  attn_prob    device fp32 [T, K]: e.g. the attn_prob output of dsa_sparse_mla_bwd
 *  topk_score   device fp32 [T, K] or NULL: the scores I_j of the slots, e.g. the
 *               topk_score output of dsa_indexer_topk_scored for this topk_idx.
 *               Given, they are read instead of formed again (one pass over the
 *               selected keys instead of two); the ReLU masks of the gradient are
 *               formed from the keys as always.  NULL: I_j is formed here.
 *  coeff        the loss coefficient (the pages train with 0.001); the gradients
 *               are those of coeff * sum_t kl[t]
 *  kl           device fp32 [T] (out);  dq_idx device bf16 [T, Hi, Di] (out)
 *  dw           device fp32 [T, Hi] (out)
 *  dk_idx_accum device fp32 [T_k, Di]: zeroed first when accumulate == 0
 *  workspace    >= dsa_indexer_kl_workspace_size() bytes
 * Indices outside [-1, T_k) are masked and reported through the device error
 * word.  Summation order of dk_idx_accum across rows is not deterministic.
 */
size_t dsa_indexer_kl_workspace_size(int32_t T, int32_t K);
dsa_status_t dsa_indexer_kl(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_idx, const float* head_weights,
                            const int32_t* topk_idx, const int32_t* topk_len, const float* attn_prob,
                            const float* topk_score, int32_t T, int32_t T_k, int32_t Hi, int32_t Di, int32_t K,
                            float coeff, float* kl,
                            dsa_bf16_t* dq_idx, float* dw, float* dk_idx_accum, int32_t accumulate,
                            void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * k-pool selection (GLM-5.3-Flash).  Source: [NoPE-PR] "Why" (the k-pool
 * selection appends the query's incomplete tail pool, so the top-k width is
 * 2048 + 3 = 2051) and "Comparing against cuDNN" (the k-pool path makes its own
 * selection instead of the token-level top-k).  The pages define nothing more;
 * readings taken: a pool is P consecutive tokens of one packed sequence counted
 * from its start (P = 4: an incomplete pool holds at most 3 tokens), numbered
 * across the sequences in order; a pooled row is the bf16 mean of its P token
 * rows; query t keeps the K complete pools of its sequence that end at or
 * before t with the best indexer score against the pooled keys, then the tokens
 * of its incomplete pool; attention runs over [pooled kv; token kv] (pool p at
 * row p, token s at row total_pools + s) with the sparse MLA entries unchanged,
 * and a token's key gradient is its row's plus 1/P of its pool's.
 */

/*
 * dsa_kpool_metadata -- pool coordinates of a packed batch.  For sequence i
 * (L_i tokens) and token t of it at position u = t - cu_seqlens[i]:
 *   pool_cu[i] = sum_{j<i} floor(L_j / P),  pool_cu[num_seqs] = total pools,
 *   pool_start[t] = pool_cu[i],  n_pools[t] = floor((u + 1) / P) (complete pools
 *   ending at or before t),  tail_start[t] = cu_seqlens[i] + P n_pools[t] (the
 *   first token of t's incomplete pool; t + 1 when t closes a pool).
 *  cu_seqlens   device int32 [num_seqs + 1], from 0, non-decreasing, ending at total_tokens
 *  pool         P >= 1
 *  pool_cu      device int32 [num_seqs + 1] (out)
 *  pool_start, n_pools, tail_start  device int32 [total_tokens] (out)
 *  total_pools_host  host int32 (out), may be NULL
 * Performs one device-to-host synchronisation to validate cu_seqlens
 * (DSA_ERR_INVALID_ARGUMENT when a rule above is broken; outputs untouched).
 */
dsa_status_t dsa_kpool_metadata(const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens, int32_t pool,
                                int32_t* pool_cu, int32_t* pool_start, int32_t* n_pools, int32_t* tail_start,
                                int32_t* total_pools_host, dsa_stream_t stream);

/*
 * dsa_kpool_pool -- pooled rows: out[pool_cu[i] + p, :] = bf16(sum_{r<P}
 * x[cu_seqlens[i] + P p + r, :] / P) (fp32 sum, round to nearest even) for every
 * complete pool p of every sequence i.  For the index keys (D = 128) and the kv
 * latents (D = 576 or 512).
 *  x            device bf16 [total_tokens, D], D a multiple of 8, 16-byte aligned
 *  cu_seqlens, pool_cu, num_seqs, pool, total_pools  as dsa_kpool_metadata
 *  out          device bf16 [total_pools, D] (out), 16-byte aligned
 */
dsa_status_t dsa_kpool_pool(const dsa_bf16_t* x, int32_t total_tokens, int32_t D, const int32_t* cu_seqlens,
                            const int32_t* pool_cu, int32_t num_seqs, int32_t pool, int32_t total_pools,
                            dsa_bf16_t* out, dsa_stream_t stream);

/*
 * dsa_kpool_topk -- per query row t: the K pools of [pool_start[t],
 * pool_start[t] + n_pools[t] - 1] with the highest indexer score (the score and
 * ranking of dsa_indexer_topk, ties to the lower pool) against the pooled keys,
 * ascending, then the rows total_pools + s for s = tail_start[t] .. t, then -1,
 * in rows of width K + pool - 1; topk_len[t] = the valid count.
 *  q_idx, head_weights  as dsa_indexer_topk (T query rows, Hi in [1, 64], Di = 128)
 *  k_pool       device bf16 [total_pools, Di] (dsa_kpool_pool of the index keys)
 *  pool_start, n_pools, tail_start  device int32 [T] (dsa_kpool_metadata)
 *  K            in [1, 2048] (2048 for GLM-5.3-Flash)
 *  topk_idx     device int32 [T, K + pool - 1] (out);  topk_len device int32 [T] (out) or NULL
 *  workspace    >= dsa_kpool_topk_workspace_size(T, K) bytes; its first word is
 *               the device error word (dsa_read_device_status)
 */
size_t dsa_kpool_topk_workspace_size(int32_t T, int32_t K);
dsa_status_t dsa_kpool_topk(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_pool, const float* head_weights,
                            const int32_t* pool_start, const int32_t* n_pools, const int32_t* tail_start, int32_t T,
                            int32_t total_pools, int32_t Hi, int32_t Di, int32_t K, int32_t pool, int32_t* topk_idx,
                            int32_t* topk_len, void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_kpool_unpool_grad -- token key gradient from the gradient of the attended
 * rows (the adjoint of x -> [pooled rows; x], without the bf16 rounding):
 *   dx[t, :] = dcat[total_pools + t, :] + dcat[pool(t), :] / P if t lies in a
 *   complete pool (pool(t) = pool_cu[i] + floor((t - cu_seqlens[i]) / P)),
 *   else dcat[total_pools + t, :].
 *  dcat         device fp32 [total_pools + total_tokens, D] (e.g. the dkv
 *               accumulator of dsa_sparse_mla_bwd over [pooled kv; kv]), D a
 *               multiple of 4, 16-byte aligned
 *  dx           device fp32 [total_tokens, D] (out), 16-byte aligned, not overlapping dcat
 */
dsa_status_t dsa_kpool_unpool_grad(const float* dcat, int32_t total_tokens, int32_t D, const int32_t* cu_seqlens,
                                   const int32_t* pool_cu, int32_t num_seqs, int32_t pool, int32_t total_pools,
                                   float* dx, dsa_stream_t stream);

/*
 * dsa_sparse_mla_fwd -- absorbed sparse MLA forward (MQA over one latent KV).
 * Source: [DSA-blog] "How DSA works" and "Why DSA needs fused kernels";
 * [cudnn_dsa] cudnn_sparse_attention / _CudnnSparseAttention.forward (q
 * [T, H, 576], kv_latent [T_k, 1, 576], int32 indices with -1 invalid, optional
 * topk_length, explicit softmax_scale, output [T, H, 512]); [NoPE-PR] "Change"
 * (value = kv[..., :512], NoPE width 512, unaligned top-k widths).
 * Slot j of row t is valid iff topk_idx[t,j] >= 0 and (topk_len == NULL or
 * j < topk_len[t]); per (t, h):
 *   z_j = softmax_scale * <q[t,h,:], kv[idx_j,:]>,  lse[t,h] = ln sum_j exp(z_j),
 *   out[t,h,:] = sum_j exp(z_j - lse) * kv[idx_j, 0:Dv].
 * A row with no valid slot gets out = 0 and lse = -inf.  Indices >= T_k or
 * < -1 are masked and reported through the device error word.
 * Attention sink ([cudnn_dsa] _pad_attention_heads pads a sink [H] with q;
 * the pages print no formula; reading taken): attn_sink[h] is one more logit
 * of every row of head h, in the units of z, with no value row:
 *   lse[t,h] = ln(sum_j exp(z_j) + exp(attn_sink[h])),  out as above,
 * so a row with no valid slot gets out = 0 and lse = attn_sink[h].  A sink of
 * -inf is no sink; NaN or +inf sinks are outside the contract.
 *  q        device bf16 [T, H, Dqk], Dqk in {512, 576};  kv device bf16 [T_k, Dqk]
 *  topk_idx device int32 [T, K], any K >= 1;  topk_len device int32 [T] or NULL
 *  attn_sink device fp32 [H] or NULL (no sink)
 *  out      device bf16 [T, H, Dv] (out), Dv = 512;  lse device fp32 [T, H] (out)
 *  out_lo   device bf16 [T, H, Dv] (out) or NULL: the rounding residual
 *           bf16(O - out) of the fp32 result O (P.V runs on bf16 hi + lo parts
 *           of P, so O is accurate to about fp32).  Passing it on to the
 *           backward makes D = <dout, O> use that O instead of the rounded out
 *           (library addition; the pages' interface returns out only).
 *  workspace >= dsa_sparse_mla_fwd_workspace_size() bytes
 * Query chunking ([Chunk-PR] "Summary"): rows are independent, so a chunk is a
 * call on row-offset pointers of q/topk_idx/out/lse with the full kv.
 */
size_t dsa_sparse_mla_fwd_workspace_size(int32_t T, int32_t H);
dsa_status_t dsa_sparse_mla_fwd(const dsa_bf16_t* q, const dsa_bf16_t* kv, const int32_t* topk_idx,
                                const int32_t* topk_len, int32_t T, int32_t T_k, int32_t H, int32_t Dqk,
                                int32_t Dv, int32_t K, float softmax_scale, const float* attn_sink, dsa_bf16_t* out,
                                dsa_bf16_t* out_lo, float* lse, void* workspace, size_t workspace_bytes,
                                dsa_stream_t stream);

/*
 * dsa_sparse_mla_bwd -- analytic backward of dsa_sparse_mla_fwd.
 * Source: [cudnn_dsa] _CudnnSparseAttention.backward (gradients for the query
 * [T, H, 576] and the latent KV from grad_output [T, H, 512]); [Chunk-PR]
 * "Summary" (query chunks are independent, key gradients sum).
 * With P_j = exp(z_j - lse), D = <dout, out>, dP_j = <dout, kv[idx_j,:Dv]>,
 * dS_j = P_j (dP_j - D):
 *   dq[t,h,:]         = softmax_scale * sum_j dS_j kv[idx_j, :]
 *   dkv_accum[idx_j,:] += softmax_scale * sum_h dS_j q[t,h,:]
 *   dkv_accum[idx_j,0:Dv] += sum_h P_j dout[t,h,:]
 * and with a sink, P_sink = exp(attn_sink[h] - lse[t,h]):
 *   d_sink[h] += -sum_t P_sink[t,h] D[t,h]
 *  q, kv, topk_idx, topk_len, sizes, softmax_scale, attn_sink: as in the forward call
 *  out, lse       device: the forward's outputs for these rows
 *  out_lo         device bf16 [T, H, Dv]: the forward's residual, or NULL (then D
 *                 is computed from the rounded out)
 *  dout           device bf16 [T, H, Dv]
 *  dq             device bf16 [T, H, Dqk] (out)
 *  dkv_accum      device fp32 [T_k, Dqk]: zeroed first when accumulate == 0,
 *                 added to when accumulate == 1 (query chunks)
 *  d_sink         device fp32 [H] or NULL (needs attn_sink): zeroed first when
 *                 accumulate == 0, added to when accumulate == 1
 *  attn_prob      device fp32 [T, K] (out) or NULL: the head-averaged attention
 *                 probability of every slot, (1/H) sum_h P[t,h,j] (0 for an
 *                 invalid slot), the target distribution of dsa_indexer_kl;
 *                 computed from the P the backward already forms
 *  dkv_bf16       device bf16 [T_k, Dqk] (out, rounded copy of dkv_accum) or NULL
 *  workspace      >= dsa_sparse_mla_bwd_workspace_size(T, H, K) bytes: the
 *                 error word, 256 scratch-slot flags, D (T*H fp32) and the
 *                 scratch slots for the bf16 dS of one row's tiles (256 slots
 *                 x ceil(K/128) x 16 KiB; a CTA claims a free slot and
 *                 releases it on exit).  One workspace serves one call at a
 *                 time: calls whose executions overlap must not share it.
 * Summation order of dkv_accum (and d_sink) across rows is not deterministic
 * (fp32 atomics).
 */
size_t dsa_sparse_mla_bwd_workspace_size(int32_t T, int32_t H, int32_t K);
dsa_status_t dsa_sparse_mla_bwd(const dsa_bf16_t* q, const dsa_bf16_t* kv, const int32_t* topk_idx,
                                const int32_t* topk_len, int32_t T, int32_t T_k, int32_t H, int32_t Dqk,
                                int32_t Dv, int32_t K, float softmax_scale, const float* attn_sink,
                                const dsa_bf16_t* out, const dsa_bf16_t* out_lo, const float* lse,
                                const dsa_bf16_t* dout, dsa_bf16_t* dq, float* dkv_accum, float* d_sink,
                                float* attn_prob, int32_t accumulate, dsa_bf16_t* dkv_bf16, void* workspace,
                                size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_sparse_mla_bwd_noalloc -- dsa_sparse_mla_bwd without a caller workspace.
 * The pages have no counterpart: this is a library addition for callers that
 * cannot allocate device memory (runtimes that reserve all device memory in
 * their own pool and forbid other allocations, or plug-ins whose host program
 * owns every allocation) and so cannot supply the workspace.  Arguments,
 * semantics and results are those of dsa_sparse_mla_bwd.
 *  - Scratch is a fixed 84 MiB + 1280 B device array built into the library,
 *    held by every GPU that loads it until the process exits; K must not
 *    exceed dsa_sparse_mla_bwd_noalloc_max_topk() (2176), else
 *    DSA_ERR_WORKSPACE is returned and nothing is launched.  Its D part holds
 *    4 Mi (row, head) pairs: longer calls run in row chunks of
 *    floor(4 Mi / H) rows, one after the other on `stream`, with dkv_accum
 *    and d_sink accumulating over the chunks.
 *  - The call allocates nothing.  The first call on a device (and again after
 *    the device's context is replaced) looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture.
 *  - Every call uses the same array: calls whose executions overlap on the
 *    GPU race on it and must be ordered by the caller (same stream or events).
 *    Each call clears the array's error word and slot flags; the device error
 *    word is read with dsa_sparse_mla_bwd_noalloc_read_status.
 */
int32_t dsa_sparse_mla_bwd_noalloc_max_topk(void);
dsa_status_t dsa_sparse_mla_bwd_noalloc(const dsa_bf16_t* q, const dsa_bf16_t* kv, const int32_t* topk_idx,
                                        const int32_t* topk_len, int32_t T, int32_t T_k, int32_t H, int32_t Dqk,
                                        int32_t Dv, int32_t K, float softmax_scale, const float* attn_sink,
                                        const dsa_bf16_t* out, const dsa_bf16_t* out_lo, const float* lse,
                                        const dsa_bf16_t* dout, dsa_bf16_t* dq, float* dkv_accum, float* d_sink,
                                        float* attn_prob, int32_t accumulate, dsa_bf16_t* dkv_bf16,
                                        dsa_stream_t stream);
/*
 * dsa_sparse_mla_bwd_noalloc_read_status -- the no-alloc backward's device
 * error word: synchronise `stream`, read and clear the word in the built-in
 * array and store it in *status_host (DSA_OK, DSA_ERR_DEVICE_INDEX or
 * DSA_ERR_TIMEOUT), as dsa_read_device_status does for a workspace.  No
 * counterpart on the pages (library addition).
 */
dsa_status_t dsa_sparse_mla_bwd_noalloc_read_status(dsa_stream_t stream, int32_t* status_host);

/*
 * The serving step: rows of a paged cache, prepared, selected and attended to.
 *
 * A paged cache is a contiguous bf16 array [num_pages, page_size, D]; request b's
 * token at position p is row block_table[b, p / page_size] * page_size + p %
 * page_size of it.  The calls read lengths and tables on the device and never
 * synchronise, so a step can be captured into a graph and replayed while the
 * lengths change.  For the same reason they do NOT clear the device error word of
 * their workspace: zero the workspace's first 256 bytes once when it is made;
 * the first failure stays there until dsa_read_device_status reads and clears it.
 * One workspace serves one call at a time; calls on one stream may share it.
 */

/*
 * dsa_paged_slots -- pages and cache rows of a step's new tokens, from the
 * requests' lengths.  Request b holds s = seq_lens[b] tokens in ceil(s / P) pages
 * and gets n = new_lens[b] more (1 when new_lens is NULL).  Its fresh pages, numbers
 * ceil(s / P) .. ceil((s + n) / P) - 1 of block_table[b, :], are taken from
 * free_pages in request order; other entries of the table are left as they are.
 * The new tokens are packed in request order: token t = cu_new[b] + j has
 *   positions[t] = s + j,
 *   slot_map[t] = block_table[b, positions[t] / P] * P + positions[t] % P,
 * and the entries t >= cu_new[B] are -1 in both.
 *  seq_lens     device int32 [B], >= 0;  new_lens device int32 [B], >= 0, or NULL
 *  B            in [0, 8192];  N >= 0: entries of slot_map and positions
 *  free_pages   device int32 [F]
 *  block_table  device int32 [B, max_pages] (in, out)
 *  seq_lens_out device int32 [B] (out) = s + n;  cu_new device int32 [B + 1] (out)
 *  slot_map, positions  device int32 [N] (out);  pages_taken device int32 [1] (out)
 *  workspace    >= 256 bytes (the error word)
 * All or nothing: when a length is negative, a request needs more than max_pages
 * pages, the fresh pages are more than F or the new tokens more than N, no request
 * gets a token (slot_map, positions -1; cu_new, pages_taken 0; seq_lens_out =
 * seq_lens; block_table untouched) and DSA_ERR_CAPACITY is recorded.  A token whose
 * page number is negative, or whose row is above 2^31 - 1, gets slot -1 and
 * DSA_ERR_DEVICE_INDEX is recorded.  Outputs must not overlap inputs or each other.
 */
dsa_status_t dsa_paged_slots(const int32_t* seq_lens, const int32_t* new_lens, int32_t B, int32_t N, int32_t page_size,
                             int32_t max_pages, const int32_t* free_pages, int32_t F, int32_t* block_table,
                             int32_t* seq_lens_out, int32_t* cu_new, int32_t* slot_map, int32_t* positions,
                             int32_t* pages_taken, void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_norm_rope_fwd -- the norm of a row's first channels and the rotation of its
 * positions in one pass.  For every row (t, h) of width D:
 *   norm 1 (rms):   y_c = x_c r weight_c, r = 1 / sqrt(mean x^2 + eps)
 *   norm 2 (layer): y_c = (x_c - mean) r weight_c + bias_c, r = 1 / sqrt(var + eps)
 *   norm 0:         y_c = x_c                          (mean, var over c < norm_dim)
 * (squares are summed in fp32, so that a norm's rows have |x_c| < 2^57 and, with eps = 0, a largest one above 2^-58)
 * for c < norm_dim, y_c = x_c above; then the rope_dim channels from rope_start are
 * turned in pairs (a, b), number i = 0 .. rope_dim / 2 - 1, by the angle
 * positions[t] * inv_freq[i] (formed exactly, whatever the position):
 *   (a, b) -> rope_scale (cos a - sin b, sin a + cos b)
 * where a pair is the channels (2i, 2i + 1) (interleaved 1) or (i, i + rope_dim / 2).
 * For the latent rows (norm 1 of 512, rotation of the last 64 of 576), the index
 * keys (norm 2 of 128, rotation of 64), per-head norms of queries and keys, and the
 * position channels of wider query rows (a strided view; out may be x itself).
 *  x            device bf16, row (t, h) at x + t x_stride_t + h x_stride_h (elements; >= 0,
 *               0 repeats a row), channels contiguous; T >= 0, H >= 1, T H <= 2^31 - 65,
 *               D in [1, 1024]
 *  weight, bias device fp32 [norm_dim] or NULL (1 and 0)
 *  positions    device int32 [T];  inv_freq device fp32 [rope_dim / 2] (both may be NULL
 *               when rope_dim is 0)
 *  out          device bf16, row (o, h) at out + o out_stride_t + h out_stride_h, with o = t,
 *               or o = out_rows[t] when out_rows (device int32 [T]) is given: -1 writes no
 *               row, other values outside [0, num_out_rows) are skipped and reported
 *               (DSA_ERR_DEVICE_INDEX); a row named twice gets each channel from one of
 *               the two results, in no order.  The rows of out must not overlap; out may equal x with the same strides
 *               and no out_rows, and must not overlap x otherwise.
 *  workspace    >= 256 bytes (the error word)
 */
dsa_status_t dsa_norm_rope_fwd(const dsa_bf16_t* x, int64_t x_stride_t, int64_t x_stride_h, int32_t T, int32_t H,
                               int32_t D, int32_t norm, int32_t norm_dim, const float* weight, const float* bias,
                               float eps, int32_t rope_start, int32_t rope_dim, int32_t interleaved,
                               const int32_t* positions, const float* inv_freq, float rope_scale, dsa_bf16_t* out,
                               int64_t out_stride_t, int64_t out_stride_h, const int32_t* out_rows,
                               int64_t num_out_rows, void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_norm_rope_bwd -- gradient of dsa_norm_rope_fwd (without out_rows): dx, and
 * with a norm the sums over all rows dweight[c] and dbias[c] (layer norm).
 *  dout, x      device bf16 with element strides as in the forward (x may be NULL without a norm)
 *  dx           device bf16 (out), its rows must not overlap; may equal dout or x with the same strides
 *  dweight, dbias  device fp32 [norm_dim] (out) or NULL: overwritten when accumulate == 0,
 *               added to when accumulate == 1
 *  workspace    >= dsa_norm_rope_bwd_workspace_size(norm_dim) bytes
 * The sums' order is fixed: equal calls give equal bits.
 */
size_t dsa_norm_rope_bwd_workspace_size(int32_t norm_dim);
dsa_status_t dsa_norm_rope_bwd(const dsa_bf16_t* dout, int64_t dout_stride_t, int64_t dout_stride_h,
                               const dsa_bf16_t* x, int64_t x_stride_t, int64_t x_stride_h, int32_t T, int32_t H,
                               int32_t D, int32_t norm, int32_t norm_dim, const float* weight, float eps,
                               int32_t rope_start, int32_t rope_dim, int32_t interleaved, const int32_t* positions,
                               const float* inv_freq, float rope_scale, dsa_bf16_t* dx, int64_t dx_stride_t,
                               int64_t dx_stride_h, float* dweight, float* dbias, int32_t accumulate, void* workspace,
                               size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_rope_frequencies -- host table of inverse frequencies base^(-2i / rope_dim),
 * and, for a context stretched by `factor` > 1, scaled by parts (the published
 * YaRN rule): pairs that turn more than beta_fast times over original_context keep
 * their frequency, those that turn fewer than beta_slow times are divided by
 * factor, with a linear ramp between; *rope_scale_host = 0.1 ln(factor) + 1 (1 when
 * factor is 1).
 *  inv_freq_host  host fp32 [rope_dim / 2] (out);  rope_scale_host host fp32 (out)
 */
dsa_status_t dsa_rope_frequencies(int32_t rope_dim, double base, double factor, int32_t original_context,
                                  double beta_fast, double beta_slow, float* inv_freq_host, float* rope_scale_host);

/*
 * dsa_paged_mla -- attention of new tokens over a paged latent cache, absorbed MLA
 * as in dsa_sparse_mla_fwd.  Request b has n = cu_q[b + 1] - cu_q[b] new tokens (one
 * each when cu_q is NULL), the last n of its seq_lens[b] cached ones: token cu_q[b] + j
 * sees the v = seq_lens[b] - n + j + 1 positions 0 .. v - 1 (none when v <= 0), or of them
 * those that its list topk_idx[token, :] names.  With those positions' rows kv:
 *   z_p = softmax_scale <q[t,h,:], kv_p>,  lse[t,h] = ln(sum_p exp(z_p) [+ exp(attn_sink[h])]),
 *   out[t,h,:] = sum_p exp(z_p - lse) kv_p[0:Dv];
 * a token that sees nothing gets out = 0 and lse = -inf (or attn_sink[h]).
 * What a position holds, infinities and NaN too, reaches the tokens that see it and no other.  (To one of them whose
 * score for it is -inf an infinite latent adds NaN, or nothing where another new token of the request does not see it.)
 *  q            device bf16 [N, H, Dqk], Dqk in {512, 576}
 *  cache        device bf16 [num_pages, page_size, Dqk]; rows that no token sees are not read
 *  block_table  device int32 [B, max_pages];  seq_lens device int32 [B]
 *  cu_q         device int32 [B + 1], non-decreasing, within [0, N], or NULL (then N = B);
 *               rows of out and lse outside [cu_q[0], cu_q[B]) are left as they are
 *  topk_idx     device int32 [N, K] positions, -1 for no entry, in any order, or NULL with K = 0
 *               (e.g. of dsa_paged_indexer_topk); an entry named twice counts twice
 *  topk_len     device int32 [N] or NULL: only the first topk_len[t] entries are looked at
 *  attn_sink    device fp32 [H] or NULL
 *  out          device bf16 [N, H, Dv] (out), Dv = 512;  lse device fp32 [N, H] (out);  N H < 2^31
 *  workspace    >= dsa_paged_mla_workspace_size() bytes, whatever the sizes
 * Positions beyond the table (p / page_size >= max_pages), entries outside [-1, v) and pages
 * outside [0, num_pages) are masked and reported (DSA_ERR_DEVICE_INDEX).  The result does not
 * depend on timing: equal calls on equal devices give equal bits.
 */
size_t dsa_paged_mla_workspace_size(void);
dsa_status_t dsa_paged_mla(const dsa_bf16_t* q, const dsa_bf16_t* cache, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* cu_q, const int32_t* topk_idx,
                           const int32_t* topk_len, int32_t N, int32_t B, int32_t H, int32_t Dqk, int32_t Dv,
                           int32_t K, int32_t num_pages, int32_t page_size, int32_t max_pages, float softmax_scale,
                           const float* attn_sink, dsa_bf16_t* out, float* lse, void* workspace,
                           size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_paged_indexer_topk -- the selection of new tokens over paged index keys: the
 * score and ranking of dsa_indexer_topk,
 *   score(t, p) = sum_h head_weights[t,h] * max(0, <q_idx[t,h,:], k_p>),
 * over the positions p that token t sees (as in dsa_paged_mla), summed in fp32.  The
 * n = min(K, positions seen) highest (ties to the lower position; NaN above all) are
 * written ascending to topk_idx[t, 0:n], then -1 up to K: the lists of dsa_paged_mla.
 *  q_idx        device bf16 [N, Hi, Di]; Hi in [1, 64], Di = 128
 *  k_cache      device bf16 [num_pages, page_size, Di]
 *  head_weights device fp32 [N, Hi]
 *  block_table, seq_lens, cu_q  as dsa_paged_mla
 *  K            in [1, 2048]
 *  max_len      no request is longer (the workspace holds N rows of that many scores);
 *               at most 2^30
 *  topk_idx     device int32 [N, K] (out);  topk_len device int32 [N] (out) or NULL;
 *               rows outside [cu_q[0], cu_q[B]) are left as they are
 *  workspace    >= dsa_paged_indexer_topk_workspace_size(N, max_len) bytes
 * Positions beyond max_len or the table are not ranked, and keys on pages outside
 * [0, num_pages) count as zero rows; both are reported (DSA_ERR_DEVICE_INDEX).
 */
size_t dsa_paged_indexer_topk_workspace_size(int32_t N, int32_t max_len);
dsa_status_t dsa_paged_indexer_topk(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_cache, const float* head_weights,
                                    const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, int32_t N,
                                    int32_t B, int32_t Hi, int32_t Di, int32_t K, int32_t num_pages, int32_t page_size,
                                    int32_t max_pages, int32_t max_len, int32_t* topk_idx, int32_t* topk_len,
                                    void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * Rows of a quantised cache.  The first quant_dim channels of a row of D are held as
 * codes, the others in bf16; a quantised channel's value is code * s (8 bits) or
 * code * block * s (4 bits).  A row's bytes, for Q = quant_dim (a multiple of 64, D - Q a
 * multiple of 8, D <= 1024):
 *   8 bits: Q codes e4m3, s (fp32), zero bytes up to a multiple of 16, 2 (D - Q) bytes of the
 *           other channels, zero bytes up to a multiple of 16;
 *   4 bits: Q / 2 bytes of codes e2m1 (channel 2i in the low half of byte i, 2i + 1 in the
 *           high), Q / 16 block scales e4m3 (one for each 16 channels, >= 0), then s and the
 *           rest as above.
 * s is a power of two in [2^-48, 2^48], or NaN: then all Q channels of the row are NaN.
 * Codes and block scales are finite (no byte 0x7f or 0xff among the e4m3 ones).
 * For the latents (D = 576, Q = 512) a row has 656 bytes of 8 bits, 432 of 4 bits, in place of 1152.
 */

/* Bytes of a row (a multiple of 16); 0 when D, quant_dim and bits (8 or 4) are not as above. */
size_t dsa_paged_quant_row_bytes(int32_t D, int32_t quant_dim, int32_t bits);

/*
 * dsa_paged_quantize -- rows quantised as they are written to a cache.  For row x with the
 * largest magnitude a over its first Q channels:
 *   s = the smallest power of two (at least 2^-48) with a <= 448 s (8 bits), a <= 2688 s (4 bits);
 *   8 bits: code = e4m3(x / s);
 *   4 bits: block = e4m3(a_block / (6 s)), code = e2m1(x / (block s)) (0 where block is 0),
 * rounded to nearest, ties to even, magnitudes past the largest code to that code.  A row with a
 * channel among the Q that is not finite, or too large for s = 2^48, gets s = NaN.
 *  x            device bf16, row t at x + t x_stride_t (elements; >= 0), channels contiguous; T >= 0
 *  cache        device bytes [num_rows, row bytes] (out), 16-byte aligned: the pages' rows laid end to end
 *  out_rows     device int32 [T] or NULL (row t): as in dsa_norm_rope_fwd (-1 writes no row; other
 *               values outside [0, num_rows) are skipped and reported, DSA_ERR_DEVICE_INDEX); a row
 *               named twice holds bytes of both results, in no order
 *  workspace    >= 256 bytes (the error word)
 * x and cache must not overlap.  Rows that are not named are left as they are.
 */
dsa_status_t dsa_paged_quantize(const dsa_bf16_t* x, int64_t x_stride_t, int32_t T, int32_t D, int32_t quant_dim,
                                int32_t bits, uint8_t* cache, int64_t num_rows, const int32_t* out_rows,
                                void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_paged_dequantize -- rows of requests read back: row cu_rows[b] + j of out is the row of
 * request b's position first[b] + j (j when first is NULL), rounded to bf16 (rows that
 * dsa_paged_quantize wrote are exact).  Rows named one by one are a request with pages of one row:
 * the list is then its block table.
 *  cache        device bytes [num_pages, page_size, row bytes], 16-byte aligned
 *  block_table  device int32 [B, max_pages];  first device int32 [B] or NULL
 *  cu_rows      device int32 [B + 1], non-decreasing, within [0, N]; rows of out outside
 *               [cu_rows[0], cu_rows[B]) are left as they are
 *  out          device bf16 (out), row t at out + t out_stride_t (>= D), channels contiguous
 *  workspace    >= 256 bytes (the error word)
 * Positions that are negative or beyond the table and pages outside [0, num_pages) give rows of
 * zeros and are reported (DSA_ERR_DEVICE_INDEX).  out must not overlap the cache.
 */
dsa_status_t dsa_paged_dequantize(const uint8_t* cache, const int32_t* block_table, const int32_t* first,
                                  const int32_t* cu_rows, int32_t N, int32_t B, int32_t D, int32_t quant_dim,
                                  int32_t bits, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                  dsa_bf16_t* out, int64_t out_stride_t, void* workspace, size_t workspace_bytes,
                                  dsa_stream_t stream);

/*
 * dsa_paged_mla_quant -- dsa_paged_mla over a cache of quantised latents (quant_dim = 512): the same
 * attention, with the rows' values as defined above for kv.  Queries, tables, lists, sink, out and lse
 * as there.  Scores and sums are fp32.  4 bits: products of the scores are exact for query channels down to
 * 2^-31 of a, the row's largest one among the first 512 (2^-24 of its largest position channel where that is
 * more); smaller ones are off by 2^-39 a at most.  A weight has 11 bits (down to 2^-32 of the largest weight
 * times s).  8 bits: a query row counts to 2^-17 of its largest channel among the first 512, a weight to
 * 2^-11 of itself (2^-28 of the largest weight times s).  The output's sums are 6
 * additions for 64 (8 bits) or 96 (4 bits) positions of a CTA's share, each off by 2^-23 of the sum at most.
 *  cache        device bytes [num_pages, page_size, dsa_paged_quant_row_bytes(Dqk, 512, bits)], 16-byte aligned
 *  bits         8 or 4
 *  workspace    >= dsa_paged_mla_quant_workspace_size() bytes, whatever the sizes
 * A row whose s is NaN makes the tokens NaN that see it and no other; a row of zero bytes, which nothing
 * was written to, holds zeros.  A query with a channel that is not finite touches no row of out and lse
 * but its own (8 bits: that becomes NaN if the channel is among the first 512).  4 bits: position channels
 * count divided by s, and overflow above 2^82 s (2^106 s for queries whose position channels are not larger
 * than the others).  num_pages * page_size < 2^31.  The result does not depend on timing: equal calls on equal
 * devices give equal bits.
 */
size_t dsa_paged_mla_quant_workspace_size(void);
dsa_status_t dsa_paged_mla_quant(const dsa_bf16_t* q, const uint8_t* cache, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* cu_q, const int32_t* topk_idx,
                                 const int32_t* topk_len, int32_t N, int32_t B, int32_t H, int32_t Dqk, int32_t Dv,
                                 int32_t bits, int32_t K, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                 float softmax_scale, const float* attn_sink, dsa_bf16_t* out, float* lse,
                                 void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * dsa_set_wait_limit_cycles -- the cycle limit of every bounded device-side
 * wait of the kernels launched after the call (process-wide; the default is
 * 2^31 SM cycles, about one second).  A wait that runs past it records
 * DSA_ERR_TIMEOUT in the device error word and its CTA leaves its work and
 * exits cleanly; 0 gives up at the first wait whose phase has not completed,
 * which lets a test drive every timeout path on purpose.  A negative value
 * restores the default.  Returns the previous limit.  Library addition with
 * no counterpart on the pages.
 */
int64_t dsa_set_wait_limit_cycles(int64_t cycles);

/*
 * dsa_read_device_status -- synchronise `stream`, read and clear the device
 * error word at the start of `workspace`, and store it in *status_host
 * (DSA_OK, DSA_ERR_DEVICE_INDEX or DSA_ERR_TIMEOUT).  Library addition with no
 * counterpart on the pages: it surfaces the bounded-wait and index checks.
 */
dsa_status_t dsa_read_device_status(void* workspace, dsa_stream_t stream, int32_t* status_host);

#ifdef __cplusplus
}
#endif
#endif /* DSA_H_ */
