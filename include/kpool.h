/*
 * kpool.h - C ABI of the MI355X (gfx950) k-pool DSA indexer selection.
 *
 * The selection a DSA indexer makes for each query row (pages: Atlas
 * inference docs, spark_model/layers/glm5next_dsa/tp.rs, module doc "Why the
 * indexer is REPLICATED, not sharded"; Megatron-LM PR #8299, sections
 * "Mechanism" and "Change"):
 *
 *   1. pool the keys over kpool consecutive tokens            kpool_pool_keys
 *   2. score every causally visible pool of row i as
 *        S[i,p] = sum_h w[i,h] * relu(scale * <q[i,h,:], kp[p,:]>)
 *      and keep the best `budget` pools, higher score first and the
 *      smaller pool index on equal scores                     kpool_score_topk
 *   3. expand the kept pools to token ids p*kpool + j and drop the tokens
 *      that come after the row                                kpool_expand
 *
 * Conventions shared by every entry point
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory, keeps no pointer after it returns and never
 *     synchronises: all work is enqueued on `stream` (a hipStream_t; NULL is
 *     the default stream).  Results are ready when the stream reaches them.
 *   - bf16 tensors are passed as their uint16_t bit patterns.  Tensors are
 *     row-major and contiguous; q, kp, k and w must be 16-byte aligned.
 *   - Packed variable-length batches ("THD") are described by cu_seqlens:
 *     sequence s holds the global rows [cu_seqlens[s], cu_seqlens[s+1]).
 *     Positions, pool ids and token ids are SEQUENCE-LOCAL: row i of
 *     sequence s sits at t = i - cu_seqlens[s], and sees the pools p with
 *     p*kpool <= t.  A single sequence is nseq = 1, cu_seqlens = {0, T}.
 *     `cu_seqlens_host` is a host copy used to validate and plan launches;
 *     `cu_seqlens_dev` / `cu_pools_dev` hold the same arrays on the device.
 *   - Every entry point validates its arguments before it launches anything
 *     and returns KPOOL_OK (0) or a negative kpool_status; the reason is then
 *     in kpool_last_error() (thread-local).  Nothing is thrown across the ABI.
 *     Launch failures map to KPOOL_EHIP; faults that happen while a kernel
 *     runs surface at the caller's next synchronisation.
 *   - Every setting is an argument: there is no process-wide switch.  Calls on
 *     one stream are ordered.  The library's only lasting state is, per caller
 *     stream that asked for the chunk overlap (KPOOL_FLAG_OVERLAP), one helper
 *     stream (default priority) with two events, created on first use and kept
 *     until the process ends; the helper joins back into the caller's stream
 *     before the call returns, so results are ordered on the caller's stream as
 *     usual.  Calls on different caller streams use different helpers.  Besides
 *     that, per device and once: the number of score workgroups the device runs
 *     at once (an occupancy query, used to plan launches) and, for
 *     kpool_score_topk_noalloc, its static scratch array's device address.  The
 *     optional profiler below is per host thread.
 */
#ifndef KPOOL_H
#define KPOOL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KPOOL_OK = 0,
  KPOOL_EINVAL = -1,       /* bad argument: range, size, pointer, alignment */
  KPOOL_EUNSUPPORTED = -2, /* head count / head dim not compiled in */
  KPOOL_EWORKSPACE = -3,   /* workspace smaller than one score row */
  KPOOL_EHIP = -4          /* a HIP launch or runtime call failed */
} kpool_status;

/* Message for the last non-OK return on this thread ("" if none). */
const char *kpool_last_error(void);

/* ABI version (major*100 + minor): 300. */
int kpool_version(void);

/* Tail mode (flags bit of kpool_count_pools, kpool_pool_keys(_gated),
 * kpool_score_topk(_noalloc) and kpool_expand; pass the same choice to all of
 * them).  Megatron-LM PR #8299 "Change" names a "tail append" between pool
 * expansion and mask filtering but does not define it; this library's reading:
 * a sequence of L tokens has only its L / kpool full pools (the pool count of
 * the Atlas tp.rs module doc, seq / kpool), and its remaining L mod kpool
 * tokens, the tail, are appended to every row's expanded token ids and filtered
 * causally like them.  Without the flag a trailing partial pool is a pool of its
 * own and there is no tail. */
#define KPOOL_FLAG_TAIL 2u

/* Pool bookkeeping on the host (Atlas tp.rs module doc: a sequence of L
 * tokens has L/kpool pools).
 *   flags            0: ceil(L / kpool) pools, a trailing partial pool kept;
 *                    KPOOL_FLAG_TAIL: floor(L / kpool), full pools only
 *   cu_pools_host[s] = sum over s' < s of the pool counts, [nseq + 1] (nullable)
 *   *max_pools_out   = the largest pool count of one sequence (nullable)
 * Returns the total pool count P_tot (>= 0) or a negative kpool_status. */
int64_t kpool_count_pools(const int32_t *cu_seqlens_host, int32_t nseq, int32_t kpool,
                          uint32_t flags, int32_t *cu_pools_host, int32_t *max_pools_out);

/* Step 1 - pooled keys (Megatron-LM PR #8299 "Mechanism": rows score the
 * pooled keys).  For pool p of sequence s, with n = min(kpool, L_s - p*kpool):
 *   kp[cu_pools[s] + p, d] = bf16_rne( fp32( (sum_j k[cu_seqlens[s] + p*kpool + j, d]) / n ) )
 * where the sum is taken in fp32 in token order starting from +0.
 *   k   bf16 [T, D]  one key per token (the indexer's key projection has no head axis)
 *   kp  bf16 [P_tot, D] output, P_tot from kpool_count_pools with the same flags
 *   flags 0 or KPOOL_FLAG_TAIL (full pools only; cu_pools_dev must count the same way)
 * D must be a multiple of 8 (<= 1024); kpool >= 1. */
int kpool_pool_keys(const uint16_t *k, const int32_t *cu_seqlens_host,
                    const int32_t *cu_seqlens_dev, const int32_t *cu_pools_dev,
                    int32_t nseq, int32_t D, int32_t kpool, uint32_t flags, uint16_t *kp,
                    void *stream);

/* Step 1, gated variant - the GLM-5.3 indexer's k-pool compression (Atlas inference
 * docs, glm5next_dsa/tp.rs: the shard plan's indexer tensors include a compression
 * gate [index_head_dim, hidden] and a slot embedding [index_kpool, index_head_dim];
 * Megatron-LM PR #8299 "Mechanism": gate scores are an input of the op).  The pages
 * give no formula; this library's reading, for pool p of sequence s with tokens
 * t_j = cu_seqlens[s] + p*kpool + j, j < n = min(kpool, L_s - p*kpool), and each dim d:
 *   z_j = g[t_j, d] + ape[j, d],  m = max_j z_j,  e_j = exp(z_j - m)
 *   kp[cu_pools[s] + p, d] = bf16_rne( (sum_j e_j * k[t_j, d]) / (sum_j e_j) )
 * in fp64, rounded once to bf16 (sums in slot order; a trailing partial pool uses
 * ape[0 .. n-1]).
 *   k    bf16 [T, D]      keys
 *   g    bf16 [T, D]      gate scores (the gate projection's output per token and dim)
 *   ape  fp32 [kpool, D]  slot embeddings
 *   kp   bf16 [P_tot, D]  output, laid out as for kpool_pool_keys
 * flags: 0 or KPOOL_FLAG_TAIL, as for kpool_pool_keys.
 * k, g, ape and kp must be 16-byte aligned; D a multiple of 8 (<= 1024); kpool >= 1.
 * Inputs must be finite. */
int kpool_pool_keys_gated(const uint16_t *k, const uint16_t *g, const float *ape,
                          const int32_t *cu_seqlens_host, const int32_t *cu_seqlens_dev,
                          const int32_t *cu_pools_dev, int32_t nseq, int32_t D, int32_t kpool,
                          uint32_t flags, uint16_t *kp, void *stream);

/* Workspace for kpool_score_topk over rows [q_lo, q_hi): per query row of a
 * chunk, one fp32 score row at a pitch of max_pools rounded up to 64 plus one
 * fp32 maximum per 16 pools of it; the score rows of one chunk are capped at
 * 2 GiB (Megatron-LM PR #8299 "Change": the chunked score path caps its score
 * buffer at 2 GiB per chunk).  With nbuf = 2 the size covers two such chunk
 * buffers when the range needs more than one chunk (for KPOOL_FLAG_OVERLAP:
 * two chunks are then in flight, up to 2 x 2 GiB of scores); with nbuf = 1, one.
 * Returns 0 for an empty range or an nbuf other than 1 or 2. */
size_t kpool_workspace_bytes(int64_t q_lo, int64_t q_hi, int32_t max_pools, int32_t nbuf);

/* Flags of kpool_score_topk. */
#define KPOOL_FLAG_OVERLAP 1u /* two chunk buffers, chunks alternating between two streams */

/* The chunk plan kpool_score_topk follows for a sequence of at most max_pools pools
 * (per kpool_count_pools with the same tail flag), a workspace of workspace_bytes and
 * these flags: returns the rows per chunk (> 0; each chunk's fp32 scores at most
 * 2 GiB) and writes the number of chunk buffers (1, or 2 with KPOOL_FLAG_OVERLAP and
 * room for two rows) to *nbuf_out (nullable).  Returns a negative kpool_status for
 * max_pools < 1, unknown flags, or a workspace smaller than one row. */
int64_t kpool_chunk_rows(int32_t max_pools, size_t workspace_bytes, uint32_t flags,
                         int32_t *nbuf_out);

/* Step 2 - score and select, for the global rows [q_lo, q_hi).
 * (Megatron-LM PR #8299 "Change": one rank's contiguous slice of query rows
 * goes through the chunked score/top-k path; per row the result equals the
 * unsliced one.  Atlas tp.rs module doc: the score formula and tie-break.)
 *   q        bf16 [T, H, D]    index queries
 *   kp       bf16 [P_tot, D]   pooled keys from kpool_pool_keys
 *   w        fp32 [T, H]       per-row head weights (any sign)
 *            (of q and w the rows [q_lo, q_hi) are read and no others)
 *   scale    > 0, usually 1/sqrt(D)
 *   budget   pools kept per row, 1..2048 (index_topk / kpool; 2048 for the per-token
 *            indexer, kpool = 1)
 *   workspace, workspace_bytes: device scratch of at least one row
 *            (kpool_workspace_bytes(q_lo, q_lo + 1, max_pools, 1)).  Each chunk
 *            has as many rows as the 2 GiB score cap and its buffer allow.
 *            Contents are scratch on return.
 *   flags    KPOOL_FLAG_OVERLAP and/or KPOOL_FLAG_TAIL.  Without OVERLAP: one
 *            chunk buffer; every launch on the caller's stream, one after the other
 *            (each kernel runs alone, which per-kernel timing needs).  With
 *            KPOOL_FLAG_OVERLAP: a workspace of two rows or more is split into two
 *            chunk buffers, and consecutive chunks alternate between the caller's
 *            stream and its helper stream, so one chunk's selection runs beside the
 *            next chunk's scoring; each buffer keeps the 2 GiB cap.  Results are
 *            bitwise the same either way.  KPOOL_FLAG_TAIL: full pools only (kp
 *            pooled with the same flag), so a row sees min(t / kpool + 1, L / kpool)
 *            pools.  Unknown bits return KPOOL_EINVAL.
 *   pool_ids int32 [q_hi - q_lo, budget] output: sequence-local pool ids,
 *            best first by (score desc, pool asc), -1 after the visible pools
 *            run out.  -0.0 ranks equal to +0.0; NaN ranks below -inf.  q, kp and
 *            w must be finite (the score's ReLU does not propagate NaN).
 *   scores_out NULLABLE fp32 [q_hi - q_lo, max_pools] (max_pools of
 *            kpool_count_pools with the same tail flag): the fp32 scores the
 *            selection ranked, -inf where the pool is not visible.
 * Supported (H, D): (4, 16) and (32, 128).  q_lo == q_hi is a no-op.
 * Sizes: one sequence's pooled keys must stay below 4 GiB (fewer than 2^24 pools
 * at D = 128) and one fp32 score row within 2 GiB; larger returns
 * KPOOL_EUNSUPPORTED. */
int kpool_score_topk(const uint16_t *q, const uint16_t *kp, const float *w,
                     const int32_t *cu_seqlens_host, const int32_t *cu_seqlens_dev,
                     int32_t nseq, int32_t H, int32_t D, int32_t kpool, float scale,
                     int64_t q_lo, int64_t q_hi, int32_t budget,
                     void *workspace, size_t workspace_bytes, uint32_t flags,
                     int32_t *pool_ids, float *scores_out, void *stream);

/* kpool_score_topk for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, and harnesses that forbid hipMalloc.  Same
 * arguments and results as kpool_score_topk (flags: KPOOL_FLAG_TAIL as there;
 * KPOOL_FLAG_OVERLAP has no effect here) but without a workspace argument: the workspace is a
 * static device array of KPOOL_NOALLOC_SCRATCH_BYTES (64 MiB) inside the library:
 * each GPU the library runs on holds its own copy until the process ends.  The call
 * allocates nothing (no hipMalloc / hipFree, no stream or event creation; the profiler
 * is bypassed); its chunks, as many rows each as one 64 MiB workspace holds, run on
 * `stream` one after the other.
 *   - A sequence whose score row (its pools rounded up to 64, plus one maximum per
 *     16 of them, 4 bytes each) exceeds the scratch, i.e. more than about 15.79M
 *     pools, returns KPOOL_EWORKSPACE with a message saying so.
 *   - All calls on one GPU share that GPU's array, which keeps the last call's
 *     contents (nothing in it needs clearing between calls).  Calls that overlap on
 *     one GPU (different streams or host threads at once) race on it: order them. */
#define KPOOL_NOALLOC_SCRATCH_BYTES (64u << 20)
int kpool_score_topk_noalloc(const uint16_t *q, const uint16_t *kp, const float *w,
                             const int32_t *cu_seqlens_host, const int32_t *cu_seqlens_dev,
                             int32_t nseq, int32_t H, int32_t D, int32_t kpool, float scale,
                             int64_t q_lo, int64_t q_hi, int32_t budget, uint32_t flags,
                             int32_t *pool_ids, float *scores_out, void *stream);

/* Step 3 - expansion and causal filter (Megatron-LM PR #8299 "Change": pool
 * expansion and mask filtering run after the pool ids are known).
 *   token_ids[i - q_lo, b*kpool + j] = p*kpool + j   if p = pool_ids[i - q_lo, b] >= 0
 *                                                    and p*kpool + j <= t(i)
 *                                    = -1            otherwise
 *   flags 0 or KPOOL_FLAG_TAIL.  Tail mode appends kpool - 1 slots per row: with
 *   a = (L / kpool) * kpool for the row's sequence of L tokens,
 *   token_ids[i - q_lo, budget*kpool + j] = a + j if a + j < L and a + j <= t(i), else -1.
 *   pool_ids  int32 [q_hi - q_lo, budget];
 *   token_ids int32 [q_hi - q_lo, budget*kpool (+ kpool - 1 in tail mode)], 16-byte
 *   aligned when kpool = 4 without tail mode. */
int kpool_expand(const int32_t *pool_ids, const int32_t *cu_seqlens_host,
                 const int32_t *cu_seqlens_dev, int32_t nseq, int32_t kpool,
                 int64_t q_lo, int64_t q_hi, int32_t budget, uint32_t flags,
                 int32_t *token_ids, void *stream);

/* The selection step alone, over caller-provided fp32 scores (the second
 * half of the chunk loop, exposed so it can be checked on its own).
 *   scores   fp32 [rows, ld], ld % 4 == 0, 16-byte aligned
 *   n_valid  int32 [rows] device: row r ranks scores[r, 0 .. n_valid[r]),
 *            0 <= n_valid[r] <= ld (a value outside is clamped to that range: a
 *            negative count selects nothing, one past ld ranks the whole row)
 *   budget   1..2048, as for kpool_score_topk
 *   pool_ids int32 [rows, budget]: same ordering and padding as kpool_score_topk */
int kpool_topk(const float *scores, int64_t ld, const int32_t *n_valid, int64_t rows,
               int32_t budget, int32_t *pool_ids, void *stream);

/* Attention of query rows over keys and values - what the selection is made for
 * (Megatron-LM PR #8299 "Mechanism": the selected tokens are what a row attends to).
 * For token row i of sequence s, query head h and key head g = h / (Hq / Hkv):
 *   o[i,h,:] = sum_j softmax_j(scale * <q[i,h,:], k[j,g,:]>) v[j,g,:]
 *   lse[i,h] = log sum_j exp(scale * <q[i,h,:], k[j,g,:]>)
 * over the tokens j that the row sees; kpool_attend: every j <= t(i).
 *   q        bf16, token row i at q + i * q_stride elements, its heads [Hq, D] contiguous;
 *            k, v likewise with [Hkv, D] (a slice of a fused projection needs no copy)
 *   cu_q     sequence s has the query rows [cu_q[s], cu_q[s+1]) and the keys
 *   cu_k     [cu_k[s], cu_k[s+1]); its queries are the LAST rows of its keys: with Lq
 *            queries and Lk keys, query n sits at position t = Lk - Lq + n.  A whole prompt
 *            has cu_q = cu_k; a chunk of a prompt, or one new token a sequence, fewer
 *            queries than keys.  Any lengths, 0 included; Lq > Lk leaves the first rows
 *            without keys.  Host and device copies hold the same values.  The launch is planned
 *            from the host's, so a captured call replays with the lengths it was captured with:
 *            new lengths (a decoding step) take a new call or a new capture.
 *   o        bf16 [Tq, Hq, D] contiguous, Tq = cu_q[nseq]; rows past Tq are not touched
 *   lse      NULLABLE fp32 [Tq, Hq]
 * A row that sees nothing gets o = 0 and lse = -inf.  Sums and statistics are fp32; the
 * weights are rounded to bf16 for the product with v, and o once.  q, k and v must be finite
 * in the rows of the sequences; nothing outside them is read.  Outputs and the workspace
 * overlap neither inputs nor one another.  The same call gives the same bits every time.
 * Sizes: D a multiple of 8 up to 128; Hq a multiple of Hkv; strides multiples of 8 from
 * H * D to 2^24; q, k, v, o and the workspace 16-byte aligned.
 *   workspace  kpool_attend_workspace_bytes(the same sizes) bytes (may be 0: then it is
 *            not read): the parts of the key axis where there are few query rows, as many for
 *            every row as the longest sequence has; scratch. */
size_t kpool_attend_workspace_bytes(const int32_t *cu_q_host, const int32_t *cu_k_host, int32_t nseq,
                                    int32_t Hq, int32_t Hkv, int32_t D);
int kpool_attend(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                 const uint16_t *v, int64_t v_stride, const int32_t *cu_q_host,
                 const int32_t *cu_q_dev, const int32_t *cu_k_host, const int32_t *cu_k_dev,
                 int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D, float scale, void *workspace,
                 size_t workspace_bytes, uint16_t *o, float *lse, void *stream);

/* Gradients of kpool_attend.  With P = exp(scale * q k^T - lse) over what a row sees and
 * delta[i,h] = <d_o[i,h,:], o[i,h,:]> (rows that see few keys, up to 512, where o's rounding
 * would show, take it as sum_j P[i,j] <d_o[i], v[j]>, which is the same):
 *   dv[j] = sum_i P[i,j] d_o[i]        dS[i,j] = P[i,j] (<d_o[i], v[j]> - delta[i])
 *   dk[j] = scale sum_i dS[i,j] q[i]   dq[i] = scale sum_j dS[i,j] k[j]
 * where dk and dv of a key head sum over its Hq / Hkv query heads.
 *   d_o, o   bf16 [Tq, Hq, D] contiguous; o and lse (fp32 [Tq, Hq]) from kpool_attend
 *   dq       bf16 [Tq, Hq, D];  dk, dv  bf16 [Tk, Hkv, D], contiguous, overwritten (0 for a
 *            row that sees nothing and a key that no row sees)
 *   workspace  kpool_attend_backward_workspace_bytes bytes, 16-byte aligned; scratch
 * The other arguments are the forward call's, and d_o must be finite as well; the outputs and
 * the workspace overlap neither inputs nor one another.  Sums are fp32 in a fixed order (no
 * atomics): the same call gives the same bits. */
size_t kpool_attend_backward_workspace_bytes(const int32_t *cu_q_host, const int32_t *cu_k_host,
                                             int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D);
int kpool_attend_backward(const uint16_t *d_o, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                          int64_t k_stride, const uint16_t *v, int64_t v_stride, const uint16_t *o,
                          const float *lse, const int32_t *cu_q_host, const int32_t *cu_q_dev,
                          const int32_t *cu_k_host, const int32_t *cu_k_dev, int32_t nseq, int32_t Hq,
                          int32_t Hkv, int32_t D, float scale, void *workspace,
                          size_t workspace_bytes, uint16_t *dq, uint16_t *dk, uint16_t *dv,
                          void *stream);

/* kpool_attend over the tokens a row selected: row i sees the tokens token_ids[i, 0 .. width)
 * that lie in 0 .. t(i) (kpool_expand's output; other entries, -1 among them, stand for
 * nothing, wherever they are in the list).  A token that is listed twice counts twice.
 *   token_ids  int32 [Tq, width], sequence-local token ids, any order
 * The other arguments, the outputs and what holds for them are kpool_attend's; only the
 * listed tokens' keys and values have to be finite, as no others are read. */
size_t kpool_attend_selected_workspace_bytes(int64_t Tq, int32_t nseq, int32_t width, int32_t Hq,
                                             int32_t Hkv, int32_t D);
int kpool_attend_selected(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                          const uint16_t *v, int64_t v_stride, const int32_t *token_ids,
                          int32_t width, const int32_t *cu_q_host, const int32_t *cu_q_dev,
                          const int32_t *cu_k_host, const int32_t *cu_k_dev, int32_t nseq, int32_t Hq,
                          int32_t Hkv, int32_t D, float scale, void *workspace,
                          size_t workspace_bytes, uint16_t *o, float *lse, void *stream);

/* Latent attention with its keys and values expanded for each head - prompts and training (Atlas
 * inference docs, glm5next_dsa/tp.rs: the shard plan's q_b_proj, kv_b_proj and kv_a_proj_with_mqa):
 * kpool_attend with keys that have a positional part besides, P values a token that all heads share,
 *   s[i,h,j] = scale * (<q[i,h,:D], k[j,g,:]> + <q[i,h,D:], k_pe[j,:]>)
 *   o[i,h,:] = sum_j softmax_j(s) v[j,g,:]        lse[i,h] = log sum_j exp(s)
 *   q        bf16, token row i at q + i * q_stride elements, its heads [Hq, D + P] contiguous
 *   k, v     bf16, head g of token j at k + j * k_stride + g * k_head_stride (v likewise): heads may lie
 *            side by side with the values, as one projection gives them
 *   k_pe     bf16, token j's at k_pe + j * pe_stride
 *   o        bf16 [Tq, Hq, D] contiguous;  lse NULLABLE fp32 [Tq, Hq]
 * cu_q, cu_k, scale, the workspace and what holds for rows, sums, bits and overlaps are kpool_attend's.
 * One kernel for all numbers of rows: new tokens over a cache take kpool_attend_latent.
 * Sizes: D a multiple of 8 up to 128, P one from 8 to 64; Hq a multiple of Hkv; strides multiples of 8 up to
 * 2^24, q's from Hq * (D + P), k's and v's from (Hkv - 1) * their head stride + D, head strides from D,
 * pe_stride from P; q, k, k_pe, v, o and the workspace 16-byte aligned. */
size_t kpool_attend_expanded_workspace_bytes(const int32_t *cu_q_host, const int32_t *cu_k_host,
                                             int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D, int32_t P);
int kpool_attend_expanded(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                          int64_t k_head_stride, const uint16_t *k_pe, int64_t pe_stride,
                          const uint16_t *v, int64_t v_stride, int64_t v_head_stride,
                          const int32_t *cu_q_host, const int32_t *cu_q_dev, const int32_t *cu_k_host,
                          const int32_t *cu_k_dev, int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D,
                          int32_t P, float scale, void *workspace, size_t workspace_bytes, uint16_t *o,
                          float *lse, void *stream);

/* Its gradients, by kpool_attend_backward's formulas: dq [Tq, Hq, D + P], dk and dv [Tk, Hkv, D] and
 *   dk_pe[j] = scale * sum_h sum_i dS[i,h,j] q[i,h,D:]        [Tk, P]
 * summed over all query heads in fp32; all bf16, contiguous, overwritten (0 for a row that sees nothing and a
 * key that no row sees).  d_o and o bf16 [Tq, Hq, D] and lse fp32 [Tq, Hq] contiguous; the other arguments
 * are the forward call's, and what holds for kpool_attend_backward holds here. */
size_t kpool_attend_expanded_backward_workspace_bytes(const int32_t *cu_q_host, const int32_t *cu_k_host,
                                                      int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D,
                                                      int32_t P);
int kpool_attend_expanded_backward(const uint16_t *d_o, const uint16_t *q, int64_t q_stride,
                                   const uint16_t *k, int64_t k_stride, int64_t k_head_stride,
                                   const uint16_t *k_pe, int64_t pe_stride, const uint16_t *v,
                                   int64_t v_stride, int64_t v_head_stride, const uint16_t *o,
                                   const float *lse, const int32_t *cu_q_host, const int32_t *cu_q_dev,
                                   const int32_t *cu_k_host, const int32_t *cu_k_dev, int32_t nseq,
                                   int32_t Hq, int32_t Hkv, int32_t D, int32_t P, float scale,
                                   void *workspace, size_t workspace_bytes, uint16_t *dq, uint16_t *dk,
                                   uint16_t *dk_pe, uint16_t *dv, void *stream);

/* Latent attention over a cache - the absorbed form (Atlas inference docs, glm5next_dsa/tp.rs: the
 * shard plan's kv_a_proj_with_mqa and kv_b_proj): one row of R + P values a token is the key of every
 * head, its first R values are the value.  For token row i of sequence s and head h
 *   o[i,h,:] = sum_j softmax_j(scale * <q[i,h,:], c[j,:]>) c[j,:R]
 *   lse[i,h] = log sum_j exp(scale * <q[i,h,:], c[j,:]>)
 * over the tokens j <= t(i), or, kpool_attend_latent_selected, over the tokens token_ids[i, 0 .. width)
 * that lie in 0 .. t(i) (as for kpool_attend_selected: other entries stand for nothing, a token that is
 * listed twice counts twice).
 *   q        bf16, token row i at q + i * q_stride elements, its heads [H, R + P] contiguous (the latent
 *            part, absorbed, then the positional part)
 *   cache    bf16, row r at cache + r * cache_stride elements, cache_rows of them
 *   page_table  int32 [nseq, pages_per_seq] device: token j of sequence s is the cache's row
 *            page_table[s, j / page_size] * page_size + j % page_size; or NULL:
 *   k_starts int32 [nseq] device: token j is row k_starts[s] + j (not read with a page table); a negative
 *            start stands for no tokens at all
 *   k_lens   int32 [nseq] device: the sequence's tokens, those of its queries among them; its queries
 *            are the LAST of them: with Lq queries, query n sits at position t = k_lens[s] - Lq + n.
 *            Lengths, page table and starts are read when the call runs on the device: a captured
 *            call replays with what they hold then.  Lengths are taken as at most max_len (and what
 *            pages_per_seq pages hold) and at least 0.  Tokens whose page or row the cache does not
 *            have stand for nothing; entries of the page table past a sequence's tokens are not read.
 *   cu_q     sequence s has the query rows [cu_q[s], cu_q[s+1]), any numbers, 0 among them; host and device
 *            copies hold the same values
 *   o        bf16 [Tq, H, R] contiguous, Tq = cu_q[nseq]; rows past Tq are not touched
 *   lse      NULLABLE fp32 [Tq, H]
 * A row that sees nothing gets o = 0 and lse = -inf.  Sums and statistics are fp32; the weights are
 * rounded to bf16 for the product with the values, and o once.  q and the cache rows of the tokens that
 * some row sees must be finite; no other rows are read.  Outputs and the workspace overlap neither inputs
 * nor one another.  The same call gives the same bits every time.
 * Sizes: R a multiple of 8 up to 512; P a multiple of 8 up to 64, or 0; strides multiples of 8 (q's from
 * H * (R + P) to 2^24, the cache's from R + P to 2^24); q, cache, o and the workspace 16-byte aligned; at
 * most 2^31 - 1 cache rows and tokens in pages_per_seq pages, max_len at most 2^31 - 256; tiles (16
 * to 64 rows of a sequence by 64 tokens) of all sequences below 2^28.
 *   workspace  kpool_attend_latent(_selected)_workspace_bytes(the same sizes) bytes (may be 0: then it is
 *            not read); scratch.  It does not depend on what k_lens holds. */
size_t kpool_attend_latent_workspace_bytes(const int32_t *cu_q_host, int32_t nseq, int32_t max_len,
                                           int32_t H, int32_t R, int32_t P);
int kpool_attend_latent(const uint16_t *q, int64_t q_stride, const uint16_t *cache,
                        int64_t cache_stride, int64_t cache_rows, const int32_t *page_table,
                        int32_t pages_per_seq, int32_t page_size, const int32_t *k_starts,
                        const int32_t *k_lens, int32_t max_len, const int32_t *cu_q_host,
                        const int32_t *cu_q_dev, int32_t nseq, int32_t H, int32_t R, int32_t P,
                        float scale, void *workspace, size_t workspace_bytes, uint16_t *o, float *lse,
                        void *stream);
size_t kpool_attend_latent_selected_workspace_bytes(int64_t Tq, int32_t width, int32_t H, int32_t R,
                                                    int32_t P);
int kpool_attend_latent_selected(const uint16_t *q, int64_t q_stride, const uint16_t *cache,
                                 int64_t cache_stride, int64_t cache_rows, const int32_t *page_table,
                                 int32_t pages_per_seq, int32_t page_size, const int32_t *k_starts,
                                 const int32_t *k_lens, const int32_t *token_ids, int32_t width,
                                 const int32_t *cu_q_host, const int32_t *cu_q_dev, int32_t nseq,
                                 int32_t H, int32_t R, int32_t P, float scale, void *workspace,
                                 size_t workspace_bytes, uint16_t *o, float *lse, void *stream);

/* Layer norm of rows - the indexer's keys pass one with weight and bias before they are
 * pooled (Atlas inference docs, glm5next_dsa/tp.rs: the indexer's k_norm among the shard
 * plan's tensors).  For row r and column j < N:
 *   mean = sum_j x[r,j] / N,   rstd = 1 / sqrt(sum_j (x[r,j] - mean)^2 / N + eps)
 *   y[r,j] = (x[r,j] - mean) * rstd * weight[j] + bias[j]
 * the mean in 64 bits, the rest in fp32, rounded once to the output's type (a constant row's
 * x - mean is 0 exactly; the mean that is returned is rounded to fp32).
 *   dtype    of x, y, dy and dx: KPOOL_DTYPE_BF16 or KPOOL_DTYPE_F32
 *   x        [rows, N], row r at x + r * x_stride elements (x_stride >= N): a slice of a
 *            wider projection needs no copy
 *   weight   fp32 [N], NULL for ones;  bias fp32 [N], NULL for zeros
 *   eps      finite, >= 0 (a constant row with eps = 0 gives the formula's NaN)
 *   y        [rows, N] contiguous
 *   mean, rstd  NULLABLE fp32 [rows]: what the backward pass reads
 * The outputs overlap neither inputs nor one another.
 * rows 0 is a no-op; N in [1, 2^26].  Any alignment of whole elements is taken; rows that start
 * at 16-byte bounds and hold whole 16-byte pieces are the fastest. */
#define KPOOL_DTYPE_BF16 0
#define KPOOL_DTYPE_F32 1
int kpool_layer_norm(const void *x, int64_t x_stride, const float *weight, const float *bias,
                     int64_t rows, int32_t N, float eps, int32_t dtype, void *y, float *mean,
                     float *rstd, void *stream);

/* Its backward pass.  With xh = (x - mean) * rstd and g = dy * weight:
 *   dx[r,j] = rstd * (g - sum_j(g) / N - xh * sum_j(g * xh) / N)
 *   dweight[j] = sum_r dy * xh,   dbias[j] = sum_r dy            (fp32 sums)
 *   dy       [rows, N] contiguous;  x, x_stride, weight as in the forward call
 *   mean, rstd  fp32 [rows] from it
 *   dx       NULLABLE [rows, N] contiguous
 *   dweight, dbias  NULLABLE fp32 [N], overwritten
 *   workspace  kpool_layer_norm_backward_workspace_bytes(rows, N) bytes where dweight or
 *            dbias is given (NULL and 0 otherwise), 16-byte aligned; scratch on return
 * The outputs and the workspace overlap neither inputs nor one another.  The sums over rows
 * run in a fixed order: the same inputs give the same bits.  rows 0 writes zeros to dweight
 * and dbias. */
size_t kpool_layer_norm_backward_workspace_bytes(int64_t rows, int32_t N);
int kpool_layer_norm_backward(const void *dy, const void *x, int64_t x_stride, const float *weight,
                              const float *mean, const float *rstd, int64_t rows, int32_t N,
                              int32_t dtype, void *workspace, size_t workspace_bytes, void *dx,
                              float *dweight, float *dbias, void *stream);

/* Rotary positions of rows of heads - what the indexer's and the attention's queries and keys
 * pass before they meet (Atlas inference docs, glm5next_dsa/tp.rs: the shard plan's q_b_proj and
 * kv_a_proj_with_mqa carry the positional part).  With theta = positions[r] * freqs[j], pair j of
 * each head of row r becomes
 *   (a, b) -> factor * (a cos(theta) - b sin(theta), a sin(theta) + b cos(theta))
 * and the head's other values are copied.
 *   pairs    1 .. (D - begin) / 2.  Without KPOOL_ROTARY_INTERLEAVED pair j is the elements
 *            begin + j and begin + pairs + j of a head, with it begin + 2 j and begin + 2 j + 1
 *   KPOOL_ROTARY_INVERSE  turns by -theta: the backward pass (dx from dy; freqs, positions and factor
 *            as in the forward call)
 *   x        [rows, heads, D], row r at x + r * x_stride elements, its heads contiguous
 *   positions  int32 [rows] device, any value;  freqs  fp64 [pairs] device, radians a token, finite:
 *            scaled for long contexts as the model has it;  factor finite (1, or the scaling's)
 *   dtype    of x and y
 *   y        like x at its own stride; or x itself (the same pointer and stride): in place.  Rows of
 *            x and y may share a wider row side by side; they do not overlap otherwise, nor does y
 *            overlap positions or freqs.
 * Angles are 64-bit turns, sines and cosines fp32, as the products; one rounding to the output's type.
 * D up to 1024.  rows 0 is a no-op.  Any alignment of whole elements; 16-byte bounds are the fastest. */
#define KPOOL_ROTARY_INTERLEAVED 1u
#define KPOOL_ROTARY_INVERSE 2u
int kpool_rotary(const void *x, int64_t x_stride, const int32_t *positions, const double *freqs,
                 int64_t rows, int32_t heads, int32_t D, int32_t begin, int32_t pairs, float factor,
                 int32_t dtype, uint32_t flags, void *y, int64_t y_stride, void *stream);

/* Optional per-kernel device timing, per host thread.  While enabled on a
 * thread, every launch that thread's calls make is bracketed by HIP events on
 * its stream.  kpool_profile_collect waits for the events the calling thread
 * recorded, adds each kernel kind's elapsed time (ms) and launch count into
 * ms[kind] / launches[kind] (arrays of KPOOL_PROFILE_KINDS) and forgets them.
 * Other threads' records and switches are untouched.  Event spans of
 * overlapped chunks (KPOOL_FLAG_OVERLAP) include whatever else the GPU runs
 * meanwhile; time kernels with flags = 0. */
#define KPOOL_PROFILE_KINDS 5 /* 0 pool_keys, 1 score, 2 topk, 3 expand, 4 scores_out copy */
int kpool_profile_enable(int on);
int kpool_profile_collect(double *ms, int64_t *launches);
/* The same for the calls around the selection (a call's launches as one), which
 * kpool_profile_collect neither reports nor forgets: arrays of
 * KPOOL_LAYER_PROFILE_KINDS. */
#define KPOOL_LAYER_PROFILE_KINDS 2 /* 0 layer norm and rotary positions, 1 attention */
int kpool_layer_profile_collect(double *ms, int64_t *launches);

#ifdef __cplusplus
}
#endif

#endif /* KPOOL_H */
