/*
 * kda_hybrid.h -- C ABI of the operators of libkda.so that stand beside KDA
 * in a hybrid stack: the plan of a serving step, a paged key/value cache held
 * in 4 bits with the attention that reads it, and a gated linear recurrence
 * with its gradients.
 *
 * The conventions are those of kda.h: device pointers, C-contiguous and
 * 16-byte aligned (int32 arrays need 4-byte alignment, int64 arrays 8-byte),
 * an asynchronous call on `stream`, memory owned by the caller, nothing
 * launched after a refused argument, nothing on the stream but kernel
 * launches (so every call can be captured into a HIP graph and replayed).
 * Outputs may not overlap each other or the inputs except where a call says
 * so, and a workspace serves one call at a time.  A launch holds fewer than
 * 2^32 threads; a problem that takes more is KDA_ERR_UNSUPPORTED.
 * What lies in device memory is not checked by the host; where a value there
 * is an index (lengths, offsets, pages, slots), the kernels bound it, so that
 * no value makes an access leave the arrays.
 *
 * Sources: devpress.csdn.net K3 article §十四 (KDA state checkpoints under
 * the same paged management as the attention layers' cache), §三 (the hybrid
 * of KDA and full attention); zuoshipin.com/article/18261 §二 (channel-wise
 * retention with a lower bound, full-rank output gate).  The pages print no
 * formula; those below define the calls.
 */
#ifndef KDA_HYBRID_H_
#define KDA_HYBRID_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the plan of a serving step --------------------------------------------
 * One step serves n_req requests; request r has past_lens[r] tokens cached
 * and brings new_lens[r] more (negative lengths count as 0).  Its tokens lie
 * in pages of page_size tokens that block_table[r, :] names.  From the
 * lengths alone the call writes
 *   cu_seqlens [n_req+1] int32: offsets of the requests' new tokens in the
 *     packed batch, cut off at `tokens` -- what the kda_varlen_* calls, the
 *     attention and the recurrence take (the attention with other lengths
 *     where a request was cut off, see below);
 *   total_lens [n_req] int32: past + new (at most INT32_MAX);
 *   block_table [n_req, max_pages] int32, in place: the entries of the pages
 *     that the new tokens begin, taken off free_pages [n_free] in the order
 *     of the requests, -1 where the list has ended; no other entry changes;
 *   slot_map [tokens] int64: page * page_size + offset of every new token, -1
 *     where it has no page (a negative entry of the table, the list ended,
 *     max_pages passed) and for the rows behind the last request's;
 *   pages_taken [1] int32: how many pages the step needs (at most INT32_MAX);
 *     more than n_free means that the list was too short.
 * The list is read, not changed: the caller drops its first pages_taken
 * entries.
 * Where the new lengths add up to more than `tokens` (in a replayed graph the
 * host cannot see it), the last requests are cut off: request r keeps the rows
 * kept_r = cu_seqlens[r+1] - cu_seqlens[r] < new_lens[r], which is how a kernel
 * tells.  total_lens, block_table and pages_taken still go by new_lens.  Such a
 * request's total_lens[r] counts tokens that have no row and no slot, so it is
 * no input for the attention, which takes a sequence's rows for its newest
 * tokens: give it past_lens[r] + kept_r, which is total_lens[r] for every other
 * request.  page_size is a power of two, 16 to 256; n_req <= 8192, and
 * tokens, n_free and n_req * max_pages <= INT32_MAX (more: KDA_ERR_UNSUPPORTED). */
kda_status kda_plan_requests(int64_t n_req, int64_t tokens, int32_t page_size, int32_t max_pages,
                             const int32_t* past_lens, const int32_t* new_lens, int32_t* block_table,
                             int64_t n_free, const int32_t* free_pages, int32_t* cu_seqlens, int32_t* total_lens,
                             int64_t* slot_map, int32_t* pages_taken, void* stream);

/* ---- a key/value cache held in 4 bits ---------------------------------------
 * Every 32 channels of a row share a power of two, 2^(scale - 127); a value is
 * one of 0, 1/2, 1, 3/2, 2, 3, 4, 6 with a sign (e2m1: sign, two exponent bits,
 * one mantissa bit) times it, two values a byte, the even channel in the low
 * half.  A scale of 255 stands for 32 NaN. */
typedef struct {
    int64_t pages;          /* pages in the cache                               */
    int32_t page_size;      /* tokens per page: a power of two, 16 to 256       */
    int32_t heads;          /* key/value heads                                  */
    int32_t d;              /* head dim, 64 or 128                              */
    void* k;                /* [pages, heads, page_size, d/2]  uint8            */
    void* k_scale;          /* [pages, heads, page_size, d/32] uint8            */
    void* v;                /* as k                                             */
    void* v_scale;          /* as k_scale                                       */
} kda_cache4;

/* Rounds k, v [tokens, heads, d] (io_dtype) into the cache at slot_map
 * [tokens].  The scale of 32 channels whose largest magnitude is m is 2^e
 * with e = floor(log2 m) - 2, one more where m > 7 * 2^e, kept within
 * [-125, 125]; values round to nearest, halves to the even code, magnitudes
 * over 6 to 6.  Channels with an Inf or NaN among their 32 become NaN.  Rows
 * whose slot lies outside the cache are dropped.  No two rows may name the
 * same slot (the slot would hold a mix of them). */
kda_status kda_cache4_append(const kda_cache4* c, int64_t tokens, kda_dtype io_dtype, const void* k, const void* v,
                             const int64_t* slot_map, void* stream);

/* The rows at slot_map [tokens] as the values they stand for (all exact in
 * bf16 and fp32), into k, v [tokens, heads, d] (io_dtype); zeros where a slot
 * lies outside the cache. */
kda_status kda_cache4_read(const kda_cache4* c, int64_t tokens, kda_dtype io_dtype, const int64_t* slot_map, void* k,
                           void* v, void* stream);

typedef struct {
    int64_t n_seq;          /* sequences                                         */
    int64_t tokens;         /* rows of q, g and out                              */
    int32_t heads;          /* query heads, a multiple of the cache's heads      */
    int32_t max_pages;      /* row length of block_table                         */
    int64_t max_q;          /* about the most queries of a sequence, >= 1  (these two   */
    int64_t max_len;        /* about the longest sequence, >= 0     steer the split only) */
    kda_dtype io_dtype;     /* dtype of q, g and out                             */
    float scale;            /* of the scores; 0 or 2^-126 to 2^127 in size       */
} kda_cache4_attention_problem;

/* Bytes of partial results; 0 where the call needs none, or p or c is invalid. */
size_t kda_cache4_attention_workspace_size(const kda_cache4* c, const kda_cache4_attention_problem* p);

/* Causal grouped-query attention over the cache, for packed queries.
 * Sequence s holds total_lens[s] tokens, in the pages block_table[s, :]
 * (at most max_pages * page_size of them, itself at most INT32_MAX - 256:
 * more is KDA_ERR_UNSUPPORTED), the newest of which are its
 * queries: rows [cu_seqlens[s], cu_seqlens[s+1]) of q, or row s alone where
 * cu_seqlens is NULL (one new token each; then tokens == n_seq).  Query i of
 * m sees the tokens at positions <= total_lens[s] - m + i:
 *   out[row, h] = softmax_t(scale * q[row, h] . K[t, h / group]) V[t, h / group]
 *                 * sigmoid(g[row, h])
 * q, g, out: [tokens, heads, d] io_dtype; g may be NULL (no gate).  A query
 * that sees nothing gives 0.  Pages outside the cache are left out, as if
 * their tokens were masked.  Rows of no sequence are not written.  Scores,
 * softmax and sums are fp32.  With bf16 the probabilities round to bf16 for
 * the product with the values; with fp32 the products take the queries and
 * probabilities in three bf16 parts, which is fp32 accuracy (4-bit values are
 * exact in bf16).  cu_seqlens must not decrease (offsets are bounded; others
 * give unspecified rows). */
kda_status kda_cache4_attention(const kda_cache4* c, const kda_cache4_attention_problem* p, const void* q,
                                const int32_t* block_table, const int32_t* total_lens, const int32_t* cu_seqlens,
                                const void* g, void* out, void* workspace, size_t workspace_bytes, void* stream);

/* The same for groups of sequences that share their first tokens, which are read
 * once for all of a group's rows: the sequences [group_offsets[j],
 * group_offsets[j+1]) have the same first prefix_lens[j] tokens, and those are
 * read where the group's first sequence has them (the other rows of block_table
 * need not name them; they may begin with the same pages).  Sequences of no
 * group, and groups of one, attend by themselves.  Where prefix_lens[j] passes
 * what a query of the group sees, or ends, only the tokens that all its queries
 * have behind them count as shared: the tables of the others have to name the
 * tokens from there on.
 *   group_offsets: [n_groups + 1], prefix_lens: [n_groups] int32 in device
 *   memory (bounded, as all indices are; offsets must not decrease, others give
 *   unspecified rows).
 *   p->max_len: about the most tokens of a sequence behind its prefix,
 *   max_prefix: about the longest prefix, >= 0 (both steer the split only).
 * n_groups == 0 is kda_cache4_attention; at most 2^23, and n_groups * p->heads at
 * most 2^30 (more: KDA_ERR_UNSUPPORTED).  Everything else is as there. */
size_t kda_cache4_shared_attention_workspace_size(const kda_cache4* c, const kda_cache4_attention_problem* p,
                                                  int64_t n_groups, int64_t max_prefix);
kda_status kda_cache4_shared_attention(const kda_cache4* c, const kda_cache4_attention_problem* p, const void* q,
                                       const int32_t* block_table, const int32_t* total_lens, int64_t n_groups,
                                       const int32_t* prefix_lens, const int32_t* group_offsets, int64_t max_prefix,
                                       const int32_t* cu_seqlens, const void* g, void* out, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* ---- a gated linear recurrence -----------------------------------------------
 * Per batch row and channel, a state h (fp32), and for token t
 *   lambda = max(log_alpha_t, log_alpha_min)
 *   h     <- exp(lambda) h + x_t
 *   out_t  = h * sigmoid(g_t)            (g NULL: out_t = h)
 * KDA's retention and output gate on a diagonal memory.  Rows are
 * independent; a packed batch (batch == 1, cu_seqlens of n_seq + 1 offsets,
 * as for kda_varlen_prepare) starts a state at each sequence's first token.
 * log_alpha is at most 0, as in kda.h (not checked); NaN acts as the floor.
 * An infinite state stays infinite under every finite lambda; with lambda =
 * -inf, which leaves nothing of a finite state, it gives NaN. */
typedef struct {
    int64_t batch;          /* rows; 1 for a packed batch                        */
    int64_t seqlen;         /* tokens of a row                                   */
    int64_t width;          /* channels, >= 1                                    */
    int64_t n_seq;          /* sequences of a packed batch; -1: not packed       */
    kda_dtype io_dtype;     /* dtype of x, g, out and their gradients            */
    float log_alpha_min;    /* retention floor in log space, < 0; -inf for none  */
} kda_recurrence_problem;

/* Bytes of scratch for the calls below; 0 where none is needed or p is invalid. */
size_t kda_recurrence_workspace_size(const kda_recurrence_problem* p);
size_t kda_recurrence_backward_workspace_size(const kda_recurrence_problem* p);

/*   x, g, out: [batch, seqlen, width] io_dtype; log_alpha: the same, fp32;
 *   state_in, state_out: [batch or n_seq, width] fp32, either may be NULL and
 *   they may be one array; cu_seqlens: NULL where p->n_seq is -1.  Tokens of
 *   no sequence are not written; an empty sequence passes its state through. */
kda_status kda_recurrence_prefill(const kda_recurrence_problem* p, const void* x, const float* log_alpha,
                                  const void* g, const float* state_in, const int32_t* cu_seqlens, void* out,
                                  float* state_out, void* workspace, size_t workspace_bytes, void* stream);

/* The same, leaving in a backward workspace the states that
 * kda_recurrence_backward continues from. */
kda_status kda_recurrence_prefill_for_backward(const kda_recurrence_problem* p, const void* x,
                                               const float* log_alpha, const void* g, const float* state_in,
                                               const int32_t* cu_seqlens, void* out, float* state_out,
                                               void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of <d_out, out> + <d_state, final states>, from the same inputs
 * and the workspace that the call above filled with them (state_in unchanged
 * too: not the array that state_out went to).  Where log_alpha <=
 * log_alpha_min, or is NaN, dlog_alpha is 0.  d_out, d_state may be NULL
 * (zero); dg is written where g is given and may be NULL otherwise;
 * d_state_in may be NULL.  Outputs are overwritten; tokens of no sequence are
 * not written.  The workspace can serve further backward calls. */
kda_status kda_recurrence_backward(const kda_recurrence_problem* p, const void* x, const float* log_alpha,
                                   const void* g, const float* state_in, const int32_t* cu_seqlens,
                                   const void* d_out, const float* d_state, void* dx, float* dlog_alpha, void* dg,
                                   float* d_state_in, void* workspace, size_t workspace_bytes, void* stream);

/* One token of each of N sequences: x, g, out [N, width], log_alpha fp32,
 * state [N, width] fp32 in place. */
kda_status kda_recurrence_step(int64_t N, int64_t width, kda_dtype io_dtype, float log_alpha_min, const void* x,
                               const float* log_alpha, const void* g, float* state, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_HYBRID_H_ */
