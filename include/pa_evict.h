/*
 * pa_evict.h -- C ABI of eviction from the paged cache: the attention weight
 * every cached token has received, the choice of the tokens worth keeping, and
 * the move that packs them.
 *
 * Each KV head keeps its own tokens: a page holds the rows of one head, so slot
 * t of a sequence may hold one token for one head and another for the next, and
 * the block table, the length and the attention kernels know nothing of it
 * (keys are rotated before they are cached, so a row may lie anywhere).  All
 * heads of a sequence keep the same number.
 *
 * The weights ("mass") are fp32 [num_seqs][num_kv_heads][mass_stride], token t of
 * a sequence at index t; row s goes with row s of the block tables.
 *
 * The conventions of pa.h hold (device pointers, 16-byte alignment of the pools
 * and of q, asynchronous on `stream`, checks on the host, values only the device
 * sees checked by the kernels).
 */
#ifndef PA_EVICT_H_
#define PA_EVICT_H_

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pa_attention_mass -- add to every cached token the softmax weights a step's
 * queries gave it.  Query i of sequence s (row cu_q_lens[s] + i, position
 * c + i with c = context_lens[s] - n) sees keys 0 .. c + i, as in
 * pa_chunked_prefill:
 *     mass_out[s][g][t] = mass_in[s][g][t]
 *         + sum_{i: c + i >= t} sum_{h of group g} exp(scale * q[r][h] . K_s[g][t] - lse[r][h])
 *
 *   q            bf16 [total_q][num_q_heads][head_dim], token stride q_stride;
 *                total_q >= 1.
 *   lse          float [total_q][num_q_heads]: the log-sum-exp of these rows over
 *                the keys they see here, as pa_decode and pa_chunked_prefill return
 *                it (an infinite one: the row adds nothing, whatever its scores are).
 *                pa_tree_attention's is that of a row whose mask is the chain of its
 *                own and all earlier tokens.  The row of a token on a branch has not
 *                seen the other branches, whose weights here would have no bound: pass
 *                the accepted branch instead, after pa_compact_tokens has packed it
 *                behind the cache -- its rows of q and lse in order, n its tokens,
 *                context_lens the cached ones and those -- where each row sees just
 *                what it saw in the tree.
 *   cu_q_lens    int32 [num_seqs + 1], device; or NULL: a decode step, row s is
 *                sequence s's only query (total_q = num_seqs, max_q_len = 1).
 *   max_q_len    host bound on any n (larger ones are left out); at most
 *                PA_MASS_MAX_QUERIES.
 *   mass_in      the weights so far, of every t < context_len (a token that this
 *                step wrote: 0, or see pa_attention_mass_ex), or NULL for none.
 *   mass_out     may be mass_in.  Entries at and past a sequence's length are
 *                not written.
 *   mass_stride  floats between two heads of both, >= every context length.
 * A sequence with inconsistent values (cu_q_lens not ascending within
 * [0, total_q], n > max_q_len, n > context_len, a context beyond the table or
 * mass_stride) is left out and sets PA_DEV_ERR_CONTEXT.  The tokens of a bad
 * block id add nothing (mass_out = mass_in) and set PA_DEV_ERR_BLOCK_ID.
 * A sum runs over the rows in a fixed order: equal inputs give equal bits.
 * Stream order: as with pa_tree_attention (nothing is read or written before the
 * kernel before has finished).
 */
#define PA_MASS_MAX_QUERIES (1 << 20)

PA_API int pa_attention_mass(const void* q, int64_t q_stride, const float* lse,
                             const int32_t* cu_q_lens, int32_t total_q, int32_t max_q_len,
                             const void* k_pool, pa_pool_desc pool, const int32_t* block_tables,
                             int32_t max_blocks_per_seq, const int32_t* context_lens,
                             int32_t num_seqs, int32_t num_q_heads, float scale,
                             const float* mass_in, float* mass_out, int64_t mass_stride,
                             void* stream);

/*
 * pa_attention_mass_ex -- pa_attention_mass with flags (0: as above).
 *   PA_MASS_OWN_FROM_ZERO  a step's own tokens (t >= c) had no weight before it:
 *     mass_in is read for t < c only.  Without it mass_in[t] of a token written this
 *     step has to be 0, which it is not behind an eviction that packed the weights in
 *     place, nor where a rejected draft's token lay.
 */
#define PA_MASS_OWN_FROM_ZERO 0x1

PA_API int pa_attention_mass_ex(const void* q, int64_t q_stride, const float* lse,
                                const int32_t* cu_q_lens, int32_t total_q, int32_t max_q_len,
                                const void* k_pool, pa_pool_desc pool,
                                const int32_t* block_tables, int32_t max_blocks_per_seq,
                                const int32_t* context_lens, int32_t num_seqs,
                                int32_t num_q_heads, float scale, const float* mass_in,
                                float* mass_out, int64_t mass_stride, uint32_t flags,
                                void* stream);

/*
 * pa_evict -- bring every sequence down to its budget.  Of L = context_lens[s]
 * tokens each KV head keeps
 *     keep = min(L, budgets[s], kept_stride, mass_out_stride):
 * the first min(sink, keep), the last min(recent, what is left), and the heaviest
 * others, the lowest index first among equal weights (NaN counts as
 * less than -inf).
 * Kept tokens stay in order: token kept[s][g][i] (ascending in i) becomes token
 * i, in the sequence's own blocks or in those of new_tables.
 *
 *   new_tables   int32 [num_seqs][new_max_blocks], or NULL to pack in place.  The
 *                blocks it names (ceil(keep / block_size) per sequence) must be
 *                no block of block_tables in use; a sequence whose blocks other
 *                sequences share must be packed this way.  In place, a sequence's
 *                blocks must be its own.
 *   kept         int32 [num_seqs][num_kv_heads][kept_stride], out; kept_stride >= 1
 *                (a budget of 0 empties a sequence).
 *   new_lens     int32 [num_seqs], out; must not be context_lens.
 *   mass_out     float [num_seqs][num_kv_heads][mass_out_stride], out: the kept
 *                tokens' weights, packed alike (-0 becomes 0, a NaN the canonical
 *                one).  May be mass with the same stride.
 * Entries of kept and mass_out past keep, rows of the cache past it, and blocks
 * of the table that are no longer needed are left as they were (so the tokens written
 * there next have no weight of their own yet: see PA_MASS_OWN_FROM_ZERO).  A length
 * outside [0, max_blocks_per_seq * block_size] or beyond mass_stride counts as 0
 * and sets PA_DEV_ERR_CONTEXT; a bad block id leaves its rows unmoved and sets
 * PA_DEV_ERR_BLOCK_ID.
 */
PA_API int pa_evict(const float* mass, int64_t mass_stride, void* k_pool, void* v_pool,
                    pa_pool_desc pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
                    const int32_t* context_lens, const int32_t* budgets, int32_t sink,
                    int32_t recent, const int32_t* new_tables, int32_t new_max_blocks,
                    int32_t* kept, int32_t kept_stride, int32_t* new_lens, float* mass_out,
                    int64_t mass_out_stride, int32_t num_seqs, void* stream);

/*
 * pa_compact_tokens -- the move alone: for every sequence s, KV head g and
 * i < counts[s], row base[s] + i takes K and V of row base[s] + kept[s][g][i].
 * With base[s] the cached length and kept the accepted branch of a drafted tree,
 * it packs what verification accepted.
 *
 *   new_tables   as in pa_evict (rows base + i of new_tables are written); NULL:
 *                in place.
 *   base         int32 [num_seqs], device, or NULL for zeros.
 *   kept         int32 [num_seqs][kept_heads][kept_stride]; kept_heads is
 *                num_kv_heads, or 1 for a list all heads share.  Strictly ascending
 *                in i and not below 0 (which makes the move in place independent
 *                of its order); kept_stride is at most 2^30.
 *   counts       int32 [num_seqs]; beyond [0, kept_stride] they are clamped, with
 *                PA_DEV_ERR_CONTEXT.
 * A row outside its table is left out, with PA_DEV_ERR_CONTEXT.
 */
PA_API int pa_compact_tokens(void* k_pool, void* v_pool, pa_pool_desc pool,
                             const int32_t* block_tables, int32_t max_blocks_per_seq,
                             const int32_t* new_tables, int32_t new_max_blocks,
                             const int32_t* base, const int32_t* kept, int32_t kept_heads,
                             int32_t kept_stride, const int32_t* counts, int32_t num_seqs,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_EVICT_H_ */
