/*
 * pa_tree.h -- C ABI of attention for a tree of drafted tokens over the paged
 * cache (the verification step of speculative decoding).
 *
 * Sequence s owns query rows cu_q_lens[s] .. cu_q_lens[s+1]-1, its n drafted
 * tokens, on top of c = context_lens[s] - n cached ones; the drafted tokens' own
 * K/V sit at positions c .. c+n-1 of the cache (pa_rope_and_cache or
 * pa_reshape_and_cache wrote them).  Row i sees every cached token and the
 * drafted tokens j whose bit is set in its mask, itself included only if bit i
 * is set:
 *     visible(i) = { t < c } u { c + j : bit j of tree_mask[row i], j < n }
 *     out[r][h] = sum_{t in visible} softmax(scale * q[r][h] . K_s[g][t]) V_s[g][t]
 *     lse[r][h] = log(sum_{t in visible} exp(scale * q[r][h] . K_s[g][t]))
 * A row that sees nothing gets out = 0 and lse = -inf.  A tree's mask has, in
 * row i, the bits of token i and of its ancestors; any other pattern (several
 * trees, a window, a chain) is as good.
 *
 * The conventions of pa.h hold (device pointers, 16-byte alignment, strides in
 * elements and multiples of 8, asynchronous on `stream`, checks on the host,
 * values only the device sees checked by the kernel).
 */
#ifndef PA_TREE_H_
#define PA_TREE_H_

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Drafted tokens of one sequence at most. */
#define PA_TREE_MAX_TOKENS 4096

/*
 * pa_tree_attention
 *
 *   q            bf16 [total_q][num_q_heads][head_dim], token stride q_stride.
 *   cu_q_lens    int32 [num_seqs + 1], device; cu_q_lens[0] = 0,
 *                cu_q_lens[num_seqs] = total_q.  Rows past the last sequence's
 *                are not written.
 *   max_q_len    host bound on any n, 1 .. PA_TREE_MAX_TOKENS.
 *   tree_mask    int64 [total_q][mask_words], device: bit j % 64 of word j / 64 of
 *                a row is drafted token j of the row's own sequence; bits from n
 *                on are ignored.  64 * mask_words >= max_q_len.
 *   context_lens int32 [num_seqs], device, including the drafted tokens.
 *   out          bf16 [total_q][num_q_heads][head_dim], packed; must not overlap q.
 *   lse          float [total_q][num_q_heads], or NULL.
 *   workspace    device scratch of at least pa_tree_workspace_size() bytes, for
 *                the partial results of contexts that several CTAs share; its
 *                contents need no initialisation and are garbage afterwards.
 *                Calls that overlap on the GPU must not share a workspace.
 *
 * A sequence with inconsistent values (cu_q_lens not ascending within
 * [0, total_q], n > max_q_len, n > context_len, a context beyond the table) is
 * left out: its rows are not written and PA_DEV_ERR_CONTEXT is set.  A bad block
 * id leaves its tokens out of the softmax and sets PA_DEV_ERR_BLOCK_ID.
 *
 * Infinities and NaN: in K they reach only the rows that see the token.  In V of
 * a cached token they reach every row's output (every row sees it).  A drafted
 * token whose V holds one makes the outputs of the rows that see it NaN (all
 * head_dim values) and leaves the other rows as they are.
 *
 * Stream order: the call's first kernel may be set up while the kernel before it on
 * `stream` ends, but reads and writes nothing before it has finished: any argument may
 * be the result of the kernel directly before, and the workspace its scratch.
 *
 * Precision: scores and the P.V product accumulate in fp32, the running maximum
 * and sum are fp32, and the softmax weights enter P.V as their nearest bf16 and the
 * nearest bf16 of what that leaves (within 2^-17 of the weight); out is rounded once.
 * Weights reach 2^16 before the division by their sum, so |V| has to stay below 2^90
 * (with up to 2^20 keys) for the sums to stay finite.
 */
PA_API size_t pa_tree_workspace_size(int32_t max_q_len, int32_t num_q_heads, pa_pool_desc pool);

PA_API int pa_tree_attention(const void* q, int64_t q_stride, const int32_t* cu_q_lens,
                             int32_t total_q, int32_t max_q_len, const int64_t* tree_mask,
                             int32_t mask_words, const void* k_pool, const void* v_pool,
                             pa_pool_desc pool, const int32_t* block_tables,
                             int32_t max_blocks_per_seq, const int32_t* context_lens,
                             int32_t num_seqs, int32_t num_q_heads, float scale, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_TREE_H_ */
