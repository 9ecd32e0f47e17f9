/*
 * pa_rope.h -- C ABI of rotary positions and of the pass that prepares a
 * step's q, K and V for the paged cache: norms per head, rotation, cache write.
 *
 * Rotation.  The first rot_dim dims of a head row form rot_dim/2 pairs; pair i
 * of a token at position p turns by a = p * inv_freq[i]:
 *     y0 = factor * (x0 cos a - x1 sin a)
 *     y1 = factor * (x1 cos a + x0 sin a)
 * where (x0, x1) are dims (i, i + rot_dim/2) in the half layout and dims
 * (2i, 2i+1) in the interleaved one.  Dims rot_dim and up pass unchanged (no
 * factor).  The angle is formed and reduced to one turn in fp64, so positions
 * of millions keep the accuracy of small ones; cos, sin and the products are
 * fp32, and each output is rounded to bf16 once.
 *
 * Norm.  With a weight w (bf16 [head_dim], shared by the heads of q or of K)
 * every head row is first x * w / sqrt(mean(x^2) + eps), in fp32 and not
 * rounded before the rotation.
 *
 * The conventions of pa.h hold (device pointers, 16-byte alignment, strides in
 * elements and multiples of 8, asynchronous on `stream`, checks on the host).
 * Compiled sizes: head_dim 64 or 128; rot_dim a multiple of 16 from 0 (norm
 * and copy only; positions and inv_freq may be NULL) to head_dim; up to
 * PA_ROPE_MAX_HEADS heads.  Other sizes return PA_ERR_UNSUPPORTED.
 */
#ifndef PA_ROPE_H_
#define PA_ROPE_H_

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_ROPE_MAX_HEADS 4096
#define PA_ROPE_HALF 0        /* pairs (i, i + rot_dim/2) */
#define PA_ROPE_INTERLEAVED 1 /* pairs (2i, 2i + 1) */

/*
 * pa_rope -- rotate q rows and k rows.
 *
 *   q, k       bf16 [num_tokens][num_q_heads or num_kv_heads][head_dim], token
 *              strides q_stride and k_stride, heads packed.  k may be NULL with
 *              num_kv_heads 0.
 *   q_out, k_out  the same shapes with their own token strides; may be the
 *              inputs themselves (same pointer and stride), but must not
 *              otherwise overlap them.
 *   positions  int64 [num_tokens], device; any value.
 *   inv_freq   double [rot_dim / 2], device, in radians per position.
 */
PA_API int pa_rope(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                   int32_t num_q_heads, const void* k, int64_t k_stride, void* k_out,
                   int64_t k_out_stride, int32_t num_kv_heads, int32_t head_dim,
                   const int64_t* positions, const double* inv_freq, int32_t rot_dim,
                   int32_t layout, float factor, int32_t num_tokens, void* stream);

/*
 * pa_rope_and_cache -- norm and rotate q, norm and rotate K and write it with V
 * into the pools (pa_reshape_and_cache of the prepared K), in one launch.
 *
 *   key, value bf16 [num_tokens][num_kv_heads][head_dim], token strides
 *              k_stride and v_stride.
 *   q_weight, k_weight  bf16 [head_dim], or NULL: that side is not normed.
 *   slot_mapping  as in pa_reshape_and_cache: a negative slot is padding, its K
 *              and V are not written (its q row is still prepared); a slot >=
 *              num_blocks * block_size is skipped and sets PA_DEV_ERR_SLOT.
 *   q, q_out, positions, inv_freq  as in pa_rope.
 * K and V must not overlap the pools or q_out.
 */
PA_API int pa_rope_and_cache(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                             int32_t num_q_heads, const void* key, int64_t k_stride,
                             const void* value, int64_t v_stride, const void* q_weight,
                             const void* k_weight, float eps, const int64_t* positions,
                             const double* inv_freq, int32_t rot_dim, int32_t layout,
                             float factor, void* k_pool, void* v_pool, pa_pool_desc pool,
                             const int64_t* slot_mapping, int32_t num_tokens, void* stream);

/*
 * pa_rope_frequencies -- inv_freq (HOST, double [rot_dim / 2]) of a base, scaled
 * for contexts `scale` times longer than original_max_position, and the factor
 * that goes with it (HOST, may be NULL).  With f_i = base^(-2i / rot_dim):
 *   PA_ROPE_SCALE_NONE    f_i; factor 1.
 *   PA_ROPE_SCALE_LINEAR  f_i / scale (positions interpolated); factor 1.
 *   PA_ROPE_SCALE_BASE    f_i of the base * scale^(rot_dim / (rot_dim - 2)): the
 *                         slowest pair is stretched by scale, the fastest kept;
 *                         factor 1.
 *   PA_ROPE_SCALE_RAMP    by the turns r_i = original_max_position * f_i / 2 pi a
 *                         pair makes over the original context: f_i where r_i >=
 *                         high_turns, f_i / scale where r_i <= low_turns, a linear
 *                         blend of the two between; factor 0.1 ln(scale) + 1 (1
 *                         for scale <= 1).  (A checkpoint whose blend is linear in
 *                         the pair's index i instead needs an array of its own.)
 * low_turns, high_turns and original_max_position are read by
 * PA_ROPE_SCALE_RAMP only.  PA_ERR_ARG on an odd or non-positive rot_dim, a
 * base <= 1, a scale <= 0, or high_turns <= low_turns; PA_ROPE_SCALE_BASE needs
 * rot_dim > 2.
 */
#define PA_ROPE_SCALE_NONE 0
#define PA_ROPE_SCALE_LINEAR 1
#define PA_ROPE_SCALE_BASE 2
#define PA_ROPE_SCALE_RAMP 3

PA_API int pa_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double scale,
                               double original_max_position, double low_turns, double high_turns,
                               double* inv_freq_host, double* factor_host);

#ifdef __cplusplus
}
#endif

#endif /* PA_ROPE_H_ */
