/*
 * hkv_train.h - C ABI of the training operators that stand between a table's
 * find and its assign (libhkv_train.so, gfx950).
 *
 * Rows found in a table score candidates: logits x[t][v], one row a decision.
 * The operators turn logits and feedback into gradients and bound them:
 *   - hkv_token_logprobs / _backward: log-probability of each row's label;
 *   - hkv_preference_loss: loss on pairs of sequences, of which one was
 *     preferred, from the ratios to a reference; value and gradient;
 *   - hkv_policy_loss: clipped policy-gradient loss with a divergence (KL)
 *     term; value and gradient;
 *   - hkv_clip_grad_norm: global norm of many gradient tensors, and clipping.
 *
 * Notation: tau = temperature, y = labels[t],
 *   lse_t  = log sum_v exp(x[t][v] / tau),   logp_t = x[t][y] / tau - lse_t.
 *
 * A row is left out when its label is negative (its logits are not read) or
 * when all its logits are -inf (it has no distribution): its logp is 0, it
 * adds nothing to a loss, and its gradient is zeros. Its lse is 0 for a
 * negative label and -inf for a row of -inf. A label >= vocab makes its row's
 * results NaN, and so does a NaN or +inf among its logits. A label whose own
 * logit is -inf beside finite ones has logp -inf. An lse or logp past
 * float32's range is written as an infinity (to the backward call an lse of
 * -inf is a row left out). A row whose coefficient g_t
 * is exactly 0 gets zeros for its gradient whatever its logits are.
 *
 * Conventions shared with hkv.h: status codes; asynchronous on `stream`;
 * arguments checked before anything is enqueued; array arguments in memory
 * that the GPU can access (the GPU of the logits, or of the first gradient);
 * no C++ exception crosses the boundary. Differences:
 *   - There is no handle. Calls keep nothing from one to the next and allocate
 *     nothing: where scratch is needed, it comes from the caller (`workspace`,
 *     16-byte aligned, at least hkv_train_workspace_bytes(...) bytes, any
 *     contents) and must stay the call's own until the stream has passed it.
 *     Every call can be captured into a HIP graph.
 *   - Logits and gradients are [rows][vocab] arrays of HKV_F32, HKV_BF16 or
 *     HKV_F16 whose rows are *_stride elements apart (stride >= vocab; any
 *     alignment of the element type). A gradient may overwrite its logits (same
 *     address, same stride) or lie beside them (other columns of the same wider
 *     rows: same stride, no common element); no other overlap of the memory
 *     from an array's first element to its last is allowed.
 *   - Results are deterministic: no sum depends on the order of execution. (It
 *     does depend on how a row is aligned, in its last bits.)
 * Limits: rows < 2^31, vocab < 2^29, pairs < 2^30, tensors < 2^20, strides up
 * to 2^40 elements, (rows - 1) * stride up to 2^60.
 */
#ifndef HKV_TRAIN_H_
#define HKV_TRAIN_H_

#include "hkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HKV_F32 0u
#define HKV_BF16 1u
#define HKV_F16 2u

/* Bytes of workspace that a call needs: rows of logits, pairs for
 * hkv_preference_loss, tensors for hkv_clip_grad_norm, 0 for what the call does
 * not have. (hkv_token_logprobs_backward needs none, hkv_token_logprobs only for
 * fewer than 64 rows of more than 256 KiB: its workspace may be NULL otherwise.) */
uint64_t hkv_train_workspace_bytes(uint64_t rows, uint64_t pairs, uint64_t tensors);

/*
 * hkv_token_logprobs - logp_t and lse_t.
 *   logits   [rows][vocab] dtype, input
 *   labels   [rows] int64, input
 *   logp_out [rows] float32, output
 *   lse_out  [rows] float32, output, nullable
 */
hkv_status hkv_token_logprobs(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                              uint64_t logits_stride, const int64_t* labels, float temperature, float* logp_out,
                              float* lse_out, void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/*
 * hkv_token_logprobs_backward - gradient of sum_t g_t logp_t:
 *   dx[t][v] = g_t / tau ([v = y] - exp(min(x[t][v] / tau - lse_t, 1))).
 * (The bound matters for a row of values so low that lse as a float does not
 * tell their exponents.)
 *   lse       [rows] float32, input: what hkv_token_logprobs gave
 *   grad_logp [rows] float32, input: g_t
 *   grad_out  [rows][vocab] dtype, output
 */
hkv_status hkv_token_logprobs_backward(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                       uint64_t logits_stride, const int64_t* labels, float temperature,
                                       const float* lse, const float* grad_logp, void* grad_out,
                                       uint64_t grad_stride, hipStream_t stream);

/*
 * hkv_preference_loss - sequences 2p (preferred) and 2p+1 (not preferred) are
 * rows [cu[s], cu[s+1]) each. With D_s = sum over a sequence's rows that are
 * not left out of logp_t - ref_logp_t,
 *   reward_s = beta D_s,   m_p = reward_2p - reward_2p+1,
 *   l_p = (1 - label_smoothing) log(1 + e^-m_p) + label_smoothing log(1 + e^m_p),
 *   loss = mean_p l_p (0 without pairs).
 * grad_out = grad_scale * d loss / d logits; rows in no sequence get zeros.
 * Offsets are used clamped to [0, rows], an end below its start as the start.
 *   cu_seqlens  [2*pairs+1] int64, input, not decreasing
 *   ref_logp    [rows] float32, input, nullable (all 0)
 *   loss_out    [1] float32, output
 *   losses_out  [pairs] float32, output
 *   rewards_out [2*pairs] float32, output
 *   logp_out    [rows] float32, output
 *   grad_out    [rows][vocab] dtype, output, nullable (no gradient is computed)
 */
hkv_status hkv_preference_loss(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                               uint64_t logits_stride, const int64_t* labels, float temperature, uint64_t pairs,
                               const int64_t* cu_seqlens, const float* ref_logp, float beta, float label_smoothing,
                               float grad_scale, float* loss_out, float* losses_out, float* rewards_out,
                               float* logp_out, void* grad_out, uint64_t grad_stride, void* workspace,
                               uint64_t workspace_bytes, hipStream_t stream);

/*
 * hkv_policy_loss - with r = exp(logp_t - old_logp_t), A = advantages[t],
 * d = ref_logp_t - logp_t:
 *   kl_t = exp(d) - d - 1 (0 without ref_logp)
 *   l_t  = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + kl_coef kl_t
 *   loss = sum_t weights[t] l_t.
 * grad_out = grad_scale * d loss / d logits, where the clamped side of the
 * minimum has no slope and at equality the other side is taken.
 * A label whose own logit is -inf beside finite ones (logp -inf) has r = 0; with
 * a finite ref_logp its d is +inf and its kl, inf - inf, NaN. Without kl_coef that
 * stays in kl_out; with one, l_t and the loss are NaN and the row's coefficient is
 * infinite: a program that masks labels leaves such rows out by a negative label.
 *   old_logp, advantages, weights [rows] float32, input
 *   ref_logp       [rows] float32, input, nullable (then kl_coef must be 0)
 *   loss_out       [1] float32, output
 *   token_loss_out [rows] float32, output: l_t
 *   kl_out         [rows] float32, output
 *   logp_out       [rows] float32, output
 *   grad_out       [rows][vocab] dtype, output, nullable (no gradient is computed)
 */
hkv_status hkv_policy_loss(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits, uint64_t logits_stride,
                           const int64_t* labels, float temperature, const float* old_logp, const float* advantages,
                           const float* weights, const float* ref_logp, float clip_low, float clip_high,
                           float kl_coef, float grad_scale, float* loss_out, float* token_loss_out, float* kl_out,
                           float* logp_out, void* grad_out, uint64_t grad_stride, void* workspace,
                           uint64_t workspace_bytes, hipStream_t stream);

/*
 * hkv_clip_grad_norm - n = sqrt of the sum of squares over all elements of all
 * tensors, held in 64 bits; then every tensor is multiplied by
 *   c = 1 where n <= max_norm, max_norm / n elsewhere
 * (a NaN norm makes c NaN, an infinite one makes it 0). Tensor i has numel[i]
 * contiguous elements of dtypes[i] at grads[i]; the product goes to outs[i], of
 * the same type, or in place when outs is NULL or outs[i] == grads[i]. Where
 * c is 1, what is in place is not written.
 *   grads, outs, numel, dtypes: arrays of `tensors` entries in HOST memory,
 *   read during the call; the tensors themselves are the GPU's. Tensors may
 *   not overlap each other where one of them is written.
 *   norm_out [1] float32, output: n (+inf past the type's range)
 * max_norm >= 0; +inf computes the norm and copies.
 */
hkv_status hkv_clip_grad_norm(uint64_t tensors, void* const* grads, void* const* outs, const uint64_t* numel,
                              const uint8_t* dtypes, float max_norm, float* norm_out, void* workspace,
                              uint64_t workspace_bytes, hipStream_t stream);

/* Description of the last failure of a call in this header on the calling thread. */
const char* hkv_train_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* HKV_TRAIN_H_ */
