/*
 * nvfp4_answer -- the operators of a training step on a model's own answers, on AMD Instinct
 * MI355X (gfx950): products of a few rows with packed NVFP4 weights, log probabilities of given
 * tokens with entropy and top alternatives and their gradient, the global gradient norm and
 * clipping.
 *
 * A student that was distilled to W4A16 (the Nemotron 3.5 Lightning NVFP4 news page, "two-stage
 * QAD") answers a token at a time from the packed weights of nvfp4_amax.h, its tokens are scored
 * under itself and its teacher, and the loss on these scores goes back through the logits into
 * the AdamW step of nvfp4_train.h, whose grad_scale is the clipping coefficient.
 *
 * Types, rounding, ownership, ordering, errors: as in nvfp4_train.h.  Pointers are device
 * pointers owned by the caller unless marked as host memory; the library allocates nothing and
 * keeps no state; all work is enqueued on `stream`, the calls return at once and may be captured
 * in a HIP graph.  Tensors need the alignment of their element type only, unless stated
 * otherwise.  Argument errors come back before anything is enqueued and leave the outputs
 * untouched.  Results depend on the arguments alone: the same call gives the same bits on the
 * same device.  Status texts: nvfp4_train_status_str.
 */
#ifndef NVFP4_ANSWER_H
#define NVFP4_ANSWER_H

#include "nvfp4_train.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_ANSWER_ABI_VERSION 1

/* Types of indices (experts, tokens). */
typedef enum { NVFP4_I32 = 0, NVFP4_I64 = 1 } nvfp4_index;

/* ABI version (NVFP4_ANSWER_ABI_VERSION). */
int nvfp4_answer_abi_version(void);

/* Products of a few rows with packed NVFP4 weights:
 *   y[t][i][j] = round(alpha[e] * sum_c x[t][c] * val(codes[e][j][c]) * dec(scales[e][j][c / 16])),
 *   e = expert[t][i]
 * (expert NULL: E = picks = 1 and e = 0).  The product of a code and its scale is exact; the sum is
 * binary32, multiplied by alpha and rounded once (the weights are not rounded to bf16 as
 * nvfp4_dequantize rounds them).  A non-finite x, scale or alpha reaches the outputs as IEEE
 * arithmetic has it; the sum is taken before alpha, so that |x| beyond 1e30 may overflow in it, and what a binary32 x has
 * below 2^-133 is cut off.
 * A row whose expert lies outside 0 .. E - 1 is zero.
 * x [tokens][cols] of `xtype` with row stride x_stride (elements, >= cols); codes [E][rows][cols/2]
 * (8-byte aligned), scales [E][rows][cols/16] and alpha [E] as nvfp4_quantize_batched writes them;
 * expert [tokens][picks] of `itype`; y [tokens][picks][rows] of `ytype`, contiguous.  y overlaps
 * nothing.  tokens >= 0, tokens * picks <= NVFP4_MATVEC_MAX_ROWS, 1 <= rows <= 2^26, cols % 16 == 0,
 * cols <= 2^27, 1 <= E <= 65535.
 * One launch. */
#define NVFP4_MATVEC_MAX_ROWS 1024
nvfp4_status nvfp4_packed_matvec(const void* x, int64_t x_stride, const uint8_t* codes,
                                 const uint8_t* scales, const float* alpha, const void* expert,
                                 int64_t tokens, int64_t picks, int64_t E, int64_t rows,
                                 int64_t cols, nvfp4_type xtype, nvfp4_type ytype,
                                 nvfp4_index itype, void* y, hipStream_t stream);

/* Log probabilities of given tokens under p = softmax(logits / T), per row:
 *   m = max_j x_j,  z = ln sum_j exp((x_j - m) / T)          (stats[row] = {m, z})
 *   logp[i] = (x[tokens[i]] - m) / T - z                     i = 0 .. given - 1
 *   entropy = z - sum_j p_j (x_j - m) / T                    (every term >= 0)
 *   top_index[0 .. top - 1]: the largest logits in falling order, the lowest index first among
 *   equals (-0 equals 0); top_logp: their log probabilities.
 *   - A token of -1 (any negative one) is none: its logp is 0.  A row with given > 0 that has no token
 *     is not read: logp, entropy, stats and top_logp are 0, top_index -1.  A token beyond the
 *     vocabulary has a logp of NaN.
 *   - Entries of -inf have probability 0 and log probability -inf.
 *   - A row with a NaN, a +inf, or no entry above -inf has no distribution: its results are NaN, its
 *     top_index -1.
 * logits [rows][vocab] of `type` with row stride `stride` (elements, >= vocab); tokens [rows][given]
 * of `itype` (NULL where given is 0); logp float [rows][given]; entropy float [rows] or NULL;
 * top_logp float and top_index int64 [rows][top] (NULL where top is 0); stats float [rows][2].
 * 0 <= given, top <= NVFP4_LOGPROBS_MAX, top <= vocab, 1 <= vocab <= 2^28, 0 <= rows <= 2^30; T > 0 and
 * log2(e) / T < 3e38 (T from 4.9e-39 on), T finite.  workspace: nvfp4_token_logprobs_workspace(...) bytes, 16-byte aligned, any content (may
 * be NULL where that is 0).  One launch; two for few long rows, which several workgroups share. */
#define NVFP4_LOGPROBS_MAX 64
int64_t nvfp4_token_logprobs_workspace(int64_t rows, int64_t vocab, int64_t top);
nvfp4_status nvfp4_token_logprobs(const void* logits, int64_t stride, const void* tokens,
                                  int64_t rows, int64_t vocab, int64_t given, int64_t top,
                                  nvfp4_type type, nvfp4_index itype, float temperature,
                                  float* logp, float* entropy, float* top_logp,
                                  int64_t* top_index, float* stats, void* workspace,
                                  hipStream_t stream);

/* Their gradient: with g_i = dlogp[i] (0 for a token of -1) and h = dentropy (0 where NULL), per row
 *   grad_j = round((sum_i g_i [tokens[i] == j] - p_j (sum_i g_i + h (ln p_j + entropy))) / T),
 *   ln p_j = (x_j - m) / T - z
 * p_j below 2^-126 counts as 0.  A finite gradient is found for every T where the sums of |g_i| and |h| entropy, and
 * 111 |h|, are below 3e38.
 * A row that was not read has a gradient of 0.  A row without a distribution, or with a token beyond
 * the vocabulary, has one of NaN.  Equal tokens of a row add up.
 * logits, tokens, given >= 1, vocab, T as in the forward call, which wrote stats and entropy
 * (entropy is NULL where dentropy is); dlogp float [rows][given], dentropy float [rows]; grad
 * [rows][vocab] of `type` with row stride grad_stride.  grad may equal logits (same stride); any other
 * overlap with it is rejected.  One launch. */
nvfp4_status nvfp4_token_logprobs_backward(const void* logits, int64_t stride, const void* tokens,
                                           const float* stats, const float* entropy,
                                           const float* dlogp, const float* dentropy,
                                           int64_t rows, int64_t vocab, int64_t given,
                                           nvfp4_type type, nvfp4_index itype, float temperature,
                                           void* grad, int64_t grad_stride, hipStream_t stream);

/* The 2-norm over all elements of many tensors, and the coefficient that clips it:
 *   norm[0] = sqrt(sum_i sum_j grad_i[j]^2),   scale[0] = min(1, max_norm / (norm + eps))
 * (1 where all three are 0).
 * Squares and sums are binary64 (no binary32 input overflows or vanishes), in an order that the
 * sizes fix; both results are rounded once.  An infinite sum of gradients gives norm inf and scale
 * 0, a NaN gives NaN in both.  scale (may be NULL) is what nvfp4_adamw_step takes as grad_scale.
 * `tensors`: host array of `count` entries, read before the call returns; empty ones are skipped and
 * may have NULL pointers.  All have `type`.  numel <= 2^36.  max_norm >= 0, eps >= 0, finite.
 * workspace: NVFP4_GRAD_NORM_WORKSPACE(count) bytes, 16-byte aligned, any content.  One launch per
 * 200 tensors, and one. */
#define NVFP4_GRAD_NORM_WORKSPACE(count) (16384 * ((int64_t)(count) / 200 + 1))
typedef struct {
  void* grad;          /* [numel] float or bf16 */
  int64_t numel;
} nvfp4_grad_tensor;
nvfp4_status nvfp4_grad_norm(const nvfp4_grad_tensor* tensors, int64_t count, nvfp4_type type,
                             double max_norm, double eps, float* norm, float* scale,
                             void* workspace, hipStream_t stream);

/* out_i = round(grad_i * scale[0]) over many tensors.  `out`: host array of entries like `tensors`
 * with the same sizes, or NULL: in place, where a scale of 1 leaves the tensors alone.  An entry of
 * `out` may be that of `tensors`; any other overlap of a written tensor with a written or read one (the
 * same tensor twice) is rejected.  One launch per 140 tensors (200 in place). */
nvfp4_status nvfp4_clip_grads(const nvfp4_grad_tensor* tensors, const nvfp4_grad_tensor* out,
                              int64_t count, nvfp4_type type, const float* scale,
                              hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_ANSWER_H */
