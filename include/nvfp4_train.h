/*
 * nvfp4_train -- the operators of a quantization-aware distillation (QAD) step around the
 * simulated quantization of nvfp4_amax.h, on AMD Instinct MI355X (gfx950): layer norm forward
 * and backward, the distillation loss with its gradient, and an AdamW step over many tensors.
 *
 * The QAD student forward runs through nvfp4_fakequant and is trained on
 * L = D_KL(p_teacher || p_student) of the logits ("Quantization-Aware Distillation for NVFP4
 * Inference Accuracy Recovery", gist.science explainer, method section; Nemotron 3.5 Lightning
 * NVFP4 news page, "two-stage QAD").  Layer norm produces the activations that it quantizes and
 * AdamW writes the weights that it quantizes; both can also deliver the absolute maximum of
 * what they write, which nvfp4_fakequant_from_amax / nvfp4_quantize_from_amax take in place of
 * the amax pass over the tensor, with the same result bit for bit.
 *
 * Types are NVFP4_T_BF16 (bf16 bit patterns) or NVFP4_T_F32.  All sums, statistics and
 * exponentials are binary32 or wider; a bf16 output is rounded once, to nearest even, unless
 * stated otherwise.
 *
 * Ownership, ordering, errors: as in nvfp4_amax.h.  Pointers are device pointers owned by the
 * caller unless marked as host memory; the library allocates nothing and keeps no state; all
 * work is enqueued on `stream` and the calls return at once and may be captured in a HIP graph
 * (which replays the numbers given by the host, such as AdamW's step, as they were).
 * Tensors need the alignment of their element type only.  Argument errors come back before
 * anything is enqueued and leave the outputs untouched.  Results depend on the arguments alone
 * (no atomics whose order matters): the same call gives the same bits on the same device.
 */
#ifndef NVFP4_TRAIN_H
#define NVFP4_TRAIN_H

#include "nvfp4_amax.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_TRAIN_ABI_VERSION 1

typedef enum { NVFP4_T_BF16 = 0, NVFP4_T_F32 = 1 } nvfp4_type;

/* These entry points return NVFP4_OK, NVFP4_ERR_NULL, NVFP4_ERR_SHAPE, NVFP4_ERR_ENUM (a type
 * that is not listed for the argument), NVFP4_ERR_ALIGN, NVFP4_ERR_ALIAS, NVFP4_ERR_HIP, or
 * NVFP4_ERR_VALUE: a number (eps, temperature, beta, step, ...) outside its range. */
#define NVFP4_ERR_VALUE ((nvfp4_status)9)

/* ABI version (NVFP4_TRAIN_ABI_VERSION) and a static description of a status of these calls. */
int nvfp4_train_abi_version(void);
const char* nvfp4_train_status_str(nvfp4_status status);

/* Layer norm over the last dimension, with an optional residual add in front:
 *   h    = round(x + residual)              (h = x without residual)
 *   mean = sum_j h_j / cols                 (0 where center == 0: root-mean-square norm)
 *   rstd = 1 / sqrt(sum_j (h_j - mean)^2 / cols + eps)
 *   y    = round((h - mean) * rstd * weight + bias)
 * (in binary32: where |h - mean| passes 2^64 the sum of squares is infinite and rstd 0).
 * x, residual [rows][cols] of `type` with row strides in elements (>= cols); h and y [rows][cols]
 * of `type`, contiguous; weight and bias (may be NULL) [cols] of `wtype`; mean (NULL where
 * center == 0) and rstd float [rows].  h is required with residual and must be NULL without.
 * h may equal x or residual where that is contiguous, and y may equal x, where no h is written
 * in its place; any other overlap with an output is rejected.
 * out_amax (may be NULL): float [1], max |y| over all rows as nvfp4_amax defines it (0 for no
 * rows).  rows >= 0, 1 <= cols <= 2^30, eps >= 0.  One launch, two with out_amax. */
nvfp4_status nvfp4_layernorm_forward(const void* x, int64_t x_stride, const void* residual,
                                     int64_t residual_stride, const void* weight,
                                     const void* bias, int64_t rows, int64_t cols,
                                     nvfp4_type type, nvfp4_type wtype, int center, float eps,
                                     void* y, void* h, float* mean, float* rstd,
                                     float* out_amax, hipStream_t stream);

/* Its gradient.  With xh = (h - mean) * rstd and g = dy * weight, per row:
 *   dx = round(rstd * (g - mean_j(g) - xh * mean_j(g * xh)) + dres)
 * (without the mean_j(g) term where mean is NULL: root-mean-square norm), and over the rows
 *   dweight = sum dy * xh,   dbias = sum dy      (dbias may be NULL)
 * summed in binary32 in an order that the shape and the device fix, rounded once to `wtype`.
 * dy, h, dres (may be NULL: the gradient that reaches h past the norm) [rows][cols] of `type`,
 * dx [rows][cols]; all contiguous.  dx may equal dy or dres.  dx is the gradient of x and of the
 * residual alike.  workspace: nvfp4_layernorm_backward_workspace(...) bytes, 16-byte aligned, any
 * content.  rows == 0 gives dweight = dbias = 0.  Two launches; three where a row is more than a
 * workgroup holds (16384 columns; 8192 binary32 ones that are no multiple of 1024). */
int64_t nvfp4_layernorm_backward_workspace(int64_t rows, int64_t cols);
nvfp4_status nvfp4_layernorm_backward(const void* dy, const void* h, const void* weight,
                                      const float* mean, const float* rstd, const void* dres,
                                      int64_t rows, int64_t cols, nvfp4_type type,
                                      nvfp4_type wtype, void* dx, void* dweight, void* dbias,
                                      void* workspace, hipStream_t stream);

/* Distillation loss and its gradient.  Per row, with p = softmax(teacher / T), q =
 * softmax(student / T) and a weight w (1 where `weight` is NULL):
 *   loss = w * sum_j p_j (log p_j - log q_j),   grad_j = round((w / T) (q_j - p_j))
 * evaluated as sum_j (q_j - p_j + p_j (log p_j - log q_j)), whose terms are all >= 0: a student
 * near its teacher keeps its relative precision.
 *   - A row of weight 0 is not read: loss 0, gradient 0, whatever its logits hold.
 *   - Entries of -inf have probability 0.  p_j = 0 contributes nothing, also where q_j = 0;
 *     p_j > 0 where the student is -inf makes the loss +inf.  Where the student is a finite value far
 *     below (the type's lowest) log q_j is that value's, though q_j comes out as 0.
 *   - A row with a NaN, a +inf, or no entry above -inf (in teacher or student) has no
 *     distribution: its loss and its whole gradient are NaN.
 * student, teacher [rows][vocab] of `stype`, `ttype` with row strides in elements (>= vocab);
 * weight float [rows] or NULL; loss float [rows]; grad [rows][vocab] of `stype` with row stride
 * grad_stride, or NULL (loss only).  grad may equal student (same stride).  temperature > 0, and 1 / T
 * finite.
 * workspace: nvfp4_distill_loss_workspace(...) bytes, 16-byte aligned, any content (may be NULL
 * where that is 0).  rows >= 0, 1 <= vocab <= 2^28.  One launch; two for few long rows, which several
 * workgroups share. */
int64_t nvfp4_distill_loss_workspace(int64_t rows, int64_t vocab);
nvfp4_status nvfp4_distill_loss(const void* student, int64_t student_stride, const void* teacher,
                                int64_t teacher_stride, const float* weight, int64_t rows,
                                int64_t vocab, nvfp4_type stype, nvfp4_type ttype,
                                float temperature, float* loss, void* grad, int64_t grad_stride,
                                void* workspace, hipStream_t stream);

/* One AdamW step over many tensors, in place.  Per element, in binary32 with one rounding per
 * operation as written (the quotient within 2 ulp where its divisor is within 2^-126 .. 2^126):
 *   g = grad * grad_scale[0]                  (grad_scale: device float, NULL = no factor)
 *   m = m * beta1 + g * (1 - beta1)
 *   v = v * beta2 + (g * g) * (1 - beta2)
 *   p = p * (1 - lr * weight_decay)
 *       - (m / (sqrt(v) * (1 / sqrt(1 - beta2^step)) + eps)) * (lr / (1 - beta1^step))
 * Parameters: float; or bf16 with a float master copy (master non-NULL: the update runs on it and
 * param is it rounded to nearest even; param is not read); or bf16 alone (master NULL), rounded
 * stochastically, because most updates are smaller than half a bf16 step.
 * States: float; or 8 bits, per block of NVFP4_ADAMW_BLOCK consecutive elements of the tensor
 * one float scale = max / 448 and E4M3 codes of m / scale and sqrt(v) / scale (v is read back as the binary32 square
 * of code * scale, 0 where that is below 2^-75).  Codes are rounded
 * stochastically (round-to-nearest would hold v still: beta2 near 1 moves it by less than half
 * a step); sqrt(v) > 0 never becomes 0, and an m whose block stays below 2^-100 does.  The update of p uses m and v before that rounding.  A block
 * with a non-finite value reads back as non-finite.
 * Stochastic rounding adds random bits below the kept ones and truncates.  The bits are
 * hash32(element + key) with key = hash32(hash32(hash32(seed) ^ step) ^ tensor index), see
 * csrc/adamw.hip: no state, the same on every run, and different for each step.  One word serves an
 * element's m (bits 0..19), sqrt(v) (bits 12..31) and bf16 parameter (the upper half of the word times
 * 0x9E3779B1): each rounding is unbiased by itself, the three are not independent of each other.
 * `tensors`: host array of `count` entries, read before the call returns.  Empty tensors
 * (numel 0) are skipped and may have NULL pointers.  All tensors of a call have one parameter type, gradient
 * type, state kind, and either all or none a master copy.  Different tensors must not overlap
 * (not checked).  numel <= 2^36.
 * out_amax: device float [count] or NULL; max |param| as written, per tensor (0 if empty).
 * betas in [0, 1), eps >= 0, step >= 1.  One launch per 58 tensors, one more with out_amax. */
#define NVFP4_ADAMW_BLOCK 128
typedef enum { NVFP4_STATE_F32 = 0, NVFP4_STATE_E4M3 = 1 } nvfp4_state;
typedef struct {
  void* param;         /* [numel] float or bf16 */
  const void* grad;    /* [numel] float or bf16 */
  void* exp_avg;       /* m: [numel] float, or E4M3 bytes */
  void* exp_avg_sq;    /* v: [numel] float, or E4M3 bytes of sqrt(v) / scale */
  float* master;       /* [numel] or NULL */
  float* avg_scale;    /* [ceil(numel / NVFP4_ADAMW_BLOCK)] for 8-bit states, else NULL */
  float* sq_scale;     /* the same */
  int64_t numel;
} nvfp4_adamw_tensor;
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;        /* 1 for the first step; < 2^32 */
  uint32_t seed;
} nvfp4_adamw_args;
nvfp4_status nvfp4_adamw_step(const nvfp4_adamw_tensor* tensors, int64_t count, nvfp4_type ptype,
                              nvfp4_type gtype, nvfp4_state state, const nvfp4_adamw_args* args,
                              const float* grad_scale, float* out_amax, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_TRAIN_H */
