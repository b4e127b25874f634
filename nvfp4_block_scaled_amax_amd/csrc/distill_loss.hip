// The distillation loss KL(softmax(teacher / T) || softmax(student / T)) per row and its
// gradient for gfx950 (include/nvfp4_train.h defines the operation).
//
// Each row is read twice: once for both maxima and both sums of exponentials together (running
// maximum and sum, so one pass serves), and once, from the caches where the row fits, for the
// loss and the gradient.  Exponentials are powers of two of (x - max) * log2(e) / T; the
// subtraction comes first, so that logits of any size (the lowest finite value, too) keep their
// differences.  The loss is summed in the second pass as q - p + p (log p - log q), whose sum
// over a row is that of the plain definition but whose terms are all >= 0.
//
// With rows for every compute unit a workgroup takes a row.  With fewer, a row is split over
// several workgroups in two launches: partial statistics, then gradient and partial losses,
// which the last workgroup of a row adds in order.
#include "train_common.h"

namespace train {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e38f;

struct Distill {
  const void* student;
  const void* teacher;
  const float* weight;
  float* loss;
  void* grad;
  float* stats;           // split rows: [rows][splits][4]
  float* part;            // split rows: [rows][splits] losses
  uint32_t* arrived;      // split rows: [rows]
  int64_t student_stride, teacher_stride, grad_stride, rows, vocab;
  int64_t split_size;     // elements of a split, a multiple of 8
  int splits;
  float c, inv_t;         // log2(e) / T and 1 / T
};

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_(float x) { return __builtin_amdgcn_logf(x); }

// max x, and the sum of 2^((x - max) c).  An empty one has max = the lowest finite value and
// sum 0; an entry of -inf adds 0 to any.
struct Stat {
  float m, z;
  __device__ __forceinline__ void join(float m2, float z2, float c) {
    const float top = fmaxf(m, m2);
    z = z * exp2_((m - top) * c) + z2 * exp2_((m2 - top) * c);
    m = top;
  }
  template <typename T>
  __device__ __forceinline__ void add(const Vec8<T>& v, float c) {
    float top = fmaxf(m, v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, v[i]);
    z *= exp2_((m - top) * c);
    m = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) z += exp2_((v[i] - top) * c);
  }
  __device__ __forceinline__ void add(float v, float c) { join(v, 1.0f, c); }
};

// Statistics of elements [lo, hi) of a row, over the workgroup; every thread gets them.
template <typename S, typename T>
__device__ __forceinline__ void row_stats(const S* s, const T* t, int64_t lo, int64_t hi, float c,
                                          Stat& qs, Stat& ps, float (*slots)[4]) {
  qs = ps = Stat{kLowest, 0.0f};
  const int64_t whole = lo + (hi - lo) / 8 * 8;
  for (int64_t at = lo + threadIdx.x * 8; at < whole; at += kThreads * 8) {
    const Vec8<S> a = load_vec(s + at);
    const Vec8<T> b = load_vec(t + at);
    qs.add(a, c);
    ps.add(b, c);
  }
  if (whole + threadIdx.x < hi) {     // the last up to 7
    const float a = to_f32(s[whole + threadIdx.x]), b = to_f32(t[whole + threadIdx.x]);
    if (a != -INFINITY) qs.add(a, c);
    if (b != -INFINITY) ps.add(b, c);
  }
  // over the wavefront, then over the workgroup
  const float mq = reduce64(qs.m, Max()), mp = reduce64(ps.m, Max());
  const float zq = reduce64(qs.z * exp2_((qs.m - mq) * c), Sum());
  const float zp = reduce64(ps.z * exp2_((ps.m - mp) * c), Sum());
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    slots[wave][0] = mq;
    slots[wave][1] = zq;
    slots[wave][2] = mp;
    slots[wave][3] = zp;
  }
  __syncthreads();
  qs = Stat{slots[0][0], slots[0][1]};
  ps = Stat{slots[0][2], slots[0][3]};
  for (int i = 1; i < kWaves; ++i) {
    qs.join(slots[i][0], slots[i][1], c);
    ps.join(slots[i][2], slots[i][3], c);
  }
}

// The second pass over elements [lo, hi): writes the gradient, returns the workgroup's part of
// the loss (without the row's weight) to every thread.
template <typename S, typename T>
__device__ __forceinline__ float row_grad(const S* s, const T* t, S* grad, int64_t lo, int64_t hi,
                                          float c, Stat qs, Stat ps, float scale, float* slots) {
  const float lq = log2_(qs.z), lp = log2_(ps.z);
  float flat = 0.0f, bent = 0.0f;    // sums of q - p and of p (log2 p - log2 q)
  auto one = [&](float a, float b) {
    const float y = (a - qs.m) * c - lq, x = (b - ps.m) * c - lp;
    const float q = exp2_(y), p = exp2_(x);
    flat += q - p;
    bent += p == 0.0f ? 0.0f : p * (x - y);
    return (q - p) * scale;
  };
  const int64_t whole = lo + (hi - lo) / 8 * 8;
  for (int64_t at = lo + threadIdx.x * 8; at < whole; at += kThreads * 8) {
    const Vec8<S> a = load_vec(s + at);
    const Vec8<T> b = load_vec(t + at);
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = one(a[i], b[i]);
    if (grad) store_vec(grad + at, make_vec(g, S()));
  }
  const int64_t at = whole + threadIdx.x;
  if (at < hi) {
    const float g = one(to_f32(s[at]), to_f32(t[at]));
    if (grad) grad[at] = from_f32<S>(g);
  }
  return reduce_group<kWaves>(flat + kLn2 * bent, Sum(), slots);
}

template <typename S>
__device__ __forceinline__ void zero_grad(S* grad, int64_t lo, int64_t hi) {
  const int64_t whole = lo + (hi - lo) / 8 * 8;
  const Vec8<S> z = zero_vec<S>();
  for (int64_t at = lo + threadIdx.x * 8; at < whole; at += kThreads * 8) store_vec(grad + at, z);
  if (whole + threadIdx.x < hi) grad[whole + threadIdx.x] = from_f32<S>(0.0f);
}

template <typename S, typename T>
__global__ __launch_bounds__(kThreads) void row_kernel(const Distill a) {
  __shared__ float slots[kWaves][4], sums[kWaves];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float w = a.weight ? a.weight[row] : 1.0f;
    S* grad = a.grad ? (S*)a.grad + row * a.grad_stride : nullptr;
    if (w == 0.0f) {
      if (grad) zero_grad(grad, 0, a.vocab);
      if (threadIdx.x == 0) a.loss[row] = 0.0f;
      continue;
    }
    const S* s = (const S*)a.student + row * a.student_stride;
    const T* t = (const T*)a.teacher + row * a.teacher_stride;
    Stat qs, ps;
    row_stats(s, t, 0, a.vocab, a.c, qs, ps, slots);
    const float loss = row_grad(s, t, grad, 0, a.vocab, a.c, qs, ps, w * a.inv_t, sums);
    if (threadIdx.x == 0) a.loss[row] = w * loss;
    __syncthreads();
  }
}

template <typename S, typename T>
__global__ __launch_bounds__(kThreads) void split_stats_kernel(const Distill a) {
  __shared__ float slots[kWaves][4];
  const int64_t row = blockIdx.y;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.arrived[row] = 0u;
  if (a.weight && a.weight[row] == 0.0f) return;
  const int64_t lo = min(blockIdx.x * a.split_size, a.vocab), hi = min(lo + a.split_size, a.vocab);
  Stat qs, ps;
  row_stats((const S*)a.student + row * a.student_stride,
            (const T*)a.teacher + row * a.teacher_stride, lo, hi, a.c, qs, ps, slots);
  if (threadIdx.x == 0) {
    float* out = a.stats + (row * a.splits + blockIdx.x) * 4;
    out[0] = qs.m;
    out[1] = qs.z;
    out[2] = ps.m;
    out[3] = ps.z;
  }
}

template <typename S, typename T>
__global__ __launch_bounds__(kThreads) void split_grad_kernel(const Distill a) {
  __shared__ float sums[kWaves];
  const int64_t row = blockIdx.y;
  const int64_t lo = min(blockIdx.x * a.split_size, a.vocab), hi = min(lo + a.split_size, a.vocab);
  const float w = a.weight ? a.weight[row] : 1.0f;
  S* grad = a.grad ? (S*)a.grad + row * a.grad_stride : nullptr;
  if (w == 0.0f) {
    if (grad) zero_grad(grad, lo, hi);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.loss[row] = 0.0f;
    return;
  }
  const float* in = a.stats + row * a.splits * 4;
  Stat qs{in[0], in[1]}, ps{in[2], in[3]};
  for (int i = 1; i < a.splits; ++i) {
    qs.join(in[4 * i], in[4 * i + 1], a.c);
    ps.join(in[4 * i + 2], in[4 * i + 3], a.c);
  }
  const float loss = row_grad((const S*)a.student + row * a.student_stride,
                              (const T*)a.teacher + row * a.teacher_stride, grad, lo, hi, a.c, qs,
                              ps, w * a.inv_t, sums);
  if (threadIdx.x == 0) {
    float* part = a.part + row * a.splits;
    __hip_atomic_store(part + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t before = __hip_atomic_fetch_add(a.arrived + row, 1u, __ATOMIC_ACQ_REL,
                                                   __HIP_MEMORY_SCOPE_AGENT);
    if (before + 1 == (uint32_t)a.splits) {      // every part is there
      float sum = 0.0f;
      for (int i = 0; i < a.splits; ++i)
        sum += __hip_atomic_load(part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      a.loss[row] = w * sum;
    }
  }
}

// Workgroups per row: one where there are rows for the 256 compute units, else enough for
// them, each with two vectors per thread at the least.
int splits_of(int64_t rows, int64_t vocab) {
  if (rows <= 0 || rows >= 192) return 1;
  const int64_t want = (256 + rows - 1) / rows, most = (vocab + 16383) / 16384;
  return (int)(want < most ? want : most);
}

template <typename S, typename T>
void launch(const Distill& a, hipStream_t stream) {
  if (a.splits == 1) {
    row_kernel<S, T><<<(unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20)), kThreads, 0, stream>>>(a);
  } else {
    const dim3 grid((unsigned)a.splits, (unsigned)a.rows);
    split_stats_kernel<S, T><<<grid, kThreads, 0, stream>>>(a);
    split_grad_kernel<S, T><<<grid, kThreads, 0, stream>>>(a);
  }
}

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT int64_t nvfp4_distill_loss_workspace(int64_t rows, int64_t vocab) {
  const int64_t splits = vocab < 1 ? 1 : splits_of(rows, vocab);
  return splits == 1 ? 0 : rows * (splits * 5 + 1) * 4;
}

NVFP4_EXPORT nvfp4_status nvfp4_distill_loss(const void* student, int64_t student_stride,
                                             const void* teacher, int64_t teacher_stride,
                                             const float* weight, int64_t rows, int64_t vocab,
                                             nvfp4_type stype, nvfp4_type ttype,
                                             float temperature, float* loss, void* grad,
                                             int64_t grad_stride, void* workspace,
                                             hipStream_t stream) {
  if (!known(stype) || !known(ttype)) return NVFP4_ERR_ENUM;
  if (!shape_ok(rows, vocab, student_stride) || !shape_ok(rows, vocab, teacher_stride) ||
      (grad && !shape_ok(rows, vocab, grad_stride)))
    return NVFP4_ERR_SHAPE;
  const float inv_t = 1.0f / temperature, c = (float)(1.4426950408889634 / (double)temperature);
  if (!(temperature > 0.0f) || !(inv_t > 0.0f) || !(c < 3.0e38f)) return NVFP4_ERR_VALUE;
  if (rows == 0) return NVFP4_OK;
  const int64_t need = nvfp4_distill_loss_workspace(rows, vocab);
  if (!student || !teacher || !loss || (need && !workspace)) return NVFP4_ERR_NULL;
  const int64_t es = size_of(stype), et = size_of(ttype);
  if (!aligned(student, es) || !aligned(grad, es) || !aligned(teacher, et) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const Range in[] = {range(student, extent(rows, vocab, student_stride, es)),
                      range(teacher, extent(rows, vocab, teacher_stride, et)),
                      range(weight, rows * 4)};
  const Range out[] = {range(grad, extent(rows, vocab, grad_stride, es)), range(loss, rows * 4),
                       range(need ? workspace : nullptr, need)};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i)
      if (!(o == 0 && i == 0 && grad == student && grad_stride == student_stride) &&
          overlap(out[o], in[i]))
        return NVFP4_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return NVFP4_ERR_ALIAS;
  }
  const int splits = splits_of(rows, vocab);
  float* ws = (float*)workspace;
  Distill a = {student, teacher, weight, loss, grad, ws, ws + rows * splits * 4,
               (uint32_t*)(ws + rows * splits * 5), student_stride, teacher_stride, grad_stride,
               rows, vocab, ((vocab + splits - 1) / splits + 7) / 8 * 8, splits, c, inv_t};
  (void)hipGetLastError();
  if (stype == NVFP4_T_BF16 && ttype == NVFP4_T_BF16) launch<bf16, bf16>(a, stream);
  else if (stype == NVFP4_T_BF16) launch<bf16, float>(a, stream);
  else if (ttype == NVFP4_T_BF16) launch<float, bf16>(a, stream);
  else launch<float, float>(a, stream);
  return launched();
}
