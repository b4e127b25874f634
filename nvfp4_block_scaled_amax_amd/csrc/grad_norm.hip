// The 2-norm of many tensors, the coefficient that clips it, and the scaled tensors, for gfx950
// (include/nvfp4_answer.h defines the operations).
//
// Squares and sums are binary64, which multiplies and adds at binary32's rate here: nothing
// overflows, vanishes or needs a second pass.  Workgroups take chunks of the tensors in turn and leave
// one sum each, which a last workgroup adds in a fixed order.  The tensors' table travels as a kernel
// argument: nothing is copied ahead and a captured graph holds it.
//
// Bound by the tensors' bytes, read once by the norm, read and written once by the clipping, which goes through
// them from the end.  Measured on one MI355X: norm of 224 million bf16 elements in tensors of all sizes 77 + 4.7 us
// (5.8 TB/s), of 64 x 2048 x 5120 bf16 221 us (6.1 TB/s), clipping these into other tensors 480 us (5.6 TB/s).
#include <stdlib.h>

#include <algorithm>

#include "nvfp4_answer.h"
#include "train_common.h"

namespace train {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 200, kTableTo = 140;          // tensors of a launch: below 4 KB
constexpr int kGroups = 2048;                        // workgroups of a launch, at most
constexpr int kDeep = 4;                             // vectors of a thread in a chunk
constexpr int64_t kCached = int64_t(128) << 20;       // bytes that are likely to stay in the last-level cache
constexpr int64_t kMaxNumel = int64_t(1) << 36;
constexpr int64_t kMaxCount = int64_t(1) << 24;

template <typename T>
constexpr int64_t kChunk = (int64_t)kThreads * kDeep * (16 / sizeof(T));
static_assert(kTable * (kMaxNumel / kChunk<float> + 1) < (int64_t(1) << 32) - kGroups, "chunks of a launch");

struct Entry {
  const void* grad;
  int64_t numel;
};
struct EntryTo {
  const void* grad;
  int64_t numel;
  void* out;
};
template <typename E, int SIZE>
struct Batch {
  E t[SIZE];
  uint32_t first[SIZE + 1];                  // first chunk of each tensor, and the number of all
  int count;
  const float* scale;
  double* part;
};
typedef Batch<Entry, kTable> NormBatch;
typedef Batch<EntryTo, kTableTo> ToBatch;
static_assert(NVFP4_GRAD_NORM_WORKSPACE(kTable - 1) == kGroups * 8 && NVFP4_GRAD_NORM_WORKSPACE(kTable) == 2 * kGroups * 8,
              "a sum for each workgroup of each launch");
static_assert(sizeof(NormBatch) <= 4096 && sizeof(ToBatch) <= 4096, "kernel arguments");

// The tensor of a chunk, from one that is not after it (uniform).
template <typename B>
__device__ __forceinline__ int find(const B& a, uint32_t chunk) {
  int lo = 0, hi = a.count;                  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_kernel(const NormBatch a) {
  constexpr int N = 16 / sizeof(T);
  __shared__ double slots[kThreads / 64];
  double sum = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < a.first[a.count]; chunk += gridDim.x) {
    const int i = find(a, chunk);
    const T* g = (const T*)a.t[i].grad;
    const int64_t n = a.t[i].numel, at = (int64_t)(chunk - a.first[i]) * kChunk<T> + threadIdx.x * N;
    Vec<T, N> v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) v[k] = load_vec<N, kAny>(g, at + k * kThreads * N, n);
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const double x = (double)v[k][j];
        sum = __builtin_fma(x, x, sum);
      }
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = (slots[0] + slots[1]) + (slots[2] + slots[3]);
}

__global__ __launch_bounds__(1024) void norm_end_kernel(const double* part, int64_t count, double max_norm,
                                                        double eps, float* norm, float* scale) {
  __shared__ double slots[16];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += 1024) sum += part[i];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < 16; ++w) sum += slots[w];
    const double all = sqrt(sum);
    *norm = (float)all;
    // (a NaN goes on; 0 / 0 does not arise)
    if (scale) *scale = max_norm >= all + eps ? 1.0f : (float)(max_norm / (all + eps));
  }
}

// STREAM: past the caches, for what is more than they hold (64 x 2048 x 5120 bf16 into other tensors, with the norm:
// 708 us, 743 through them, where writing drives out what the norm's pass left).
template <typename T, typename B, bool TO, bool STREAM>
__global__ __launch_bounds__(kThreads) void scale_kernel(const B a) {
  constexpr int N = 16 / sizeof(T);
  const float s = *a.scale;
  if (!TO && s == 1.0f) return;
  // from the end: it is what the norm's pass left in the caches
  const uint32_t total = a.first[a.count];
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    const uint32_t chunk = total - 1 - c;
    const int i = find(a, chunk);
    const T* g = (const T*)a.t[i].grad;
    T* to;
    if constexpr (TO) to = (T*)a.t[i].out;
    else to = (T*)const_cast<void*>(a.t[i].grad);
    const int64_t n = a.t[i].numel, at = (int64_t)(chunk - a.first[i]) * kChunk<T> + threadIdx.x * N;
    Vec<T, N> v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) v[k] = load_vec<N, kAny>(g, at + k * kThreads * N, n);
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      float r[N];
#pragma unroll
      for (int j = 0; j < N; ++j) r[j] = v[k][j] * s;
      store_vec<kAny, STREAM>(to, at + k * kThreads * N, n, make_vec<T>(r));
    }
  }
}

template <typename B, bool TO>
void scale_batch(const B& b, unsigned groups, nvfp4_type type, bool stream_out, hipStream_t s) {
  if (type == NVFP4_T_BF16) {
    if (stream_out) scale_kernel<bf16, B, TO, true><<<groups, kThreads, 0, s>>>(b);
    else scale_kernel<bf16, B, TO, false><<<groups, kThreads, 0, s>>>(b);
  } else {
    if (stream_out) scale_kernel<float, B, TO, true><<<groups, kThreads, 0, s>>>(b);
    else scale_kernel<float, B, TO, false><<<groups, kThreads, 0, s>>>(b);
  }
}

int64_t chunk_of(nvfp4_type type) { return type == NVFP4_T_BF16 ? kChunk<bf16> : kChunk<float>; }

// f(batch, workgroups) for one launch after the other.
template <typename B, int SIZE, typename Fill, typename F>
nvfp4_status batches(const nvfp4_grad_tensor* t, int64_t count, nvfp4_type type, Fill fill, F f) {
  const int64_t chunk = chunk_of(type);
  B b;
  int64_t at = 0;
  while (at < count) {
    int64_t chunks = 0;
    b.count = 0;
    for (; at < count && b.count < SIZE; ++at) {
      if (t[at].numel == 0) continue;
      b.first[b.count] = (uint32_t)chunks;
      b.t[b.count].grad = t[at].grad;
      b.t[b.count].numel = t[at].numel;
      fill(b.t[b.count], at);
      ++b.count;
      chunks += (t[at].numel + chunk - 1) / chunk;      // all of them fit 32 bits
    }
    b.first[b.count] = (uint32_t)chunks;
    if (chunks == 0) continue;
    f(b, (unsigned)(chunks < kGroups ? chunks : kGroups));
    const nvfp4_status st = launched();
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}

nvfp4_status look(const nvfp4_grad_tensor* t, int64_t count, int64_t es) {
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].numel < 0 || t[i].numel > kMaxNumel) return NVFP4_ERR_SHAPE;
    if (t[i].numel == 0) continue;
    if (!t[i].grad) return NVFP4_ERR_NULL;
    if (!aligned(t[i].grad, es)) return NVFP4_ERR_ALIGN;
  }
  return NVFP4_OK;
}

// Whether what is written (out, or the tensors themselves) overlaps nothing else that is written or read.
nvfp4_status apart(const nvfp4_grad_tensor* in, const nvfp4_grad_tensor* out, int64_t count, int64_t es) {
  struct Part {
    uintptr_t lo, hi;
    bool written;
  };
  Part* part = (Part*)malloc((size_t)(count ? count : 1) * 2 * sizeof(Part));
  if (!part) return NVFP4_ERR_HIP;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (in[i].numel == 0) continue;
    const Range from = range(in[i].grad, in[i].numel * es), to = out ? range(out[i].grad, in[i].numel * es) : from;
    part[n++] = {to.lo, to.hi, true};
    if (to.lo != from.lo) part[n++] = {from.lo, from.hi, false};
  }
  std::sort(part, part + n, [](const Part& a, const Part& b) { return a.lo < b.lo; });
  uintptr_t written = 0, read = 0;                     // the furthest ends so far
  bool ok = true;
  for (int64_t i = 0; i < n && ok; ++i) {
    ok = part[i].lo >= written && (!part[i].written || part[i].lo >= read);
    uintptr_t& end = part[i].written ? written : read;
    if (part[i].hi > end) end = part[i].hi;
  }
  free(part);
  return ok ? NVFP4_OK : NVFP4_ERR_ALIAS;
}

bool size_ok(double v) { return v >= 0.0 && v < 3.0e38; }

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT nvfp4_status nvfp4_grad_norm(const nvfp4_grad_tensor* tensors, int64_t count,
                                          nvfp4_type type, double max_norm, double eps, float* norm,
                                          float* scale, void* workspace, hipStream_t stream) {
  if (!known(type)) return NVFP4_ERR_ENUM;
  if (count < 0 || count > kMaxCount) return NVFP4_ERR_SHAPE;
  if ((count && !tensors) || !norm || !workspace) return NVFP4_ERR_NULL;
  if (!size_ok(max_norm) || !size_ok(eps)) return NVFP4_ERR_VALUE;
  if (!aligned(norm, 4) || !aligned(scale, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  const int64_t es = size_of(type);
  nvfp4_status st = look(tensors, count, es);
  if (st != NVFP4_OK) return st;
  const Range out[] = {range(norm, 4), range(scale, 4),
                       range(workspace, NVFP4_GRAD_NORM_WORKSPACE(count))};
  for (int o = 0; o < 3; ++o) {
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return NVFP4_ERR_ALIAS;
    for (int64_t i = 0; i < count; ++i)
      if (tensors[i].numel && overlap(out[o], range(tensors[i].grad, tensors[i].numel * es))) return NVFP4_ERR_ALIAS;
  }
  (void)hipGetLastError();
  double* part = (double*)workspace;
  int64_t parts = 0;
  st = batches<NormBatch, kTable>(tensors, count, type, [](Entry&, int64_t) {}, [&](NormBatch& b, unsigned groups) {
    b.part = part + parts;
    parts += groups;
    if (type == NVFP4_T_BF16) norm_kernel<bf16><<<groups, kThreads, 0, stream>>>(b);
    else norm_kernel<float><<<groups, kThreads, 0, stream>>>(b);
  });
  if (st != NVFP4_OK) return st;
  norm_end_kernel<<<1, 1024, 0, stream>>>(part, parts, max_norm, eps, norm, scale);
  return launched();
}

NVFP4_EXPORT nvfp4_status nvfp4_clip_grads(const nvfp4_grad_tensor* tensors, const nvfp4_grad_tensor* out,
                                           int64_t count, nvfp4_type type, const float* scale,
                                           hipStream_t stream) {
  if (!known(type)) return NVFP4_ERR_ENUM;
  if (count < 0 || count > kMaxCount) return NVFP4_ERR_SHAPE;
  if ((count && !tensors) || !scale) return NVFP4_ERR_NULL;
  if (!aligned(scale, 4)) return NVFP4_ERR_ALIGN;
  const int64_t es = size_of(type);
  nvfp4_status st = look(tensors, count, es);
  if (st == NVFP4_OK && out) st = look(out, count, es);
  if (st != NVFP4_OK) return st;
  const Range by = range(scale, 4);
  for (int64_t i = 0; i < count; ++i) {
    if (out && out[i].numel != tensors[i].numel) return NVFP4_ERR_SHAPE;
    if (tensors[i].numel && overlap(by, range(out ? out[i].grad : tensors[i].grad, tensors[i].numel * es)))
      return NVFP4_ERR_ALIAS;
  }
  st = apart(tensors, out, count, es);
  if (st != NVFP4_OK) return st;
  (void)hipGetLastError();
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) bytes += tensors[i].numel * es;
  const bool stream_out = bytes > kCached;
  if (!out)
    return batches<NormBatch, kTable>(tensors, count, type, [](Entry&, int64_t) {}, [&](NormBatch& b, unsigned groups) {
      b.scale = scale;
      scale_batch<NormBatch, false>(b, groups, type, stream_out, stream);
    });
  return batches<ToBatch, kTableTo>(tensors, count, type, [&](EntryTo& e, int64_t i) { e.out = out[i].grad; },
                                    [&](ToBatch& b, unsigned groups) {
    b.scale = scale;
    scale_batch<ToBatch, true>(b, groups, type, stream_out, stream);
  });
}
