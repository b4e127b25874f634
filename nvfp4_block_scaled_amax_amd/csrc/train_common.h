// What the training operators' kernels share: element types, vectors of eight elements at any
// element alignment, reductions, and the host's argument checks.
#ifndef NVFP4_TRAIN_COMMON_H
#define NVFP4_TRAIN_COMMON_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_train.h"

#define NVFP4_EXPORT extern "C" __attribute__((visibility("default")))

namespace train {

// ------------------------------------------------------------------------- element types
struct bf16 {
  uint16_t bits;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }

// Two binary32 values to bf16, round to nearest even (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2));
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) {
  return bf16{(uint16_t)pack_bf16(v, 0.0f)};
}

// v rounded to T and back.
template <typename T>
__device__ __forceinline__ float rounded(float v) {
  return to_f32(from_f32<T>(v));
}

// ----------------------------------------------------------------- vectors of N elements
// Rows of an odd length, and parts of tensors, start at any element: gfx950 loads and stores
// 16 bytes at any byte address, so one vector form serves every alignment.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

template <typename T, int N>
struct Vec {
  static constexpr int kWords = N * (int)sizeof(T) / 4;      // 2, 4 or 8
  uint32_t w[kWords];
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(sizeof(T) == 4 ? w[i % kWords]
                           : (i & 1)      ? w[i / 2 % kWords] & 0xFFFF0000u
                                          : w[i / 2 % kWords] << 16);
  }
};

// STREAM: past the caches, for data that is not likely to be found there when it is wanted next.
template <int N, bool STREAM = false, typename T>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p) {
  constexpr int words = Vec<T, N>::kWords;
  Vec<T, N> r;
  if constexpr (words == 2) {
    typedef u32x2 half __attribute__((aligned(2)));
    const u32x2 v = *reinterpret_cast<const half*>(p);
    r.w[0] = v[0], r.w[1] = v[1];
  } else {
#pragma unroll
    for (int k = 0; k < words; k += 4) {
      const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p) + k / 4;
      const u32x4 v = STREAM ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[k + i] = v[i];
    }
  }
  return r;
}
template <bool STREAM = false, typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& r) {
  static_assert(Vec<T, N>::kWords >= 4, "");
#pragma unroll
  for (int k = 0; k < Vec<T, N>::kWords; k += 4) {
    u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p) + k / 4;
    const u32x4 v = {r.w[k], r.w[k + 1], r.w[k + 2], r.w[k + 3]};
    if (STREAM) __builtin_nontemporal_store(v, q);
    else *q = v;
  }
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> make_vec(const float (&v)[N]) {
  Vec<T, N> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> zero_vec() {
  Vec<T, N> r;
#pragma unroll
  for (int i = 0; i < Vec<T, N>::kWords; ++i) r.w[i] = 0u;
  return r;
}

// Makes the compiler forget how v came about (no instruction): what was computed from it
// before is computed again rather than kept in registers.
template <typename T, int N>
__device__ __forceinline__ void opaque(Vec<T, N>& v) {
#pragma unroll
  for (int i = 0; i < Vec<T, N>::kWords; ++i) asm("" : "+v"(v.w[i]));
}

// The same, and not before `after` is there.
template <typename T, int N>
__device__ __forceinline__ void opaque(Vec<T, N>& v, float after) {
#pragma unroll
  for (int i = 0; i < Vec<T, N>::kWords; ++i) asm("" : "+v"(v.w[i]) : "v"(after));
}
// v is in its registers, before anything that follows and has an effect (a barrier, a volatile asm): the
// others may be moved past these.
template <typename T, int N>
__device__ __forceinline__ void arrived(Vec<T, N>& v) {
#pragma unroll
  for (int i = 0; i < Vec<T, N>::kWords; ++i) asm volatile("" : "+v"(v.w[i]));
}
__device__ __forceinline__ void opaque(uint32_t& v, float after) { asm volatile("" : "+v"(v) : "v"(after)); }

// Elements by..N-1 moved to the front, zeros behind them (by in 1..N-1).
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> shift(Vec<T, N> v, int by) {
  constexpr int words = Vec<T, N>::kWords;
  if (sizeof(T) == 2) {
    if (by & 1) {
#pragma unroll
      for (int i = 0; i < words; ++i)
        v.w[i] = (v.w[i] >> 16) | (i + 1 < words ? v.w[(i + 1) % words] << 16 : 0u);
    }
    by >>= 1;
  }
#pragma unroll
  for (int d = 1; d < words; d *= 2)
    if (by & d) {
#pragma unroll
      for (int i = 0; i < words; ++i) v.w[i] = i + d < words ? v.w[(i + d) % words] : 0u;
    }
  return v;
}

// How a row's end falls on its vectors: there is none (every vector is in the row); on a
// boundary; anywhere, in a row of N elements or more; anywhere.
enum End { kFull, kWhole, kCut, kAny };

// Elements [at, at + N) of a row of n, zeros past its end.  A vector that the end cuts is loaded
// (kCut) from the last N elements and shifted, which takes no further loads and registers.
template <int N, End E, bool STREAM = false, typename T, typename I>
__device__ __forceinline__ Vec<T, N> load_vec(const T* row, I at, I n) {
  if (E == kFull) return load_vec<N, STREAM>(row + at);
  Vec<T, N> r = zero_vec<T, N>();
  if (E == kWhole) {
    if (at < n) r = load_vec<N, STREAM>(row + at);
  } else if (E == kCut) {
    if (at < n) {
      const I from = at < n - N ? at : n - N;
      r = load_vec<N, STREAM>(row + from);
      if (at != from) r = shift(r, (int)(at - from));
    }
  } else if (at + N <= n) {
    r = load_vec<N, STREAM>(row + at);
  } else if (at < n) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = at + i < n ? to_f32(row[at + i]) : 0.0f;
    r = make_vec<T>(v);
  }
  return r;
}
template <End E, bool STREAM = false, typename T, typename I, int N>
__device__ __forceinline__ void store_vec(T* row, I at, I n, const Vec<T, N>& v) {
  if (E == kFull) {
    store_vec<STREAM>(row + at, v);
  } else if (E == kWhole) {
    if (at < n) store_vec<STREAM>(row + at, v);
  } else if (at + N <= n) {
    store_vec<STREAM>(row + at, v);
  } else if (at < n) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at + i < n) row[at + i] = from_f32<T>(v[i]);
  }
}

// ---------------------------------------------------------------------------- reductions
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
// A rotation of each row of 16 lanes by N.
template <int N, typename V>
__device__ __forceinline__ V rotate16(V v) {
  return dpp<0x120 + N>(v);
}
struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
// Over each row of 16 lanes: every lane gets the result.
template <typename Op, typename V>
__device__ __forceinline__ V reduce16(V v, Op op) {
  v = op(v, rotate16<8>(v));
  v = op(v, rotate16<4>(v));
  v = op(v, rotate16<2>(v));
  return op(v, rotate16<1>(v));
}
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
// A barrier for shared memory alone: __syncthreads would also wait for vector memory in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Over the wavefront: every lane gets the result.  All 64 lanes must be active.
template <typename Op, typename V>
__device__ __forceinline__ V reduce64(V v, Op op) {
  v = reduce16(v, op);
  return op(op(read_lane(v, 0), read_lane(v, 16)), op(read_lane(v, 32), read_lane(v, 48)));
}
// Over groups of N neighbouring lanes that hold N values, repeated: every lane gets the result.
template <int N, typename Op, typename V>
__device__ __forceinline__ V reduce_few(V v, Op op) {
  if (N >= 16) v = op(v, rotate16<8>(v));
  if (N >= 8) v = op(v, rotate16<4>(v));
  if (N >= 4) v = op(v, rotate16<2>(v));
  if (N >= 2) v = op(v, rotate16<1>(v));
  return v;
}
// Over a workgroup of WAVES (a power of two) wavefronts through `slots` (WAVES entries of LDS):
// every lane gets the result.  The caller keeps a barrier between two uses of the same slots.
template <int WAVES, typename Op, typename V>
__device__ __forceinline__ V reduce_group(V v, Op op, V* slots) {
  v = reduce64(v, op);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  return reduce_few<WAVES>(slots[threadIdx.x % WAVES], op);
}

// A workgroup's part of a tensor's maximum: on the bits, where inf and NaN sort above the rest.
// Atomics on one word take turns (2048 of them 15 us or so), so one that cannot raise the word is
// left out: after the first few that is most of them.  The maximum does not depend on who came first.
template <int WAVES>
__device__ __forceinline__ void publish_amax(uint32_t m, uint32_t* amax, uint32_t* slots) {
  m = reduce_group<WAVES>(m, Max(), slots);
  if (threadIdx.x == 0 && m > __hip_atomic_load(amax, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
    atomicMax(amax, m);
}

__global__ void clear_words(uint32_t* p, int64_t n);

// ---------------------------------------------------------------------------------- host
// Dynamic shared memory that a kernel with a little static one may ask for without being told.
constexpr int kPlainLds = 65536 - 1024;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Range {
  uintptr_t lo, hi;
};
inline Range range(const void* p, int64_t bytes) {
  return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)(p ? bytes : 0)};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool known(nvfp4_type t) { return t == NVFP4_T_BF16 || t == NVFP4_T_F32; }
inline int64_t size_of(nvfp4_type t) { return t == NVFP4_T_BF16 ? 2 : 4; }

// Bytes of a [rows][cols] array whose rows are `stride` elements apart.
inline int64_t extent(int64_t rows, int64_t cols, int64_t stride, int64_t esize) {
  return rows <= 0 ? 0 : ((rows - 1) * stride + cols) * esize;
}
// Keeps every byte offset below 2^62.
inline bool shape_ok(int64_t rows, int64_t cols, int64_t stride) {
  return rows >= 0 && cols >= 1 && stride >= cols && stride < (int64_t(1) << 40) &&
         (rows == 0 || rows < (int64_t(1) << 59) / stride);
}

inline nvfp4_status launched() {
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status clear(uint32_t* p, int64_t n, hipStream_t stream);

}  // namespace train
#endif
