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

// -------------------------------------------------------------- vectors of eight elements
// Rows of an odd length, and parts of tensors, start at any element: gfx950 loads and stores
// 16 bytes at any byte address, so one vector form serves every alignment.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

template <typename T>
struct Vec8;
template <>
struct Vec8<bf16> {
  u32x4 w;
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct Vec8<float> {
  u32x4 w, w2;
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i < 4 ? w[i & 3] : w2[i & 3]);
  }
};

__device__ __forceinline__ Vec8<bf16> load_vec(const bf16* p) {
  return {*reinterpret_cast<const u32x4_a2*>(p)};
}
__device__ __forceinline__ Vec8<float> load_vec(const float* p) {
  const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
  return {q[0], q[1]};
}
__device__ __forceinline__ Vec8<bf16> make_vec(const float (&v)[8], bf16) {
  Vec8<bf16> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  return r;
}
__device__ __forceinline__ Vec8<float> make_vec(const float (&v)[8], float) {
  Vec8<float> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.w[i] = __float_as_uint(v[i]);
    r.w2[i] = __float_as_uint(v[i + 4]);
  }
  return r;
}
__device__ __forceinline__ void store_vec(bf16* p, const Vec8<bf16>& v) {
  *reinterpret_cast<u32x4_a2*>(p) = v.w;
}
__device__ __forceinline__ void store_vec(float* p, const Vec8<float>& v) {
  u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
  q[0] = v.w;
  q[1] = v.w2;
}

// Four binary32 elements, where a lane's 16 bytes are to touch its neighbours'.
struct Vec4 {
  u32x4 w;
  __device__ __forceinline__ float operator[](int i) const { return __uint_as_float(w[i]); }
};

// Makes the compiler forget how v came about (no instruction): what was computed from it
// before is computed again rather than kept in registers.
__device__ __forceinline__ void opaque(Vec8<bf16>& v) { asm("" : "+v"(v.w)); }
__device__ __forceinline__ void opaque(Vec8<float>& v) { asm("" : "+v"(v.w), "+v"(v.w2)); }
__device__ __forceinline__ void opaque(Vec4& v) { asm("" : "+v"(v.w)); }

// The same past the caches, for data that no later kernel is likely to find there.
__device__ __forceinline__ void store_stream(bf16* p, const Vec8<bf16>& v) {
  __builtin_nontemporal_store(v.w, reinterpret_cast<u32x4_a2*>(p));
}
__device__ __forceinline__ void store_stream(float* p, const Vec8<float>& v) {
  u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
  __builtin_nontemporal_store(v.w, q);
  __builtin_nontemporal_store(v.w2, q + 1);
}
__device__ __forceinline__ Vec8<bf16> load_stream(const bf16* p) {
  return {__builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p))};
}
__device__ __forceinline__ Vec8<float> load_stream(const float* p) {
  const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
  return {__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)};
}

template <typename T>
__device__ __forceinline__ Vec8<T> zero_vec() {
  const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  return make_vec(z, T());
}

// Elements by..7 moved to the front, zeros behind them (by in 1..7).
__device__ __forceinline__ Vec8<bf16> shift(Vec8<bf16> v, int by) {
  u32x4 w = v.w;
  if (by & 1) w = {(w[0] >> 16) | (w[1] << 16), (w[1] >> 16) | (w[2] << 16),
                   (w[2] >> 16) | (w[3] << 16), w[3] >> 16};
  if (by & 2) w = {w[1], w[2], w[3], 0u};
  if (by & 4) w = {w[2], w[3], 0u, 0u};
  return {w};
}
__device__ __forceinline__ Vec8<float> shift(Vec8<float> v, int by) {
  u32x4 a = v.w, b = v.w2;
  if (by & 1) a = {a[1], a[2], a[3], b[0]}, b = {b[1], b[2], b[3], 0u};
  if (by & 2) a = {a[2], a[3], b[0], b[1]}, b = {b[2], b[3], 0u, 0u};
  if (by & 4) a = b, b = {0u, 0u, 0u, 0u};
  return {a, b};
}

// How a row's end falls on its vectors: on a boundary; anywhere, in a row of 8 elements or more;
// anywhere.
enum End { kWhole, kCut, kAny };

// Elements [at, at + 8) of a row of n, zeros past its end.  A vector that the end cuts is loaded
// (kCut) from the last 8 elements and shifted, which takes no further loads and registers.
template <End E, typename T, typename I>
__device__ __forceinline__ Vec8<T> load_vec(const T* row, I at, I n) {
  Vec8<T> r = zero_vec<T>();
  if (E == kWhole) {
    if (at < n) r = load_vec(row + at);
  } else if (E == kCut) {
    if (at < n) {
      const I from = at < n - 8 ? at : n - 8;
      r = load_vec(row + from);
      if (at != from) r = shift(r, (int)(at - from));
    }
  } else if (at + 8 <= n) {
    r = load_vec(row + at);
  } else if (at < n) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = at + i < n ? to_f32(row[at + i]) : 0.0f;
    r = make_vec(v, T());
  }
  return r;
}
template <End E, typename T, typename I>
__device__ __forceinline__ void store_vec(T* row, I at, I n, const Vec8<T>& v) {
  if (E == kWhole) {
    if (at < n) store_vec(row + at, v);
  } else if (at + 8 <= n) {
    store_vec(row + at, v);
  } else if (at < n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
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

__global__ void clear_words(uint32_t* p, int64_t n);

// ---------------------------------------------------------------------------------- host
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
