// One AdamW step over many tensors for gfx950 (include/nvfp4_train.h defines the update).
//
// A launch takes up to 58 tensors, whose table travels as a kernel argument: no copy to the
// device, no state, nothing to go stale.  A workgroup takes one chunk of one tensor; a lane
// takes eight consecutive elements at a time, so that 16 neighbouring lanes hold one block of
// an 8-bit state and its maximum is four rotations within a row of lanes.
//
// 8-bit states: m and sqrt(v) as E4M3 times a scale per block of 128.  With the square root
// their 17 octaves span 34 octaves of v.  Codes are rounded stochastically on the bits:
// random bits below the kept ones, then truncation, with values under 2^-6 moved up by 2^-6
// first so that the same 20 bits are cut from the subnormal steps of 2^-9.
#include "train_common.h"

namespace train {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kStep = kThreads * 8;                // elements of a workgroup at a time
constexpr int kSteps = 4;                              // of them in a chunk of a large launch
constexpr int kTable = 58;                             // tensors: Batch stays below 4 KB
constexpr float kTiny = 7.8886090522101180541e-31f;    // 2^-100

struct Batch {
  nvfp4_adamw_tensor t[kTable];
  uint32_t first[kTable + 1];         // first chunk of each tensor
  int count, index;                   // tensors, and the index of the first in the call
  int steps;                          // of kStep elements: a chunk
  float beta1, beta2, rest1, rest2, keep, rate, root, eps;
  uint32_t key;
  const float* grad_scale;
  uint32_t* amax;
};

static_assert(sizeof(Batch) <= 4096 && kTable <= 64, "kernel arguments; a lane per entry");

// Two rounds of xor-shift and multiply: every input bit reaches every output bit.  Shifts and factors are a
// published set of low bias (C. Wellons, "Prospecting for Hash Functions", 2018, public domain).
__host__ __device__ __forceinline__ uint32_t hash32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x7FEB352Du;
  h ^= h >> 15;
  h *= 0x846CA68Bu;
  return h ^ (h >> 16);
}

enum Param { kF32, kMaster, kAlone };       // float; bf16 with a master copy; bf16 alone

// y >= 0 (or NaN) -> the value above or below it in E4M3's steps, up as often as the 20 random bits say.
__device__ __forceinline__ float round_e4m3(float y, uint32_t bits) {
  const float up = y < 0.015625f ? 0.015625f : 0.0f;
  const float cut = __uint_as_float((__float_as_uint(y + up) + bits) & 0xFFF00000u);
  return cut - up;
}

// sqrt(v) rounded to nearest, for v = 0, inf and v >= 2^-96.  The hardware's root is within one step, and the
// sign of v - s' s tells on which side of the midpoint between a neighbour s' and s the root lies (Tuckerman's
// test: Agarwal et al., "New scalar and vector elementary functions for the IBM System/370", 1986).  With
// s >= 2^-48 the residual is a multiple of 2^-142, so that no sign is lost.  (That of 0 and inf is NaN,
// tells nothing and changes nothing.)
__device__ __forceinline__ float root(float v) {
  const float s = __builtin_amdgcn_sqrtf(v);
  const float below = __uint_as_float(__float_as_uint(s) - 1u);
  const float above = __uint_as_float(__float_as_uint(s) + 1u);
  const float r = fmaf(-below, s, v) <= 0.0f ? below : s;
  return fmaf(-above, s, v) > 0.0f ? above : r;
}

// The same for every v.  The hardware takes a subnormal v for 0; what is below 2^-96 is taken 2^96
// times, which is exact, in a branch that ordinary second moments do not enter.
__device__ __forceinline__ void roots(const float (&v)[8], float (&r)[8]) {
  float least = v[0];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = root(v[i]);
    least = fminf(least, v[i]);
  }
  if (least < 0x1p-96f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v[i] > 0.0f && v[i] < 0x1p-96f) r[i] = root(v[i] * 0x1p96f) * 0x1p-48f;
  }
}

// Eight values over 16 lanes to a block scale and eight E4M3 bytes.
template <bool POSITIVE>
__device__ __forceinline__ u32x2 encode(const float (&x)[8], const uint32_t (&bits)[8], float& scale) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const float top = __uint_as_float(reduce16(most, Max()));
  scale = top < kTiny ? 0.0f : top * (1.0f / 448.0f);
  const float inv = scale == 0.0f ? 0.0f : 1.0f / scale;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = x[i] * inv;
    // at the most 448; and for the root, which is divided by, at the least 2^-9 where it is not 0: the
    // median with 2^-9 and a bound that is 0 for 0, else above 2^-9 and s rounded up (the smallest
    // root of all, 2^-74.5, over the largest, 2^64, is s = 2^-129.7, and 2^127 times that 2^-2.7)
    if (POSITIVE)
      y[i] = __builtin_amdgcn_fmed3f(round_e4m3(s, bits[i] >> 12), 0.001953125f,
                                     fminf(s * 0x1p127f, 448.0f));
    else
      y[i] = copysignf(fminf(round_e4m3(fabsf(s), bits[i] & 0xFFFFFu), 448.0f), s);
  }
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
    r[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w, true);
  }
  return r;
}
__device__ __forceinline__ void decode(u32x2 w, float scale, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    x[4 * i] = lo[0] * scale;
    x[4 * i + 1] = lo[1] * scale;
    x[4 * i + 2] = hi[0] * scale;
    x[4 * i + 3] = hi[1] * scale;
  }
}

// Eight bytes of a row of n, zeros past its end.
__device__ __forceinline__ u32x2 load_bytes(const uint8_t* p, int64_t at, int64_t n) {
  u32x2 r = {0, 0};
  if (at + 8 <= n) {
    r = *reinterpret_cast<const u32x2_a1*>(p + at);
  } else if (at < n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i < n) r[i >> 2] |= (uint32_t)p[at + i] << (8 * (i & 3));
  }
  return r;
}
__device__ __forceinline__ void store_bytes(uint8_t* p, int64_t at, int64_t n, u32x2 v) {
  if (at + 8 <= n) {
    *reinterpret_cast<u32x2_a1*>(p + at) = v;
  } else if (at < n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i < n) p[at + i] = (uint8_t)(v[i >> 2] >> (8 * (i & 3)));
  }
}

// p <- p (1 - lr decay) - lr m^ / (sqrt(v^) + eps), the corrections of m and v being in rate and
// root, and the running means as given in the header; everything in binary32 until it is stored.
//
// With binary32 states the memory bounds it: bf16 parameters with a master copy and bf16
// gradients, 28 bytes an element, 671 million of them in 3.59 ms (5.2 TB/s, as a copy).  8-bit
// states leave 10 bytes and 80 issue slots an element (95 before the codes were rounded on their
// bits): 224 million in 490 us a call, 467 of it the large tensors' launch at its best, where 39.3 T slots a
// second allow 456.  bf16 parameters alone with binary32 states: 201 million in 836 us (22 bytes, 5.3 TB/s).  A
// step of a small model is the latency of one chunk: 24 x 65536 elements, all in 32 bits, in 10.7 us.
template <Param P, typename G, bool E4M3, bool AMAX>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Batch a) {
  __shared__ uint32_t slots[kThreads / 64];
  // the chunk's tensor: the last one whose first chunk is not after it (the lanes look at an
  // entry each)
  const uint32_t lane = threadIdx.x & 63;
  const bool before = lane < (uint32_t)a.count && a.first[lane < kTable ? lane : 0] <= blockIdx.x;
  const int lo = __builtin_amdgcn_readfirstlane(__popcll(__ballot(before)) - 1);
  const nvfp4_adamw_tensor& t = a.t[lo];
  const int64_t n = t.numel, base = (int64_t)(blockIdx.x - a.first[lo]) * (a.steps * kStep);
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  uint32_t key = hash32(a.key ^ (uint32_t)(a.index + lo));
  if (base >> 32) key = hash32(key ^ (uint32_t)(base >> 32));    // chunks do not cross 2^32
  uint32_t most = 0;
#pragma unroll 1
  for (int step = 0; step < a.steps; ++step) {
    const int64_t at = base + (int64_t)(step * kThreads + threadIdx.x) * 8;
    if (base + step * kStep >= n) break;
    const Vec<G, 8> g8 = load_vec<8, kAny>((const G*)t.grad, at, n);
    float m[8], v[8], p[8];
    if (E4M3) {
      const int64_t block = at / NVFP4_ADAMW_BLOCK;
      const float ms = at < n ? t.avg_scale[block] : 0.0f, vs = at < n ? t.sq_scale[block] : 0.0f;
      decode(load_bytes((const uint8_t*)t.exp_avg, at, n), ms, m);
      decode(load_bytes((const uint8_t*)t.exp_avg_sq, at, n), vs, v);
    } else {
      const Vec<float, 8> m8 = load_vec<8, kAny>((const float*)t.exp_avg, at, n);
      const Vec<float, 8> v8 = load_vec<8, kAny>((const float*)t.exp_avg_sq, at, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = m8[i];
        v[i] = v8[i];
      }
    }
    if (P == kAlone) {
      const Vec<bf16, 8> p8 = load_vec<8, kAny>((const bf16*)t.param, at, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = p8[i];
    } else {
      const Vec<float, 8> p8 = load_vec<8, kAny>(P == kF32 ? (const float*)t.param : t.master, at, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = p8[i];
    }
    uint32_t bits[8];
    if (E4M3 || P == kAlone) {
#pragma unroll
      for (int i = 0; i < 8; ++i) bits[i] = hash32((uint32_t)at + i + key);
    }
    float low[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = a.grad_scale ? g8[i] * gs : g8[i];
      const float sq = E4M3 ? v[i] * v[i] : v[i];
      m[i] = m[i] * a.beta1 + g * a.rest1;
      v[i] = sq * a.beta2 + (g * g) * a.rest2;
      if (!E4M3) low[i] = sqrtf(v[i]);
    }
    if (E4M3) roots(v, low);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = p[i] * a.keep - (m[i] * __builtin_amdgcn_rcpf(low[i] * a.root + a.eps)) * a.rate;
    if (E4M3) {
      float ms, vs;
      const u32x2 mc = encode<false>(m, bits, ms), vc = encode<true>(low, bits, vs);
      store_bytes((uint8_t*)t.exp_avg, at, n, mc);
      store_bytes((uint8_t*)t.exp_avg_sq, at, n, vc);
      if ((threadIdx.x & 15) == 0 && at < n) {
        t.avg_scale[at / NVFP4_ADAMW_BLOCK] = ms;
        t.sq_scale[at / NVFP4_ADAMW_BLOCK] = vs;
      }
    } else {
      store_vec<kAny>((float*)t.exp_avg, at, n, make_vec<float>(m));
      store_vec<kAny>((float*)t.exp_avg_sq, at, n, make_vec<float>(v));
    }
    if (P == kMaster) store_vec<kAny>(t.master, at, n, make_vec<float>(p));
    if (P == kAlone) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = __float_as_uint(p[i]);
        const uint32_t up = (w & 0x7FFFFFFFu) + ((bits[i] * 0x9E3779B1u) >> 16);
        p[i] = p[i] == p[i] ? __uint_as_float((up & 0xFFFF0000u) | (w & 0x80000000u)) : p[i];
      }
    }
    if (P == kF32) {
      store_vec<kAny>((float*)t.param, at, n, make_vec<float>(p));
    } else {
      const Vec<bf16, 8> out = make_vec<bf16>(p);
      store_vec<kAny>((bf16*)t.param, at, n, out);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = out[i];
    }
    if (AMAX) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < n) most = max(most, __float_as_uint(p[i]) & 0x7FFFFFFFu);
    }
  }
  if (AMAX) publish_amax<kThreads / 64>(most, a.amax + a.index + lo, slots);
}

template <Param P, typename G, bool E4M3>
void launch(const Batch& b, uint32_t chunks, hipStream_t s) {
  if (b.amax) adamw_kernel<P, G, E4M3, true><<<chunks, kThreads, 0, s>>>(b);
  else adamw_kernel<P, G, E4M3, false><<<chunks, kThreads, 0, s>>>(b);
}
template <Param P, typename G>
void launch(const Batch& b, uint32_t chunks, nvfp4_state state, hipStream_t s) {
  if (state == NVFP4_STATE_E4M3) launch<P, G, true>(b, chunks, s);
  else launch<P, G, false>(b, chunks, s);
}
template <Param P>
void launch(const Batch& b, uint32_t chunks, nvfp4_type gtype, nvfp4_state state, hipStream_t s) {
  if (gtype == NVFP4_T_BF16) launch<P, bf16>(b, chunks, state, s);
  else launch<P, float>(b, chunks, state, s);
}

constexpr int64_t kMaxNumel = int64_t(1) << 36;
constexpr int64_t kMaxChunks = int64_t(1) << 23;       // of a launch: threads stay below 2^32

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT nvfp4_status nvfp4_adamw_step(const nvfp4_adamw_tensor* tensors, int64_t count,
                                           nvfp4_type ptype, nvfp4_type gtype, nvfp4_state state,
                                           const nvfp4_adamw_args* args, const float* grad_scale,
                                           float* out_amax, hipStream_t stream) {
  if (!known(ptype) || !known(gtype) || (state != NVFP4_STATE_F32 && state != NVFP4_STATE_E4M3))
    return NVFP4_ERR_ENUM;
  if (count < 0 || count > (int64_t(1) << 24)) return NVFP4_ERR_SHAPE;
  if (!args || (count && !tensors)) return NVFP4_ERR_NULL;
  const auto beta_ok = [](double b) { return b >= 0.0 && b < 1.0; };
  const auto finite = [](double v) { return v > -3.0e38 && v < 3.0e38; };
  if (!beta_ok(args->beta1) || !beta_ok(args->beta2) || !(args->eps >= 0.0) ||
      !finite(args->eps) || !finite(args->lr) || !finite(args->weight_decay) || args->step < 1 ||
      args->step > 0xFFFFFFFFll)
    return NVFP4_ERR_VALUE;
  const int64_t ps = size_of(ptype), gs = size_of(gtype), ss = state == NVFP4_STATE_F32 ? 4 : 1;
  int master = -1;
  if (!aligned(grad_scale, 4) || !aligned(out_amax, 4)) return NVFP4_ERR_ALIGN;
  for (int64_t i = 0; i < count; ++i) {
    const nvfp4_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || t.numel > kMaxNumel) return NVFP4_ERR_SHAPE;
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return NVFP4_ERR_NULL;
    if (state == NVFP4_STATE_E4M3 && (!t.avg_scale || !t.sq_scale)) return NVFP4_ERR_NULL;
    if (master >= 0 && master != (t.master != nullptr)) return NVFP4_ERR_NULL;
    master = t.master != nullptr;
    if (master && ptype == NVFP4_T_F32) return NVFP4_ERR_ENUM;
    if (!aligned(t.param, ps) || !aligned(t.grad, gs) || !aligned(t.exp_avg, ss) ||
        !aligned(t.exp_avg_sq, ss) || !aligned(t.master, 4) || !aligned(t.avg_scale, 4) ||
        !aligned(t.sq_scale, 4))
      return NVFP4_ERR_ALIGN;
    const int64_t blocks = (t.numel + NVFP4_ADAMW_BLOCK - 1) / NVFP4_ADAMW_BLOCK;
    const bool scaled = state == NVFP4_STATE_E4M3;
    const Range r[] = {range(t.param, t.numel * ps), range(t.exp_avg, t.numel * ss),
                       range(t.exp_avg_sq, t.numel * ss), range(t.master, t.numel * 4),
                       range(scaled ? t.avg_scale : nullptr, blocks * 4),
                       range(scaled ? t.sq_scale : nullptr, blocks * 4),
                       range(out_amax, count * 4), range(t.grad, t.numel * gs),
                       range(grad_scale, 4)};
    for (int x = 0; x < 9; ++x)
      for (int y = 0; y < x && y < 7; ++y)
        if (overlap(r[x], r[y])) return NVFP4_ERR_ALIAS;
  }
  (void)hipGetLastError();
  if (out_amax) {
    const nvfp4_status st = clear((uint32_t*)out_amax, count, stream);
    if (st != NVFP4_OK) return st;
  }
  const double t = (double)args->step;
  Batch b;
  b.beta1 = (float)args->beta1;
  b.beta2 = (float)args->beta2;
  b.rest1 = (float)(1.0 - args->beta1);
  b.rest2 = (float)(1.0 - args->beta2);
  b.keep = (float)(1.0 - args->lr * args->weight_decay);
  b.rate = (float)(args->lr / (1.0 - __builtin_pow(args->beta1, t)));
  b.root = (float)(1.0 / __builtin_sqrt(1.0 - __builtin_pow(args->beta2, t)));
  b.eps = (float)args->eps;
  b.key = hash32(hash32(args->seed) ^ (uint32_t)args->step);
  b.grad_scale = grad_scale;
  b.amax = (uint32_t*)out_amax;
  int64_t at = 0;
  while (at < count) {
    // chunks of one step where there are few elements, for the latency; of more where there are
    // many, for fewer workgroups
    int64_t elements = 0;
    for (int64_t i = at; i < count && i < at + kTable; ++i) elements += tensors[i].numel;
    b.steps = elements <= kStep * 2048 ? 1 : kSteps;
    const int64_t chunk = b.steps * kStep;
    int64_t chunks = 0;
    b.count = 0;
    b.index = (int)at;
    for (; at < count && b.count < kTable; ++at) {
      const int64_t need = (tensors[at].numel + chunk - 1) / chunk;
      if (b.count && chunks + need > kMaxChunks) break;
      b.first[b.count] = (uint32_t)chunks;
      b.t[b.count++] = tensors[at];
      chunks += need;
    }
    b.first[b.count] = (uint32_t)chunks;
    if (chunks == 0) continue;
    if (ptype == NVFP4_T_F32) launch<kF32>(b, (uint32_t)chunks, gtype, state, stream);
    else if (master > 0) launch<kMaster>(b, (uint32_t)chunks, gtype, state, stream);
    else launch<kAlone>(b, (uint32_t)chunks, gtype, state, stream);
    const nvfp4_status st = launched();
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}
