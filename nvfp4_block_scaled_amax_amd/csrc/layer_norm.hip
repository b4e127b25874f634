// Layer norm forward and backward for gfx950 (include/nvfp4_train.h defines the operation).
//
// Both directions move bytes and little else: the forward pass reads x (and the residual) and
// writes y (and h) once, the backward pass reads dy and h (and dres) and writes dx once.  So a row
// is held in registers while its sums are made: up to 512 columns by 16, 32 or 64 lanes of a
// wavefront, eight elements each (in the backward pass up to 1024 of bf16, sixteen each); up to
// 16384 by one workgroup of as many wavefronts as the row fills.  The variance is the mean square
// of what is held less the mean (not E[x^2] - mean^2, which cancels).  Longer rows are read again
// for each step.  The backward pass keeps, next to the row, its share of the column sums (dweight,
// dbias) in registers over all the rows that a workgroup takes, leaves them as one partial row per
// workgroup in the workspace, and a second launch adds those in a fixed order.  Loads are 16
// bytes a lane, at any alignment of the element.
#include <type_traits>

#include "train_common.h"

namespace train {
namespace {

constexpr int kMaxHeldCols = 16384;

struct Forward {
  const void* x;
  const void* residual;
  const void* weight;
  const void* bias;
  void* y;
  void* h;
  float* mean;
  float* rstd;
  uint32_t* amax;
  int64_t x_stride, residual_stride, rows;
  int cols, center;
  float eps;
};

struct Backward {
  const void* dy;
  const void* h;
  const void* weight;
  const float* mean;
  const float* rstd;
  const void* dres;
  void* dx;
  float* partial;     // [groups][sums][cols]: dweight, and with sums == 2 dbias
  int64_t rows;
  int cols, sums;
};

// A lane's vector: 16 bytes of T, so that a wavefront's loads are next to each other.
template <typename T>
constexpr int kVec = 16 / sizeof(T);
template <typename T>
constexpr int kUnits = 8 / kVec<T>;

// A lane's vector of a row of `cols` elements that is held: where it is, and where it is loaded
// from.  No load depends on a condition (the compiler can then count the loads in flight, and wait
// for the first of them alone): a vector past the row's end, or cut by it, is loaded from the last
// N elements, and settled when it is used.  (Rows that may have fewer than N, kAny, do without.)
template <int N, End E>
struct Place {
  uint32_t at, from, end;
  __device__ __forceinline__ Place(uint32_t at_, uint32_t cols)
      : at(at_), from(E == kFull || E == kAny || at_ < cols - N ? at_ : cols - N), end(cols) {}
  template <typename T>
  __device__ __forceinline__ Vec<T, N> load(const T* row) const {
    if (E == kAny) return load_vec<N, E>(row, at, end);
    return load_vec<N>(row + from);
  }
  // zeros past the row's end (kCut; with kWhole a vector is in the row or not: see in())
  template <typename T>
  __device__ __forceinline__ void settle(Vec<T, N>& v) const {
    if (E == kCut && at != from) v = at - from < N ? shift(v, (int)(at - from)) : zero_vec<T, N>();
  }
  __device__ __forceinline__ bool in(uint32_t cols) const { return E == kFull || at < cols; }
  __device__ __forceinline__ bool in(uint32_t cols, int i) const {
    return E == kFull || (E == kWhole ? at < cols : at + i < cols);
  }
};

// A value that the whole wavefront wants from memory that no kernel in flight writes, through the
// scalar cache.
__device__ __forceinline__ float scalar_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

// The sum over groups of LANES lanes, to every lane.
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
  if (LANES == 64) return reduce64(v, Sum());
  v = reduce16(v, Sum());
  if (LANES == 32) v += __shfl_xor(v, 16, 32);
  return v;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// y = (h - mean) rstd weight + bias.  Rows of up to 512 columns take a wavefront each, those of up
// to 256 and 128 a half and a quarter of one (LANES; 262144 x 128 bf16 26.8 us, 52.4 with a wavefront
// each); longer ones a workgroup (LANES == 0).  A lane holds K vectors, and where that is eight
// elements (HOLD) also its weights for all the rows that it comes by (bf16, 8192 x 4097 30.5 us, 41.0 if
// they are read for each; 8192 x 4104 with residual 49.9 and 57.0; f32 the same).  Rows of bf16 that
// fill the workgroup, without a residual, are an exception while the tensors are of the last-level
// cache's size; why has not been shown (us, weights held and read for each row: 16384 x 2048 26.7 and
// 24.4, 6553 x 5120 30.4 and 26.5, 8192 x 4096 27.2 and 23.4, 4096 x 8192 27.3 and 23.0, 512 x 4096 4.6
// and 4.8).  For larger ones it is the slower way: 32768 x 4096 100 and 113.
//
// The memory bounds it: 8192 x 4096 bf16 with residual and h 49.5 us (268 MB, 5.4 TB/s; a copy of
// that size 5.4), without 23.3 (134 MB, half of it in the last-level cache), f32 47.5; 65536 x 512
// bf16 27.2 us, 4.9 TB/s.  An odd width costs bf16 rows the alignment of every other one
// (8192 x 4097: 30.6 us).  One row is the launch: 2.6 us of kernel.
template <typename T, typename W, int THREADS, int K, End E, int LANES, bool HOLD>
__global__ __launch_bounds__(THREADS) void forward_kernel(const Forward a) {
  constexpr int N = kVec<T>, ROWS = LANES ? THREADS / (LANES ? LANES : 1) : 1;    // at a time
  __shared__ float slots[2][2][16];
  __shared__ uint32_t top[16];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lanes = LANES ? LANES : blockDim.x, lane = LANES ? threadIdx.x % lanes : threadIdx.x;
  const uint32_t first = LANES == 64 ? wave : LANES ? threadIdx.x / lanes : 0;
  const uint32_t cols = a.cols;
  const float inv = 1.0f / (float)a.cols;
  auto vector = [&](const void* v, int k) {
    const Place<N, E> at((k * lanes + lane) * N, cols);
    Vec<W, N> r = v ? at.load((const W*)v) : zero_vec<W, N>();
    at.settle(r);
    return r;
  };
  Vec<W, N> weight[HOLD ? K : 1], bias[HOLD ? K : 1];
#pragma unroll
  for (int k = 0; k < (HOLD ? K : 0); ++k) weight[k] = vector(a.weight, k), bias[k] = vector(a.bias, k);
  if (!LANES) {
    if (threadIdx.x < 64) ((float*)slots)[threadIdx.x] = 0.0f;      // those of wavefronts not there
    if (threadIdx.x < 16) top[threadIdx.x] = 0u;
    __syncthreads();
  }
  // over the row; the slots of two rows in turn
  auto total = [&](float v, float* part) {
    if (LANES) return sum_lanes<LANES ? LANES : 64>(v);
    v = reduce64(v, Sum());
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    lds_barrier();
    return reduce16(part[threadIdx.x % 16], Sum());
  };
  uint32_t most = 0;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + first; row < a.rows; row += step, turn ^= 1) {
    const T* x = (const T*)a.x + row * a.x_stride;
    Vec<T, N> q[K];
    float v[K][N];
#pragma unroll
    for (int k = 0; k < K; ++k) q[k] = Place<N, E>((k * lanes + lane) * N, cols).load(x);
    if (a.residual) {
      const T* r = (const T*)a.residual + row * a.residual_stride;
      T* h = (T*)a.h + row * cols;
      Vec<T, N> p[K];
#pragma unroll
      for (int k = 0; k < K; ++k) p[k] = Place<N, E>((k * lanes + lane) * N, cols).load(r);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Place<N, E> at((k * lanes + lane) * N, cols);
        at.settle(q[k]);
        at.settle(p[k]);
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = q[k][i] + p[k][i];
        q[k] = make_vec<T>(v[k]);
        store_vec<E, true>(h, at.at, cols, q[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) Place<N, E>((k * lanes + lane) * N, cols).settle(q[k]);
    }
    float mean = 0.0f, sum = 0.0f, sq = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Place<N, E> at((k * lanes + lane) * N, cols);
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[k][i] = q[k][i];
        part += v[k][i];
      }
      sum += at.in(cols) ? part : 0.0f;
    }
    if (a.center) mean = total(sum, slots[turn][0]) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Place<N, E> at((k * lanes + lane) * N, cols);
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[k][i] -= mean;
        const float d = E < kCut || at.in(cols, i) ? v[k][i] : 0.0f;
        part = fmaf(d, d, part);
      }
      sq += at.in(cols) ? part : 0.0f;
    }
    const float rstd = 1.0f / sqrtf(total(sq, slots[turn][1]) * inv + a.eps);
    if (lane == 0) {
      a.rstd[row] = rstd;
      if (a.center) a.mean[row] = mean;
    }
    T* y = (T*)a.y + row * cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Place<N, E> at((k * lanes + lane) * N, cols);
      const Vec<W, N> w = HOLD ? weight[HOLD ? k : 0] : vector(a.weight, k);
      const Vec<W, N> b = HOLD ? bias[HOLD ? k : 0] : vector(a.bias, k);
#pragma unroll
      for (int i = 0; i < N; ++i) v[k][i] = fmaf(v[k][i] * rstd, w[i], b[i]);
      const Vec<T, N> out = make_vec<T>(v[k]);
      store_vec<E, true>(y, at.at, cols, out);
      if (a.amax) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at.in(cols, i)) most = max(most, abs_bits(out[i]));
      }
    }
  }
  if (a.amax) publish_amax<LANES ? THREADS / 64 : 16>(most, a.amax, top);
}

// Rows longer than the registers hold: three passes over the row, of which the caches serve some
// (1024 x 32768 bf16 49.5 us, f32 77: 2.7 and 3.5 TB/s of one read and one write).
template <typename T, typename W>
__global__ __launch_bounds__(1024) void forward_long_kernel(const Forward a) {
  __shared__ float slots[2][16];
  __shared__ uint32_t top[16];
  const float inv = 1.0f / (float)a.cols;
  uint32_t most = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.x_stride;
    const T* r = a.residual ? (const T*)a.residual + row * a.residual_stride : nullptr;
    auto held = [&](int64_t at, float (&v)[8]) {
      const Vec<T, 8> q = load_vec<8, kAny>(x, at, (int64_t)a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q[i];
      if (r) {
        const Vec<T, 8> p = load_vec<8, kAny>(r, at, (int64_t)a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = rounded<T>(v[i] + p[i]);
      }
    };
    float mean = 0.0f, sum = 0.0f, sq = 0.0f, v[8];
    if (a.center) {
      for (int64_t at = threadIdx.x * 8; at < a.cols; at += 8192) {
        held(at, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[i];
      }
      mean = reduce_group<16>(sum, Sum(), slots[0]) * inv;
    }
    for (int64_t at = threadIdx.x * 8; at < a.cols; at += 8192) {
      held(at, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = at + i < a.cols ? v[i] - mean : 0.0f;
        sq += d * d;
      }
    }
    const float var = reduce_group<16>(sq, Sum(), slots[1]) * inv;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
      a.rstd[row] = rstd;
      if (a.center) a.mean[row] = mean;
    }
    for (int64_t at = threadIdx.x * 8; at < a.cols; at += 8192) {
      held(at, v);
      if (r) store_vec<kAny>((T*)a.h + row * a.cols, at, (int64_t)a.cols, make_vec<T>(v));
      const Vec<W, 8> w = load_vec<8, kAny>((const W*)a.weight, at, (int64_t)a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (v[i] - mean) * rstd * w[i];
      if (a.bias) {
        const Vec<W, 8> b = load_vec<8, kAny>((const W*)a.bias, at, (int64_t)a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
      }
      const Vec<T, 8> out = make_vec<T>(v);
      store_vec<kAny>((T*)a.y + row * a.cols, at, (int64_t)a.cols, out);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < a.cols) most = max(most, abs_bits(out[i]));
    }
    __syncthreads();
  }
  if (a.amax) publish_amax<16>(most, a.amax, top);
}

// A row in a wavefront or a part of it: K vectors per lane.  Each group of LANES goes its own way
// to the end, where the workgroup adds their column sums in order.  Bound by the memory, at two
// workgroups a compute unit: 65536 x 512 bf16 42 us, 262144 x 128 42.4 (86 with a wavefront for
// each row), 4.8 TB/s with the column sums' launch; 262144 x 512 150 (5.4), and 164 with half as
// many threads.
template <typename T, typename W, int THREADS, int K, End E, int LANES>
__global__ __launch_bounds__(THREADS) void backward_wave_kernel(const Backward a) {
  constexpr int N = kVec<T>, ROWS = THREADS / LANES;
  __shared__ float part[ROWS][LANES * N];
  const uint32_t lane = threadIdx.x % LANES, cols = a.cols;
  const uint32_t first = LANES == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : threadIdx.x / LANES;
  const float inv = 1.0f / (float)a.cols;
  float dw[K][N], db[K][N];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[k][i] = db[k][i] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + first; row < a.rows;
       row += (int64_t)gridDim.x * ROWS) {
    Vec<T, N> dy[K], h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t at = (k * LANES + lane) * N;
      dy[k] = load_vec<N, E>((const T*)a.dy + row * a.cols, at, cols);
      h[k] = load_vec<N, E>((const T*)a.h + row * a.cols, at, cols);
    }
    const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint32_t at = (k * LANES + lane) * N;
      asm volatile("" : "+v"(at));       // read again for each row: not worth registers
      const Vec<W, N> w = load_vec<N, E>((const W*)a.weight, at, cols);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (h[k][i] - mean) * rstd, d = dy[k][i], g = d * w[i];
        s1 += g;
        s2 = fmaf(g, xh, s2);
        dw[k][i] = fmaf(d, xh, dw[k][i]);
        db[k][i] += d;
        asm volatile("" : "+v"(s1), "+v"(s2), "+v"(dw[k][i]), "+v"(db[k][i]));   // here, not later
      }
    }
    // dx = rstd (g - c1 - xh c2), with both constants times rstd
    const float c1 = a.mean ? sum_lanes<LANES>(s1) * inv * rstd : 0.0f;
    const float c2 = sum_lanes<LANES>(s2) * inv * rstd * rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint32_t at = (k * LANES + lane) * N;
      opaque(at, c2);
      opaque(dy[k], c2);  // unpacked again from here: the floats need not live across the sums
      opaque(h[k], c2);
      const Vec<W, N> w = load_vec<N, E>((const W*)a.weight, at, cols);
      float d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        d[i] = fmaf(mean - h[k][i], c2, fmaf(dy[k][i] * w[i], rstd, -c1));
      }
      if (a.dres) {
        const Vec<T, N> r = load_vec<N, E>((const T*)a.dres + row * a.cols, at, cols);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] += r[i];
      }
      store_vec<E, true>((T*)a.dx + row * a.cols, at, cols, make_vec<T>(d));
    }
  }
  float* out = a.partial + (int64_t)blockIdx.x * a.sums * a.cols;
  for (int v = 0; v < a.sums; ++v, out += cols) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[first][lane * N + i] = v ? db[k][i] : dw[k][i];
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < LANES * N; c += THREADS) {
        float s = part[0][c];
#pragma unroll
        for (int r = 1; r < ROWS; ++r) s += part[r][c];
        if (k * LANES * N + c < cols) out[k * LANES * N + c] = s;
      }
      __syncthreads();
    }
  }
}

// Longer rows: a workgroup takes one at a time, K vectors a lane, and loads the next one meanwhile
// (AHEAD).  Nothing may stand between those loads and their use a row later that waits for vector
// memory in order, or that the compiler cannot count: the weights lie in shared memory, the
// statistics come through the scalar cache, and no load or store depends on a condition.  Where the
// row does not fill the workgroup (not FULL), a vector past the row's end, or cut by it, is the last
// N elements instead.  Its lane then computes and writes what its neighbours do, the same
// bits, and its weights are zero in the row's sums for the elements that are not its own.
//
// Bound by the memory: 8192 x 4096 bf16 with dres 50.3 us (268 MB, 5.3 TB/s), without 39 (5.2), and
// the column sums' launch.  2051 x 14336 bf16 takes 38 us (4.6 TB/s): 256 workgroups of 896 threads,
// of which three take a ninth row.
template <typename T, typename W, int K, bool FULL, bool RES>
__global__ __launch_bounds__(1024) void backward_kernel(const Backward a) {
  constexpr int N = kVec<T>;
  constexpr bool AHEAD = K * N == 8 || sizeof(T) == 2;      // there are registers for two rows
  __shared__ float slots[2][2][16];
  extern __shared__ __align__(16) char dynamic[];
  Vec<W, N>* const weight = (Vec<W, N>*)dynamic + threadIdx.x;       // [K][threads], by vectors
  const uint32_t threads = blockDim.x, cols = a.cols;
  const float inv = 1.0f / (float)a.cols;
  auto own = [&](int k) { return (k * threads + threadIdx.x) * N; };        // the vector's place
  auto from = [&](int k) { return FULL || own(k) < cols - N ? own(k) : cols - N; };
  float dw[K][N], db[K][N];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    weight[k * threads] = load_vec<N>((const W*)a.weight + from(k));
#pragma unroll
    for (int i = 0; i < N; ++i) dw[k][i] = db[k][i] = 0.0f;
  }
  if (threadIdx.x < 64) ((float*)slots)[threadIdx.x] = 0.0f;         // those of wavefronts not there
  __syncthreads();
  const int64_t step = gridDim.x, last = a.rows - 1;
  Vec<T, N> dy[K], h[K], dy2[K], h2[K], res[K];
  auto load = [&](const void* base, int64_t row, Vec<T, N> (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = load_vec<N>((const T*)base + row * cols + from(k));
  };
  if (AHEAD) {
    load(a.dy, blockIdx.x, dy2);
    load(a.h, blockIdx.x, h2);
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row <= last; row += step, turn ^= 1) {
    if (AHEAD) {
#pragma unroll
      for (int k = 0; k < K; ++k) dy[k] = dy2[k], h[k] = h2[k];
    } else {
      load(a.dy, row, dy);
      load(a.h, row, h);
    }
    if (RES && AHEAD) load(a.dres, row, res);
    if (AHEAD) {
      const int64_t next = row + step <= last ? row + step : last;   // one too many at the end
      load(a.dy, next, dy2);
      load(a.h, next, h2);
    }
    const float mean = a.mean ? scalar_load(a.mean + row) : 0.0f, rstd = scalar_load(a.rstd + row);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Vec<W, N> w = weight[k * threads];
      if (!FULL && own(k) != from(k)) {        // zero before its own elements
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = i < (int)(own(k) - from(k)) ? 0.0f : w[i];
        w = make_vec<W>(f);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (h[k][i] - mean) * rstd, d = dy[k][i], g = d * w[i];
        s1 += g;
        s2 = fmaf(g, xh, s2);
        dw[k][i] = fmaf(d, xh, dw[k][i]);
        db[k][i] += d;
        asm volatile("" : "+v"(s1), "+v"(s2), "+v"(dw[k][i]), "+v"(db[k][i]));   // here, not later
      }
    }
    // dres is here before the barrier, behind which another lane may write over it (a vector past the
    // row's end, or cut by it, is its neighbours').  What is loaded of dy and h is used before the barrier.
    if (RES && !FULL) {
      static_assert(AHEAD || FULL, "");
#pragma unroll
      for (int k = 0; k < K; ++k) opaque(res[k], s2);      // as late as can be
#pragma unroll
      for (int k = 0; k < K; ++k) arrived(res[k]);
    }
    // the slots of two rows in turn: one barrier per row is enough
    s1 = reduce64(s1, Sum());
    s2 = reduce64(s2, Sum());
    if ((threadIdx.x & 63) == 0) {
      slots[turn][0][threadIdx.x >> 6] = s1;
      slots[turn][1][threadIdx.x >> 6] = s2;
    }
    lds_barrier();
    s1 = reduce16(slots[turn][0][threadIdx.x % 16], Sum());
    s2 = reduce16(slots[turn][1][threadIdx.x % 16], Sum());
    // dx = rstd (g - c1 - xh c2), with both constants times rstd
    const float c1 = a.mean ? s1 * inv * rstd : 0.0f, c2 = s2 * inv * rstd * rstd;
    T* dx = (T*)a.dx + row * cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float d[N];
      opaque(dy[k], c2);      // unpacked again from here: the floats need not live across the sums
      opaque(h[k], c2);
      const Vec<W, N> w = weight[k * threads];
      if (RES && !AHEAD) res[k] = load_vec<N>((const T*)a.dres + row * cols + from(k));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        d[i] = fmaf(mean - h[k][i], c2, fmaf(dy[k][i] * w[i], rstd, -c1));
        if (RES) d[i] += res[k][i];
      }
      store_vec<true>(dx + from(k), make_vec<T>(d));
    }
  }
  float* out = a.partial + (int64_t)blockIdx.x * a.sums * cols;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (FULL || own(k) == from(k)) {
      store_vec(out + own(k), make_vec<float>(dw[k]));
      if (a.sums == 2) store_vec(out + cols + own(k), make_vec<float>(db[k]));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= (int)(own(k) - from(k))) {
          out[from(k) + i] = dw[k][i];
          if (a.sums == 2) out[cols + from(k) + i] = db[k][i];
        }
    }
}

// Rows longer than the registers hold: dx from two passes over the row (with the column sums, which
// read dy and h a third time, 1024 x 32768 bf16 102 us, f32 180) ...
template <typename T, typename W>
__global__ __launch_bounds__(1024) void backward_long_kernel(const Backward a) {
  __shared__ float slots[2][16];
  const float inv = 1.0f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = (const T*)a.dy + row * a.cols;
    const T* h = (const T*)a.h + row * a.cols;
    const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t at = threadIdx.x * 8; at < a.cols; at += 8192) {
      const Vec<T, 8> d = load_vec<8, kAny>(dy, at, (int64_t)a.cols), x = load_vec<8, kAny>(h, at, (int64_t)a.cols);
      const Vec<W, 8> w = load_vec<8, kAny>((const W*)a.weight, at, (int64_t)a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = d[i] * w[i];
        s1 += g;
        s2 = fmaf(g, (x[i] - mean) * rstd, s2);
      }
    }
    s1 = reduce_group<16>(s1, Sum(), slots[0]);
    s2 = reduce_group<16>(s2, Sum(), slots[1]);
    const float c1 = a.mean ? s1 * inv : 0.0f, c2 = s2 * inv;
    for (int64_t at = threadIdx.x * 8; at < a.cols; at += 8192) {
      const Vec<T, 8> d = load_vec<8, kAny>(dy, at, (int64_t)a.cols), x = load_vec<8, kAny>(h, at, (int64_t)a.cols);
      const Vec<W, 8> w = load_vec<8, kAny>((const W*)a.weight, at, (int64_t)a.cols);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = rstd * (d[i] * w[i] - c1 - (x[i] - mean) * rstd * c2);
      if (a.dres) {
        const Vec<T, 8> r = load_vec<8, kAny>((const T*)a.dres + row * a.cols, at, (int64_t)a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      store_vec<kAny>((T*)a.dx + row * a.cols, at, (int64_t)a.cols, make_vec<T>(v));
    }
    __syncthreads();
  }
}

// ... and the column sums by themselves, before dx may overwrite dy: a workgroup takes 2048
// columns (x) of every gridDim.y-th row.
template <typename T>
__global__ __launch_bounds__(256) void backward_long_columns_kernel(const Backward a) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  float dw[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const Vec<T, 8> d = load_vec<8, kAny>((const T*)a.dy + row * a.cols, at, (int64_t)a.cols);
    const Vec<T, 8> x = load_vec<8, kAny>((const T*)a.h + row * a.cols, at, (int64_t)a.cols);
    const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = fmaf(d[i], (x[i] - mean) * rstd, dw[i]);
      db[i] += d[i];
    }
  }
  float* out = a.partial + (int64_t)blockIdx.y * a.sums * a.cols;
  store_vec<kAny>(out, at, (int64_t)a.cols, make_vec<float>(dw));
  if (a.sums == 2) store_vec<kAny>(out + a.cols, at, (int64_t)a.cols, make_vec<float>(db));
}

// dweight (y == 0) and dbias (y == 1): a lane adds a column, the 16 wavefronts of a workgroup
// take every 16th partial row, and their sums are added in order.  Short: 512 partial rows of both
// sums of 4096 columns 4.6 us, 256 of one of 14336 4.6, 64 of 256 columns 2.5, most of it the launch.
template <typename W>
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ partial,
                                                           int groups, int cols, W* dweight,
                                                           W* dbias) {
  __shared__ float part[16][64];
  W* out = blockIdx.y ? dbias : dweight;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t first = (int64_t)blockIdx.x * 64; first < cols; first += (int64_t)gridDim.x * 64) {
    const int64_t c = first + lane;
    float s = 0.0f;
    if (c < cols) {
      const float* p = partial + (int64_t)blockIdx.y * cols + c;
#pragma unroll 16
      for (int g = wave; g < groups; g += 16) s += p[(int64_t)g * gridDim.y * cols];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < cols) {
#pragma unroll
      for (int i = 1; i < 16; ++i) s += part[i][lane];
      out[c] = from_f32<W>(s);
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------------------------- host
// Workgroups of `threads` in the forward pass: 1536 threads on each of 256 compute units, and two
// workgroups at the least, so that one loads while the other adds up.  More is no faster with a
// residual (8192 x 4096 bf16 50.0 us, 50.7 for 2048 threads) and worse where the last one does not
// fit (6144 x 5120: 49.9 us for two of 640 threads, 60.7 for three).
constexpr int64_t resident(int threads) {
  return (int64_t)256 * (threads > 768 ? 2 : 1536 / threads);
}

// Rows that a workgroup holds.
bool held(int64_t cols) { return cols <= kMaxHeldCols; }

// Threads for a row with `per` elements each: whole wavefronts.
int threads_for(int64_t cols, int per) { return (int)((cols + 64 * per - 1) / (64 * per)) * 64; }

// How the end of held rows falls on vectors of N elements, `per` of them in a lane.
template <int N>
End end_of(int64_t cols, int per) {
  return cols % (64 * per) == 0 ? kFull : cols % N == 0 ? kWhole : kCut;
}

// Lanes of a wavefront for a row of up to 512 columns: eight elements each.
int lanes_for(int64_t cols) { return cols <= 128 ? 16 : cols <= 256 ? 32 : 64; }

// Calls f(std::integral_constant) for a runtime End.
template <typename F>
void with_end(End e, F f) {
  if (e == kFull) f(std::integral_constant<End, kFull>());
  else if (e == kWhole) f(std::integral_constant<End, kWhole>());
  else f(std::integral_constant<End, kCut>());
}

// Calls f(lanes, end) for a row of up to 512 columns in vectors of N elements.
template <int N, typename F>
void with_lanes(int64_t cols, F f) {
  const int lanes = lanes_for(cols);
  if (cols < 8) return f(std::integral_constant<int, 16>(), std::integral_constant<End, kAny>());
  with_end(cols == lanes * 8 ? kFull : cols % N == 0 ? kWhole : kCut, [&](auto e) {
    if (lanes == 16) f(std::integral_constant<int, 16>(), e);
    else if (lanes == 32) f(std::integral_constant<int, 32>(), e);
    else f(std::integral_constant<int, 64>(), e);
  });
}

template <typename T, typename W>
void forward(const Forward& a, hipStream_t s) {
  constexpr int N = kVec<T>, k = kUnits<T>;
  const auto grid = [&](int threads, int rows) {
    const int64_t groups = (a.rows + rows - 1) / rows, most = resident(threads);
    return (unsigned)(groups < most ? groups : most);
  };
  const auto launch = [&](auto kernel, int threads, int rows) {
    kernel<<<grid(threads, rows), threads, 0, s>>>(a);
  };
  if (!held(a.cols)) {
    launch(forward_long_kernel<T, W>, 1024, 1);
  } else if (a.cols <= 512) {           // a wavefront or part of one; a workgroup of four of them
    with_lanes<N>(a.cols, [&](auto lanes, auto e) {
      constexpr int L = decltype(lanes)::value;
      launch(forward_kernel<T, W, 256, k, decltype(e)::value, L, true>, 256, 256 / L);
    });
  } else if (a.cols <= 8192) {          // eight elements a lane
    const int threads = threads_for(a.cols, 8);
    with_end(end_of<N>(a.cols, 8), [&](auto e) {
      constexpr End E = decltype(e)::value;
      if (E == kFull && sizeof(T) == 2 && !a.residual)
        launch(forward_kernel<T, W, 1024, k, E, 0, !(E == kFull && sizeof(T) == 2)>, threads, 1);
      else
        launch(forward_kernel<T, W, 1024, k, E, 0, true>, threads, 1);
    });
  } else {                              // thirty-two: 2051 x 14336 bf16 24.5 us, with sixteen 27.7
    const int threads = threads_for(a.cols, 32);
    with_end(end_of<N>(a.cols, 32), [&](auto e) {
      launch(forward_kernel<T, W, 512, 4 * k, decltype(e)::value, 0, false>, threads, 1);
    });
  }
}

// Rows that a workgroup of the backward pass takes at a time, and the most workgroups: they fill
// the chip once, and are also the partial rows of the column sums.
struct Split {
  int rows, most;
};
// Rows that a workgroup of the backward pass holds: long binary32 ones only if they fill it (the
// others would need more than 1024 threads' 128 registers; read again they take 2048 x 10001 110 us,
// 12000 123 and 16383 176, where the held 2048 x 12288 takes 67 and 16384 90).
bool backward_held(int64_t cols, int64_t esize) {
  return held(cols) && (esize == 2 || cols <= 8192 || cols % 1024 == 0);
}
// Rows that a wavefront takes by itself: one vector a lane, or two of bf16 (16384 x 1024 22.7 us,
// 28.7 with a workgroup each; 2048 x 1024 8.0 and 11.2; but 65536 x 1024 84 and 82).  binary32 would
// take four (16384 x 1024 with dres 58 us, and 55), and bf16 of 2048 columns, too (46 and 45).
bool backward_wave(int64_t cols, int64_t esize) { return cols <= 512 || (esize == 2 && cols <= 1024); }
Split backward_split(int64_t cols, int64_t esize, bool dres) {
  if (!backward_held(cols, esize)) return {1, 256};
  if (cols <= 512) return {1024 / lanes_for(cols), 512};
  if (backward_wave(cols, esize)) return {8, 512};
  // What a compute unit has in flight: 512 threads with 48 or 64 bytes each, 1024 with 32.  More
  // is no faster and leaves more partial rows (8192 x 4096 bf16: with dres 52.8 us for 512
  // threads and 57.8 for 1024, without 53.5 and 43.9).
  const int threads = threads_for(cols, cols <= 8192 ? 8 : 16), fill = esize == 4 || dres ? 512 : 1024;
  return {1, 256 * (fill > threads ? fill / threads : 1)};
}
// A workgroup for each compute unit, then four rows at the least to a partial row (bf16, 2048
// columns: 1024 rows 10.7 us, 14.0 with a workgroup for each of them; 2051 rows 13.5 and 16.1).
int backward_groups(int64_t rows, int64_t cols, int64_t esize, bool dres) {
  const Split d = backward_split(cols, esize, dres);
  const int64_t all = (rows + d.rows - 1) / d.rows, few = (rows + 3) / 4 > 256 ? (rows + 3) / 4 : 256;
  const int64_t groups = all < few ? all : few;
  return (int)(groups < d.most ? groups : d.most);
}

template <typename T, typename W, int K>
void backward_held(const Backward& a, int groups, hipStream_t s) {
  constexpr int per = K * kVec<T>, most = 1024 * per * sizeof(W);
  const bool full = a.cols % (64 * per) == 0;
  auto kernel = a.dres ? backward_kernel<T, W, K, true, true> : backward_kernel<T, W, K, true, false>;
  if constexpr (per == 8 || sizeof(T) == 2)
    if (!full)
      kernel = a.dres ? backward_kernel<T, W, K, false, true> : backward_kernel<T, W, K, false, false>;
  const int threads = threads_for(a.cols, per), bytes = threads * per * (int)sizeof(W);
  if (most > kPlainLds && bytes > kPlainLds)
    (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, most);
  kernel<<<groups, threads, bytes, s>>>(a);
}
template <typename T, typename W>
void backward(const Backward& a, int groups, void* dweight, void* dbias, hipStream_t s) {
  constexpr int N = kVec<T>, k = kUnits<T>;
  if (groups == 0) {
  } else if (!backward_held(a.cols, sizeof(T))) {
    const dim3 grid((unsigned)((a.cols + 2047) / 2048), (unsigned)groups);
    backward_long_columns_kernel<T><<<grid, 256, 0, s>>>(a);
    backward_long_kernel<T, W><<<(unsigned)(a.rows < 512 ? a.rows : 512), 1024, 0, s>>>(a);
  } else if (a.cols <= 512) {
    with_lanes<N>(a.cols, [&](auto lanes, auto e) {
      backward_wave_kernel<T, W, 1024, k, decltype(e)::value, decltype(lanes)::value>
          <<<groups, 1024, 0, s>>>(a);
    });
  } else if (backward_wave(a.cols, sizeof(T))) {
    if constexpr (sizeof(T) == 2)
      with_end(a.cols == 1024 ? kFull : a.cols % N == 0 ? kWhole : kCut, [&](auto e) {
        backward_wave_kernel<T, W, 512, 2 * k, decltype(e)::value, 64><<<groups, 512, 0, s>>>(a);
      });
  } else if (a.cols <= 8192) {
    backward_held<T, W, k>(a, groups, s);
  } else {
    backward_held<T, W, 2 * k>(a, groups, s);
  }
  const int64_t columns = ((int64_t)a.cols + 63) / 64, most = 1 << 20;    // threads stay below 2^32
  const dim3 grid((unsigned)(columns < most ? columns : most), dbias ? 2 : 1);
  column_sums_kernel<W><<<grid, 1024, 0, s>>>(a.partial, groups, a.cols, (W*)dweight, (W*)dbias);
}

constexpr int64_t kMaxCols = int64_t(1) << 30;

}  // namespace

__global__ void clear_words(uint32_t* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0u;
}
nvfp4_status clear(uint32_t* p, int64_t n, hipStream_t stream) {
  if (n <= 0) return NVFP4_OK;
  clear_words<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(p, n);
  return launched();
}

}  // namespace train

using namespace train;

NVFP4_EXPORT int nvfp4_train_abi_version(void) { return NVFP4_TRAIN_ABI_VERSION; }

NVFP4_EXPORT const char* nvfp4_train_status_str(nvfp4_status st) {
  switch ((int)st) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_NULL: return "null pointer argument";
    case NVFP4_ERR_SHAPE: return "bad shape or row stride";
    case NVFP4_ERR_ENUM: return "type or state kind out of range";
    case NVFP4_ERR_ALIGN: return "pointer not aligned to its element type (workspace: 16 B)";
    case NVFP4_ERR_ALIAS: return "overlapping arguments";
    case NVFP4_ERR_HIP: return "HIP kernel launch failed";
    case (int)NVFP4_ERR_VALUE: return "a number is outside its range";
  }
  return "unknown status";
}

NVFP4_EXPORT nvfp4_status nvfp4_layernorm_forward(
    const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
    const void* weight, const void* bias, int64_t rows, int64_t cols, nvfp4_type type,
    nvfp4_type wtype, int center, float eps, void* y, void* h, float* mean, float* rstd,
    float* out_amax, hipStream_t stream) {
  if (!known(type) || !known(wtype)) return NVFP4_ERR_ENUM;
  if (cols > kMaxCols || !shape_ok(rows, cols, x_stride)) return NVFP4_ERR_SHAPE;
  if (residual && !shape_ok(rows, cols, residual_stride)) return NVFP4_ERR_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return NVFP4_ERR_VALUE;
  if (!weight || (!!residual != !!h) || (center && rows && !mean)) return NVFP4_ERR_NULL;
  if (rows && (!x || !y || !rstd)) return NVFP4_ERR_NULL;
  const int64_t es = size_of(type), ws = size_of(wtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(h, es) ||
      !aligned(weight, ws) || !aligned(bias, ws) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(out_amax, 4))
    return NVFP4_ERR_ALIGN;
  const Range in[] = {range(x, extent(rows, cols, x_stride, es)),
                      range(residual, extent(rows, cols, residual_stride, es)),
                      range(weight, cols * ws), range(bias, cols * ws)};
  const Range out[] = {range(y, extent(rows, cols, cols, es)), range(h, extent(rows, cols, cols, es)),
                       range(center ? mean : nullptr, rows * 4), range(rstd, rows * 4),
                       range(out_amax, 4)};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 4; ++i) {
      const bool same = (i == 0 && x_stride == cols && (o == 1 ? h == x : o == 0 && !h && y == x)) ||
                        (i == 1 && o == 1 && residual_stride == cols && h == residual);
      if (!same && overlap(out[o], in[i])) return NVFP4_ERR_ALIAS;
    }
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return NVFP4_ERR_ALIAS;
  }
  (void)hipGetLastError();
  if (out_amax) {
    const nvfp4_status st = clear((uint32_t*)out_amax, 1, stream);
    if (st != NVFP4_OK) return st;
  }
  if (rows == 0) return NVFP4_OK;
  const Forward a = {x, residual, weight, bias, y, h, mean, rstd, (uint32_t*)out_amax,
                     x_stride, residual_stride, rows, (int)cols, center ? 1 : 0, eps};
  if (type == NVFP4_T_BF16 && wtype == NVFP4_T_BF16) forward<bf16, bf16>(a, stream);
  else if (type == NVFP4_T_BF16) forward<bf16, float>(a, stream);
  else if (wtype == NVFP4_T_BF16) forward<float, bf16>(a, stream);
  else forward<float, float>(a, stream);
  return launched();
}

NVFP4_EXPORT int64_t nvfp4_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols < 1 || cols > kMaxCols) return 0;
  const int a = backward_groups(rows, cols, 2, false), b = backward_groups(rows, cols, 4, false);
  return (int64_t)(a > b ? a : b) * 2 * cols * 4;
}

NVFP4_EXPORT nvfp4_status nvfp4_layernorm_backward(const void* dy, const void* h,
                                                   const void* weight, const float* mean,
                                                   const float* rstd, const void* dres,
                                                   int64_t rows, int64_t cols, nvfp4_type type,
                                                   nvfp4_type wtype, void* dx, void* dweight,
                                                   void* dbias, void* workspace,
                                                   hipStream_t stream) {
  if (!known(type) || !known(wtype)) return NVFP4_ERR_ENUM;
  if (cols > kMaxCols || !shape_ok(rows, cols, cols)) return NVFP4_ERR_SHAPE;
  if (!weight || !dweight) return NVFP4_ERR_NULL;
  if (rows && (!dy || !h || !rstd || !dx || !workspace)) return NVFP4_ERR_NULL;
  const int64_t es = size_of(type), ws = size_of(wtype), n = extent(rows, cols, cols, es);
  if (!aligned(dy, es) || !aligned(h, es) || !aligned(dres, es) || !aligned(dx, es) ||
      !aligned(weight, ws) || !aligned(dweight, ws) || !aligned(dbias, ws) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const Range in[] = {range(dy, n), range(dres, n), range(h, n), range(weight, cols * ws),
                      range(mean, rows * 4), range(rstd, rows * 4)};
  const Range out[] = {range(dx, n), range(dweight, cols * ws), range(dbias, cols * ws),
                       range(workspace, nvfp4_layernorm_backward_workspace(rows, cols))};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 6; ++i)
      if (!(o == 0 && i < 2 && dx == (i ? dres : dy)) && overlap(out[o], in[i]))
        return NVFP4_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return NVFP4_ERR_ALIAS;
  }
  (void)hipGetLastError();
  const Backward a = {dy, h, weight, mean, rstd, dres, dx, (float*)workspace, rows, (int)cols,
                      dbias ? 2 : 1};
  const int groups = rows ? backward_groups(rows, cols, es, dres != nullptr) : 0;
  if (type == NVFP4_T_BF16 && wtype == NVFP4_T_BF16) backward<bf16, bf16>(a, groups, dweight, dbias, stream);
  else if (type == NVFP4_T_BF16) backward<bf16, float>(a, groups, dweight, dbias, stream);
  else if (wtype == NVFP4_T_BF16) backward<float, bf16>(a, groups, dweight, dbias, stream);
  else backward<float, float>(a, groups, dweight, dbias, stream);
  return launched();
}
