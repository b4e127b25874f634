// Layer norm forward and backward for gfx950 (include/nvfp4_train.h defines the operation).
//
// A row is held in registers by one wavefront (up to 1024 columns) or one workgroup (up to
// 16384), eight consecutive elements per lane and step, so that x is read once: the mean and then
// the centred sum of squares come from the registers.  Longer rows are read again for each of
// the three steps.  The backward pass keeps, next to the row, its share of the column sums
// (dweight, dbias) in registers over all the rows that a workgroup takes, leaves them as one
// partial row per workgroup in the workspace, and a second launch adds those in a fixed order.
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
  float* partial;     // [groups][2][cols]: dweight, dbias
  int64_t rows;
  int cols;
};

// The columns of a held row: known to be in 8 .. TPR * K * 8, so that offsets take 32 bits.
template <int TPR, int K>
__device__ __forceinline__ uint32_t held_cols(int cols) {
  __builtin_assume(cols >= 8 && cols <= TPR * K * 8);
  return (uint32_t)cols;
}
// Which row of the workgroup's this thread is at, as a scalar.
template <int TPR>
__device__ __forceinline__ uint32_t wave_of() {
  return TPR < 256 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0u;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// A workgroup's part of the tensor maximum: on the bits, where inf and NaN sort above the rest.
template <int WAVES>
__device__ __forceinline__ void publish_amax(uint32_t m, uint32_t* amax, uint32_t* slots) {
  m = reduce_group<WAVES>(m, Max(), slots);
  if (threadIdx.x == 0 && m != 0) atomicMax(amax, m);
}

// One row: TPR lanes hold K vectors each.  With TPR == 64 a workgroup takes 4 rows at a time.
template <typename T, typename W, int TPR, int K, End E>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void forward_kernel(const Forward a) {
  constexpr int WAVES = TPR / 64, ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float slots[2][WAVES];
  __shared__ uint32_t top[TPR < 256 ? 4 : WAVES];
  const uint32_t lane = threadIdx.x % TPR, cols = held_cols<TPR, K>(a.cols);
  const float inv = 1.0f / (float)a.cols;
  uint32_t most = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + wave_of<TPR>(); row < a.rows;
       row += (int64_t)gridDim.x * ROWS) {
    const T* x = (const T*)a.x + row * a.x_stride;
    float v[K][8];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Vec8<T> q = load_vec<E>(x, (k * TPR + lane) * 8, cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = q[i];
    }
    if (a.residual) {
      const T* r = (const T*)a.residual + row * a.residual_stride;
      T* h = (T*)a.h + row * a.cols;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint32_t at = (k * TPR + lane) * 8;
        const Vec8<T> q = load_vec<E>(r, at, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] += q[i];
        const Vec8<T> s = make_vec(v[k], T());
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = s[i];
        store_vec<E>(h, at, cols, s);
      }
    }
    float mean = 0.0f;
    if (a.center) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[k][i];
      mean = reduce_group<WAVES>(sum, Sum(), slots[0]) * inv;
    }
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = (k * TPR + lane) * 8 + i < cols ? v[k][i] - mean : 0.0f;
        sq += d * d;
      }
    const float var = reduce_group<WAVES>(sq, Sum(), slots[1]) * inv;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (lane == 0) {
      a.rstd[row] = rstd;
      if (a.center) a.mean[row] = mean;
    }
    T* y = (T*)a.y + row * a.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t at = (k * TPR + lane) * 8;
      const Vec8<W> w = load_vec<E>((const W*)a.weight, at, cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = (v[k][i] - mean) * rstd * w[i];
      if (a.bias) {
        const Vec8<W> b = load_vec<E>((const W*)a.bias, at, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] += b[i];
      }
      const Vec8<T> out = make_vec(v[k], T());
      store_vec<E>(y, at, cols, out);
      if (a.amax) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < cols) most = max(most, abs_bits(out[i]));
      }
    }
    if (WAVES > 1) __syncthreads();     // the slots are free for the next row
  }
  if (a.amax) publish_amax<(TPR < 256 ? 4 : WAVES)>(most, a.amax, top);
}

// Rows longer than the registers hold (and those under 8 columns): three passes over the row.
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
      const Vec8<T> q = load_vec<kAny>(x, at, (int64_t)a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q[i];
      if (r) {
        const Vec8<T> p = load_vec<kAny>(r, at, (int64_t)a.cols);
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
      if (r) store_vec<kAny>((T*)a.h + row * a.cols, at, (int64_t)a.cols, make_vec(v, T()));
      const Vec8<W> w = load_vec<kAny>((const W*)a.weight, at, (int64_t)a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (v[i] - mean) * rstd * w[i];
      if (a.bias) {
        const Vec8<W> b = load_vec<kAny>((const W*)a.bias, at, (int64_t)a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
      }
      const Vec8<T> out = make_vec(v, T());
      store_vec<kAny>((T*)a.y + row * a.cols, at, (int64_t)a.cols, out);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < a.cols) most = max(most, abs_bits(out[i]));
    }
    __syncthreads();
  }
  if (a.amax) publish_amax<16>(most, a.amax, top);
}

template <typename T, typename W, int TPR, int K, End E>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void backward_kernel(const Backward a) {
  constexpr int WAVES = TPR / 64, ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float slots[2][2][WAVES];
  const uint32_t lane = threadIdx.x % TPR, sub = wave_of<TPR>();
  const uint32_t cols = held_cols<TPR, K>(a.cols);
  const float inv = 1.0f / (float)a.cols;
  // 1024 threads have 128 registers each: there the weights are read again for every use
  constexpr bool HOLD = TPR < 1024;
  auto weight = [&](int k) {
    uint32_t at = (k * TPR + lane) * 8;
    if (!HOLD) asm volatile("" : "+v"(at));          // not taken out of the row loop
    return load_vec<E>((const W*)a.weight, at, cols);
  };
  Vec8<W> held[HOLD ? K : 1];
  float dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (HOLD) held[k] = weight(k);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + sub; row < a.rows;
       row += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    Vec8<T> dy[K], h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t at = (k * TPR + lane) * 8;
      dy[k] = load_vec<E>((const T*)a.dy + row * a.cols, at, cols);
      h[k] = load_vec<E>((const T*)a.h + row * a.cols, at, cols);
    }
    const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Vec8<W> w = HOLD ? held[HOLD ? k : 0] : weight(k);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (h[k][i] - mean) * rstd, g = dy[k][i] * w[i];
        s1 += g;
        s2 = fmaf(g, xh, s2);
        dw[k][i] = fmaf(dy[k][i], xh, dw[k][i]);
        db[k][i] += dy[k][i];
        asm volatile("" : "+v"(dw[k][i]), "+v"(db[k][i]));   // here, not at the loop's end
      }
    }
    // the slots of two rows in turn: one barrier per row is enough
    s1 = reduce64(s1, Sum());
    s2 = reduce64(s2, Sum());
    if (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) {
        slots[turn][0][threadIdx.x >> 6] = s1;
        slots[turn][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = reduce_few<WAVES>(slots[turn][0][threadIdx.x % WAVES], Sum());
      s2 = reduce_few<WAVES>(slots[turn][1][threadIdx.x % WAVES], Sum());
    }
    const float c1 = a.mean ? s1 * inv : 0.0f, c2 = s2 * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t at = (k * TPR + lane) * 8;
      float d[8];
      opaque(dy[k]);      // unpacked again from here: the floats need not live across the sums
      opaque(h[k]);
      const Vec8<W> w = HOLD ? held[HOLD ? k : 0] : weight(k);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (h[k][i] - mean) * rstd, g = dy[k][i] * w[i];
        d[i] = rstd * (g - c1 - xh * c2);
      }
      if (a.dres) {
        const Vec8<T> r = load_vec<E>((const T*)a.dres + row * a.cols, at, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += r[i];
      }
      store_vec<E>((T*)a.dx + row * a.cols, at, cols, make_vec(d, T()));
    }
  }
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
  if (ROWS > 1) {       // the four wavefronts' sums, added in their order
    __shared__ float part[ROWS > 1 ? ROWS : 1][2][ROWS > 1 ? TPR * K * 8 : 1];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        part[sub][0][(k * TPR + lane) * 8 + i] = dw[k][i];
        part[sub][1][(k * TPR + lane) * 8 + i] = db[k][i];
      }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < cols; c += blockDim.x) {
      float s = 0.0f, t = 0.0f;
      for (int r = 0; r < ROWS; ++r) {
        s += part[r][0][c];
        t += part[r][1][c];
      }
      out[c] = s;
      out[cols + c] = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t at = (k * TPR + lane) * 8;
      store_vec<E>(out, at, cols, make_vec(dw[k], 0.0f));
      store_vec<E>(out + cols, at, cols, make_vec(db[k], 0.0f));
    }
  }
}

// Rows longer than the registers hold (and those under 8 columns): dx from two passes over the row ...
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
      const Vec8<T> d = load_vec<kAny>(dy, at, (int64_t)a.cols), x = load_vec<kAny>(h, at, (int64_t)a.cols);
      const Vec8<W> w = load_vec<kAny>((const W*)a.weight, at, (int64_t)a.cols);
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
      const Vec8<T> d = load_vec<kAny>(dy, at, (int64_t)a.cols), x = load_vec<kAny>(h, at, (int64_t)a.cols);
      const Vec8<W> w = load_vec<kAny>((const W*)a.weight, at, (int64_t)a.cols);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = rstd * (d[i] * w[i] - c1 - (x[i] - mean) * rstd * c2);
      if (a.dres) {
        const Vec8<T> r = load_vec<kAny>((const T*)a.dres + row * a.cols, at, (int64_t)a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      store_vec<kAny>((T*)a.dx + row * a.cols, at, (int64_t)a.cols, make_vec(v, T()));
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
    const Vec8<T> d = load_vec<kAny>((const T*)a.dy + row * a.cols, at, (int64_t)a.cols);
    const Vec8<T> x = load_vec<kAny>((const T*)a.h + row * a.cols, at, (int64_t)a.cols);
    const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = fmaf(d[i], (x[i] - mean) * rstd, dw[i]);
      db[i] += d[i];
    }
  }
  float* out = a.partial + (int64_t)blockIdx.y * 2 * a.cols;
  store_vec<kAny>(out, at, (int64_t)a.cols, make_vec(dw, 0.0f));
  store_vec<kAny>(out + a.cols, at, (int64_t)a.cols, make_vec(db, 0.0f));
}

// dweight (y == 0) and dbias (y == 1): a lane adds a column, the 16 wavefronts of a workgroup
// take every 16th partial row, and their sums are added in order.
template <typename W>
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ partial,
                                                           int groups, int cols, W* dweight,
                                                           W* dbias) {
  __shared__ float part[16][64];
  W* out = blockIdx.y ? dbias : dweight;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols) {
    const float* p = partial + (int64_t)blockIdx.y * cols + c;
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) s += p[(int64_t)g * 2 * cols];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    out[c] = from_f32<W>(s);
  }
}

// ----------------------------------------------------------------------------------- host
constexpr int64_t kForwardGroups = 2048;

// Rows that a workgroup holds.
bool held(int64_t cols) { return cols >= 8 && cols <= kMaxHeldCols; }

template <typename T, typename W, int TPR, int K, End E>
void forward_held(const Forward& a, hipStream_t s) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  const int64_t groups = (a.rows + ROWS - 1) / ROWS;
  forward_kernel<T, W, TPR, K, E><<<(unsigned)(groups < kForwardGroups ? groups : kForwardGroups),
                                    TPR < 256 ? 256 : TPR, 0, s>>>(a);
}
template <typename T, typename W, End E>
void forward(const Forward& a, hipStream_t s) {
  if (a.cols <= 512) return forward_held<T, W, 64, 1, E>(a, s);
  if (a.cols <= 1024) return forward_held<T, W, 64, 2, E>(a, s);
  if (a.cols <= 2048) return forward_held<T, W, 256, 1, E>(a, s);
  if (a.cols <= 4096) return forward_held<T, W, 256, 2, E>(a, s);
  if (a.cols <= 8192) return forward_held<T, W, 512, 2, E>(a, s);
  forward_held<T, W, 1024, 2, E>(a, s);
}
template <typename T, typename W>
void forward(const Forward& a, hipStream_t s) {
  if (!held(a.cols)) {
    const int64_t groups = a.rows < kForwardGroups ? a.rows : kForwardGroups;
    forward_long_kernel<T, W><<<(unsigned)groups, 1024, 0, s>>>(a);
  } else if (a.cols % 8) {
    forward<T, W, kCut>(a, s);
  } else {
    forward<T, W, kWhole>(a, s);
  }
}

// Partial rows of the column sums, which is also the grid of the backward pass.
int backward_groups(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 1024 ? 4 : 1;
  const int64_t groups = (rows + per - 1) / per;
  const int64_t most = cols <= 4096 ? 512 : 256;
  return (int)(groups < most ? groups : most);
}

template <typename T, typename W, int TPR, int K, End E>
void backward_held(const Backward& a, int groups, hipStream_t s) {
  backward_kernel<T, W, TPR, K, E><<<groups, TPR < 256 ? 256 : TPR, 0, s>>>(a);
}
template <typename T, typename W, End E>
void backward(const Backward& a, int groups, hipStream_t s) {
  if (a.cols <= 512) return backward_held<T, W, 64, 1, E>(a, groups, s);
  if (a.cols <= 1024) return backward_held<T, W, 64, 2, E>(a, groups, s);
  if (a.cols <= 2048) return backward_held<T, W, 256, 1, E>(a, groups, s);
  if (a.cols <= 4096) return backward_held<T, W, 256, 2, E>(a, groups, s);
  if (a.cols <= 8192) return backward_held<T, W, 512, 2, E>(a, groups, s);
  backward_held<T, W, 1024, 2, E>(a, groups, s);
}
template <typename T, typename W>
void backward(const Backward& a, int groups, void* dweight, void* dbias, hipStream_t s) {
  if (groups == 0) {
  } else if (!held(a.cols)) {
    const dim3 grid((unsigned)((a.cols + 2047) / 2048), (unsigned)groups);
    backward_long_columns_kernel<T><<<grid, 256, 0, s>>>(a);
    backward_long_kernel<T, W><<<(unsigned)(a.rows < 512 ? a.rows : 512), 1024, 0, s>>>(a);
  } else if (a.cols % 8) {
    backward<T, W, kCut>(a, groups, s);
  } else {
    backward<T, W, kWhole>(a, groups, s);
  }
  const dim3 grid((unsigned)((a.cols + 63) / 64), dbias ? 2 : 1);
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
  return (int64_t)backward_groups(rows, cols) * 2 * cols * 4;
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
  const Backward a = {dy, h, weight, mean, rstd, dres, dx, (float*)workspace, rows, (int)cols};
  const int groups = rows ? backward_groups(rows, cols) : 0;
  if (type == NVFP4_T_BF16 && wtype == NVFP4_T_BF16) backward<bf16, bf16>(a, groups, dweight, dbias, stream);
  else if (type == NVFP4_T_BF16) backward<bf16, float>(a, groups, dweight, dbias, stream);
  else if (wtype == NVFP4_T_BF16) backward<float, bf16>(a, groups, dweight, dbias, stream);
  else backward<float, float>(a, groups, dweight, dbias, stream);
  return launched();
}
