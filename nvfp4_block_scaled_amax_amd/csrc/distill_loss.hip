// The distillation loss KL(softmax(teacher / T) || softmax(student / T)) per row and its
// gradient for gfx950 (include/nvfp4_train.h defines the operation).
//
// Each row is read twice: once for both sums of exponentials, and once, from the caches where
// the row fits, for the loss and the gradient.  All exponentials are powers of two,
//   2^(fma(x, c, -R)),  c = log2(e) / T,
// with R the rounded product of c and some entry near the row's largest: whatever float R is, it
// cancels exactly between an entry and its sum, so one fma per exponent loses nothing.
//   first pass:   Zq = sum 2^(fma(s, c, -Rq)), Zp = sum 2^(fma(t, c, -Rp)); a lane moves its R
//                 only when an entry passes it by 2^16, which is rare after the first steps
//   in between:   Rq moves by log2(Zq / Zp) (the rounding of that sum is kept), so that both
//                 probabilities come out over the same 1 / Zp and log2 p - log2 q is X - Y
//   second pass:  Y, X the exponents of both; q - p = (2^Y - 2^X) / Zp;
//                 loss = sum (q - p) + ln 2 sum p (X - Y)
// The sum of q - p is zero in exact arithmetic.  With it, the terms are all >= 0, and an error
// that q's normalization brings into both its parts cancels to second order: the loss of a
// student near its teacher keeps its precision.
//
// Where c x is 2^14 or more (logits of 11000, a temperature of 1/100; rows of the lowest finite value,
// where it overflows) the fast form has too few bits for what lies between R and log2 Z, or no sum;
// such a row is done again with (x - max) c, which keeps the differences, element by element (a call
// of such rows alone, 4096 x 128000 bf16, 3.4 ms).
//
// With rows for the compute units a workgroup takes a row and holds what it can of it between
// the passes: 64 registers per thread, and up to 128 KB of a compute unit's shared memory.  The
// more workgroups share a compute unit the better their passes overlap, so a row gets as few
// threads as can hold it, and no more registers than it fills, since what is loaded past its end
// is not free (8192 x 1000 bf16 14.3 us with 128 threads of one vector each, 19.5 with 256, 31 with
// 256 of eight; 8192 x 6000 52 with four vectors, 58 with eight; 4000 x 8191 with four 43, 59 with eight):
// 128 threads to 1024 bf16 logits, 256 (4 workgroups a compute unit) to 16384, 512 (2) to
// 32768, or 49152 with shared memory; and 512 up to twice that, the rest being read again, before
// 1024 (1), which hold 98304, or with 88 registers per thread 122880, where the row has as many.
// bf16, us per call: 8192 x 32000 270 with 512 threads, 437 with 1024; 4096 x 60000 330 and 383,
// 98000 534 and 556, 128000 686 and 649; 88 registers 110000 594 and 577 with 64, 128000 649 and
// 657, 200192 1050 and 1120.  Without holding anything, 4096 x 128000 took 805 us with one
// workgroup a compute unit and 985 with two, whose rows together pass the last-level cache: the
// second reading is what costs, not the exponentials.  Loads and stores bypass the caches (660
// against 692 us; the rest of a long row, which is read again, does not).  Rows of an odd length
// start at odd addresses, where 16-byte accesses are slow (4096 x 127999: 827 us).  Starting each row's units
// at a 16-byte boundary (707 us) would let its last bits depend on where it lies; loading from the
// boundary below and shifting words into the same units would not, and is not built.
//
// What bounds it is the memory: 4096 x 128000 bf16 reads and writes 3146 MB in 647 us, 4.86 TB/s,
// where a copy of that size runs at 4.8.  Without the gradient 541 us (2097 MB read, 3.9 TB/s).
//
// Where the rows are few and long, a row is split over several workgroups in two launches:
// partial statistics, then gradient and partial losses, which the last workgroup of a row adds
// in order.
#include "train_common.h"

namespace train {
namespace {

constexpr int kThreads = 1024;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e38f;

struct Distill {
  const void* student;
  const void* teacher;
  const float* weight;
  float* loss;
  void* grad;
  float* stats;           // split rows: [rows][splits][2] of Split
  float* part;            // split rows: [rows][splits] losses
  uint32_t* arrived;      // split rows: [rows]
  int64_t student_stride, teacher_stride, grad_stride, rows;
  uint32_t vocab;
  uint32_t split_size;    // elements of a split, a multiple of 8
  int splits;
  float c, temperature;   // log2(e) / T, T
};

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kSlack = 16.0f;      // how far (in powers of two) entries may pass a lane's R

// A unit is what a lane loads of both logits at once: eight elements, or four where both are
// binary32, so that a wavefront's 16-byte loads are next to each other.
template <typename S, typename T>
constexpr int kUnit = sizeof(S) == 4 && sizeof(T) == 4 ? 4 : 8;
// sum 2^(fma(x, c, -r)).  An empty one has r = the lowest finite value and sum 0; an entry of
// -inf adds 0 to any.  r is c times some entry, rounded; m is the largest entry.
struct Stat {
  float r, z, m;
  __device__ __forceinline__ void join(Stat o) {
    m = fmaxf(m, o.m);
    const float top = fmaxf(r, o.r);
    z = z * exp2_(r - top) + o.z * exp2_(o.r - top);
    r = top;
  }
  template <typename T, int N>
  __device__ __forceinline__ void add(const Vec<T, N>& v, float c) {
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
    m = fmaxf(m, top);
    top *= c;
    if (top > r + kSlack) {
      z *= exp2_(r - top);
      r = top;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) z += exp2_(fmaf(v[i], c, -r));
  }
  // Whether the fast form can go on from here: z is a number that a ratio has room for (a row's is
  // between 2^-1 and 2^16 times its length while r is small), and r is so small that log2 of a ratio
  // added to it is rounded by 2^-11 at the most, whose square row_grad leaves out.
  __device__ __forceinline__ bool good() const {
    return z > 0x1p-60f && z < 0x1p60f && fabsf(r) < 16384.0f;
  }
};

// One entry: its term is 1 but for what r is rounded by (0 for one near the lowest value).
__device__ __forceinline__ Stat single(float x, float c) {
  const float r = fmaxf(x * c, kLowest);
  return Stat{r, exp2_(fmaf(x, c, -r)), x};
}

// The same with exact differences: max x, and sum 2^((x - max) c).
struct Exact {
  float m, z;
  __device__ __forceinline__ void join(Exact o, float c) {
    const float top = fmaxf(m, o.m);
    z = z * exp2_((m - top) * c) + o.z * exp2_((o.m - top) * c);
    m = top;
  }
};

// r and z of both over a workgroup of WAVES wavefronts; every thread gets them.
template <int WAVES>
__device__ __forceinline__ void join_group(Stat& q, Stat& p, float (*slots)[4]) {
  const float rq = reduce64(q.r, Max()), rp = reduce64(p.r, Max());
  const float zq = reduce64(q.z * exp2_(q.r - rq), Sum());
  const float zp = reduce64(p.z * exp2_(p.r - rp), Sum());
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    slots[wave][0] = rq;
    slots[wave][1] = zq;
    slots[wave][2] = rp;
    slots[wave][3] = zp;
  }
  __syncthreads();
  const float* mine = slots[threadIdx.x % WAVES];
  q.r = reduce_few<WAVES>(mine[0], Max());
  p.r = reduce_few<WAVES>(mine[2], Max());
  q.z = reduce_few<WAVES>(mine[1] * exp2_(mine[0] - q.r), Sum());
  p.z = reduce_few<WAVES>(mine[3] * exp2_(mine[2] - p.r), Sum());
}

// A row's elements [lo, hi) as the threads of a workgroup hold them between the two passes.
// The first REGS units of each thread stay in registers, the next LDS ones in shared memory, the
// rest is read again; the up to 7 elements behind the last unit are single threads'.
template <typename S, typename T, int THREADS, int REGS, int LDS>
struct Row {
  const S* s;
  const T* t;
  uint32_t lo, hi, whole;      // whole: end of the last unit
  static constexpr int N = kUnit<S, T>;
  typedef Vec<S, N> VS;
  typedef Vec<T, N> VT;
  VS a[REGS > 0 ? REGS : 1];
  VT b[REGS > 0 ? REGS : 1];

  static constexpr int64_t kBytes = (int64_t)LDS * THREADS * N * (sizeof(S) + sizeof(T));

  __device__ __forceinline__ Row(const S* s_, const T* t_, uint32_t lo_, uint32_t hi_)
      : s(s_), t(t_), lo(lo_), hi(hi_), whole(lo_ + (hi_ - lo_) / N * N) {}
  __device__ __forceinline__ uint32_t place(int k) const {
    return lo + (k * THREADS + threadIdx.x) * N;
  }
  // where a vector is loaded from: one past the row's end from its beginning, at a 16-byte boundary
  // (unused, but no branch stands between the loads; 2000 x 17001 bf16 53 us, 62 from odd addresses)
  template <typename V>
  __device__ __forceinline__ uint32_t inside(const V* row, int k) const {
    const uint32_t at = place(k);
    const uint32_t even = lo + (uint32_t)(-(intptr_t)(row + lo) & 15) / sizeof(V);
    return at < whole ? at : even + N <= hi ? even : lo;
  }
  static __device__ __forceinline__ VS* lds_a(void* lds, int k) {
    return (VS*)lds + k * THREADS + threadIdx.x;
  }
  static __device__ __forceinline__ VT* lds_b(void* lds, int k) {
    return (VT*)((VS*)lds + LDS * THREADS) + k * THREADS + threadIdx.x;
  }

  // First pass: f(vector of s, vector of t) for every vector, then g(s, t) for the singles.
  template <typename F, typename G>
  __device__ __forceinline__ void load(void* lds, F f, G g) {
    if (lo < whole) {
#pragma unroll
      for (int k = 0; k < REGS; ++k) {
        a[k] = load_vec<N, true>(s + inside(s, k));
        b[k] = load_vec<N, true>(t + inside(t, k));
      }
#pragma unroll
      for (int k = 0; k < LDS; ++k) {
        const VS x = load_vec<N, true>(s + inside(s, REGS + k));
        const VT y = load_vec<N, true>(t + inside(t, REGS + k));
        *lds_a(lds, k) = x;
        *lds_b(lds, k) = y;
        if (place(REGS + k) < whole) f(x, y);
      }
#pragma unroll
      for (int k = 0; k < REGS; ++k)
        if (place(k) < whole) f(a[k], b[k]);
    }
    for (uint32_t at = place(REGS + LDS); at < whole; at += THREADS * N)
      f(load_vec<N>(s + at), load_vec<N>(t + at));
    const uint32_t at = whole + threadIdx.x;
    if (at < hi) g(to_f32(s[at]), to_f32(t[at]));
  }
  // Second pass: f(place, vectors), g(place, s, t).
  template <typename F, typename G>
  __device__ __forceinline__ void again(void* lds, F f, G g) {
#pragma unroll
    for (int k = 0; k < REGS; ++k)
      if (place(k) < whole) {
        opaque(a[k]);       // unpacked again: the floats do not stay in registers, too
        opaque(b[k]);
        f(place(k), a[k], b[k]);
      }
#pragma unroll
    for (int k = 0; k < LDS; ++k)
      if (place(REGS + k) < whole) f(place(REGS + k), *lds_a(lds, k), *lds_b(lds, k));
    for (uint32_t at = place(REGS + LDS); at < whole; at += THREADS * N)
      f(at, load_vec<N>(s + at), load_vec<N>(t + at));
    const uint32_t at = whole + threadIdx.x;
    if (at < hi) g(at, to_f32(s[at]), to_f32(t[at]));
  }
};

// Sums of a row's elements.
template <int THREADS, typename R>
__device__ __forceinline__ void row_stats(R& row, void* lds, float c, Stat& q, Stat& p,
                                          float (*slots)[4]) {
  q = p = Stat{kLowest, 0.0f, kLowest};
  row.load(lds, [&](const auto& a, const auto& b) { q.add(a, c), p.add(b, c); },
           [&](float a, float b) {
             if (a != -INFINITY) q.join(single(a, c));
             if (b != -INFINITY) p.join(single(b, c));
           });
  join_group<THREADS / 64>(q, p, slots);
}

// The same with exact differences, for the rare row.
template <int THREADS, typename S>
__device__ __forceinline__ Exact row_exact(const S* s, uint32_t lo, uint32_t hi, float c, float* slots) {
  Exact e{kLowest, 0.0f};
#pragma unroll 1
  for (uint32_t at = lo + threadIdx.x; at < hi; at += THREADS) {
    const float a = to_f32(s[at]);
    if (a != -INFINITY) e.join(Exact{a, 1.0f}, c);
  }
  const float m = reduce_group<THREADS / 64>(e.m, Max(), slots);
  const float z = e.z * exp2_((e.m - m) * c);
  __syncthreads();
  e = Exact{m, reduce_group<THREADS / 64>(z, Sum(), slots)};
  __syncthreads();
  return e;
}

// An entry that the student excludes by a finite value (the type's lowest, -1e36): from X - Y = kFar on,
// Zp p (X - Y) may overflow where the loss does not, and Y itself does.  There p (log p - log q) is -p s / T,
// infinite where s is: the rest of X - Y is no part of it in 32 bits.  The sum of the loss is kept
// kDown times, where Zp p is below 1.
constexpr float kFar = 0x1p100f, kDown = 0x1p-64f;
__device__ __forceinline__ float far_part(float ep, float c, float s) {
  return ep * (c * kLn2) * (-s * kDown);
}

// The second pass: writes the gradient, returns the workgroup's part of the loss (with the row's
// weight) to every thread.
template <int THREADS, typename S, typename R>
__device__ __forceinline__ float row_grad(R& row, void* lds, S* grad, float c, float temperature,
                                          float weight, Stat q, Stat p, float* slots) {
  constexpr int N = R::N;
  // R of the student + log2(Zq / Zp) = r + off, r rounded
  const float by = log2f(q.z / p.z), r = q.r + by;
  const float part = r - q.r, off = (q.r - (r - part)) + (by - part);
  const float scale = weight / (temperature * p.z);
  const float back = 1.0f - off * kLn2;       // 2^-off: |off| <= 2^-11, see good()
  // Zp sum of (q - p) + ln 2 p (X - Y): both parts of a unit meet before they are added to the
  // others, because their sums over the row are far larger than the loss
  float sum = 0.0f;
  row.again(
      lds,
      [&](uint32_t at, const auto& a, const auto& b) {
        float x[N], y[N], g[N], least = INFINITY, flat = 0.0f, bent = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          y[i] = fmaf(a[i], c, -r);
          x[i] = fmaf(b[i], c, -p.r);
          least = fminf(least, fminf(x[i], y[i]));
        }
        if (least < -kFar) {          // log2 p - log2 q counts where p is not 0
          bool far = false;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float eq = exp2_(y[i]), ep = exp2_(x[i]), d = fmaf(eq, back, -ep);
            const float gap = x[i] - y[i];
            far |= gap > kFar && ep != 0.0f;
            bent += ep == 0.0f || gap > kFar ? 0.0f : ep * gap;
            flat += d;
            g[i] = d * scale;
          }
          if (far)            // seldom: read again (not yet written over), there are no registers for them
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
              const float s = to_f32(row.s[at + i]), x = fmaf(to_f32(row.t[at + i]), c, -p.r);
              if (exp2_(x) != 0.0f && x - fmaf(s, c, -r) > kFar) sum += far_part(exp2_(x), c, s);
            }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float eq = exp2_(y[i]), ep = exp2_(x[i]), d = fmaf(eq, back, -ep);
            bent = fmaf(ep, x[i] - y[i], bent);
            flat += d;
            g[i] = d * scale;
          }
        }
        sum = fmaf(kDown, fmaf(kLn2, bent, flat), sum);
        if (grad) store_vec<true>(grad + at, make_vec<S>(g));
      },
      [&](uint32_t at, float a, float b) {
        const float y = fmaf(a, c, -r), x = fmaf(b, c, -p.r);
        const float eq = exp2_(y), ep = exp2_(x), d = fmaf(eq, back, -ep);
        const float gap = x - y;
        if (ep != 0.0f && gap > kFar) sum += far_part(ep, c, a);
        sum = fmaf(kDown, fmaf(kLn2, ep == 0.0f || gap > kFar ? 0.0f : ep * gap, d), sum);
        if (grad) grad[at] = from_f32<S>(d * scale);
      });
  // What is missing: log2 p - log2 q is X - Y + off, and `back` is rounded.  The p and the q add up
  // to 1 each, so that is ln 2 off + (2^-off - back) = 1 - back.
  const float all = reduce_group<THREADS / 64>(weight * (sum / (p.z * kDown)), Sum(), slots);
  return row.lo == 0 ? fmaf(weight, 1.0f - back, all) : all;
}

// The same from the sums with exact differences.
template <int THREADS, typename S, typename T>
__device__ __forceinline__ float row_grad_exact(const S* s, const T* t, S* grad, uint32_t lo,
                                             uint32_t hi, float c, float temperature, float weight,
                                             Exact q, Exact p, float* slots) {
  const float lq = log2f(q.z), lp = log2f(p.z), scale = weight / temperature;
  float sum = 0.0f;
#pragma unroll 1
  for (uint32_t at = lo + threadIdx.x; at < hi; at += THREADS) {
    const float y = (to_f32(s[at]) - q.m) * c - lq, x = (to_f32(t[at]) - p.m) * c - lp;
    const float eq = exp2_(y), ep = exp2_(x), b = to_f32(s[at]);
    // (top - s in halves: it may be up to twice the largest number)
    const float bent = y < -kFar ? ep * (0.5f * q.m - 0.5f * b) * (c * kLn2) * 2.0f : kLn2 * ep * (x - y);
    sum += (eq - ep) + (ep == 0.0f ? 0.0f : bent);
    if (grad) grad[at] = from_f32<S>((eq - ep) * scale);
  }
  return reduce_group<THREADS / 64>(weight * sum, Sum(), slots);
}

template <int THREADS, typename S>
__device__ __forceinline__ void zero_grad(S* grad, uint32_t lo, uint32_t hi) {
  const uint32_t whole = lo + (hi - lo) / 8 * 8;
  const Vec<S, 8> z = zero_vec<S, 8>();
  for (uint32_t at = lo + threadIdx.x * 8; at < whole; at += THREADS * 8) store_vec(grad + at, z);
  if (whole + threadIdx.x < hi) grad[whole + threadIdx.x] = from_f32<S>(0.0f);
}

template <typename S, typename T, int THREADS, int REGS, int LDS>
__global__ __launch_bounds__(THREADS) void row_kernel(const Distill a) {
  __shared__ float slots[THREADS / 64][4], sums[THREADS / 64];
  extern __shared__ __align__(16) char held[];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const float w = a.weight ? a.weight[row] : 1.0f;
  S* grad = a.grad ? (S*)a.grad + row * a.grad_stride : nullptr;
  if (w == 0.0f) {
    if (grad) zero_grad<THREADS>(grad, 0, a.vocab);
    if (threadIdx.x == 0) a.loss[row] = 0.0f;
    return;
  }
  const S* s = (const S*)a.student + row * a.student_stride;
  const T* t = (const T*)a.teacher + row * a.teacher_stride;
  Row<S, T, THREADS, REGS, LDS> r(s, t, 0, a.vocab);
  Stat q, p;
  row_stats<THREADS>(r, held, a.c, q, p, slots);
  float loss;
  if (q.good() && p.good()) {
    loss = row_grad<THREADS>(r, held, grad, a.c, a.temperature, w, q, p, sums);
  } else {
    const Exact eq = row_exact<THREADS>(s, 0, a.vocab, a.c, sums);
    const Exact ep = row_exact<THREADS>(t, 0, a.vocab, a.c, sums);
    loss = row_grad_exact<THREADS>(s, t, grad, 0, a.vocab, a.c, a.temperature, w, eq, ep, sums);
  }
  if (threadIdx.x == 0) a.loss[row] = loss;
}

// What a split of a row leaves for both of its logits: r and z of Stat, m and z of Exact, since
// another split of the row can be one that the fast form has no sum of.
struct Split {
  float r, z, m, e;
};

// A good sum, and the same over 2^((x - m) c): times 2^(r - c m), of which 2^(c m - r) is the
// largest term of the sum (in halves: it may have no reciprocal).
__device__ __forceinline__ Exact to_exact(Stat s, float m, float c) {
  const float half = exp2_(-0.5f * fmaf(m, c, -s.r));
  return Exact{m, s.z * half * half};
}

template <typename S, typename T>
__global__ __launch_bounds__(kThreads) void split_stats_kernel(const Distill a) {
  __shared__ float slots[kThreads / 64][4], sums[kThreads / 64];
  const int64_t row = blockIdx.y;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.arrived[row] = 0u;
  if (a.weight && a.weight[row] == 0.0f) return;
  const uint32_t lo = min(blockIdx.x * a.split_size, a.vocab), hi = min(lo + a.split_size, a.vocab);
  const S* s = (const S*)a.student + row * a.student_stride;
  const T* t = (const T*)a.teacher + row * a.teacher_stride;
  Stat q, p;
  Row<S, T, kThreads, 0, 0> r(s, t, lo, hi);
  row_stats<kThreads>(r, nullptr, a.c, q, p, slots);
  const float mq = reduce_group<kThreads / 64>(q.m, Max(), sums);
  __syncthreads();
  const float mp = reduce_group<kThreads / 64>(p.m, Max(), sums);
  __syncthreads();
  const Exact eq = q.good() ? to_exact(q, mq, a.c) : row_exact<kThreads>(s, lo, hi, a.c, sums);
  const Exact ep = p.good() ? to_exact(p, mp, a.c) : row_exact<kThreads>(t, lo, hi, a.c, sums);
  if (threadIdx.x == 0) {
    Split* out = (Split*)a.stats + (row * a.splits + blockIdx.x) * 2;
    out[0] = Split{q.r, q.z, eq.m, eq.z};
    out[1] = Split{p.r, p.z, ep.m, ep.z};
  }
}

template <typename S, typename T>
__global__ __launch_bounds__(kThreads) void split_grad_kernel(const Distill a) {
  __shared__ float sums[kThreads / 64];
  const int64_t row = blockIdx.y;
  const uint32_t lo = min(blockIdx.x * a.split_size, a.vocab), hi = min(lo + a.split_size, a.vocab);
  const float w = a.weight ? a.weight[row] : 1.0f;
  S* grad = a.grad ? (S*)a.grad + row * a.grad_stride : nullptr;
  if (w == 0.0f) {
    if (grad) zero_grad<kThreads>(grad, lo, hi);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.loss[row] = 0.0f;
    return;
  }
  const S* s = (const S*)a.student + row * a.student_stride;
  const T* t = (const T*)a.teacher + row * a.teacher_stride;
  const Split* in = (const Split*)a.stats + row * a.splits * 2;
  Stat q{in[0].r, in[0].z, 0.0f}, p{in[1].r, in[1].z, 0.0f};
  Exact eq{in[0].m, in[0].e}, ep{in[1].m, in[1].e};
  for (int i = 1; i < a.splits; ++i) {
    q.join(Stat{in[2 * i].r, in[2 * i].z, 0.0f});
    p.join(Stat{in[2 * i + 1].r, in[2 * i + 1].z, 0.0f});
    eq.join(Exact{in[2 * i].m, in[2 * i].e}, a.c);
    ep.join(Exact{in[2 * i + 1].m, in[2 * i + 1].e}, a.c);
  }
  Row<S, T, kThreads, 0, 0> r(s, t, lo, hi);
  const float loss =
      q.good() && p.good()
          ? row_grad<kThreads>(r, nullptr, grad, a.c, a.temperature, w, q, p, sums)
          : row_grad_exact<kThreads>(s, t, grad, lo, hi, a.c, a.temperature, w, eq, ep, sums);
  if (threadIdx.x == 0) {
    float* part = a.part + row * a.splits;
    __hip_atomic_store(part + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t before = __hip_atomic_fetch_add(a.arrived + row, 1u, __ATOMIC_ACQ_REL,
                                                   __HIP_MEMORY_SCOPE_AGENT);
    if (before + 1 == (uint32_t)a.splits) {      // every part is there
      float sum = 0.0f;
      for (int i = 0; i < a.splits; ++i)
        sum += __hip_atomic_load(part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      a.loss[row] = sum;
    }
  }
}

// Places within a row fit 32 bits, their bytes and those of a whole split past them too.
constexpr int64_t kMaxVocab = int64_t(1) << 28;

// Workgroups per row: few rows that are long enough to be worth two launches get as many as the
// 256 compute units have room for at one each, and two units per thread.  bf16, us, one workgroup
// and several: 3 x 32000 9.6 and 11.6, 8 x 40000 11.8 and 11.2, 8 x 64000 19.3 and 11.9, 8 x 128000
// 30.0 and 14.0, 64 x 64000 20.0 and 16.7, 100 x 64000 20.7 and 19.5, 100 x 256000 67 and 52, 127 x
// 64000 21.5 and 22.7, 127 x 256000 69 and 67.
int splits_of(int64_t rows, int64_t vocab) {
  if (rows <= 0 || rows > 100 || vocab <= 32768) return 1;
  const int64_t want = 256 / rows, most = (vocab + 16383) / 16384;
  return (int)(want < most ? want : most);
}

template <typename S, typename T, int THREADS, int REGS, int LDS>
void launch_rows(const Distill& a, hipStream_t stream) {
  const int bytes = (int)Row<S, T, THREADS, REGS, LDS>::kBytes;
  auto kernel = row_kernel<S, T, THREADS, REGS, LDS>;
  if (bytes > 65536 - 512)
    (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  constexpr int64_t kLine = 1 << 20;                // workgroups in x: threads stay below 2^32
  const dim3 grid((unsigned)(a.rows < kLine ? a.rows : kLine), (unsigned)((a.rows + kLine - 1) / kLine));
  kernel<<<grid, THREADS, bytes, stream>>>(a);
}

template <typename S, typename T>
void launch(const Distill& a, hipStream_t stream) {
  // units that a thread holds: 64 registers, and of 1024 threads 128 KB of shared memory; 88
  // registers for rows that fill them (shorter ones would wait for loads of nothing)
  constexpr int unit = kUnit<S, T>, bytes = unit * (sizeof(S) + sizeof(T));
  constexpr int regs = 256 / bytes, lds = 128 / bytes, more = 352 / bytes;
  if (a.splits > 1) {
    const dim3 grid((unsigned)a.splits, (unsigned)a.rows);
    split_stats_kernel<S, T><<<grid, kThreads, 0, stream>>>(a);
    split_grad_kernel<S, T><<<grid, kThreads, 0, stream>>>(a);
  } else if (a.vocab <= 128 * unit) {
    launch_rows<S, T, 128, 1, 0>(a, stream);
  } else if (a.vocab <= 256 * unit) {
    launch_rows<S, T, 256, 1, 0>(a, stream);
  } else if (a.vocab <= 256 * unit * 2) {
    launch_rows<S, T, 256, 2, 0>(a, stream);
  } else if (a.vocab <= 256 * unit * 4) {
    launch_rows<S, T, 256, 4, 0>(a, stream);
  } else if (a.vocab <= 256 * unit * regs) {
    launch_rows<S, T, 256, regs, 0>(a, stream);
  } else if (a.vocab <= 512 * unit * regs) {
    launch_rows<S, T, 512, regs, 0>(a, stream);
  } else if (a.vocab <= 2 * 512 * unit * (regs + lds)) {
    launch_rows<S, T, 512, regs, lds>(a, stream);
  } else if (a.vocab <= 1024 * unit * (more + lds)) {
    launch_rows<S, T, 1024, regs, lds>(a, stream);
  } else {
    launch_rows<S, T, 1024, more, lds>(a, stream);
  }
}

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT int64_t nvfp4_distill_loss_workspace(int64_t rows, int64_t vocab) {
  const int64_t splits = vocab < 1 ? 1 : splits_of(rows, vocab);
  return splits == 1 ? 0 : rows * (splits * 9 + 1) * 4;
}

NVFP4_EXPORT nvfp4_status nvfp4_distill_loss(const void* student, int64_t student_stride,
                                             const void* teacher, int64_t teacher_stride,
                                             const float* weight, int64_t rows, int64_t vocab,
                                             nvfp4_type stype, nvfp4_type ttype,
                                             float temperature, float* loss, void* grad,
                                             int64_t grad_stride, void* workspace,
                                             hipStream_t stream) {
  if (!known(stype) || !known(ttype)) return NVFP4_ERR_ENUM;
  if (vocab > kMaxVocab || !shape_ok(rows, vocab, student_stride) || !shape_ok(rows, vocab, teacher_stride) ||
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
  Distill a = {student, teacher, weight, loss, grad, ws, ws + rows * splits * 8,
               (uint32_t*)(ws + rows * splits * 9), student_stride, teacher_stride, grad_stride,
               rows, (uint32_t)vocab, (uint32_t)(((vocab + splits - 1) / splits + 7) / 8 * 8), splits,
               c, temperature};
  (void)hipGetLastError();
  if (stype == NVFP4_T_BF16 && ttype == NVFP4_T_BF16) launch<bf16, bf16>(a, stream);
  else if (stype == NVFP4_T_BF16) launch<bf16, float>(a, stream);
  else if (ttype == NVFP4_T_BF16) launch<float, bf16>(a, stream);
  else launch<float, float>(a, stream);
  return launched();
}
