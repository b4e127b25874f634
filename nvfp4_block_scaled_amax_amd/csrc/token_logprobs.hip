// Log probabilities of given tokens, entropy and top alternatives per row of logits, and their
// gradient, for gfx950 (include/nvfp4_answer.h defines the operations).
//
// Forward, one pass over a row.  Each thread keeps the largest entry m that it has seen and
//   Z = sum 2^d,  S = sum d 2^d,   d = (x - m) c,  c = log2(e) / T,
// and moves both when m grows: Z 2^-D and (S - D Z) 2^-D for m + D / c.  With exact differences the
// size of the logits costs no precision, and entropy = ln Z - ln 2 S / Z has no term below 0.
//
// Top alternatives without a sort: a column is the vectors that a few threads read; its largest
// entry and the first vector that holds it are known after the pass.  The k columns that come first by
// (entry, place) hold all of the top k: an entry of another column comes after k others.  What those
// columns hold down to the k-th column's entry is read again (20 columns of 256: a thirteenth of the
// row, from the caches), collected in shared memory, and each entry's place is the number of those
// before it.  More than fit (many equal or rising entries in few columns) are found one by one.
#include "nvfp4_answer.h"
#include "train_common.h"

namespace train {
namespace {

constexpr int kMost = NVFP4_LOGPROBS_MAX;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -1000.0f;             // 2^kNone is 0: stands for any d below

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

struct Stat {
  float m, z, s;
  // to a larger m (an empty one has Z = S = 0 and the lowest m)
  __device__ __forceinline__ void raise(float to, float c) {
    const float d = fmaxf((m - to) * c, kNone), f = exp2_(d);
    s = f * fmaf(d, z, s);
    z *= f;
    m = to;
  }
  // x: a NaN and two +inf make Z NaN
  __device__ __forceinline__ void add(float x, float c) {
    const float d = (x - m) * c, e = exp2_(d);
    z += e;
    s = fmaf(e, fmaxf(d, kNone), s);
  }
  __device__ __forceinline__ bool good() const { return z > 0.0f && z < INFINITY; }
};

// Over a workgroup; every thread gets it.  slots: WAVES of Stat.
template <int WAVES>
__device__ __forceinline__ Stat join_group(Stat a, float c, Stat* slots) {
  a.raise(reduce64(a.m, Max()), c);
  a.z = reduce64(a.z, Sum());
  a.s = reduce64(a.s, Sum());
  if (WAVES == 1) return a;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = a;
  __syncthreads();
  a = slots[threadIdx.x % WAVES];
  a.raise(reduce_few<WAVES>(a.m, Max()), c);
  a.z = reduce_few<WAVES>(a.z, Sum());
  a.s = reduce_few<WAVES>(a.s, Sum());
  return a;
}

// An entry and its place as one number: larger entries above smaller ones, lower places above higher
// ones among equals.  0 is below all (the place is never 2^32 - 1).
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);          // -0 is 0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float entry(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t at) { return (uint64_t)order(x) << 32 | (uint32_t)~at; }

struct Args {
  const void* logits;
  const void* tokens;
  float* logp;
  float* entropy;
  float* top_logp;
  int64_t* top_index;
  float* stats;
  float* part;              // split rows: [rows][splits][4] m, z, s
  uint64_t* keys;           // split rows: [rows][splits][top]
  int64_t stride, rows;
  uint32_t vocab, split_size;
  int given, top, splits, wide;
  float c, inv_t;
};

__device__ __forceinline__ int64_t token(const void* tokens, int wide, int64_t i) {
  return wide ? ((const int64_t*)tokens)[i] : (int64_t)((const int32_t*)tokens)[i];
}

// Whether a row has any token, seen by every thread.
__device__ __forceinline__ bool is_read(const void* tokens, int wide, int given, int64_t row) {
  if (given == 0) return true;
  const int lane = threadIdx.x & 63;
  return __ballot(lane < given && token(tokens, wide, row * given + lane) >= 0) != 0;
}

__device__ __forceinline__ void skip_row(const Args& a, int64_t row) {
  const int i = threadIdx.x;
  if (i < a.given) a.logp[row * a.given + i] = 0.0f;
  if (i < a.top) {
    a.top_logp[row * a.top + i] = 0.0f;
    a.top_index[row * a.top + i] = -1;
  }
  if (i < 2) a.stats[row * 2 + i] = 0.0f;
  if (i == 0 && a.entropy) a.entropy[row] = 0.0f;
}

// What a row's statistics give, but for the top alternatives; returns ln Z (NaN: no distribution).
template <typename T>
__device__ __forceinline__ float finish_row(const Args& a, int64_t row, Stat t) {
  const float z = t.good() ? logf(t.z) : NAN, m = t.good() ? t.m : NAN;
  const int i = threadIdx.x;
  if (i < a.given) {
    const int64_t id = token(a.tokens, a.wide, row * a.given + i);
    float v = 0.0f;
    if (id >= a.vocab) v = NAN;
    else if (id >= 0) v = (to_f32(((const T*)a.logits)[row * a.stride + id]) - m) * a.inv_t - z;
    a.logp[row * a.given + i] = v;
  }
  if (i == 0) {
    a.stats[row * 2] = m;
    a.stats[row * 2 + 1] = z;
    if (a.entropy) a.entropy[row] = fmaf(-kLn2, t.s / t.z, z);
  }
  return z;
}

constexpr int kColumns = 256;
constexpr int kHeld = 1024;               // candidates in shared memory

struct TopShared {
  uint64_t column[kColumns];
  uint64_t held[kHeld];
  uint32_t owner[kMost];
  uint64_t limit, best[16];
  int count;
};

// The places of `count` numbers among themselves: put(place, number) for the first `top`.
template <int THREADS, typename Put>
__device__ __forceinline__ void rank(const uint64_t* held, int count, int top, Put put) {
  for (int i = threadIdx.x; i < count; i += THREADS) {
    const uint64_t mine = held[i];
    int before = 0;
    for (int j = 0; j < count; ++j) before += held[j] > mine;
    if (before < top) put(before, mine);
  }
}

// The top entries of a row's part [lo, hi), from each thread's largest entry and its place.
// put(place, key) for all of them, at most once each.
template <typename T, int THREADS, typename Put>
__device__ __forceinline__ void find_top(const T* row, uint32_t lo, uint32_t hi, int top, uint64_t mine,
                                         TopShared& sh, Put put) {
  constexpr int N = 16 / sizeof(T);
  constexpr int kPer = THREADS > kColumns ? THREADS / kColumns : 1;      // threads of a column
  constexpr int kHave = THREADS / kPer;
  // columns of neighbouring threads
#pragma unroll
  for (int d = 1; d < kPer; d *= 2) {
    const uint64_t other = __shfl_xor((unsigned long long)mine, d);
    mine = other > mine ? other : mine;
  }
  if (threadIdx.x % kPer == 0) sh.column[threadIdx.x / kPer] = mine;
  if (threadIdx.x == 0) sh.count = 0, sh.limit = 0;
  if (threadIdx.x < kMost) sh.owner[threadIdx.x] = ~0u;
  __syncthreads();
  if (threadIdx.x < kHave) {
    const uint64_t k = sh.column[threadIdx.x];
    if (k) {
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < kHave; ++j) before += sh.column[j] > k;
      if (before < top) sh.owner[before] = threadIdx.x;
      if (before == top - 1) sh.limit = k;
    }
  }
  __syncthreads();
  // fewer columns than `top`: everything is a candidate
  const uint64_t limit = sh.limit;
  const uint32_t low = (uint32_t)(limit >> 32), until = limit ? ~(uint32_t)limit + N : ~0u;
  const uint32_t vectors = (hi - lo + N - 1) / N;                     // of the part
  const uint32_t deep = (vectors + THREADS - 1) / THREADS;            // of a thread
  const uint32_t total = deep * kPer * top;
  const auto visit = [&](auto f) {
    for (uint32_t i = threadIdx.x; i < total; i += THREADS) {
      const uint32_t owner = sh.owner[i % top], t = i / top;
      if (owner == ~0u) continue;
      const uint32_t at = lo + ((t / kPer) * THREADS + owner * kPer + t % kPer) * N;
      if (at >= hi) continue;
      if (at + N <= hi) {
        const Vec<T, N> v = load_vec<N>(row + at);
#pragma unroll
        for (int j = 0; j < N; ++j) f(v[j], at + j);
      } else {
        for (uint32_t j = at; j < hi; ++j) f(to_f32(row[j]), j);
      }
    }
  };
  visit([&](float x, uint32_t at) {
    const uint32_t o = order(x);
    if (o > low || (o == low && at < until)) {
      const int n = atomicAdd(&sh.count, 1);
      if (n < kHeld) sh.held[n] = (uint64_t)o << 32 | (uint32_t)~at;
    }
  });
  __syncthreads();
  const int count = sh.count;
  if (count <= kHeld) {
    rank<THREADS>(sh.held, count, top, put);
    return;
  }
  uint64_t last = ~uint64_t(0);
  for (int k = 0; k < top; ++k) {
    uint64_t best = 0;
    visit([&](float x, uint32_t at) {
      const uint64_t n = key_of(x, at);
      if (n < last && n > best) best = n;
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint64_t other = __shfl_xor((unsigned long long)best, d);
      best = other > best ? other : best;
    }
    if ((threadIdx.x & 63) == 0) sh.best[threadIdx.x >> 6] = best;
    __syncthreads();
    for (int w = 0; w < THREADS / 64; ++w) best = sh.best[w] > best ? sh.best[w] : best;
    if (threadIdx.x == 0) put(k, best);
    last = best;
    __syncthreads();
  }
}

__device__ __forceinline__ void put_top(const Args& a, int64_t row, Stat t, float z, int place, uint64_t key) {
  a.top_index[row * a.top + place] = (int64_t)(uint32_t)~(uint32_t)key;
  a.top_logp[row * a.top + place] = (entry((uint32_t)(key >> 32)) - t.m) * a.inv_t - z;
}
// A row without a distribution has no order either.
__device__ __forceinline__ void no_top(const Args& a, int64_t row) {
  if (threadIdx.x < a.top) {
    a.top_index[row * a.top + threadIdx.x] = -1;
    a.top_logp[row * a.top + threadIdx.x] = NAN;
  }
}

template <typename T, int THREADS, bool TOP, bool SPLIT>
__global__ __launch_bounds__(THREADS) void forward_kernel(const Args a) {
  constexpr int N = 16 / sizeof(T);
  __shared__ Stat slots[THREADS / 64];
  __shared__ TopShared sh;
  const int64_t row = SPLIT ? (int64_t)blockIdx.y : (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  if (!is_read(a.tokens, a.wide, a.given, row)) {
    if (!SPLIT) skip_row(a, row);
    return;
  }
  const T* x = (const T*)a.logits + row * a.stride;
  const uint32_t lo = SPLIT ? min(blockIdx.x * a.split_size, a.vocab) : 0;
  const uint32_t hi = SPLIT ? min(lo + a.split_size, a.vocab) : a.vocab;
  Stat t{kLowest, 0.0f, 0.0f};
  // the thread's largest entry, and the first vector that holds it
  float most = -INFINITY;
  uint32_t place = lo + threadIdx.x * N;
  const bool any = place < hi;
  const auto unit = [&](const Vec<T, N>& v, uint32_t at) {
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
    if (top > most) {
      most = top;
      place = at;
      if (top > t.m) t.raise(top, a.c);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) t.add(v[i], a.c);
  };
  constexpr int kAhead = 4;                         // vectors in flight per thread
  uint32_t at = lo + threadIdx.x * N;
  const uint32_t step = THREADS * N;
  for (; at + (kAhead - 1) * step + N <= hi; at += kAhead * step) {
    Vec<T, N> v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = load_vec<N>(x + at + k * step);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) unit(v[k], at + k * step);
  }
  for (; at < hi; at += step) {
    if (at + N <= hi) {
      unit(load_vec<N>(x + at), at);
    } else {
      float w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = at + i < hi ? to_f32(x[at + i]) : -INFINITY;
      unit(make_vec<T>(w), at);
    }
  }
  const Stat whole = join_group<THREADS / 64>(t, a.c, slots);
  const uint64_t mine = any ? key_of(most, place) : 0;
  if (SPLIT) {
    if (threadIdx.x == 0) {
      float* out = a.part + (row * a.splits + blockIdx.x) * 4;
      out[0] = whole.m, out[1] = whole.z, out[2] = whole.s;
    }
    if (TOP) {
      uint64_t* keys = a.keys + (row * a.splits + blockIdx.x) * a.top;
      if (threadIdx.x < a.top && threadIdx.x >= hi - lo) keys[threadIdx.x] = 0;      // a short last part
      find_top<T, THREADS>(x, lo, hi, a.top, mine, sh, [&](int p, uint64_t k) { keys[p] = k; });
    }
  } else {
    const float z = finish_row<T>(a, row, whole);
    if (!TOP) return;
    if (!whole.good()) return no_top(a, row);
    find_top<T, THREADS>(x, lo, hi, a.top, mine, sh,
                         [&](int p, uint64_t k) { put_top(a, row, whole, z, p, k); });
  }
}

constexpr int kMaxSplits = 64;

// Rows of several parts: their statistics and lists become one.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const Args a) {
  __shared__ uint64_t held[kMaxSplits * kMost];
  __shared__ uint64_t limit;
  __shared__ int count;
  const int64_t row = blockIdx.x;
  if (!is_read(a.tokens, a.wide, a.given, row)) return skip_row(a, row);
  // a lane of every wavefront takes a part
  const int lane = threadIdx.x & 63;
  Stat t{kLowest, 0.0f, 0.0f};
  if (lane < a.splits) {
    const float* in = a.part + (row * a.splits + lane) * 4;
    t = Stat{in[0], in[1], in[2]};
  }
  t.raise(reduce64(t.m, Max()), a.c);
  t.z = reduce64(t.z, Sum());
  t.s = reduce64(t.s, Sum());
  const float z = finish_row<T>(a, row, t);
  if (!a.top) return;
  if (!t.good()) return no_top(a, row);
  // the k-th largest of the first few of each list is a lower bound for all
  const uint64_t* keys = a.keys + row * a.splits * a.top;
  const int first = min(a.top, max(4, (a.top + a.splits - 1) / a.splits)), some = first * a.splits;
  if (threadIdx.x == 0) limit = 1, count = 0;
  for (int i = threadIdx.x; i < some; i += 256) held[i] = keys[i / first * a.top + i % first];
  __syncthreads();
  for (int i = threadIdx.x; i < some; i += 256) {
    const uint64_t mine = held[i];
    int before = 0;
    for (int j = 0; j < some; ++j) before += held[j] > mine;
    if (before == a.top - 1 && mine) limit = mine;
  }
  __syncthreads();
  const uint64_t least = limit;
  for (int i = threadIdx.x; i < a.splits * a.top; i += 256) {
    const uint64_t k = keys[i];
    if (k >= least) held[atomicAdd(&count, 1)] = k;
  }
  __syncthreads();
  rank<256>(held, count, a.top, [&](int p, uint64_t k) { put_top(a, row, t, z, p, k); });
}

// ------------------------------------------------------------------------------- gradient
struct BackArgs {
  const void* logits;
  const void* tokens;
  const float* stats;
  const float* entropy;
  const float* dlogp;
  const float* dentropy;
  void* grad;
  int64_t stride, grad_stride, rows;
  uint32_t vocab, split_size;
  int given, wide;
  float c, inv_t;
};

// A workgroup takes a part of a row.  With y = log2 p: grad = p (A y + B), A = -h ln 2 / T,
// B = -(sum g + h entropy) / T; the given tokens' entries are read before anything is written (grad may be
// logits) and written again at the end with what their g adds.
template <typename T>
__global__ __launch_bounds__(256) void backward_kernel(const BackArgs a) {
  constexpr int N = 16 / sizeof(T), THREADS = 256;
  __shared__ int64_t id[kMost];
  __shared__ float up[kMost];
  const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (row >= a.rows) return;
  const uint32_t lo = blockIdx.x * a.split_size, hi = min(lo + a.split_size, a.vocab);
  const T* x = (const T*)a.logits + row * a.stride;
  T* grad = (T*)a.grad + row * a.grad_stride;
  const int i = threadIdx.x & 63;
  int64_t mine = -1;
  float g = 0.0f;
  if (i < a.given) {
    mine = token(a.tokens, a.wide, row * a.given + i);
    g = mine < 0 ? 0.0f : a.dlogp[row * a.given + i];
  }
  if (__ballot(mine >= 0) == 0) {
    const Vec<T, N> zero = zero_vec<T, N>();
    for (uint32_t at = lo + threadIdx.x * N; at < hi; at += THREADS * N) store_vec<kAny>(grad, at, hi, zero);
    return;
  }
  if (mine >= (int64_t)a.vocab) g = NAN;
  const float m = a.stats[row * 2], z = a.stats[row * 2 + 1];
  const float h = a.dentropy ? a.dentropy[row] : 0.0f, all = reduce64(g, Sum());
  const float A = -h * kLn2 * a.inv_t;
  float B = a.dentropy ? -fmaf(h, a.entropy[row], all) * a.inv_t : -all * a.inv_t;
  if (!(z == z)) B = NAN;                          // no distribution
  const float z2 = z * kLog2e;
  const auto value = [&](float v) {
    const float y = fmaxf(fmaf(v - m, a.c, -z2), kNone);
    return exp2_(y) * fmaf(A, y, B);
  };
  // the first of equal tokens in this part takes their sum
  float fix = 0.0f;
  bool fixes = false;
  if (threadIdx.x < 64) {
    id[i] = mine;
    up[i] = g;
  }
  __syncthreads();
  if (threadIdx.x < a.given && mine >= lo && mine < hi) {
    fixes = true;
    for (int j = 0; j < a.given; ++j)
      if (id[j] == mine) {
        fix += up[j];
        if (j < i) fixes = false;
      }
    if (fixes) fix = fmaf(fix, a.inv_t, value(to_f32(x[mine])));
  }
  __syncthreads();
  constexpr int kAhead = 4;
  uint32_t at = lo + threadIdx.x * N;
  constexpr uint32_t step = THREADS * N;
  const auto unit = [&](const Vec<T, N>& v, uint32_t to) {
    float r[N];
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = value(v[k]);
    store_vec<kAny>(grad, to, hi, make_vec<T>(r));
  };
  for (; at + (kAhead - 1) * step + N <= hi; at += kAhead * step) {
    Vec<T, N> v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = load_vec<N>(x + at + k * step);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) unit(v[k], at + k * step);
  }
  for (; at < hi; at += step) unit(load_vec<N, kAny>(x, at, hi), at);
  __syncthreads();
  if (fixes) grad[mine] = from_f32<T>(fix);
}

constexpr int64_t kMaxVocab = int64_t(1) << 28;

// Workgroups per row: few long rows are shared.
int splits_of(int64_t rows, int64_t vocab) {
  if (rows <= 0 || rows > 100 || vocab <= 16384) return 1;
  int64_t want = 512 / rows;
  const int64_t most = (vocab + 4095) / 4096;
  want = want < most ? want : most;
  return (int)(want < kMaxSplits ? want : kMaxSplits);
}

template <typename T, int THREADS, bool SPLIT>
void launch_forward(const Args& a, dim3 grid, hipStream_t s) {
  if (a.top) forward_kernel<T, THREADS, true, SPLIT><<<grid, THREADS, 0, s>>>(a);
  else forward_kernel<T, THREADS, false, SPLIT><<<grid, THREADS, 0, s>>>(a);
}

template <typename T>
void launch_forward(const Args& a, hipStream_t s) {
  if (a.splits > 1) {
    launch_forward<T, 256, true>(a, dim3((unsigned)a.splits, (unsigned)a.rows), s);
    join_kernel<T><<<(unsigned)a.rows, 256, 0, s>>>(a);
    return;
  }
  constexpr int64_t kLine = 1 << 20;                // workgroups in x: threads stay below 2^32
  const dim3 grid((unsigned)(a.rows < kLine ? a.rows : kLine), (unsigned)((a.rows + kLine - 1) / kLine));
  launch_forward<T, 256, false>(a, grid, s);
}

bool temperature_ok(float temperature, float& inv_t, float& c) {
  inv_t = 1.0f / temperature;
  c = (float)(1.4426950408889634 / (double)temperature);
  return temperature > 0.0f && inv_t > 0.0f && c < 3.0e38f;
}

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT int64_t nvfp4_token_logprobs_workspace(int64_t rows, int64_t vocab, int64_t top) {
  const int64_t splits = vocab < 1 ? 1 : splits_of(rows, vocab);
  return splits == 1 || top < 0 || top > kMost ? 0 : rows * splits * (16 + top * 8);
}

NVFP4_EXPORT nvfp4_status nvfp4_token_logprobs(const void* logits, int64_t stride, const void* tokens,
                                               int64_t rows, int64_t vocab, int64_t given, int64_t top,
                                               nvfp4_type type, nvfp4_index itype, float temperature,
                                               float* logp, float* entropy, float* top_logp,
                                               int64_t* top_index, float* stats, void* workspace,
                                               hipStream_t stream) {
  if (!known(type) || (itype != NVFP4_I32 && itype != NVFP4_I64)) return NVFP4_ERR_ENUM;
  if (vocab > kMaxVocab || !shape_ok(rows, vocab, stride) || rows >= (int64_t(1) << 40) || given < 0 ||
      given > kMost || top < 0 || top > kMost || top > vocab)
    return NVFP4_ERR_SHAPE;
  float inv_t, c;
  if (!temperature_ok(temperature, inv_t, c)) return NVFP4_ERR_VALUE;
  if (rows == 0) return NVFP4_OK;
  const int64_t need = nvfp4_token_logprobs_workspace(rows, vocab, top);
  if (!logits || !stats || (given && (!tokens || !logp)) || (top && (!top_logp || !top_index)) ||
      (need && !workspace))
    return NVFP4_ERR_NULL;
  const int64_t es = size_of(type), is = itype == NVFP4_I32 ? 4 : 8;
  if (!aligned(logits, es) || !aligned(tokens, is) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(top_logp, 4) || !aligned(top_index, 8) || !aligned(stats, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const Range in[] = {range(logits, extent(rows, vocab, stride, es)), range(tokens, rows * given * is)};
  const Range out[] = {range(logp, rows * given * 4), range(entropy, rows * 4),
                       range(top_logp, rows * top * 4), range(top_index, rows * top * 8),
                       range(stats, rows * 8), range(need ? workspace : nullptr, need)};
  for (int o = 0; o < 6; ++o) {
    for (const Range& r : in)
      if (overlap(out[o], r)) return NVFP4_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return NVFP4_ERR_ALIAS;
  }
  const int splits = splits_of(rows, vocab);
  uint64_t* keys = (uint64_t*)workspace;
  const Args a = {logits, tokens, logp, entropy, top_logp, top_index, stats,
                  (float*)(keys + (need ? rows * splits * top : 0)), keys, stride, rows, (uint32_t)vocab,
                  (uint32_t)(((vocab + splits - 1) / splits + 7) / 8 * 8), (int)given, (int)top, splits,
                  itype == NVFP4_I64, c, inv_t};
  (void)hipGetLastError();
  if (type == NVFP4_T_BF16) launch_forward<bf16>(a, stream);
  else launch_forward<float>(a, stream);
  return launched();
}

NVFP4_EXPORT nvfp4_status nvfp4_token_logprobs_backward(const void* logits, int64_t stride,
                                                        const void* tokens, const float* stats,
                                                        const float* entropy, const float* dlogp,
                                                        const float* dentropy, int64_t rows,
                                                        int64_t vocab, int64_t given, nvfp4_type type,
                                                        nvfp4_index itype, float temperature,
                                                        void* grad, int64_t grad_stride,
                                                        hipStream_t stream) {
  if (!known(type) || (itype != NVFP4_I32 && itype != NVFP4_I64)) return NVFP4_ERR_ENUM;
  if (vocab > kMaxVocab || !shape_ok(rows, vocab, stride) || !shape_ok(rows, vocab, grad_stride) ||
      rows >= (int64_t(1) << 31) || given < 1 || given > kMost)
    return NVFP4_ERR_SHAPE;
  float inv_t, c;
  if (!temperature_ok(temperature, inv_t, c)) return NVFP4_ERR_VALUE;
  if (rows == 0) return NVFP4_OK;
  if (!logits || !tokens || !stats || !dlogp || !grad || (dentropy && !entropy)) return NVFP4_ERR_NULL;
  const int64_t es = size_of(type), is = itype == NVFP4_I32 ? 4 : 8;
  if (!aligned(logits, es) || !aligned(grad, es) || !aligned(tokens, is) || !aligned(stats, 4) ||
      !aligned(entropy, 4) || !aligned(dlogp, 4) || !aligned(dentropy, 4))
    return NVFP4_ERR_ALIGN;
  const Range out = range(grad, extent(rows, vocab, grad_stride, es));
  const Range in[] = {range(logits, extent(rows, vocab, stride, es)), range(tokens, rows * given * is),
                      range(stats, rows * 8), range(entropy, rows * 4), range(dlogp, rows * given * 4),
                      range(dentropy, rows * 4)};
  for (int i = 0; i < 6; ++i)
    if (!(i == 0 && grad == logits && grad_stride == stride) && overlap(out, in[i])) return NVFP4_ERR_ALIAS;
  const uint32_t size = 16384;
  const int64_t line = rows < 32768 ? rows : 32768;
  const BackArgs a = {logits, tokens, stats, entropy, dlogp, dentropy, grad, stride, grad_stride, rows,
                      (uint32_t)vocab, size, (int)given, itype == NVFP4_I64, c, inv_t};
  const dim3 grid((unsigned)((vocab + size - 1) / size), (unsigned)line, (unsigned)((rows + line - 1) / line));
  (void)hipGetLastError();
  if (type == NVFP4_T_BF16) backward_kernel<bf16><<<grid, 256, 0, stream>>>(a);
  else backward_kernel<float><<<grid, 256, 0, stream>>>(a);
  return launched();
}
