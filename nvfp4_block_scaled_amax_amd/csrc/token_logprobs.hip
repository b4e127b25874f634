// Log probabilities of given tokens, entropy and top alternatives per row of logits, and their
// gradient, for gfx950 (include/nvfp4_answer.h defines the operations).
//
// Forward, one pass over a row.  Each thread keeps the largest entry m that it has seen and
//   Z = sum 2^d,  S = sum d 2^d,   d = (x - m) c,  c = log2(e) / T,
// and moves both when m grows: Z 2^-D and (S - D Z) 2^-D for m + D / c.  With exact differences the
// size of the logits costs no precision, and entropy = ln Z - ln 2 S / Z has no term below 0.
//
// Top alternatives without a sort: a cell is the vectors that a few threads read in a part of the row's
// length, as many cells as threads; its largest entry and the first vector that holds it are known
// after the pass.  The k cells that come first by (entry, place) hold all of the top k: an entry of
// another cell comes after k others.  A bound that a few more than k cells reach is found bit by bit, the vectors
// of these cells are read again (24 or so cells of 256: a tenth of the row, 9 % more bytes fetched), what
// reaches the bound is collected in shared memory, and each entry's place is the number of those before
// it.  More than fit (many equal or rising entries in few cells) are found one by one.  The order in which the
// collecting atomics run changes nothing: the numbers are distinct and their places follow from them.
//
// Bound by the row's bytes; the exponential of every entry hides behind them at eight workgroups a
// compute unit.  Measured on one MI355X: 4096 x 128000 bf16 185 us without alternatives, 203 us with 20 (5.2
// TB/s); 515 x 50251 binary32 of which a quarter is not read 15.5 us (5.0 TB/s); gradient, 4096 x 128000 bf16 385 us
// (5.4 TB/s).  512 x 128000 with 20 alternatives of rows of which half the entries are equal, or of which few threads
// hold all large ones, 120-140 us, of other rows 37.
#include "nvfp4_answer.h"
#include "train_common.h"

namespace train {
namespace {

constexpr int kMost = NVFP4_LOGPROBS_MAX;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -160.0f;              // 2^kNone is 0: stands for any d below

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

// A given token and its logit, a lane each.
struct Given {
  int64_t id;
  float x;
};
template <typename T>
__device__ __forceinline__ Given given_of(const Args& a, int64_t row) {
  Given g = {-1, 0.0f};
  if (threadIdx.x < a.given) {
    g.id = token(a.tokens, a.wide, row * a.given + threadIdx.x);
    if (g.id >= 0 && g.id < a.vocab) g.x = to_f32(((const T*)a.logits)[row * a.stride + g.id]);
  }
  return g;
}

// What a row's statistics give, but for the top alternatives; returns ln Z (NaN: no distribution).
__device__ __forceinline__ float finish_row(const Args& a, int64_t row, Stat t, Given g) {
  const float z = t.good() ? logf(t.z) : NAN, m = t.good() ? t.m : NAN;
  const int i = threadIdx.x;
  if (i < a.given)
    a.logp[row * a.given + i] = g.id < 0 ? 0.0f : g.id >= a.vocab ? NAN : (g.x - m) * a.inv_t - z;
  if (i == 0) {
    a.stats[row * 2] = m;
    a.stats[row * 2 + 1] = z;
    if (a.entropy) a.entropy[row] = fmaf(-kLn2, t.s / t.z, z);
  }
  return z;
}

template <int THREADS>
constexpr int kHeld = THREADS == 64 ? 512 : 1024;        // candidates in shared memory

template <int THREADS>
struct TopShared {
  uint64_t cell[THREADS], best[THREADS / 64], limit;
  uint64_t held[kHeld<THREADS>];
  u32x4 vector[kHeld<THREADS> / 4];                      // those that may hold candidates
  uint32_t place[kHeld<THREADS> / 4], owner[THREADS];
  int owners, vectors, count;
};

// A row's part in cells: the threads of a group of G neighbours, in one of G blocks of steps (a step is a
// vector of every thread).  There are as many cells as threads; a cell's vectors lie G together.
template <int THREADS, int N>
struct Cells {
  uint32_t steps, block;             // of the part; of a block, a multiple of kStepsAhead
  int bits;                          // log2 G
  static constexpr uint32_t kStepsAhead = 4;
  __device__ __forceinline__ Cells(uint32_t size) {
    steps = (size + THREADS * N - 1) / (THREADS * N);
    bits = steps < 2 * kStepsAhead ? 0 : steps < 4 * kStepsAhead ? 1 : steps < 8 * kStepsAhead ? 2 : 3;
    block = (((steps + (1u << bits) - 1) >> bits) + kStepsAhead - 1) / kStepsAhead * kStepsAhead;
  }
};

// The places of `count` numbers among themselves: put(place, number) for the first `top`.
template <int THREADS, typename Put>
__device__ __forceinline__ void rank(const uint64_t* held, int count, int top, Put put) {
  for (int i = threadIdx.x; i < count; i += THREADS) {
    const uint64_t mine = held[i];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) before += held[j] > mine;
    if (before < top) put(before, mine);
  }
}

// A lower bound for the top-th largest of PER numbers of each lane of a wavefront, none of them equal but for 0:
// `top` or somewhat more of them reach it (0 where fewer are not 0).  Bit by bit, first the entries' 32 and, where
// too many are left by equal entries, the places'.
template <int PER>
__device__ __forceinline__ uint64_t threshold(const uint64_t (&key)[PER], int top) {
  const int enough = top + 4 + top / 4;
  uint32_t t = 0;
  int have = 64 * PER;
  for (uint32_t bit = 1u << 31; bit && have > enough; bit >>= 1) {
    const uint32_t next = t | bit;
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += __popcll(__ballot((uint32_t)(key[i] >> 32) >= next));
    if (n >= top) t = next, have = n;
  }
  uint64_t low = (uint64_t)t << 32;
  if (t == 0) return low;
  for (uint32_t bit = 1u << 31; bit && have > enough; bit >>= 1) {
    const uint64_t next = low | bit;
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += __popcll(__ballot(key[i] >= next));
    if (n >= top) low = next, have = n;
  }
  return low;
}

// The top entries of a row's part [lo, hi), from each cell's largest entry and its place (sh.cell).
// put(place, key) for all of them, at most once each.
template <typename T, int THREADS, int N, typename Put>
__device__ __forceinline__ void find_top(const T* row, uint32_t lo, uint32_t hi, int top, Cells<THREADS, N> cells,
                                         TopShared<THREADS>& sh, Put put) {
  constexpr int WAVES = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  if (wave == 0) {
    uint64_t key[WAVES];
#pragma unroll
    for (int i = 0; i < WAVES; ++i) key[i] = sh.cell[i * 64 + lane];
    const uint64_t limit = threshold(key, top);
    int n = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const bool in = key[i] && key[i] >= limit;
      const uint64_t all = __ballot(in);
      if (in) sh.owner[n + __popcll(all & ((uint64_t(1) << lane) - 1))] = i * 64 + lane;
      n += __popcll(all);
    }
    if (lane == 0) sh.owners = n, sh.limit = limit, sh.count = 0, sh.vectors = 0;
  }
  __syncthreads();
  // an entry above the limit's, or equal to it and no further than its vector, is a candidate (of fewer cells
  // than `top`, and of less than that many entries at all, everything is)
  const uint64_t limit = sh.limit;
  const int owners = sh.owners;
  const uint32_t low = (uint32_t)(limit >> 32);
  const uint32_t until = (uint32_t)limit ? ~(uint32_t)limit + N : ~0u;
  const int block_bits = cells.block < 2 ? 0 : 32 - __builtin_clz(cells.block - 1);
  const int deep_bits = block_bits + cells.bits;        // vectors of a cell, of which some may not be there
  // f(vector, place) for the owners' vectors, -inf past the end
  const auto visit = [&](auto f) {
    constexpr uint32_t kAhead = 4;                     // vectors in flight per thread
    constexpr int kThreadBits = THREADS == 64 ? 6 : 8;
    static_assert(THREADS == 1 << kThreadBits, "");
    const uint32_t total = (uint32_t)owners << deep_bits;
    for (uint32_t i = threadIdx.x; i < total; i += THREADS * kAhead) {
      Vec<T, N> v[kAhead];
      uint32_t at[kAhead];
#pragma unroll
      for (uint32_t k = 0; k < kAhead; ++k) {
        const uint32_t j = i + k * THREADS, owner = j < total ? sh.owner[j >> deep_bits] : 0;
        const uint32_t t = j & ((1u << deep_bits) - 1), in = t >> cells.bits;          // step of the block
        const uint32_t group = owner & ((THREADS >> cells.bits) - 1), block = owner >> (kThreadBits - cells.bits);
        const uint32_t step = block * cells.block + in;
        at[k] = j < total && in < cells.block && step < cells.steps
                    ? lo + (step * THREADS + (group << cells.bits) + (t & ((1u << cells.bits) - 1))) * N
                    : hi;
        at[k] = min(at[k], hi);
        if (at[k] + N <= hi) v[k] = load_vec<N>(row + at[k]);
      }
#pragma unroll
      for (uint32_t k = 0; k < kAhead; ++k) {
        if (at[k] + N <= hi) {
          f(v[k], at[k]);
        } else if (at[k] < hi) {
          float w[N];
#pragma unroll
          for (int j = 0; j < N; ++j) w[j] = at[k] + j < hi ? to_f32(row[at[k] + j]) : -INFINITY;
          f(make_vec<T>(w), at[k]);
        }
      }
    }
  };
  // vectors with an entry that reaches the limit, and of these the candidates
  // (a limit below -inf's number, of which the bits that were not looked for are 0, is no entry's)
  const float least = low > order(-INFINITY) ? entry(low) : -INFINITY;
  constexpr int kVectors = kHeld<THREADS> / 4;
  visit([&](const Vec<T, N>& v, uint32_t at) {
    float most = v[0];
#pragma unroll
    for (int j = 1; j < N; ++j) most = fmaxf(most, v[j]);
    if (most > least || (most == least && at < until)) {
      const int n = atomicAdd(&sh.vectors, 1);
      if (n < kVectors) {
        sh.vector[n] = u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
        sh.place[n] = at;
      }
    }
  });
  __syncthreads();
  const int vectors = sh.vectors;
  if (vectors <= kVectors) {
    for (int i = threadIdx.x; i < vectors * N; i += THREADS) {
      const uint32_t at = sh.place[i / N];
      const T* held = (const T*)&sh.vector[i / N];
      const uint32_t o = order(to_f32(held[i % N]));
      if (at + i % N < hi && (o > low || (o == low && at + i % N < until))) {
        const int n = atomicAdd(&sh.count, 1);
        if (n < kHeld<THREADS>) sh.held[n] = (uint64_t)o << 32 | (uint32_t)~(at + i % N);
      }
    }
    __syncthreads();
    if (sh.count <= kHeld<THREADS>) {
      rank<THREADS>(sh.held, sh.count, top, put);
      return;
    }
  }
  // more than fit: one by one
  uint64_t last = ~uint64_t(0);
  for (int k = 0; k < top; ++k) {
    uint64_t best = 0;
    visit([&](const Vec<T, N>& v, uint32_t at) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint64_t n = at + j < hi ? key_of(v[j], at + j) : 0;
        if (n < last && n > best) best = n;
      }
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint64_t other = __shfl_xor((unsigned long long)best, d);
      best = other > best ? other : best;
    }
    if (lane == 0) sh.best[wave] = best;
    __syncthreads();
    for (int w = 0; w < WAVES; ++w) best = sh.best[w] > best ? sh.best[w] : best;
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

// ODD: bf16 rows some of which begin at odd 2-byte addresses, where 16-byte loads are slow: they are loaded from the
// 4-byte boundary below, with the word behind (both words hold a part of the row), and shifted: 4096 x 127999
// 182 us, loaded where they lie 217; with 20 alternatives 208 and 245.  The entries are the same and so are
// all results.
template <typename T, int THREADS, bool TOP, bool SPLIT, bool ODD>
__global__ __launch_bounds__(THREADS) void forward_kernel(const Args a) {
  constexpr int N = 16 / sizeof(T);
  __shared__ Stat slots[THREADS / 64];
  __shared__ TopShared<THREADS> sh;
  const int64_t row = SPLIT ? (int64_t)blockIdx.y : (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  if (!SPLIT && !is_read(a.tokens, a.wide, a.given, row)) return skip_row(a, row);
  const T* x = (const T*)a.logits + row * a.stride;
  const uint32_t lo = SPLIT ? min(blockIdx.x * a.split_size, a.vocab) : 0;
  const uint32_t hi = SPLIT ? min(lo + a.split_size, a.vocab) : a.vocab;
  Stat t{kLowest, 0.0f, 0.0f};
  // the thread's largest entry of a block, and the first vector that holds it
  const Cells<THREADS, N> cells(hi - lo);
  constexpr uint32_t step = THREADS * N;
  const uint32_t start = lo + threadIdx.x * N;
  float most = -INFINITY;
  uint32_t place = start;
  const auto flush = [&](uint32_t block) {            // of the block that ends; then the next begins
    uint64_t key = place < hi ? key_of(most, place) : 0;
    for (int d = 1; d < 1 << cells.bits; d *= 2) {
      const uint64_t other = __shfl_xor((unsigned long long)key, d);
      key = other > key ? other : key;
    }
    if ((threadIdx.x & ((1 << cells.bits) - 1)) == 0)
      sh.cell[(block * THREADS + threadIdx.x) >> cells.bits] = key;
    most = -INFINITY;
    place = start + (block + 1) * cells.block * step;
  };
  if (TOP) {
    sh.cell[threadIdx.x] = 0;
    __syncthreads();
  }
  const auto unit = [&](const Vec<T, N>& v, uint32_t at) {
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
    if (top > (TOP ? most : t.m)) {
      most = top;
      place = at;
      if (top > t.m) t.raise(top, a.c);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) t.add(v[i], a.c);
  };
  // vectors are loaded kAhead at a time, the next ones before these are looked at
  constexpr int kAhead = Cells<THREADS, N>::kStepsAhead;
  struct Batch {
    Vec<T, N> v[kAhead];
    uint32_t behind[ODD ? kAhead : 1];
  };
  const uint32_t shift = ODD ? (uint32_t)(uintptr_t)x & 2 : 0;
  const T* from = (const T*)((const char*)x - shift);
  const uint32_t next_word = shift ? N : 0;
  const auto fetch = [&](Batch& b, int k, uint32_t at) {
    b.v[k] = load_vec<N>(from + at);
    if constexpr (ODD) b.behind[k] = *(const uint32_t*)(from + at + next_word);
  };
  const auto vector = [&](const Batch& b, int k) {
    Vec<T, N> v = b.v[k];
    if constexpr (ODD) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v.w[i] = __builtin_amdgcn_alignbyte(i < 3 ? b.v[k].w[i + 1] : b.behind[k], b.v[k].w[i], shift);
    }
    return v;
  };
  const auto load = [&](uint32_t at) {
    Batch b;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(b, k, at + k * step);
    return b;
  };
  const auto load_rest = [&](uint32_t at) {
    Batch b = {};
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (at + k * step + N <= hi) fetch(b, k, at + k * step);
    return b;
  };
  const uint32_t batches = (hi - lo) / (step * kAhead);          // that all threads have
  uint32_t at = start, block = 0;
  Batch now = batches ? load(at) : load_rest(at);
  // (a part of a row is on its way before it is known whether the row is read)
  if (SPLIT && !is_read(a.tokens, a.wide, a.given, row)) return;
  Given given = {-1, 0.0f};
  if (!SPLIT) given = given_of<T>(a, row);
  uint32_t in = 0;
  const auto take = [&] {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) unit(vector(now, k), at + k * step);
    at += kAhead * step;
    in += kAhead;
    if (TOP && in == cells.block) {
      flush(block++);
      in = 0;
    }
  };
  if (batches) {
    for (uint32_t i = 1; i < batches; ++i) {
      const Batch next = load(at + kAhead * step);
      take();
      now = next;
    }
    const Batch next = load_rest(at + kAhead * step);
    take();
    now = next;
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const uint32_t to = at + k * step;
    if (to + N <= hi) {
      unit(vector(now, k), to);
    } else if (to < hi) {
      float w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = to + i < hi ? to_f32(x[to + i]) : -INFINITY;
      unit(make_vec<T>(w), to);
    }
  }
  if (TOP && block * cells.block < cells.steps) flush(block);
  const Stat whole = join_group<THREADS / 64>(t, a.c, slots);
  if (SPLIT) {
    if (threadIdx.x == 0) {
      float* out = a.part + (row * a.splits + blockIdx.x) * 4;
      out[0] = whole.m, out[1] = whole.z, out[2] = whole.s;
    }
    if (TOP) {
      uint64_t* keys = a.keys + (row * a.splits + blockIdx.x) * a.top;
      if (threadIdx.x < a.top && threadIdx.x >= hi - lo) keys[threadIdx.x] = 0;      // a short last part
      find_top<T, THREADS, N>(x, lo, hi, a.top, cells, sh, [&](int p, uint64_t k) { keys[p] = k; });
    }
  } else {
    const float z = finish_row(a, row, whole, given);
    if (!TOP) return;
    if (!whole.good()) return no_top(a, row);
    find_top<T, THREADS, N>(x, lo, hi, a.top, cells, sh,
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
  const Given given = given_of<T>(a, row);
  // a lane of every wavefront takes a part
  const int lane = threadIdx.x & 63;
  Stat t{kLowest, 0.0f, 0.0f};
  if (lane < a.splits) {
    const float* in = a.part + (row * a.splits + lane) * 4;
    t = Stat{in[0], in[1], in[2]};
  }
  // the k-th largest of the first few of each list is a lower bound for all
  const uint64_t* keys = a.keys + row * a.splits * a.top;
  const int first = min(a.top, 256 / a.splits), some = first * a.splits;
  uint64_t key[4] = {0, 0, 0, 0};
  if (threadIdx.x < 64) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = i * 64 + lane;
      if (j < some) key[i] = keys[j / first * a.top + j % first];
    }
  }
  t.raise(reduce64(t.m, Max()), a.c);
  t.z = reduce64(t.z, Sum());
  t.s = reduce64(t.s, Sum());
  const float z = finish_row(a, row, t, given);
  if (!a.top) return;
  if (!t.good()) return no_top(a, row);
  if (threadIdx.x < 64) {
    const uint64_t t = threshold(key, a.top);
    if (lane == 0) limit = t ? t : 1, count = 0;
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

// A workgroup takes a part of a row.  With y = log2 p: grad = p (A y + B) / T, A = -h ln 2,
// B = -(sum g + h entropy); the given tokens' entries are read before anything is written (grad may be
// logits) and written again at the end with what their g adds.  A 1 / T above 1 multiplies p, one below 1 A and B: no
// factor of a finite gradient is infinite.
// STREAM: past the caches, of a gradient that is more than they hold.  4096 x 128000 bf16 385 us, through them 403.  Of one
// that the last-level cache holds the next reader gains more than the writer loses: 128 x 151000 binary32 with the
// gradient's norm after it 50.2 us, through the caches 44.2.
template <typename T, bool STREAM>
__global__ __launch_bounds__(256) void backward_kernel(const BackArgs a) {
  constexpr int N = 16 / sizeof(T), THREADS = 256;
  __shared__ int64_t id[kMost];
  __shared__ float up[kMost];
  const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (row >= a.rows) return;
  const uint32_t lo = blockIdx.x * a.split_size, hi = min(lo + a.split_size, a.vocab);
  const T* x = (const T*)a.logits + row * a.stride;
  T* grad = (T*)a.grad + row * a.grad_stride;
  constexpr int kAhead = 4;
  // Vectors begin at a line of grad's (each entry's value is its own); the few before are a thread's each.  4096 x 127999
  // bf16 389 us, from the part's begin 463; 8192 x 8191 56 and 74; 4096 x 127999 binary32 785 and 915.
  const uint32_t before = (uint32_t)(-(uintptr_t)(grad + lo) & 127) / sizeof(T);
  const bool first = threadIdx.x < before && lo + threadIdx.x < hi;
  uint32_t at = lo + before + threadIdx.x * N;
  constexpr uint32_t step = THREADS * N;
  const auto whole_batch = [&](uint32_t at) { return at + (kAhead - 1) * step + N <= hi; };
  struct Batch {
    Vec<T, N> v[kAhead];
  };
  const auto load = [&](uint32_t at) {
    Batch b;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) b.v[k] = load_vec<N>(x + at + k * step);
    return b;
  };
  const int i = threadIdx.x & 63;
  int64_t mine = -1;
  if (i < a.given) mine = token(a.tokens, a.wide, row * a.given + i);
  if (__ballot(mine >= 0) == 0) {
    const Vec<T, N> zero = zero_vec<T, N>();
    if (first) grad[lo + threadIdx.x] = from_f32<T>(0.0f);
    for (; at < hi; at += step) store_vec<kAny>(grad, at, hi, zero);
    return;
  }
  // the first vectors are on their way while the row's numbers come
  bool more = whole_batch(at);
  Batch now = {};
  if (more) now = load(at);
  float g = mine < 0 ? 0.0f : a.dlogp[row * a.given + i];
  if (mine >= (int64_t)a.vocab) g = NAN;
  const float m = a.stats[row * 2], z = a.stats[row * 2 + 1];
  const float h = a.dentropy ? a.dentropy[row] : 0.0f, all = reduce64(g, Sum());
  const float below = fminf(a.inv_t, 1.0f), above = fmaxf(a.inv_t, 1.0f);
  const float A = -h * kLn2 * below;
  float B = a.dentropy ? -fmaf(h, a.entropy[row], all) * below : -all * below;
  if (!(z == z)) B = NAN;                          // no distribution
  const float z2 = z * kLog2e;
  const auto value = [&](float e, float by) {
    const float y = fmaxf(fmaf(e - m, a.c, -z2), kNone);
    return exp2_(y) * by * fmaf(A, y, B);
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
    if (fixes) fix = fmaf(fix, below, value(to_f32(x[mine]), 1.0f)) * above;
  }
  __syncthreads();
  const auto unit = [&](const Vec<T, N>& v, uint32_t to) {
    float r[N];
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = value(v[k], above);
    store_vec<kAny, STREAM>(grad, to, hi, make_vec<T>(r));
  };
  if (first) grad[lo + threadIdx.x] = from_f32<T>(value(to_f32(x[lo + threadIdx.x]), above));
  while (more) {
    const uint32_t then = at + kAhead * step;
    more = whole_batch(then);
    const Batch next = load(more ? then : at);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) unit(now.v[k], at + k * step);
    at = then;
    now = next;
  }
  for (; at < hi; at += step) unit(load_vec<N, kAny>(x, at, hi), at);
  __syncthreads();
  if (fixes) grad[mine] = from_f32<T>(fix);
}

constexpr int64_t kCached = int64_t(128) << 20;       // bytes that are likely to stay in the last-level cache
constexpr int64_t kMaxVocab = int64_t(1) << 28, kMaxTokenRows = int64_t(1) << 30;

// Workgroups per row: few long rows are shared by several, where that saves more than a second launch costs.  bf16 with
// 20 alternatives, one workgroup a row against several: 4 x 128000 23.5 us, 12.1; 192 x 128000 26.1, 25.6; 64 x 65536
// 16.3, 14.5; 128 x 65536 16.6, 16.1; 4 x 40960 11.5 both; 4 x 32768 10.6, 11.7; 100 x 32768 11.4, 13.7.
int splits_of(int64_t rows, int64_t vocab) {
  if (rows <= 0 || rows > 512 || vocab < 40960 || rows * 640 > vocab) return 1;
  int64_t want = 512 / rows;                            // 1 at least
  const int64_t most = (vocab + 4095) / 4096;
  want = want < most ? want : most;
  return (int)(want < kMaxSplits ? want : kMaxSplits);
}

template <typename T, int THREADS, bool SPLIT, bool ODD>
void launch_forward(const Args& a, dim3 grid, hipStream_t s) {
  if (a.top) forward_kernel<T, THREADS, true, SPLIT, ODD><<<grid, THREADS, 0, s>>>(a);
  else forward_kernel<T, THREADS, false, SPLIT, ODD><<<grid, THREADS, 0, s>>>(a);
}
template <typename T, int THREADS, bool SPLIT>
void launch_forward(const Args& a, dim3 grid, hipStream_t s) {
  const bool odd = sizeof(T) == 2 && (((uintptr_t)a.logits & 2) || (a.stride & 1));
  if (odd) launch_forward<T, THREADS, SPLIT, sizeof(T) == 2>(a, grid, s);
  else launch_forward<T, THREADS, SPLIT, false>(a, grid, s);
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
  // A wavefront to a row of up to 16 vectors a lane, where there are more rows than the compute units hold workgroups.
  // bf16, 20 alternatives, 256 threads against 64: 4096 x 512 16.4 us, 9.8; 4096 x 2048 17.7, 13.4; 4096 x 8192 26.7,
  // 26.4; 8192 x 16384 61, 77; 1024 x 2048 8.1, 8.6; 16 x 8192 7.4, 12.1; 40 alternatives of 64 cells are too
  // many (4096 x 2048: found one by one).
  if (a.rows > 2048 && a.vocab <= 64 * 16 * (16 / sizeof(T)) && a.top <= 24) launch_forward<T, 64, false>(a, grid, s);
  else launch_forward<T, 256, false>(a, grid, s);
}

template <typename T>
void launch_backward(const BackArgs& a, dim3 grid, hipStream_t s) {
  if (a.rows * a.vocab * (int64_t)sizeof(T) > kCached) backward_kernel<T, true><<<grid, 256, 0, s>>>(a);
  else backward_kernel<T, false><<<grid, 256, 0, s>>>(a);
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
  if (vocab > kMaxVocab || !shape_ok(rows, vocab, stride) || rows > kMaxTokenRows || given < 0 ||
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
      rows > kMaxTokenRows || given < 1 || given > kMost)
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
  // workgroups of up to 16384 elements, all alike (as much as eight divide)
  const int64_t parts = (vocab + 16383) / 16384;
  const uint32_t size = (uint32_t)(((vocab + parts - 1) / parts + 7) / 8 * 8);
  const int64_t line = rows < 32768 ? rows : 32768;
  const BackArgs a = {logits, tokens, stats, entropy, dlogp, dentropy, grad, stride, grad_stride, rows,
                      (uint32_t)vocab, size, (int)given, itype == NVFP4_I64, c, inv_t};
  const dim3 grid((unsigned)((vocab + size - 1) / size), (unsigned)line, (unsigned)((rows + line - 1) / line));
  (void)hipGetLastError();
  if (type == NVFP4_T_BF16) launch_backward<bf16>(a, grid, stream);
  else launch_backward<float>(a, grid, stream);
  return launched();
}
