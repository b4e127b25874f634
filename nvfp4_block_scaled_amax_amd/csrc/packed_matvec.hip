// Products of a few rows with packed NVFP4 weights for gfx950 (include/nvfp4_answer.h defines the
// operation):  y[m, j] = alpha sum_k x[m, k] code[j, k] scale[j, k / 16].
//
// The weights are 0.5625 bytes an element and are read once: with few rows of x that is the floor.
// At one to sixteen rows a 16x16x32 matrix instruction serves 512 weights in 18 cycles of a wavefront, while
// turning their codes into bf16 takes the vector unit longer than that, so the work is bound by the
// reads first and by the vector instructions soon after, never by the matrix cores.
//
// A code (2 significant bits) times its E4M3 scale (4) has 6 significant bits and lies between
// 2^-10 and 2688: exact in bf16.  So the matrix cores take the weights as bf16(code * scale), the rows
// of x as they are, and alpha comes last.  A row of binary32 x goes in as three columns of bf16 whose sum it is
// (24 bits in three times 8), split while x is staged.  Of four columns or fewer (FEW) the other twelve of a
// tile would idle: there the tile's 16 columns are 4 columns of x by 4 groups of 16 elements, zero outside
// the group's own ("block diagonal"), the codes go in alone, one conversion for two elements, and the
// four products of a block are scaled in binary32 afterwards.  4096 x 14336 by one row: 10.0 us (3.3 TB/s),
// with scaled weights 13; 50251 x 4080 by one row 28, scaled 33.
//
// A wavefront takes units of 16 weight rows by 512 elements: a lane holds 64 bytes of one row's codes
// (128 elements, eight scales), four lanes a row's 256.  Which k a lane's elements stand for does not
// matter as long as both operands agree, so the lane reads the same 32 elements at a time of its column of x,
// from shared memory, where each workgroup puts x (as much as fits) before it starts.  Loading by
// lines and transposing the codes through shared memory was not faster (50251 x 4080) or slower (64 rows).
// The last unit of a row ends with the row and overlaps the one before, with x zero there; units past
// the end are loaded from the first one, so that no branch stands between loads and the waits count them.
//
// 2^deal wavefronts share out a tile's units and add up in shared memory, in order; the other
// wavefronts of the workgroup take further tiles, which share its x.
//
// Measured on one MI355X, kernel alone, bf16 x unless it says so: 4096 x 14336 by 1 row 10.0 us; 14336 x 4096 by 16
// rows 13.0 us, by 24 rows 15.6, by 64 rows 24.4; 50251 x 4080 by 7 binary32 rows 40 us (2.9 TB/s); 24 rows to 4 of
// 64 experts of 2048 x 5120, 44 of them hit, 65 us (4.0 TB/s; the weights' loads alone, without any use
// of them, take 47); 131072 x 4096 by 16 rows 70 us (4.3 TB/s).
#include <algorithm>

#include "nvfp4_answer.h"
#include "train_common.h"

namespace train {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef u32x2 u32x2_a8 __attribute__((aligned(8)));

constexpr int kMaxRows = NVFP4_MATVEC_MAX_ROWS;
// Threads of a launch stay below 2^32, offsets within a tile of 16 rows below 2^31.
constexpr int64_t kMaxWeightRows = int64_t(1) << 26, kMaxCols = int64_t(1) << 27;
constexpr int kUnit = 512;                  // elements of 16 weight rows that a wavefront takes at a time

struct Matvec {
  const void* x;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* alpha;
  const void* expert;
  void* y;
  int64_t x_stride, rows, cols;
  int out_rows, picks, experts;             // tokens * picks
  int wide, f32;                            // 64-bit indices; binary32 y
  int lds;                                  // bytes of shared memory for x
  int deal;                                 // log2 of the wavefronts that deal a tile's units among them
};

// Eight codes as bf16.
__device__ __forceinline__ bf16x8 decode8(uint32_t w) {
  u32x4 r;
#define PAIR(SEL) \
  r[SEL] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, SEL));
  PAIR(0) PAIR(1) PAIR(2) PAIR(3)
#undef PAIR
  return __builtin_bit_cast(bf16x8, r);
}
// Eight codes times their scale, as bf16: the low half of each product is zero.
__device__ __forceinline__ bf16x8 decode8(uint32_t w, float scale) {
  u32x4 r;
#define PAIR(SEL)                                                              \
  {                                                                            \
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);    \
    r[SEL] = __builtin_amdgcn_perm(__float_as_uint(v[1] * scale),              \
                                   __float_as_uint(v[0] * scale), 0x07060302); \
  }
  PAIR(0) PAIR(1) PAIR(2) PAIR(3)
#undef PAIR
  return __builtin_bit_cast(bf16x8, r);
}
// Scales 2 `pair` and 2 `pair` + 1 of eight bytes.
__device__ __forceinline__ f32x2 scales_of(u32x2 bytes, int pair) {
  const int w = (int)bytes[pair >> 1];
  return pair & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
}

// What a lane holds of a unit: 128 elements of a weight row, and the scales that it needs.
template <int S>
struct Unit {
  u32x4 code[4];
  u32x2 scale[S];
};

// Eight binary32 values as three times eight bf16 whose sums they are: the upper 8 significant bits, the next, the
// last.
__device__ __forceinline__ void thirds(const Vec<float, 8>& v, u32x4 (&r)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[2][3];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = v[2 * i + h];
      // of an infinity and a NaN (whose lower bits may be all it has) the first part is all
      const bool odd = !(fabsf(f) < INFINITY);
      const float first = odd ? (f != f ? NAN : f) : __uint_as_float(__float_as_uint(f) & 0xFFFF0000u);
      const float rest = odd ? 0.0f : f - first;
      const float second = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u);
      w[h][0] = __float_as_uint(first);
      w[h][1] = __float_as_uint(second);
      w[h][2] = __float_as_uint(rest - second);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) r[p][i] = (w[0][p] >> 16) | (w[1][p] & 0xFFFF0000u);
  }
}

// SHORT: rows of less than a unit.
template <typename X, bool FEW, int MT, int W, bool EXPERT, bool SHORT>
__global__ __launch_bounds__(W * 64) void matvec_kernel(const Matvec a) {
  constexpr int kCols = FEW ? 4 : 16;                // of a tile
  constexpr int kGroup = sizeof(X) == 4 ? 3 : 1;     // columns of a row of x
  constexpr int S = FEW ? 4 : 1;
  extern __shared__ __align__(16) char held[];       // x, then the wavefronts' sums
  // the rows of y that go to this expert, in order, and behind the end those that go nowhere; their tokens
  __shared__ uint16_t list[EXPERT ? kMaxRows : 1], tokens[EXPERT ? kMaxRows : 1];
  __shared__ int counts[2];
  __shared__ u32x4 zeros[FEW ? 16 : 1];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int deal = 1 << a.deal, wr = wave >> a.deal, wk = wave & (deal - 1);
  const int e = EXPERT ? blockIdx.y : 0;
  const int64_t row0 = (int64_t)blockIdx.x * (W * 16 >> a.deal);      // the workgroup's first weight row
  const float alpha = a.alpha[e];
  int count = a.out_rows;
  if (EXPERT) {
    if (wave == 0) {
      int n = 0, none = 0;
      constexpr int kAhead = 4;
      for (int base = 0; base < a.out_rows; base += 64 * kAhead) {
        int64_t id[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int m = min(base + k * 64 + lane, a.out_rows - 1);
          id[k] = a.wide ? ((const int64_t*)a.expert)[m] : ((const int32_t*)a.expert)[m];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int m = base + k * 64 + lane;
          const bool mine = m < a.out_rows && id[k] == e;
          const bool lost = m < a.out_rows && e == 0 && (id[k] < 0 || id[k] >= a.experts);
          const uint64_t got = __ballot(mine), gone = __ballot(lost), below = (uint64_t(1) << lane) - 1;
          if (mine) {
            list[n + __popcll(got & below)] = (uint16_t)m;
            tokens[n + __popcll(got & below)] = (uint16_t)(m / a.picks);
          }
          if (lost) list[kMaxRows - 1 - none - __popcll(gone & below)] = (uint16_t)m;
          n += __popcll(got);
          none += __popcll(gone);
        }
      }
      if (lane == 0) counts[0] = n, counts[1] = none;
    }
    __syncthreads();
    count = counts[0];
    for (int i = 0; i < counts[1] && blockIdx.z == 0; ++i) {      // expert 0's workgroups write zeros
      const int64_t m = list[kMaxRows - 1 - i];
      for (int64_t j = row0 + threadIdx.x; j < row0 + (W * 16 >> a.deal) && j < a.rows; j += W * 64) {
        if (a.f32) ((float*)a.y)[m * a.rows + j] = 0.0f;
        else ((uint16_t*)a.y)[m * a.rows + j] = 0;
      }
    }
    if (count == 0) return;
  }
  if (FEW && threadIdx.x < 16) zeros[threadIdx.x] = u32x4{0u, 0u, 0u, 0u};
  // Units of a row.  What is left behind the whole ones is a unit that ends with the row: x is zero
  // where it overlaps the one before.
  const int cols = (int)a.cols, full = cols / kUnit, all = (cols + kUnit - 1) / kUnit;
  const auto start = [&](int unit) { return SHORT ? 0 : unit < full ? unit * kUnit : cols - kUnit; };
  // the tile's first weight row, this lane's row in it, and the rows of its scales (the last one again
  // past the end: what comes of it is not stored)
  const int64_t row_t = row0 + wr * 16 < a.rows ? row0 + wr * 16 : a.rows - 1;
  const int rows_t = (int)(a.rows - row_t < 16 ? a.rows - row_t : 16);
  const int64_t first_row = (int64_t)e * a.rows + row_t;
  const uint8_t* code = a.codes + first_row * (a.cols / 2);
  const uint8_t* scale = a.scales + first_row * (a.cols / 16);
  const uint32_t code_at = (uint32_t)min(c, rows_t - 1) * (uint32_t)(cols / 2) + g * 64;
  uint32_t scale_at[S];
#pragma unroll
  for (int i = 0; i < S; ++i)
    scale_at[i] = (uint32_t)min(FEW ? g * 4 + i : c, rows_t - 1) * (uint32_t)(cols / 16) + (FEW ? c & 3 : g) * 8;
  // A unit past this wavefront's last one is 64 bytes of its first, read by every lane: no branch stands
  // between loads and the waits can count them.
  const auto load = [&](Unit<S>& u, int unit) {
    const int at = unit < all ? start(unit) : 0;
    const uint32_t there = unit < all ? ~0u : 0u;
    const uint8_t* codes = code + at / 2;
    const uint8_t* scales = scale + at / 16;
    if constexpr (!SHORT) {
#pragma unroll
      for (int q = 0; q < 4; ++q) u.code[q] = *(const u32x4_a8*)(codes + (code_at & there) + q * 16);
#pragma unroll
      for (int i = 0; i < S; ++i) u.scale[i] = *(const u32x2_a1*)(scales + (scale_at[i] & there));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = cols - g * 128 - q * 32;
        u.code[q] = u32x4{0u, 0u, 0u, 0u};
        if (k >= 32) {
          u.code[q] = *(const u32x4_a8*)(codes + code_at + q * 16);
        } else if (k >= 16) {
          const u32x2 v = *(const u32x2_a8*)(codes + code_at + q * 16);
          u.code[q][0] = v[0], u.code[q][1] = v[1];
        }
      }
      const int n = cols / 16 - (FEW ? c & 3 : g) * 8;       // scales that are there
#pragma unroll
      for (int i = 0; i < S; ++i) {
        u.scale[i] = u32x2{0u, 0u};
        if (n >= 8) {
          u.scale[i] = *(const u32x2_a1*)(scales + scale_at[i]);
        } else if (n > 0) {
          uint32_t b[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) b[k] = scales[scale_at[i] + min(k, n - 1)];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < n) u.scale[i][k >> 2] |= b[k] << (8 * (k & 3));
        }
      }
    }
  };
  // rows of x of which a turn of the wavefronts (a unit each, where there are as many) fits: at least one
  const int turn = kUnit * deal;
  const int per_pass = min(MT * kCols, a.lds / (min(turn, all * kUnit) * 2 + 16)) / kGroup;
  for (int first = blockIdx.z * per_pass; first < count; first += per_pass * gridDim.z) {
    const int here = min(per_pass, count - first), wide = here * kGroup;
    // x: all of it, or as many elements of each column as fit, a multiple of a turn
    const int fit = (a.lds / wide - 16) / 2, chunk = (fit >= all * kUnit ? all * kUnit : fit / turn * turn) / kUnit;
    const int pitch = chunk * (kUnit * 2) + 16;
    // A wavefront stages units of rows of x: with 2^beside wavefronts to a row it takes every so-manieth unit of
    // every W / 2^beside-th row, kAhead at a time.  The first ones are asked for before the weights: loads come
    // back in order.
    constexpr int kAhead = FEW || kGroup == 3 || (W == 16 && MT > 1) ? 4 : 8;
    const int beside = 31 - __builtin_clz(min(chunk, W)), row_step = W >> beside;
    struct Place {
      int row, unit;
    };
    const Place begin = {wave >> beside, wave & ((1 << beside) - 1)};
    const auto after = [&](Place p) {
      p.row += row_step;
      if (p.row >= here) {
        p.row = begin.row;
        p.unit += 1 << beside;
      }
      return p;
    };
    Vec<X, 8> v[kAhead];
    // (a place past the last one is the last one again, and no branch stands between the loads)
    const auto fetch = [&](int from, Place p) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = first + min(p.row, here - 1), unit = min(from + min(p.unit, chunk - 1), all - 1);
        const int at = start(unit) + lane * 8;
        const int64_t row = EXPERT ? __builtin_amdgcn_readfirstlane(tokens[i]) : i;
        const X* x = (const X*)a.x + row * a.x_stride;
        v[k] = load_vec<8>(x + (uint32_t)(SHORT ? min(at, cols - 8) : at));
        const bool fresh = SHORT ? at < cols : at >= unit * kUnit;
#pragma unroll
        for (int w = 0; w < Vec<X, 8>::kWords; ++w) v[k].w[w] = fresh ? v[k].w[w] : 0u;
        p = after(p);
      }
    };
    const auto put = [&](Place p) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int col = min(p.row, here - 1) * kGroup, unit = min(p.unit, chunk - 1);
        char* to = held + col * pitch + unit * (kUnit * 2) + lane * 16;
        if constexpr (kGroup == 1) {
          *(u32x4*)to = u32x4{v[k].w[0], v[k].w[1], v[k].w[2], v[k].w[3]};
        } else {
          u32x4 r[3];
          thirds(v[k], r);
#pragma unroll
          for (int q = 0; q < 3; ++q) *(u32x4*)(to + q * pitch) = r[q];
        }
        p = after(p);
      }
      return p;
    };
    fetch(0, begin);
    Unit<S> s;
    load(s, wk);
    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // the lane's column of x: of FEW, four columns a tile, four lanes each; the lanes of group g take the
    // column's elements of group g, the others zeros
    const char* xs[MT];
    int live[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int col = m * kCols + (FEW ? c >> 2 : c);
      live[m] = !FEW || ((c & 3) == g && col < wide) ? -1 : 0;
      xs[m] = live[m] ? held + min(col, wide - 1) * pitch + g * 256 : (const char*)zeros;
    }
    const auto add = [&](const Unit<S>& u, int unit) {        // unit: in the chunk
      const char* from[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) from[m] = xs[m] + ((unit * (kUnit * 2)) & live[m]);
      f32x4 last[MT];                                // of FEW: the products of the block before
      f32x2 by[4];                                   // and the scales of two blocks
      const auto take = [&](int block) {
        if (!(block & 1))
#pragma unroll
          for (int i = 0; i < 4; ++i) by[i] = scales_of(u.scale[i % S], block >> 1);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][i] = fmaf(last[m][i], by[i][block & 1], acc[m][i]);
          // (the sums stay here: moved down behind the loop's branch they would keep every block's products)
          asm volatile("" : "+v"(acc[m]));
        }
      };
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u32x4 x[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[m][i] = *(const u32x4*)(from[m] + q * 64 + i * 16);
        if constexpr (FEW) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bf16x8 w0 = decode8(u.code[q][2 * h]), w1 = decode8(u.code[q][2 * h + 1]);
            f32x4 d[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
              d[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, __builtin_bit_cast(bf16x8, x[m][2 * h]), zero, 0,
                                                             0, 0);
              d[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, __builtin_bit_cast(bf16x8, x[m][2 * h + 1]), d[m],
                                                             0, 0, 0);
            }
            if (q + h) take(2 * q + h - 1);          // while this block's products are under way
#pragma unroll
            for (int m = 0; m < MT; ++m) last[m] = d[m];
            __builtin_amdgcn_sched_barrier(0);
          }
          if (q == 3) take(7);
        } else {
          const f32x2 by = scales_of(u.scale[0], q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bf16x8 w = decode8(u.code[q][i], by[i >> 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x[m][i]), acc[m],
                                                               0, 0, 0);
          }
        }
      }
    };
    int t = wk;
    for (int from = 0; from < all; from += chunk) {
      if (first || from) __syncthreads();            // the chunk before, or the last pass' sums, is read
      if (from) fetch(from, begin);
      for (Place p = put(begin); p.unit < chunk;) {
        fetch(from, p);
        p = put(p);
      }
      lds_barrier();
      const int until = min(from + chunk, all);
      for (; t < until; t += deal) {
        add(s, t - from);
        load(s, t + deal);
      }
    }
    __syncthreads();                                 // x is read
    // [wave][column][16 rows of the tile]
    float* part = (float*)held;
    constexpr int kPart = MT * kCols * 16;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      f32x4 v = acc[m];
      if constexpr (FEW) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] += dpp<0xB1>(v[i]);                   // the four lanes of a column
          v[i] += dpp<0x4E>(v[i]);
        }
        if ((c & 3) == 0) *(f32x4*)(part + wave * kPart + (m * 4 + (c >> 2)) * 16 + g * 4) = v;
      } else {
        *(f32x4*)(part + wave * kPart + (m * 16 + c) * 16 + g * 4) = v;
      }
    }
    __syncthreads();
    constexpr int kRowBits = 4 + (W == 16 ? 4 : W == 8 ? 3 : 2);
    const int row_bits = kRowBits - a.deal;          // the workgroup's weight rows
    for (int o = threadIdx.x; o < here << row_bits; o += W * 64) {
      const int j = o & ((1 << row_bits) - 1), i = o >> row_bits;
      if (row0 + j >= a.rows) continue;
      float sum = 0.0f;
#pragma unroll
      for (int p = kGroup - 1; p >= 0; --p) {          // the smallest part first
        const float* from = part + ((j >> 4) << a.deal) * kPart + (i * kGroup + p) * 16 + (j & 15);
        for (int w = 0; w < deal; ++w) sum += from[w * kPart];
      }
      sum *= alpha;
      const int64_t m = EXPERT ? (int)list[first + i] : first + i, to = m * a.rows + row0 + j;
      if (a.f32) ((float*)a.y)[to] = sum;
      else ((bf16*)a.y)[to] = from_f32<bf16>(sum);
    }
  }
}

constexpr int kOne = 150 * 1024, kTwo = 75 * 1024, kThree = 40 * 1024, kFour = 34 * 1024;

// `room`: shared memory for x, so that one (150 KB) to four workgroups share a compute unit.
template <typename X, bool FEW, int MT, int W, bool EXPERT, bool SHORT = false>
void launch(Matvec a, int64_t columns, int room, int deal, hipStream_t stream) {
  const int64_t tiles = (a.rows + 15) / 16, units = (a.cols + kUnit - 1) / kUnit;
  const auto turn = [](int deal) { return (kUnit * 2 << deal) + 16; };     // bytes of a turn's units of a column
  // The least room for a column: a turn, or the row where it is shorter (a turn of 8 wavefronts for rows of 5 units left
  // room for 5 of 8 columns, and the weights were read twice: 4096 x 3584 by 4 rows 8.1 us, 5.9 at once; 8960 x 2560 by 16
  // rows 23.6, 16.0; 4096 x 5120 by 3 binary32 rows 29.8, 11.3).
  const auto column = [&](int deal) { return std::min<int64_t>(turn(deal), units * (kUnit * 2) + 16); };
  const int64_t hit = a.experts < a.out_rows ? a.experts : a.out_rows;       // weights that are read
  // enough workgroups for the compute units: where the rows are few, more wavefronts deal a tile's units, as
  // far as there are units and every column fits
  constexpr int kMany = 192;
  a.deal = units > 1 ? deal : 0;
  while ((2 << a.deal) <= W && (1 << a.deal) < units && !SHORT && columns * turn(a.deal + 1) <= room &&
         hit * ((tiles << a.deal) / W) < kMany)
    ++a.deal;
  // all of x, or what there is
  const int64_t want = columns * (units * (2 * kUnit) + 16);
  const int least = 3 * (int)column(a.deal);
  a.lds = (int)(want < room ? want : room);
  if (a.lds < least) a.lds = least;
  constexpr int kSums = W * MT * (FEW ? 256 : 1024);
  static_assert(kSums <= kOne && 3 * ((kUnit * 2 * W) + 16) <= kOne, "no call asks for more than a workgroup's own");
  const int bytes = a.lds > kSums ? a.lds : kSums;
  // The passes over the rows of x (of an expert: over twice its share) go one after the other or, where that leaves
  // compute units without a workgroup, side by side: 2048 x 8192 by 64 rows 15.1 us, 40.9 one after the other with 64
  // rows a pass; 512 x 496 by 1024 rows 7.1, 246.
  constexpr int kFull = EXPERT ? 4096 : 8192;                                // wavefronts
  const int64_t per_pass = std::min<int64_t>(MT * (FEW ? 4 : 16), a.lds / column(a.deal)) / (sizeof(X) == 4 ? 3 : 1);
  const int64_t groups = (tiles + (W >> a.deal) - 1) / (W >> a.deal), full = kFull / (groups * hit * W) + 1;
  const int64_t likely = (a.out_rows * (EXPERT ? 2 : 1) + a.experts - 1) / a.experts;
  const dim3 grid((unsigned)groups, (unsigned)a.experts,
                  (unsigned)std::min<int64_t>((likely + per_pass - 1) / per_pass, full));
  const auto kernel = matvec_kernel<X, FEW, MT, W, EXPERT, SHORT>;
  if (bytes > 60 * 1024)      // (the most that any call asks for: calls of several threads agree)
    (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kOne);
  kernel<<<grid, W * 64, bytes, stream>>>(a);
}

// Which form, by sweeps of all of them over 1158 single matrices (128 to 131072 rows, 848 to 16384 columns, 1 to 256
// rows of x of both types) and 534 of 4 to 64 experts (256 to 8192 rows, 512 to 10848 columns, one token to
// 128, 1 to 8 picks, some experts picked more often), weights from memory.  The rules were fitted to 608 and 450 of these,
// where single ones are 3 % off the fastest form on average and the experts' 6 %; over all of them it is 4.5 % (57 % at
// most: 16 binary32 rows to 8960 x 1536) and 7 % (86 %: one binary32 row to 8 of 64 experts of 1408 x 2560).  The
// figures are us, geometric means of all cases that a rule takes where no size stands with them.
template <typename X>
void launch(const Matvec& a, hipStream_t stream) {
  constexpr int kGroup = sizeof(X) == 4 ? 3 : 1;
  const int64_t units = (a.cols + kUnit - 1) / kUnit;
  if (a.expert) {
    // What an expert gets is not known here: `all` / E columns on average.
    const int64_t E = a.experts, all = a.out_rows * kGroup, rows = a.rows * std::min<int64_t>(E, a.out_rows);
    const int64_t work = rows * ((all + 16 * E - 1) / (16 * E));
    if (a.cols < kUnit) launch<X, false, 1, 4, true, true>(a, 16, kOne, 0, stream);
    // Many columns, 64 a pass: 62, 32 columns 65-76, 16 82.
    else if (all >= 20 * E && work > 25000) launch<X, false, 4, 8, true>(a, 64, kOne, 0, stream);
    // Few: the scaled products, 10.7, with 8 wavefronts 11.3, scaled weights 12.4; four workgroups a compute unit (4 rows
    // to 4 of 64 experts of 2048 x 5120 25.2, three 27.9).
    else if (all * kGroup <= E && rows < 64000) launch<X, true, 1, 4, true>(a, 4, kFour, 1, stream);
    // 32 columns a pass: 53.0, 16 columns 52.9-63, 64 57.3.
    else if (units > 4 && all > 5 * E && work > 14700) launch<X, false, 2, 16, true>(a, 32, kOne, 0, stream);
    // Long rows and few of them: 16 wavefronts share a tile's units, 21.5, 8 21.2, 4 24.6 (of the first 450 cases 21.7,
    // 22.5, 26.8).
    else if (units > 4 && rows < 25000) launch<X, false, 1, 16, true>(a, 16, kOne, 0, stream);
    // The others: small workgroups, whose starts (the list of rows, x) hide behind each other's loads, 18.9, with 8
    // wavefronts 20.2, with 16 24.7.  Four workgroups a compute unit where x is short (24 rows to 4 of 64 experts of
    // 5120 x 2048 62, three 68), three where it is long (of 2048 x 5120 63.5, four 64.6).
    else launch<X, false, 1, 4, true>(a, 16, units <= 4 ? kFour : kThree, 0, stream);
    return;
  }
  const int64_t columns = a.out_rows * kGroup, work = a.rows * ((columns + 15) / 16);
  const int64_t some = std::min<int64_t>(columns, 16), x = some * units;
  if (a.cols < kUnit && columns <= 4) {
    launch<X, true, 1, 4, false, true>(a, columns, kOne, 0, stream);
  } else if (a.cols < kUnit) {
    launch<X, false, 1, 4, false, true>(a, 16, kOne, 0, stream);
  } else if (columns <= 4) {
    // The scaled products; 4 wavefronts for short rows and for so many that each workgroup's x is read often
    // (50251 x 4080 28.2, 8 wavefronts 30.4; 4096 x 1024 4.0 and 4.8), 8 for the others (8192 x 8192 11.7 and 15.5).
    if (units <= 2 || a.rows > 32768) launch<X, true, 1, 4, false>(a, columns, kOne, 1, stream);
    else launch<X, true, 1, 8, false>(a, columns, kOne, 1, stream);
  } else if (columns <= 16 || work <= 14700) {
    // 16 columns a pass, by the smallest workgroup that holds them whole: of 4 wavefronts 6.0, where 8 take 6.9 and 16
    // 9.4; of 8 8.7, where 4 take 9.9 and 16 11.5; of 16 20.7, where 8 take 20.9 and 4 24.9.
    if (x <= 36) launch<X, false, 1, 4, false>(a, some, kThree, 0, stream);
    else if (x <= 72) launch<X, false, 1, 8, false>(a, some, kTwo, 0, stream);
    // Long rows and few of them: the scaled products, 8 columns a pass, 9.1, the other forms 12.5 or more.
    else if (a.rows * ((columns + 7) / 8) <= 4100)
      launch<X, true, 2, 8, false>(a, std::min<int64_t>(columns, 8), kOne, 0, stream);
    // (more than one pass over rows of up to 10 units, by 8 wavefronts: 11.6, by 16 13.2)
    else if (columns > 16 && units <= 10) launch<X, false, 1, 8, false>(a, some, kTwo, 0, stream);
    else launch<X, false, 1, 16, false>(a, some, kOne, 0, stream);
  } else if (columns <= 32 || work <= 35000) {
    // 32 columns a pass: 21.0, 16 columns 22.6, 64 26.9.
    launch<X, false, 2, 16, false>(a, std::min<int64_t>(columns, 32), kOne, 0, stream);
  } else {
    // 64 columns a pass: 49.2, 32 columns 57.2, 16 56.9.
    launch<X, false, 4, 8, false>(a, std::min<int64_t>(columns, 64), kOne, 0, stream);
  }
}

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT int nvfp4_answer_abi_version(void) { return NVFP4_ANSWER_ABI_VERSION; }

NVFP4_EXPORT nvfp4_status nvfp4_packed_matvec(const void* x, int64_t x_stride, const uint8_t* codes,
                                              const uint8_t* scales, const float* alpha,
                                              const void* expert, int64_t tokens, int64_t picks,
                                              int64_t E, int64_t rows, int64_t cols,
                                              nvfp4_type xtype, nvfp4_type ytype,
                                              nvfp4_index itype, void* y, hipStream_t stream) {
  if (!known(xtype) || !known(ytype) || (itype != NVFP4_I32 && itype != NVFP4_I64)) return NVFP4_ERR_ENUM;
  if (tokens < 0 || tokens > kMaxRows || picks < 1 || picks > kMaxRows || tokens * picks > kMaxRows ||
      E < 1 || E > 65535 || (!expert && (E != 1 || picks != 1)) || rows < 1 || rows > kMaxWeightRows ||
      cols < 16 || cols % 16 || cols > kMaxCols || !shape_ok(tokens, cols, x_stride) ||
      E > (int64_t(1) << 58) / (rows * cols))
    return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!x || !codes || !scales || !alpha || !y) return NVFP4_ERR_NULL;
  const int64_t xs = size_of(xtype), ys = size_of(ytype), is = itype == NVFP4_I32 ? 4 : 8;
  if (!aligned(x, xs) || !aligned(codes, 8) || !aligned(alpha, 4) || !aligned(expert, is) || !aligned(y, ys))
    return NVFP4_ERR_ALIGN;
  const int64_t out_rows = tokens * picks;
  const Range in[] = {range(x, extent(tokens, cols, x_stride, xs)), range(codes, E * rows * (cols / 2)),
                      range(scales, E * rows * (cols / 16)), range(alpha, E * 4),
                      range(expert, out_rows * is)};
  for (const Range& r : in)
    if (overlap(range(y, out_rows * rows * ys), r)) return NVFP4_ERR_ALIAS;
  (void)hipGetLastError();
  const Matvec a = {x, codes, scales, alpha, expert, y, x_stride, rows, cols, (int)out_rows, (int)picks, (int)E,
                    itype == NVFP4_I64, ytype == NVFP4_T_F32, 0, 0};
  if (xtype == NVFP4_T_F32) launch<float>(a, stream);
  else launch<bf16>(a, stream);
  return launched();
}
