// Products of a few rows with packed NVFP4 weights for gfx950 (include/nvfp4_answer.h defines the
// operation).
//
// A code (2 significant bits) times its E4M3 scale (4) has 6 significant bits and lies between
// 2^-10 and 2688: exact in bf16.  So the matrix cores take the weights as
// bf16(code * scale), the rows of x as they are, and alpha comes last.  A row of binary32 x goes in
// as three rows of bf16 whose sum it is (24 bits in three times 8), which a small kernel writes first.
//
// A wavefront holds RT tiles of 16 rows of the weights and MT tiles of 16 columns (rows of x).  A
// lane loads 16 bytes of codes of one weight row at a time (32 elements, two scales); four lanes
// read 64 bytes in a row.  Their 32 elements are what four matrix instructions take: which k
// a lane's elements stand for does not matter as long as both operands agree, so the lane
// reads the same 32 elements of its column of x.  The wavefronts of a workgroup take steps of 128 elements
// in turn and add up their tiles in shared memory, in order.
#include "nvfp4_answer.h"
#include "train_common.h"

namespace train {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef u32x2 u32x2_a8 __attribute__((aligned(8)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

constexpr int kMaxRows = NVFP4_MATVEC_MAX_ROWS;
constexpr int kStepK = 128;                 // elements of a weight row that a wavefront takes at a time

struct Matvec {
  const uint16_t* x;        // bf16; binary32 rows are three each
  const uint8_t* codes;
  const uint8_t* scales;
  const float* alpha;
  const void* expert;
  void* y;
  int64_t x_stride, rows, cols;
  int out_rows, picks, experts, group;      // tokens * picks; 1 or 3 rows of x per token
  int wide, f32;                            // 64-bit indices; binary32 y
};

// Eight codes times their scale, as bf16: the low half of each product is zero.
__device__ __forceinline__ bf16x8 decode8(uint32_t w, float scale) {
  uint32_t r[4];
#define PAIR(SEL)                                                              \
  {                                                                            \
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);    \
    r[SEL] = __builtin_amdgcn_perm(__float_as_uint(v[1] * scale),              \
                                   __float_as_uint(v[0] * scale), 0x07060302); \
  }
  PAIR(0) PAIR(1) PAIR(2) PAIR(3)
#undef PAIR
  const u32x4 v = {r[0], r[1], r[2], r[3]};
  return __builtin_bit_cast(bf16x8, v);
}

template <int RT, int MT>
struct Stage {
  u32x4 code[RT];
  uint32_t scale[RT];
  u32x4 x[MT][4];
};

template <int RT, int MT, int W, int DEPTH, bool EXPERT>
__global__ __launch_bounds__(W * 64) void matvec_kernel(const Matvec a) {
  __shared__ float part[W][RT * MT][256];
  __shared__ uint16_t list[EXPERT ? kMaxRows : 1];
  __shared__ int counts[2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = EXPERT ? blockIdx.y : 0;
  const int64_t row0 = (int64_t)blockIdx.x * (RT * 16);
  int count = a.out_rows;
  if (EXPERT) {
    // the rows that go to this expert, in order; behind the end those that go nowhere (expert 0's
    // workgroups write their zeros)
    if (wave == 0) {
      int n = 0, none = 0;
      for (int base = 0; base < a.out_rows; base += 64) {
        const int m = base + lane;
        int64_t id = -1;
        if (m < a.out_rows) id = a.wide ? ((const int64_t*)a.expert)[m] : ((const int32_t*)a.expert)[m];
        const bool mine = m < a.out_rows && id == e;
        const bool lost = m < a.out_rows && e == 0 && (id < 0 || id >= a.experts);
        const uint64_t got = __ballot(mine), gone = __ballot(lost), below = (uint64_t(1) << lane) - 1;
        if (mine) list[n + __popcll(got & below)] = (uint16_t)m;
        if (lost) list[kMaxRows - 1 - none - __popcll(gone & below)] = (uint16_t)m;
        n += __popcll(got);
        none += __popcll(gone);
      }
      if (lane == 0) counts[0] = n, counts[1] = none;
    }
    __syncthreads();
    count = counts[0];
    for (int i = 0; i < counts[1]; ++i) {
      const int64_t m = list[kMaxRows - 1 - i];
      for (int64_t j = row0 + threadIdx.x; j < row0 + RT * 16 && j < a.rows; j += W * 64) {
        if (a.f32) ((float*)a.y)[m * a.rows + j] = 0.0f;
        else ((uint16_t*)a.y)[m * a.rows + j] = 0;
      }
    }
    if (count == 0) return;
  }
  const float alpha = a.alpha[e];
  const int g = lane >> 4;
  // this lane's weight rows (the last one again past the end: what comes of it is not stored)
  const uint8_t* code[RT];
  const uint8_t* scale[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t row = row0 + r * 16 + (lane & 15);
    const int64_t at = (int64_t)e * a.rows + (row < a.rows ? row : a.rows - 1);
    code[r] = a.codes + at * (a.cols / 2) + g * 16;
    scale[r] = a.scales + at * (a.cols / 16) + g * 2;
  }
  const int full = (int)(a.cols / kStepK);
  const int per_pass = MT * 16 / a.group;
  for (int first = 0; first < count; first += per_pass) {
    const int here = min(per_pass, count - first);
    const uint16_t* x[MT];
#pragma unroll
    for (int c = 0; c < MT; ++c) {
      const int col = min(c * 16 + (lane & 15), here * a.group - 1);
      const int i = first + col / a.group;
      const int token = (EXPERT ? (int)list[i] : i) / a.picks;
      x[c] = a.x + (int64_t)(token * a.group + col % a.group) * a.x_stride + g * 32;
    }
    f32x4 acc[RT][MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < MT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const auto load = [&](Stage<RT, MT>& s, int step) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        s.code[r] = *(const u32x4_a8*)(code[r] + (int64_t)step * (kStepK / 2));
        s.scale[r] = *(const u16_a1*)(scale[r] + (int64_t)step * (kStepK / 16));
      }
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s.x[c][i] = *(const u32x4_a2*)(x[c] + (int64_t)step * kStepK + i * 8);
    };
    const auto add = [&](const Stage<RT, MT>& s) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float lo = __builtin_amdgcn_cvt_f32_fp8((int)s.scale[r], 0);
        const float hi = __builtin_amdgcn_cvt_f32_fp8((int)s.scale[r], 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 w = decode8(s.code[r][i], i < 2 ? lo : hi);
#pragma unroll
          for (int c = 0; c < MT; ++c)
            acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                w, __builtin_bit_cast(bf16x8, s.x[c][i]), acc[r][c], 0, 0, 0);
        }
      }
    };
    Stage<RT, MT> s[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (wave + d * W < full) load(s[d], wave + d * W);
    for (int step = wave; step < full; step += DEPTH * W) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (step + d * W < full) {
          add(s[d]);
          if (step + (d + DEPTH) * W < full) load(s[d], step + (d + DEPTH) * W);
        }
      }
    }
    // what is left of the rows: up to 112 elements, blocks of 16 whole
    const int left = (int)(a.cols - (int64_t)full * kStepK) - g * 32;
    if (full * (int64_t)kStepK < a.cols && full % W == wave) {
      Stage<RT, MT> t;
      const int64_t step = full;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        t.code[r] = u32x4{0u, 0u, 0u, 0u};
        t.scale[r] = 0u;
        if (left >= 16) {
          const u32x2 v = *(const u32x2_a8*)(code[r] + step * (kStepK / 2));
          t.code[r][0] = v[0], t.code[r][1] = v[1];
          t.scale[r] = scale[r][step * (kStepK / 16)];
        }
        if (left >= 32) {
          const u32x2 v = *(const u32x2_a8*)(code[r] + step * (kStepK / 2) + 8);
          t.code[r][2] = v[0], t.code[r][3] = v[1];
          t.scale[r] |= (uint32_t)scale[r][step * (kStepK / 16) + 1] << 8;
        }
      }
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t.x[c][i] = u32x4{0u, 0u, 0u, 0u};
          if (left >= i * 8 + 8) t.x[c][i] = *(const u32x4_a2*)(x[c] + step * kStepK + i * 8);
        }
      add(t);
    }
    if (first) __syncthreads();               // the last pass' sums are read
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < MT; ++c) *(f32x4*)&part[wave][r * MT + c][lane * 4] = acc[r][c];
    __syncthreads();
    for (int o = threadIdx.x; o < here * (RT * 16); o += W * 64) {
      const int j = o % (RT * 16), i = o / (RT * 16);
      if (row0 + j >= a.rows) continue;
      float sum = 0.0f;
      for (int p = a.group - 1; p >= 0; --p) {         // the smallest part first
        const int col = i * a.group + p;
        const int at = ((j & 15) >> 2) * 64 + (col & 15) * 4 + (j & 3);
#pragma unroll
        for (int w = 0; w < W; ++w) sum += part[w][(j >> 4) * MT + (col >> 4)][at];
      }
      sum *= alpha;
      const int64_t m = EXPERT ? (int)list[first + i] : first + i, to = m * a.rows + row0 + j;
      if (a.f32) ((float*)a.y)[to] = sum;
      else ((bf16*)a.y)[to] = from_f32<bf16>(sum);
    }
  }
}

// binary32 rows as three bf16 rows each: the upper 8 significant bits, the next, the last.
__global__ __launch_bounds__(256) void split_kernel(const float* x, int64_t stride, int64_t cols,
                                                    uint16_t* out) {
  const int64_t row = blockIdx.y;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= cols) return;
  const Vec<float, 8> v = load_vec<8>(x + row * stride + at);
  u32x4 r[3];
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
#pragma unroll
  for (int p = 0; p < 3; ++p) *(u32x4*)(out + (row * 3 + p) * cols + at) = r[p];
}

template <int RT, int MT, int W, int DEPTH>
void launch(const Matvec& a, int64_t tiles, hipStream_t stream) {
  const dim3 grid((unsigned)((tiles + RT - 1) / RT), (unsigned)a.experts);
  if (a.expert) matvec_kernel<RT, MT, W, DEPTH, true><<<grid, W * 64, 0, stream>>>(a);
  else matvec_kernel<RT, MT, W, DEPTH, false><<<grid, W * 64, 0, stream>>>(a);
}

}  // namespace
}  // namespace train

using namespace train;

NVFP4_EXPORT int nvfp4_answer_abi_version(void) { return NVFP4_ANSWER_ABI_VERSION; }

NVFP4_EXPORT int64_t nvfp4_packed_matvec_workspace(int64_t tokens, int64_t cols, nvfp4_type xtype) {
  if (xtype != NVFP4_T_F32 || tokens <= 0 || tokens > kMaxRows || cols <= 0 || cols > (int64_t(1) << 30)) return 0;
  return tokens * cols * 6;
}

NVFP4_EXPORT nvfp4_status nvfp4_packed_matvec(const void* x, int64_t x_stride, const uint8_t* codes,
                                              const uint8_t* scales, const float* alpha,
                                              const void* expert, int64_t tokens, int64_t picks,
                                              int64_t E, int64_t rows, int64_t cols,
                                              nvfp4_type xtype, nvfp4_type ytype,
                                              nvfp4_index itype, void* y, void* workspace,
                                              hipStream_t stream) {
  if (!known(xtype) || !known(ytype) || (itype != NVFP4_I32 && itype != NVFP4_I64)) return NVFP4_ERR_ENUM;
  if (tokens < 0 || tokens > kMaxRows || picks < 1 || picks > kMaxRows || tokens * picks > kMaxRows ||
      E < 1 || E > 65535 || (!expert && (E != 1 || picks != 1)) || rows < 1 || rows > (int64_t(1) << 30) ||
      cols < 16 || cols % 16 || cols > (int64_t(1) << 30) || !shape_ok(tokens, cols, x_stride) ||
      E > (int64_t(1) << 58) / (rows * cols))
    return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  const int64_t need = nvfp4_packed_matvec_workspace(tokens, cols, xtype), out_rows = tokens * picks;
  if (!x || !codes || !scales || !alpha || !y || (need && !workspace)) return NVFP4_ERR_NULL;
  const int64_t xs = size_of(xtype), ys = size_of(ytype), is = itype == NVFP4_I32 ? 4 : 8;
  if (!aligned(x, xs) || !aligned(codes, 8) || !aligned(alpha, 4) || !aligned(expert, is) ||
      !aligned(y, ys) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const Range in[] = {range(x, extent(tokens, cols, x_stride, xs)), range(codes, E * rows * (cols / 2)),
                      range(scales, E * rows * (cols / 16)), range(alpha, E * 4),
                      range(expert, out_rows * is)};
  const Range out[] = {range(y, out_rows * rows * ys), range(need ? workspace : nullptr, need)};
  for (int o = 0; o < 2; ++o)
    for (const Range& r : in)
      if (overlap(out[o], r)) return NVFP4_ERR_ALIAS;
  if (overlap(out[0], out[1])) return NVFP4_ERR_ALIAS;
  (void)hipGetLastError();
  Matvec a = {(const uint16_t*)x, codes, scales, alpha, expert, y, x_stride, rows, cols, (int)out_rows,
              (int)picks, (int)E, 1, itype == NVFP4_I64, ytype == NVFP4_T_F32};
  if (xtype == NVFP4_T_F32) {
    split_kernel<<<dim3((unsigned)((cols + 2047) / 2048), (unsigned)tokens), 256, 0, stream>>>(
        (const float*)x, x_stride, cols, (uint16_t*)workspace);
    const nvfp4_status st = launched();
    if (st != NVFP4_OK) return st;
    a.x = (const uint16_t*)workspace;
    a.x_stride = cols;
    a.group = 3;
  }
  const int64_t tiles = (rows + 15) / 16;
  const int64_t columns = (out_rows + E - 1) / E * a.group;
  if (columns <= 16) launch<1, 1, 8, 3>(a, tiles, stream);
  else if (columns <= 32) launch<2, 2, 8, 2>(a, tiles, stream);
  else launch<2, 4, 4, 1>(a, tiles, stream);
  return launched();
}
