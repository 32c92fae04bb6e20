// Low-rank corrections of a batch whose rows use different adapters, for
// gfx950: with g the adapter of row m (a group of the plan),
//   T[m] = X[m] A_g^T                        A_g [r, K], fp32 sums
//   out[m, n] = Y[m, n] + scale_g sum_j T[m, j] B_g[n, j]
// and out[m] = Y[m] for rows without an adapter.
//
//  * down: a workgroup takes a tile of the plan (16 MT rows of one group) and
//    one block of K, up to 128 columns of r; its eight waves split the block's 32-wide
//    steps (v_mfma_f32_16x16x32_bf16, A's rows as the row operand) and add
//    their sums through LDS.  The fp32 sums of every K block go to the
//    workspace, one row per position of the plan: few rows give few tiles, so
//    K is split until the grid covers the CUs, and the second product adds
//    the blocks in order as it reads them (no third launch).
//  * up: a wave takes 16 positions and runs along N in steps of 64 features.
//    It adds the K blocks' sums of its rows once and keeps them in registers
//    as bf16 terms: two (hi + lo, 16 bits of the fp32 sum) for a bf16 output,
//    three (24 bits, all of it) for an fp32 one, so that the correction is
//    not rounded before the output is.  The products with bf16 B are exact in
//    the fp32 accumulator's inputs.  The features of a step are dealt to the
//    MFMA rows so that a lane ends with consecutive ones of one row, which it
//    reads from Y and writes to out in 16-byte pieces.  Bound by Y and out.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device.h"
#include "launchers.h"

namespace convrot {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kDownWaves = 8;
constexpr int kUpWaves = 4;
// Columns of r per down workgroup: a wave's fragments and accumulators of
// more would not fit its registers, so higher ranks read X again.
constexpr int kDownCols = 128;

struct LoraArgs {
  const __bf16* X;
  int64_t ldx;
  const __bf16* A;
  int64_t lda, stride_a;
  const __bf16* B;
  int64_t ldb, stride_b;
  const float* scales;
  const int32_t* order;
  const int32_t* offsets;
  const int32_t* list;
  const int32_t* count;
  int M, K, N, r, groups;
  int nb, spb;  // K blocks and 32-wide steps per block
  int rb;       // blocks of kDownCols columns of r
  float* P;     // [nb][M][r], rows by position
  const void* Y;
  int64_t ldy;
  void* out;
  int64_t ldo;
  int col_steps;  // 64-feature steps per wave
  int col_blocks;
  bool copy;      // rows without an adapter are copied (out is not Y)
  bool vec;       // 16-byte pieces of Y and out
};

__device__ __forceinline__ i32x4 load8(const __bf16* p, bool live) {
  return live ? *reinterpret_cast<const i32x4*>(p) : i32x4{0, 0, 0, 0};
}

template <int RT, int MT>  // 16-column tiles of r, 16-row tiles
__global__ __launch_bounds__(64 * kDownWaves) void lora_grouped_down_kernel(LoraArgs a) {
  __shared__ f32x4 partial[kDownWaves - 1][MT * RT][64];
  const int tile = blockIdx.x / (a.nb * a.rb), kb = blockIdx.x / a.rb % a.nb;
  const int c0 = blockIdx.x % a.rb * kDownCols;
  if (tile >= *a.count) return;
  const int group = a.list[2 * tile], p0 = a.list[2 * tile + 1];
  const int first = a.offsets[group], last = a.offsets[group + 1];
  const int cnt = min(plan_tile_rows(last - first, MT == 4 ? 2 : 0), last - p0);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int row = lane & 15, ch = lane >> 4;
  const int steps = (a.K + 31) / 32;
  const int b0 = kb * a.spb, b1 = min(steps, b0 + a.spb);
  const int per = (b1 - b0 + kDownWaves - 1) / kDownWaves;
  const int s0 = b0 + wid * per, s1 = min(b1, s0 + per);
  const __bf16* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    x[i] = a.X + static_cast<int64_t>(a.order[p0 + min(16 * i + row, cnt - 1)]) * a.ldx + 8 * ch;
  const __bf16* w = a.A + group * a.stride_a + (c0 + row) * a.lda + 8 * ch;
  f32x4 acc[MT][RT] = {};
  struct Frags {
    i32x4 x[MT];
    i32x4 w[RT];
  };
  auto load = [&](int st, Frags& f) {
    const int k = 32 * st;
    const bool live = k + 8 * ch < a.K;
#pragma unroll
    for (int i = 0; i < MT; ++i) f.x[i] = load8(x[i] + k, live);
#pragma unroll
    for (int j = 0; j < RT; ++j) f.w[j] = load8(w + static_cast<int64_t>(16 * j) * a.lda + k, live && c0 + 16 * j < a.r);
  };
  auto mma = [&](const Frags& f) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.w[j]),
                                                            __builtin_bit_cast(bf16x8, f.x[i]), acc[i][j], 0, 0, 0);
  };
  Frags fa, fb;
  if (s0 < s1) load(s0, fa);
  for (int st = s0; st < s1; st += 2) {
    if (st + 1 < s1) load(st + 1, fb);
    mma(fa);
    if (st + 1 >= s1) break;
    if (st + 2 < s1) load(st + 2, fa);
    mma(fb);
  }
  if (wid > 0) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) partial[wid - 1][i * RT + j][lane] = acc[i][j];
  }
  __syncthreads();
  if (wid != 0) return;
  // Lane holds position p0 + 16 i + row and columns c0 + 16 j + 4 ch + e.
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (16 * i + row >= cnt) continue;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if (c0 + 16 * j >= a.r) break;
      f32x4 v = acc[i][j];
#pragma unroll
      for (int q = 0; q < kDownWaves - 1; ++q) v += partial[q][i * RT + j][lane];
      *reinterpret_cast<f32x4*>(a.P + (static_cast<int64_t>(kb) * a.M + p0 + 16 * i + row) * a.r + c0 + 16 * j +
                                4 * ch) = v;
    }
  }
}

// OUT: 0 = fp32, 1 = bf16.  KS: 32-wide steps of r.  MT: 16-position tiles per
// workgroup; its four waves are MT position tiles x 4 / MT column ranges.
template <int OUT, int KS, int MT>
__global__ __launch_bounds__(64 * kUpWaves) void lora_grouped_up_kernel(LoraArgs a) {
  using out_t = typename std::conditional<OUT == 0, float, __bf16>::type;
  constexpr int kTerms = OUT == 0 ? 3 : 2;
  constexpr int kVec = 16 / static_cast<int>(sizeof(out_t));
  typedef out_t vec_t __attribute__((ext_vector_type(kVec)));
  const int tile = blockIdx.x / a.col_blocks;
  if (tile >= *a.count) return;
  const int group = a.list[2 * tile], p0 = a.list[2 * tile + 1];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int row = lane & 15, ch = lane >> 4;
  const int sub = wid % MT;
  const int begin = a.offsets[group], last = group < a.groups ? a.offsets[group + 1] : a.M;
  const int end = min(last, p0 + plan_tile_rows(last - begin, MT == 4 ? 2 : 0));
  const int cnt = min(16, end - p0 - 16 * sub);
  if (cnt <= 0 || (group == a.groups && !a.copy)) return;
  const int pos = p0 + 16 * sub + min(row, cnt - 1);
  const int64_t m = a.order[pos];
  const bool live_row = row < cnt;
  const out_t* y = static_cast<const out_t*>(a.Y) + m * a.ldy;
  out_t* o = static_cast<out_t*>(a.out) + m * a.ldo;

  bf16x8 t[KS][kTerms] = {};
  float scale = 0.f;
  const __bf16* bw = a.B;
  if (group < a.groups) {
    scale = a.scales[group];
    bw += group * a.stride_b;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = 32 * s + 8 * ch;
      f32x4 v[2] = {};
      if (c < a.r) {
        for (int b = 0; b < a.nb; ++b) {
          const f32x4* p = reinterpret_cast<const f32x4*>(a.P + (static_cast<int64_t>(b) * a.M + pos) * a.r + c);
          v[0] += p[0];
          v[1] += p[1];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float rest = v[e / 4][e % 4];
#pragma unroll
        for (int q = 0; q < kTerms; ++q) {
          t[s][q][e] = static_cast<__bf16>(rest);
          rest -= static_cast<float>(t[s][q][e]);
        }
      }
    }
  }

  // Step: 64 features from n0.  MFMA tile j, row i holds feature
  // n0 + kSpan (i / 4) + 4 j' + i % 4 (see feature()): a lane's accumulators
  // of kVec / 4 consecutive tiles are kVec consecutive features.
  const int first = (blockIdx.x % a.col_blocks * (kUpWaves / MT) + wid / MT) * a.col_steps * 64;
  for (int it = 0; it < a.col_steps; ++it) {
    const int n0 = first + 64 * it;
    if (n0 >= a.N) break;
    constexpr int kPer = kVec / 4;  // MFMA tiles per 16-byte piece (1 or 2)
    // First feature of lane (ch)'s piece q of the step, q < 4 / kPer.
    auto piece = [&](int q, int c) { return n0 + 4 * kVec * q + kVec * c; };
    f32x4 acc[4] = {};
    vec_t old[4 / kPer];
    bool full[4 / kPer];
#pragma unroll
    for (int q = 0; q < 4 / kPer; ++q) {
      const int n = piece(q, ch);
      full[q] = a.vec && n + kVec <= a.N;
      if (full[q]) old[q] = *reinterpret_cast<const vec_t*>(y + n);
    }
    if (group < a.groups) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int f = min(piece(j / kPer, row >> 2) + 4 * (j % kPer) + (row & 3), a.N - 1);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int c = 32 * s + 8 * ch;
          const i32x4 b = load8(bw + static_cast<int64_t>(f) * a.ldb + c, c < a.r);
#pragma unroll
          for (int q = 0; q < kTerms; ++q)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), t[s][q], acc[j], 0, 0, 0);
        }
      }
    }
    if (!live_row) continue;
#pragma unroll
    for (int q = 0; q < 4 / kPer; ++q) {
      const int n = piece(q, ch);
      if (full[q]) {
        vec_t v = old[q];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          v[e] = static_cast<out_t>(fmaf(scale, acc[q * kPer + e / 4][e % 4], static_cast<float>(v[e])));
        *reinterpret_cast<vec_t*>(o + n) = v;
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (n + e < a.N)
            o[n + e] = static_cast<out_t>(fmaf(scale, acc[q * kPer + e / 4][e % 4], static_cast<float>(y[n + e])));
      }
    }
  }
}

// Rows per tile: tiles of 64 rows where groups hold that many on average
// (less of A and B is read again), of 16 otherwise.
int tile_list(int64_t M, int64_t E) { return M / E >= 32 ? 2 : 0; }
// Down products keep 16-row tiles above rank 64, whose accumulators fill the
// registers.
int down_list(int64_t M, int64_t E, int64_t r) { return r <= 64 ? tile_list(M, E) : 0; }

int down_blocks(int64_t M, int64_t K, int64_t r, int64_t E) {
  const int64_t tiles = plan_max_tiles(M, E, down_list(M, E, r));
  const int64_t steps = (K + 31) / 32;
  int64_t nb = (2 * device_cus() + tiles - 1) / tiles;
  nb = std::min<int64_t>(nb, std::max<int64_t>(1, steps / (2 * kDownWaves)));
  nb = std::min<int64_t>(nb, 16);
  const int64_t spb = (steps + nb - 1) / nb;
  return static_cast<int>((steps + spb - 1) / spb);
}

template <int OUT, int KS>
void launch_up(LoraArgs a, const RowPlan& plan, hipStream_t stream) {
  const int b = tile_list(a.M, a.groups);
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + kPlanLists + b;  // with the tiles of rows without an adapter
  const int64_t tiles = plan_max_tiles(plan.pairs, plan.groups, b);
  const int ranges = b == 2 ? 1 : kUpWaves;  // column ranges per workgroup
  const int64_t steps = (a.N + 63) / 64;
  // Up to four steps per wave (a row's sums are read once for all of them)
  // while the grid still holds four workgroups per CU.
  int64_t per = 4;
  while (per > 1 && tiles * ((steps + per * ranges - 1) / (per * ranges)) < 4 * device_cus()) per /= 2;
  a.col_steps = static_cast<int>(per);
  a.col_blocks = static_cast<int>((steps + per * ranges - 1) / (per * ranges));
  const dim3 grid(static_cast<unsigned>(tiles * a.col_blocks));
  if (b == 2)
    hipLaunchKernelGGL((lora_grouped_up_kernel<OUT, KS, 4>), grid, dim3(64 * kUpWaves), 0, stream, a);
  else
    hipLaunchKernelGGL((lora_grouped_up_kernel<OUT, KS, 1>), grid, dim3(64 * kUpWaves), 0, stream, a);
}

template <int OUT>
void launch_up_r(const LoraArgs& a, const RowPlan& plan, hipStream_t stream) {
  if (a.r <= 32)
    launch_up<OUT, 1>(a, plan, stream);
  else if (a.r <= 64)
    launch_up<OUT, 2>(a, plan, stream);
  else if (a.r <= 128)
    launch_up<OUT, 4>(a, plan, stream);
  else
    launch_up<OUT, 8>(a, plan, stream);
}

}  // namespace

int64_t lora_grouped_ws_bytes(int64_t M, int64_t K, int64_t r, int64_t E) {
  return M == 0 || E == 0 ? 0 : 4 * down_blocks(M, K, r, E) * M * r;
}

hipError_t launch_lora_grouped(const void* X, int64_t ldx, const void* A, int64_t lda, int64_t stride_a,
                               const void* B, int64_t ldb, int64_t stride_b, const float* scales, int64_t M,
                               int64_t K, int64_t N, int64_t r, const RowPlan& plan, const void* Y, int64_t ldy,
                               void* out, int64_t ldo, Elt dt, void* ws, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  LoraArgs a{};
  a.X = static_cast<const __bf16*>(X);
  a.ldx = ldx;
  a.A = static_cast<const __bf16*>(A);
  a.lda = lda;
  a.stride_a = stride_a;
  a.B = static_cast<const __bf16*>(B);
  a.ldb = ldb;
  a.stride_b = stride_b;
  a.scales = scales;
  a.order = plan.order;
  a.offsets = plan.offsets;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.r = static_cast<int>(r);
  a.groups = plan.groups;
  a.P = static_cast<float*>(ws);
  a.Y = Y;
  a.ldy = ldy;
  a.out = out;
  a.ldo = ldo;
  a.copy = Y != out;
  const int64_t elt = dt == Elt::F32 ? 4 : 2;
  auto rows16 = [&](const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * elt) % 16 == 0;
  };
  a.vec = rows16(Y, ldy) && rows16(out, ldo);
  const int b = down_list(M, plan.groups, r);
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + b;
  a.nb = down_blocks(M, K, r, plan.groups);
  a.spb = ((a.K + 31) / 32 + a.nb - 1) / a.nb;
  a.rb = (a.r + kDownCols - 1) / kDownCols;
  const dim3 grid(static_cast<unsigned>(plan_max_tiles(plan.pairs, plan.groups, b) * a.nb * a.rb)), block(64 * kDownWaves);
#define CONVROT_DOWN(RT_, MT_) hipLaunchKernelGGL((lora_grouped_down_kernel<RT_, MT_>), grid, block, 0, stream, a)
  if (r <= 16) {
    if (b == 2) CONVROT_DOWN(1, 4); else CONVROT_DOWN(1, 1);
  } else if (r <= 32) {
    if (b == 2) CONVROT_DOWN(2, 4); else CONVROT_DOWN(2, 1);
  } else if (r <= 64) {
    if (b == 2) CONVROT_DOWN(4, 4); else CONVROT_DOWN(4, 1);
  } else {
    CONVROT_DOWN(8, 1);
  }
#undef CONVROT_DOWN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dt == Elt::F32)
    launch_up_r<0>(a, plan, stream);
  else
    launch_up_r<1>(a, plan, stream);
  return hipGetLastError();
}

}  // namespace convrot
