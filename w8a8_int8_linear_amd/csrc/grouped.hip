// Grouped linears for gfx950: rows of one packed activation that meet
// different weights of a stack (the experts' products of a routed layer).
//
//   position i of the plan's order, pair q = order[i], group e:
//   Y[dest] = act(acc(x, W_e) s_x s_w + b)    or    act(gate) * up
//
// with x the packed row of pair q (row q / per_row, row q, or row i) and dest
// row q or i.  The accumulator is the exact int32 product, and the epilogue
// is the other linears' expression in the same precision, so that a group's
// rows carry the bits that convrot_linear (_act, _gated) gives for its weight
// alone.
//
// Streaming kernel.  A workgroup takes one tile of the plan (up to 16 MT
// positions of one group) and 16 output features; its waves split K into
// runs of 64-byte steps (v_mfma_i32_16x16x64_i8, weights as the row operand)
// straight from memory into registers, add their partial sums through LDS and
// finish 16 positions per wave.  Bound by the weights' bytes where groups
// hold few rows; every group's weight is read once per tile.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "device.h"
#include "epilogue.h"
#include "launchers.h"

namespace convrot {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct GroupedArgs {
  const uint8_t* A;
  int64_t lda;
  const float* sa;
  const uint8_t* B;
  int64_t ldb;
  const float* sb;
  const float* bias;
  const uint8_t* B2;
  int64_t ldb2;
  const float* sb2;
  const float* bias2;
  const int32_t* order;
  const int32_t* offsets;
  const int32_t* list;   // tiles of the plan, {group, first position}
  const int32_t* count;  // how many of them
  int per_row;
  int source;  // RowOrder of A's rows
  int dest;    // RowOrder of C's rows
  int act;
  int N;
  int K;
  void* C;
  int64_t ldc;
  int tiles_n;   // feature blocks
  bool vec_out;  // rows of C take 16-byte stores
};

// SiLU, y / (1 + e^{-y}), with the hardware exp2 and reciprocal (at
// 2^.. = inf the reciprocal is 0).
__device__ __forceinline__ float silu(float y) {
  return y * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(y * -1.4426950408889634f));
}

__device__ __forceinline__ float apply_act(int act, float y) {
  switch (act) {  // uniform
    case 1: return activation<1>(y);
    case 2: return activation<2>(y);
    case 3: return silu(y);
    default: return y;
  }
}

__device__ __forceinline__ int64_t row_of(int order, int pos, int pair, int per_row) {
  return order == static_cast<int>(RowOrder::Sorted) ? pos
         : order == static_cast<int>(RowOrder::Pair) ? pair
                                                     : pair / per_row;
}

template <typename T>
__device__ __forceinline__ bool aligned4(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0;
}

// Four consecutive features of one output row, the columns past N dropped.
template <int OUT>
__device__ __forceinline__ void store4(void* C, int64_t at, int n, int N, const float y[4]) {
  if constexpr (OUT == 0) {
    float* out = static_cast<float*>(C) + at + n;
    if (n + 3 < N && aligned4(out)) {
      *reinterpret_cast<f32x4*>(out) = f32x4{y[0], y[1], y[2], y[3]};
    } else {
      for (int r = 0; r < 4 && n + r < N; ++r) out[r] = y[r];
    }
  } else {
    __bf16* out = static_cast<__bf16*>(C) + at + n;
    if (n + 3 < N && aligned4(out)) {
      *reinterpret_cast<bf16x4*>(out) = bf16x4{static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                                               static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
    } else {
      for (int r = 0; r < 4 && n + r < N; ++r) out[r] = static_cast<__bf16>(y[r]);
    }
  }
}

}  // namespace
}  // namespace convrot

#include "grouped_tile.h"

namespace convrot {
namespace {

template <int OUT, bool GATED, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void grouped_stream_kernel(GroupedArgs a) {
  constexpr int kW = GATED ? 2 : 1;
  constexpr int kAhead = 4;  // K steps in flight
  static_assert(MT <= WAVES, "one wave finishes each 16 positions");
  __shared__ i32x4 partial[WAVES][kW][MT][64];
  const int tile = blockIdx.x / a.tiles_n;
  if (tile >= *a.count) return;
  const int n0 = (blockIdx.x % a.tiles_n) * 16;
  const int group = a.list[2 * tile], p0 = a.list[2 * tile + 1];
  const int cnt = min(16 * MT, a.offsets[group + 1] - p0);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int row = lane & 15, ch = lane >> 4;

  // Rows past the tile's last re-read it; features past the last likewise.
  // Their results are dropped.
  const uint8_t* x[MT];
  int pos[MT], pair[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    pos[t] = p0 + min(16 * t + row, cnt - 1);
    pair[t] = a.order[pos[t]];
    x[t] = a.A + row_of(a.source, pos[t], pair[t], a.per_row) * a.lda + 16 * ch;
  }
  const int64_t wrow = static_cast<int64_t>(group) * a.N + min(n0 + row, a.N - 1);
  const uint8_t* w[kW];
  w[0] = a.B + wrow * a.ldb + 16 * ch;
  if constexpr (GATED) w[1] = a.B2 + wrow * a.ldb2 + 16 * ch;

  const int steps = (a.K + 63) / 64;
  const int per = (steps + WAVES - 1) / WAVES;
  const int s0 = wid * per, s1 = min(steps, s0 + per);
  i32x4 acc[kW][MT] = {};
  for (int s = s0; s < s1; s += kAhead) {
    i32x4 fw[kAhead][kW], fx[kAhead][MT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool live = s + u < s1 && 64 * (s + u) + 16 * ch < a.K;
      const int64_t k = 64 * static_cast<int64_t>(s + u);
#pragma unroll
      for (int j = 0; j < kW; ++j) fw[u][j] = live ? *reinterpret_cast<const i32x4*>(w[j] + k) : i32x4{};
#pragma unroll
      for (int t = 0; t < MT; ++t) fx[u][t] = live ? *reinterpret_cast<const i32x4*>(x[t] + k) : i32x4{};
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < kW; ++j)
          acc[j][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][j], fx[u][t], acc[j][t], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < kW; ++j)
#pragma unroll
    for (int t = 0; t < MT; ++t) partial[wid][j][t][lane] = acc[j][t];
  __syncthreads();
  // Lane holds position 16 t + row and features n0 + 4 ch + r.
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (wid != t || 16 * t + row >= cnt) continue;
    const float sr = a.sa[row_of(a.source, pos[t], pair[t], a.per_row)];
    const int64_t out = row_of(a.dest, pos[t], pair[t], a.per_row) * a.ldc;
    i32x4 sum[kW];
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      sum[j] = partial[0][j][t][lane];
#pragma unroll
      for (int v = 1; v < WAVES; ++v) sum[j] += partial[v][j][t][lane];
    }
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t col = static_cast<int64_t>(group) * a.N + min(n0 + 4 * ch + r, a.N - 1);
      const float z = fmaf(static_cast<float>(sum[0][r]), sr * a.sb[col], a.bias != nullptr ? a.bias[col] : 0.f);
      y[r] = apply_act(a.act, z);
      if constexpr (GATED)
        y[r] *= fmaf(static_cast<float>(sum[1][r]), sr * a.sb2[col], a.bias2 != nullptr ? a.bias2[col] : 0.f);
    }
    store4<OUT>(a.C, out, n0 + 4 * ch, a.N, y);
  }
}

template <int OUT, bool GATED>
hipError_t launch_stream(GroupedArgs a, const RowPlan& plan, hipStream_t stream) {
  // Tiles of 16 positions, or of more where groups hold more on average, so
  // that a group's weight is read by few workgroups.
  const int64_t avg = plan.pairs / plan.groups;
  const int b = avg <= 16 ? 0 : avg <= 32 ? 1 : 2;
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + b;
  a.tiles_n = (a.N + 15) / 16;
  const dim3 grid(static_cast<unsigned>(plan_max_tiles(plan.pairs, plan.groups, b) * a.tiles_n));
  // Eight waves where each still gets two K steps.
  const bool wide = a.K >= 1024;
#define CONVROT_GROUPED(MT_)                                                                              \
  if (wide)                                                                                               \
    hipLaunchKernelGGL((grouped_stream_kernel<OUT, GATED, MT_, 8>), grid, dim3(512), 0, stream, a);       \
  else                                                                                                    \
    hipLaunchKernelGGL((grouped_stream_kernel<OUT, GATED, MT_, 4>), grid, dim3(256), 0, stream, a)
  switch (b) {
    case 0: CONVROT_GROUPED(1); break;
    case 1: CONVROT_GROUPED(2); break;
    default: CONVROT_GROUPED(4); break;
  }
#undef CONVROT_GROUPED
  return hipGetLastError();
}

template <int OUT, bool GATED, bool KTAIL>
hipError_t launch_tile_typed(GroupedArgs a, const RowPlan& plan, hipStream_t stream) {
  auto kern = tile::grouped_tile_kernel<OUT, GATED, KTAIL>;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), tile::kSmem, lds_set);
  if (e != hipSuccess) return e;
  constexpr int b = 4;  // tiles of 256 positions
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + b;
  constexpr int kFeat = GATED ? tile::kRows / 2 : tile::kRows;
  a.tiles_n = (a.N + kFeat - 1) / kFeat;
  const int elt = OUT == 0 ? 4 : 2;
  a.vec_out = (reinterpret_cast<uintptr_t>(a.C) & 15) == 0 && (a.ldc * elt) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(plan_max_tiles(plan.pairs, plan.groups, b) * a.tiles_n));
  hipLaunchKernelGGL(kern, grid, dim3(tile::kThreads), tile::kSmem, stream, a);
  return hipGetLastError();
}

template <int OUT, bool GATED>
hipError_t launch_grouped(const GroupedArgs& a, const RowPlan& plan, hipStream_t stream) {
  if (plan.pairs / plan.groups < 64) return launch_stream<OUT, GATED>(a, plan, stream);
  return a.K % tile::kSlice != 0 ? launch_tile_typed<OUT, GATED, true>(a, plan, stream)
                                 : launch_tile_typed<OUT, GATED, false>(a, plan, stream);
}

}  // namespace

hipError_t launch_linear_grouped(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* sa,
                                 const float* sb, const float* bias, const int8_t* B2, int64_t ldb2, const float* sb2,
                                 const float* bias2, bool gated, Act act, const RowPlan& plan, RowOrder source,
                                 RowOrder dest, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                                 hipStream_t stream) {
  if (plan.pairs == 0 || plan.groups == 0 || N == 0) return hipSuccess;
  GroupedArgs a{};
  a.A = reinterpret_cast<const uint8_t*>(A);
  a.lda = lda;
  a.sa = sa;
  a.B = reinterpret_cast<const uint8_t*>(B);
  a.ldb = ldb;
  a.sb = sb;
  a.bias = bias;
  a.B2 = reinterpret_cast<const uint8_t*>(B2);
  a.ldb2 = ldb2;
  a.sb2 = sb2;
  a.bias2 = bias2;
  a.order = plan.order;
  a.offsets = plan.offsets;
  a.per_row = plan.per_row;
  a.source = static_cast<int>(source);
  a.dest = static_cast<int>(dest);
  a.act = static_cast<int>(act);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.C = C;
  a.ldc = ldc;
  if (out == Elt::F32)
    return gated ? launch_grouped<0, true>(a, plan, stream) : launch_grouped<0, false>(a, plan, stream);
  return gated ? launch_grouped<1, true>(a, plan, stream) : launch_grouped<1, false>(a, plan, stream);
}

}  // namespace convrot
