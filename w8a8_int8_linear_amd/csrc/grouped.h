// Operands and helpers shared by the kernels of the grouped linears.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "device.h"
#include "epilogue.h"
#include "launchers.h"

namespace convrot {

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
  int pairs;
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

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));


// SiLU, y / (1 + e^{-y}), with the hardware exp2 and reciprocal (at
// 2^.. = inf the reciprocal is 0).
__device__ __forceinline__ float silu(float y) {
  return y * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(y * -1.4426950408889634f));
}

template <int ACT>
__device__ __forceinline__ float act_of(float y) {
  if constexpr (ACT == 3)
    return silu(y);
  else
    return activation<ACT>(y);
}
template <int ACT, int N>
__device__ __forceinline__ void act_all(float* y) {
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = act_of<ACT>(y[i]);
}
// The activation of N values in place, one uniform branch for all.
template <int N>
__device__ __forceinline__ void apply_act(int act, float* y) {
  switch (act) {
    case 1: act_all<1, N>(y); break;
    case 2: act_all<2, N>(y); break;
    case 3: act_all<3, N>(y); break;
    default: break;
  }
}

__device__ __forceinline__ int row_of(int order, int pos, int pair, int per_row) {
  return order == static_cast<int>(RowOrder::Sorted) ? pos
         : order == static_cast<int>(RowOrder::Pair) ? pair
                                                     : pair / per_row;
}

// Positions of the tile of at most 16 << B positions that starts at p0.
template <int B>
__device__ __forceinline__ int tile_positions(const int32_t* offsets, int group, int p0) {
  const int first = offsets[group], end = offsets[group + 1];
  return min(plan_tile_rows(end - first, B), end - p0);
}

// Keeps the compiler from moving instructions across this point.
__device__ __forceinline__ void sched_fence() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
#endif
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

// The tiled kernel's launches (grouped_tile.hip, grouped_tile_gated.hip).
hipError_t launch_grouped_tile(GroupedArgs a, const RowPlan& plan, Elt out, hipStream_t stream);
hipError_t launch_grouped_tile_gated(GroupedArgs a, const RowPlan& plan, Elt out, hipStream_t stream);

}  // namespace convrot
