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
// Few rows per group: the weight-streaming ring (grouped_ring.h), bound by the
// weights' bytes.  Many: the tiled kernel (grouped_tile.h).
#include "grouped.h"
#include "grouped_ring.h"

namespace convrot {
namespace {

template <int OUT, bool GATED, bool KTAIL, int MT, int NW, bool SPLIT>
hipError_t launch_ring_typed(GroupedArgs a, const RowPlan& plan, hipStream_t stream) {
  auto kern = ring::grouped_ring_kernel<OUT, GATED, KTAIL, MT, NW, SPLIT>;
  constexpr int kSmem = ring::smem_bytes<MT, NW, SPLIT>();
  constexpr int b = MT == 1 ? 0 : MT == 2 ? 1 : 2;
  constexpr int kFeat = (GATED ? 16 : 32) * (SPLIT ? 1 : NW);
  a.tiles_n = (a.N + kFeat - 1) / kFeat;
  const int64_t blocks = plan_max_tiles(plan.pairs, plan.groups, b) * a.tiles_n;
  if (blocks > kMaxLaunchThreads / (64 * NW)) return hipErrorInvalidConfiguration;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), kSmem, lds_set);
  if (e != hipSuccess) return e;
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + b;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(blocks)), dim3(64 * NW), kSmem, stream, a);
  return hipGetLastError();
}

// The ring's form for a launch, by what the host knows of the groups: the
// number of pairs and groups (rows per group on average).  Measured on one
// box, 8 to 32 groups, K = 1024 to 6912 (us):
//   rows per tile, by rows per group:
//     4 rows   16: 14.0, 32: 14.6, 64: 15.6       8 rows  16: 17.8, 32: 15.9, 64: 16.9
//     32 rows  16: 24.8, 32: 21.4, 64: 23.2       64 rows 16: 34.8, 32: 28.0, 64: 26.1
//   K shared by the workgroup's waves (2, 4), with fewer workgroups than CUs:
//     72 workgroups 25.6, 17.9 (2), 16.6 (4)      128: 10.9, 9.3, 9.0
//     256: 15.1, 13.8, 15.5                       512: 26.6, 26.8, 27.8
template <int OUT, bool GATED, bool KTAIL>
hipError_t launch_ring(const GroupedArgs& a, const RowPlan& plan, hipStream_t stream) {
  constexpr int kNW = 4;
  const int64_t avg = plan.pairs / plan.groups;
  const int64_t blocks = (a.N + (GATED ? 16 : 32) * kNW - 1) / ((GATED ? 16 : 32) * kNW);
  // workgroups of a launch with tiles of 16 << b rows
  auto workgroups = [&](int b) {
    return blocks * std::max<int64_t>(std::min<int64_t>(plan.groups, plan.pairs), plan.pairs >> (4 + b));
  };
  if (avg > 40 && workgroups(2) >= 160) return launch_ring_typed<OUT, GATED, KTAIL, 4, kNW, false>(a, plan, stream);
  if (avg >= 6)
    return workgroups(1) >= 160 ? launch_ring_typed<OUT, GATED, KTAIL, 2, kNW, false>(a, plan, stream)
                                : launch_ring_typed<OUT, GATED, KTAIL, 2, 2, true>(a, plan, stream);
  const int64_t w = workgroups(0);
  return w >= 512   ? launch_ring_typed<OUT, GATED, KTAIL, 1, kNW, false>(a, plan, stream)
         : w >= 160 ? launch_ring_typed<OUT, GATED, KTAIL, 1, 2, true>(a, plan, stream)
                    : launch_ring_typed<OUT, GATED, KTAIL, 1, 4, true>(a, plan, stream);
}

// Whether the tiled kernel is the faster one.  Both costs are estimates in
// units of 0.1 us, from launches where a 128-byte slice took a CU 1.4 us for a
// tile of the tiled kernel (with 8 us for its ends, in whole rounds over the
// CUs) and 0.7 us for a 64-row tile of the ring (with 4 us per launch).  Tiles
// are counted as if every group had half a tile that is not full.  Tiled
// against ring where they meet (us; 8 or 32 groups, r rows per group):
//   gated K = 2048, N = 1024: r 96 52.9 / 45.4, 128 52.8 / 53.8, 192 55.9 / 64.7
//   K = 1024, N = 2048:       r 128 37.2 / 34.1, 192 38.3 / 42.1
//   gated K = 1152, N = 6912: r 64 39.0 / 40.1, 96 43.3 / 50.4
//   K = 6912, N = 1152 (few workgroups): r 128 67.1 / 43.1, 256 71.2 / 50.8
template <bool GATED>
bool tiled_is_faster(const GroupedArgs& a, const RowPlan& plan) {
  const int64_t cus = device_cus(), slices = (a.K + 127) / 128;
  const int64_t used = std::min<int64_t>(plan.groups, plan.pairs);
  auto tiles = [&](int64_t rows) { return std::max(used, plan.pairs / rows + used / 2); };
  auto blocks = [&](int64_t features) { return (a.N + features - 1) / features; };
  const int64_t tiled = (tiles(256) + used / 16) * blocks(GATED ? 128 : 256);
  const int64_t ring = tiles(64) * blocks(GATED ? 64 : 128);
  return (tiled + cus - 1) / cus * (14 * slices + 80) < std::max(ring, cus) * 7 * slices / cus + 40;
}

template <int OUT, bool GATED>
hipError_t launch_grouped(const GroupedArgs& a, const RowPlan& plan, hipStream_t stream) {
  if (tiled_is_faster<GATED>(a, plan)) {
    const Elt out = OUT == 0 ? Elt::F32 : Elt::BF16;
    return GATED ? launch_grouped_tile_gated(a, plan, out, stream) : launch_grouped_tile(a, plan, out, stream);
  }
  return a.K % ring::kSlice != 0 ? launch_ring<OUT, GATED, true>(a, plan, stream)
                                 : launch_ring<OUT, GATED, false>(a, plan, stream);
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
  a.pairs = static_cast<int>(plan.pairs);
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
