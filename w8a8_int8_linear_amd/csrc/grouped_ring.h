// Weight-streaming kernel of the grouped linears (grouped.hip) for gfx950:
// groups with few rows, bound by the bytes of the weights.
//
// A workgroup of NW waves takes 32 NW weight rows of one group (32 NW
// features, or 16 NW gate and 16 NW up rows of the same features) and a tile
// of up to 16 MT positions.  K runs in 128-byte slices through a ring of
// slices in LDS that global -> LDS transfers keep filled ahead of the
// multiplications: what is in flight does not cost registers, and every
// transfer moves whole 128-byte lines of eight rows.  One barrier per slice
// publishes the slice that has landed and frees the one before it.  Wave w
// owns two 16-row weight tiles (gated: a gate and its up tile) and multiplies
// them with every position tile in use (v_mfma_i32_16x16x64_i8).
//
// With fewer workgroups than keep the memory busy (SPLIT), the workgroup takes
// 32 weight rows and its waves share the slices, each with a ring of its own
// and no barrier until their sums meet in LDS.
//
// Fragments loaded straight into registers (16 rows x 64 bytes per load, K
// shared by the waves) took 31.3-32.3 us where the ring takes 26.0 (8 groups
// of 4 rows, gated, K = 1152, N = 6912: 127 MB, 4.9 TB/s).
#pragma once
#include "grouped_lds.h"

namespace convrot {
namespace {
namespace ring {

constexpr int kSlice = 128;
// Slices of the ring: two workgroups of four waves (four of two) fit a CU.
template <int MT, bool SPLIT>
constexpr int kStages = MT <= 2 && !SPLIT ? 4 : 3;
template <int MT, int RING>
constexpr int slice_bytes() {
  return (32 * RING + 16 * MT) * kSlice;
}
template <int MT, int NW, bool SPLIT>
constexpr int smem_bytes() {
  return SPLIT ? NW * kStages<MT, true> * slice_bytes<MT, 1>() : kStages<MT, false> * slice_bytes<MT, NW>();
}

// OUT: 0 = fp32, 1 = bf16.  KTAIL: K is no multiple of 128.  SPLIT: the waves
// share the slices of one 32-row block, each with a ring of its own.
template <int OUT, bool GATED, bool KTAIL, int MT, int NW, bool SPLIT>
__global__ __launch_bounds__(64 * NW, 2) void grouped_ring_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int kRing = SPLIT ? 1 : NW;                   // waves that fill a ring
  constexpr int kFeat = GATED ? 16 * kRing : 32 * kRing;  // features per workgroup
  constexpr int kS = kStages<MT, SPLIT>;
  constexpr int kBytes = slice_bytes<MT, kRing>();
  constexpr int kXAt = 32 * kRing * kSlice;            // rows behind the weights in a slice
  constexpr int kXDma = (2 * MT + kRing - 1) / kRing;  // 1 KiB transfers per wave and slice: rows
  constexpr int kDma = 4 + kXDma;                   // and in all
  // Contiguous runs of (tile, feature block) per XCD, feature blocks
  // innermost, so that tiles of one group share its weights in an L2.
  const int total = *a.count * a.tiles_n;
  const int bid = blockIdx.x;
  if (bid >= total) return;
  const int xcd = bid % 8;
  const int logical = xcd * (total / 8) + min(xcd, total % 8) + bid / 8;
  const int t_id = logical / a.tiles_n;
  const int n_blk = logical % a.tiles_n * kFeat;
  const int group = a.list[2 * t_id], p0 = a.list[2 * t_id + 1];

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int frow = lane & 15, fk = lane >> 4;
  const int slices = (a.K + kSlice - 1) / kSlice;
  // SPLIT: every NW-th slice, so that the waves together read whole rows.
  const int nk = SPLIT ? (slices - wid + NW - 1) / NW : slices;
  auto k_byte = [&](int s) { return (SPLIT ? s * NW + wid : s) * kSlice; };
  const int rid = SPLIT ? 0 : wid;  // the wave among those of its ring
  uint8_t* smem = lds + (SPLIT ? wid * kS * kBytes : 0);

  // Transfers (layout as the tiled kernel's): instruction i < 4 of a wave
  // fills rows 8 i .. 8 i + 7 of its 32 weight rows.
  const int ch16 = ((lane & 7) ^ (lane >> 3)) * 16;
  const uint8_t* w_ptr[2];  // its two 16-row tiles' bases
  uint32_t w_off[4];
  const int feat0 = GATED ? 16 * rid : 32 * rid;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool up = GATED && j == 1;
    w_ptr[j] = (up ? a.B2 : a.B) + (static_cast<int64_t>(group) * a.N + n_blk) * (up ? a.ldb2 : a.ldb);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = GATED && i >= 2;
    const int feat = feat0 + (GATED ? 8 * (i & 1) : 8 * i) + (lane >> 3);
    w_off[i] = static_cast<uint32_t>(min(feat, a.N - n_blk - 1)) * static_cast<uint32_t>(up ? a.ldb2 : a.ldb);
  }
  auto k_at = [&](int s) -> uint32_t {
    const int k = k_byte(s) + ch16;
    return KTAIL && k >= a.K ? 0 : k;
  };
  auto dma_w = [&](int s, int buf) {
    const uint32_t k = k_at(s);
    uint8_t* to = smem + buf * kBytes + rid * 32 * kSlice;
#pragma unroll
    for (int i = 0; i < 4; ++i) dma16(w_ptr[i / 2] + (w_off[i] + k), to + i * 1024);
  };
  // What the rows and the epilogue need is requested first (loads return in
  // order, so a lookup behind the transfers would wait for them), then the
  // first slices of the weights, then those of the rows.  Positions past the
  // tile's last hold other groups' rows (or the order's last); their results
  // are dropped.
  int x_pos[kXDma], x_pair[kXDma], pair[MT];
#pragma unroll
  for (int i = 0; i < kXDma; ++i) {
    const int blk = (rid + kRing * i) % (2 * MT);  // eight positions; with more waves than blocks some load one twice
    x_pos[i] = min(p0 + 8 * blk + (lane >> 3), a.pairs - 1);
    x_pair[i] = a.order[x_pos[i]];
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) pair[t] = a.order[min(p0 + 16 * t + frow, a.pairs - 1)];
  const int64_t col0 = static_cast<int64_t>(group) * a.N;
  float sc[2][4], bs[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float* sv = GATED && j == 1 ? a.sb2 : a.sb;
    const float* bv = GATED && j == 1 ? a.bias2 : a.bias;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t col = col0 + min(n_blk + feat0 + (GATED ? 0 : 16 * j) + 4 * fk + r, a.N - 1);
      sc[j][r] = sv[col];
      bs[j][r] = bv != nullptr ? bv[col] : 0.f;
    }
  }
  const int cnt = tile_positions<MT == 1 ? 0 : MT == 2 ? 1 : 2>(a.offsets, group, p0);
  sched_fence();
#pragma unroll
  for (int s = 0; s < kS - 1; ++s)
    if (s < nk) dma_w(s, s);
  sched_fence();
  const uint8_t* x_ptr[kXDma];
#pragma unroll
  for (int i = 0; i < kXDma; ++i) x_ptr[i] = a.A + row_of(a.source, x_pos[i], x_pair[i], a.per_row) * a.lda;
  auto dma_x = [&](int s, int buf) {
    const uint32_t k = k_at(s);
#pragma unroll
    for (int i = 0; i < kXDma; ++i)
      dma16(x_ptr[i] + k, smem + buf * kBytes + kXAt + (rid + kRing * i) % (2 * MT) * 1024);
  };
#pragma unroll
  for (int s = 0; s < kS - 1; ++s)
    if (s < nk) dma_x(s, s);
  sched_fence();
  const int mt = (cnt + 15) >> 4;  // position tiles in use
  float s_row[MT];
  int64_t out_row[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int pos = min(p0 + 16 * t + frow, a.pairs - 1);
    s_row[t] = a.sa[row_of(a.source, pos, pair[t], a.per_row)];
    out_row[t] = row_of(a.dest, pos, pair[t], a.per_row);
  }

  const uint32_t lds0 =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)(smem)));
  uint32_t f_off[2];
#pragma unroll
  for (int st = 0; st < 2; ++st) f_off[st] = lds0 + frow * kSlice + (((4 * st + fk) ^ (frow & 7)) << 4);
  i32x4 acc[2][MT] = {};
  int buf = 0;
  for (int s = 0; s < nk; ++s) {
    // Wait until this wave's transfers of slice s have landed.  Behind them
    // it has issued, at least: the rows of the first slices after s (whose
    // weights went ahead of all rows), then whole slices.
    if (s >= kS - 2 && s + kS - 2 < nk) {
      wait_vm<(kS - 2) * kDma>();
    } else {
      const int first = min(kS - 1, nk);
      const int behind = max(0, first - 1 - s) * kXDma + (min(nk, s + kS - 1) - max(first, s + 1)) * kDma;
      if (behind >= kXDma + kDma) wait_vm<kXDma + kDma>();
      else if (behind >= kDma) wait_vm<kDma>();
      else if (behind >= kXDma) wait_vm<kXDma>();
      else wait_vm<0>();
    }
    if constexpr (!SPLIT) barrier();
    const int free_buf = buf == 0 ? kS - 1 : buf - 1;  // slice s - 1, which every wave of the ring has read
    if (s + kS - 1 < nk) {
      dma_x(s + kS - 1, free_buf);
      dma_w(s + kS - 1, free_buf);
    }
    const uint32_t at = buf * kBytes;
    i32x4 fw[2][2], fx[2][MT];
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const uint32_t aw = f_off[st] + at + rid * 32 * kSlice, ax = f_off[st] + at + kXAt;
      lds_read16<0>(fw[st][0], aw);
      lds_read16<16 * kSlice>(fw[st][1], aw);
      static_for<MT>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        lds_read16<16 * kSlice * t>(fx[st][t], ax);
      });
    }
    wait_lds();
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      landed(fw[st][0]);
      landed(fw[st][1]);
      const bool dead = KTAIL && k_byte(s) + 64 * st + 16 * fk >= a.K;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        landed(fx[st][t]);
        if constexpr (KTAIL) fx[st][t] = dead ? i32x4{} : fx[st][t];
        if (t < mt) {
          acc[0][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[st][0], fx[st][t], acc[0][t], 0, 0, 0);
          acc[1][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[st][1], fx[st][t], acc[1][t], 0, 0, 0);
        }
      }
    }
    buf = buf == kS - 1 ? 0 : buf + 1;
  }
  if constexpr (SPLIT) {
    // The waves' partial sums meet in LDS; each finishes some position tiles
    // (and, plain, weight tiles).
    __syncthreads();  // every ring is done
    i32x4* sums = reinterpret_cast<i32x4*>(lds);
    static_assert(NW * 2 * MT * 1024 <= smem_bytes<MT, NW, SPLIT>(), "partial sums");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) sums[((wid * 2 + j) * MT + t) * 64 + lane] = acc[j][t];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        acc[j][t] = sums[(j * MT + t) * 64 + lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) acc[j][t] += sums[((v * 2 + j) * MT + t) * 64 + lane];
      }
  }
  // Lane l holds position 16 t + l % 16 and features 4 (l / 16) + r of each
  // of the wave's weight tiles.
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (16 * t + frow >= cnt || (SPLIT && t % NW != wid)) continue;
    const int n = n_blk + feat0 + 4 * fk;
    float y[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) y[j][r] = fmaf(static_cast<float>(acc[j][t][r]), s_row[t] * sc[j][r], bs[j][r]);
    apply_act<GATED ? 4 : 8>(a.act, y[0]);
    if constexpr (GATED) {
#pragma unroll
      for (int r = 0; r < 4; ++r) y[0][r] *= y[1][r];
      store4<OUT>(a.C, out_row[t] * a.ldc, n, a.N, y[0]);
    } else {
      store4<OUT>(a.C, out_row[t] * a.ldc, n, a.N, y[0]);
      store4<OUT>(a.C, out_row[t] * a.ldc, n + 16, a.N, y[1]);
    }
  }
}

}  // namespace ring
}  // namespace
}  // namespace convrot
