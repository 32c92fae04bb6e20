// Tiled matrix-core kernel of the grouped linears (grouped.hip) for gfx950:
// groups with more rows than the streaming kernel serves well.
//
// A workgroup of eight waves takes 256 weight rows of one group (256 features,
// or 128 gate and 128 up rows of the same features) and one tile of the plan,
// up to 256 positions of that group, and runs K in 128-byte slices through
// LDS: three weight slices and two row slices ([rows][128 B], 16-byte chunks
// XOR-swizzled by row & 7), filled by global -> LDS transfers.  Two waves
// share a SIMD and take turns, one in its memory phase (fragment reads of its
// next 64-byte step, its share of the transfers) while the other multiplies,
// a workgroup barrier swapping the roles; four waves lead and four run one
// phase behind.
//
// Wave w owns weight rows 64 (w % 4) .. + 63 and every other 16-position tile
// (w / 4, w / 4 + 2, ..), so that a tile of the plan with few positions
// shortens every wave's phases alike: time follows the positions in use, not
// the tile's size.  Weights are the MFMA's row operand (v_mfma_i32_16x16x64_i8),
// so a lane's four accumulators are four consecutive features of a position.
//
// Rows are gathered by the transfers themselves: a lane's source address is
// its row's, looked up once per tile.  Workgroups are dealt to the eight XCDs
// in contiguous runs of (tile, weight block), the weight blocks innermost, so
// that the blocks that read a tile's rows and the tiles that read a group's
// weights meet in one L2.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "epilogue.h"

namespace convrot {
namespace {
namespace tile {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kThreads = 512;
constexpr int kRows = 256;       // weight rows, and most positions, of a tile
constexpr int kSlice = 128;      // bytes of K
constexpr int kBuf = kRows * kSlice;
constexpr int kXBase = 3 * kBuf;  // LDS: three weight slices, then two row slices
constexpr int kSmem = 5 * kBuf;
constexpr int kDma = kRows / 64;  // 1 KiB transfers per wave, slice and operand
constexpr int kPT = 8;            // 16-position tiles per wave
static_assert(kSmem <= 160 * 1024, "LDS budget");

__device__ __forceinline__ void dma16(const uint8_t* g, uint8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_global_load_lds(g, (lds_ptr_t)lds, 16, 0, 0);
#endif
}
// 16-byte LDS read in program order; the register is only safe to use past
// wait_lds() and landed().
template <int OFF>
__device__ __forceinline__ void lds_read16(i32x4& r, uint32_t addr) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "i"(OFF) : "memory");
#endif
}
// No instruction: uses of r stay behind the wait in front of this point.
__device__ __forceinline__ void landed(i32x4& r) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(r));
#endif
}
__device__ __forceinline__ void wait_lds() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
#endif
}
// At most N of this wave's vector-memory operations outstanding.
template <int N>
__device__ __forceinline__ void wait_vm() {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(N >= 0 && N < 16, "low bits of vmcnt");
  __builtin_amdgcn_s_waitcnt(N | (7 << 4) | (15 << 8));
#endif
}
// Workgroup barrier without a fence: callers wait for what they need.
__device__ __forceinline__ void barrier() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#endif
}
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// OUT: 0 = fp32, 1 = bf16.  KTAIL: K is no multiple of 128.
template <int OUT, bool GATED, bool KTAIL>
__global__ __launch_bounds__(kThreads, 1) void grouped_tile_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int kFeat = GATED ? kRows / 2 : kRows;  // features per tile
  constexpr int kWFeat = kFeat / 4;                 // and per wave
  constexpr int kFT = kWFeat / 16;                  // 16-feature tiles per wave
  const int total = *a.count * a.tiles_n;
  const int bid = blockIdx.x;
  if (bid >= total) return;
  const int xcd = bid % 8;
  const int logical = xcd * (total / 8) + min(xcd, total % 8) + bid / 8;
  const int t_id = logical / a.tiles_n;
  const int n_blk = logical % a.tiles_n * kFeat;
  const int group = a.list[2 * t_id], p0 = a.list[2 * t_id + 1];
  const int cnt = min(kRows, a.offsets[group + 1] - p0);

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = wid >> 2;
  const int frow = lane & 15, fk = lane >> 4;
  const int nk = (a.K + kSlice - 1) / kSlice;

  // Transfers: instruction i of wave w fills rows 8 (w + 8 i) .. + 7 of a
  // slice, lane l chunk l % 8 of row l / 8, which holds chunk
  // (l % 8) ^ (l / 8).  Rows past the tile's or the weight's last re-read it;
  // transfers of positions nobody multiplies are left out.
  const int ch16 = ((lane & 7) ^ (lane >> 3)) * 16;
  const uint8_t* w_base[kDma];
  uint32_t w_off[kDma];
  const uint8_t* x_ptr[kDma];
  const int used = (cnt + 15) & ~15;
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int row0 = 8 * (wid + 8 * i);  // uniform
    const bool up = GATED && row0 % 64 >= 32;
    const int feat = (GATED ? row0 / 64 * 32 + row0 % 32 : row0) + (lane >> 3);
    const int64_t ld = up ? a.ldb2 : a.ldb;
    w_base[i] = (up ? a.B2 : a.B) + (static_cast<int64_t>(group) * a.N + n_blk) * ld;
    w_off[i] = static_cast<uint32_t>(min(feat, a.N - n_blk - 1)) * static_cast<uint32_t>(ld);
    const int pos = p0 + min(row0 + (lane >> 3), cnt - 1);
    x_ptr[i] = a.A + row_of(a.source, pos, a.source == static_cast<int>(RowOrder::Sorted) ? 0 : a.order[pos],
                            a.per_row) * a.lda;
  }
  // Byte of a row that the lane fetches of slice s (in the last slice, chunks
  // past K re-read the row's first; they are multiplied as zeros).
  auto k_at = [&](int s) -> uint32_t {
    const int k = s * kSlice + ch16;
    return KTAIL && k >= a.K ? 0 : k;
  };
  auto dma_w = [&](int s, int buf) {
    const uint32_t k = k_at(s);
#pragma unroll
    for (int i = 0; i < kDma; ++i) dma16(w_base[i] + (w_off[i] + k), smem + buf * kBuf + (wid + 8 * i) * 1024);
  };
  auto dma_x = [&](int s, int buf) {
    const uint32_t k = k_at(s);
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      if (8 * (wid + 8 * i) < used) dma16(x_ptr[i] + k, smem + kXBase + buf * kBuf + (wid + 8 * i) * 1024);
  };

  // Fragment addresses: row l % 16 of a 16-row tile, chunk l / 16 of the
  // 64-byte step (st 0 or 1 of the slice).
  const uint32_t lds0 =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)(smem)));
  uint32_t w_addr[2], x_addr[2];
#pragma unroll
  for (int st = 0; st < 2; ++st) {
    const uint32_t off = frow * kSlice + (((4 * st + fk) ^ (frow & 7)) << 4);
    w_addr[st] = lds0 + (wid & 3) * 64 * kSlice + off;
    x_addr[st] = lds0 + kXBase + grp * 16 * kSlice + off;
  }
  const int np = ((used >> 4) - grp + 1) >> 1;  // position tiles of this wave

  i32x4 acc[4][kPT] = {};
  i32x4 fw[4], fx[kPT];
  auto read_step = [&](int st, int wbuf, int xbuf) {
    const uint32_t aw = w_addr[st] + wbuf * kBuf, ax = x_addr[st] + xbuf * kBuf;
    static_for<4>([&](auto i_c) { lds_read16<16 * kSlice * decltype(i_c)::value>(fw[decltype(i_c)::value], aw); });
    static_for<kPT>([&](auto f_c) {
      constexpr int f = decltype(f_c)::value;
      if (f < np) lds_read16<32 * kSlice * f>(fx[f], ax);
    });
  };
  auto compute_step = [&](int s, int st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) landed(fw[i]);
    const bool dead = KTAIL && s * kSlice + 64 * st + 16 * fk >= a.K;
#pragma unroll
    for (int f = 0; f < kPT; ++f) {
      if (f >= np) break;
      landed(fx[f]);
      if constexpr (KTAIL) fx[f] = dead ? i32x4{} : fx[f];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fx[f], acc[i][f], 0, 0, 0);
    }
  };

  dma_w(0, 0);
  dma_x(0, 0);
  if (nk > 1) dma_w(1, 1);
  // Row scale and output row of the lane's position in each of its tiles.
  float s_row[kPT];
  int64_t out_row[kPT];
#pragma unroll
  for (int f = 0; f < kPT; ++f) {
    s_row[f] = 0.f;
    out_row[f] = 0;
    if (f < np) {
      const int pos = p0 + min(16 * (2 * f + grp) + frow, cnt - 1);
      const int pair = a.order[pos];
      s_row[f] = a.sa[row_of(a.source, pos, pair, a.per_row)];
      out_row[f] = row_of(a.dest, pos, pair, a.per_row);
    }
  }
  wait_vm<0>();
  barrier();
  if (grp == 1) barrier();  // the second four run one phase behind

  int w_cur = 0;
  for (int s = 0; s < nk; ++s) {
    const int x_cur = s & 1;
    const int w_next = w_cur == 2 ? 0 : w_cur + 1;
    const int w_after = w_next == 2 ? 0 : w_next + 1;
    // Buffers: weights of slice s + 2 go where slice s - 1 was, rows of s + 1
    // where s - 1 was; every wave's last read of those precedes the barrier
    // that opens slice s.
    read_step(0, w_cur, x_cur);
    if (s + 1 < nk) dma_x(s + 1, x_cur ^ 1);
    wait_lds();
    barrier();
    compute_step(s, 0);
    barrier();
    read_step(1, w_cur, x_cur);
    if (s + 2 < nk) dma_w(s + 2, w_after);
    // all but the transfers just issued have landed; the barrier publishes them
    if (s + 2 < nk) wait_vm<kDma>(); else wait_vm<0>();
    wait_lds();
    barrier();
    compute_step(s, 1);
    if (grp == 0 || s + 1 < nk) barrier();
    w_cur = w_next;
  }
  // (both halves have passed the same number of barriers; every slice read is
  // done, so the staging below may overwrite the slices)

  // Epilogue: lane l holds, for tiles (i, f), position 16 (2 f + grp) + l % 16
  // and features 16 i + 4 (l / 16) + r of the wave.  Scales and biases first.
  const int n_wave = n_blk + (wid & 3) * kWFeat;
  const int64_t col0 = static_cast<int64_t>(group) * a.N;
  float sc[4][4], bs[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = GATED && i >= kFT;
    const float* s = up ? a.sb2 : a.sb;
    const float* b = up ? a.bias2 : a.bias;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t col = col0 + min(n_wave + 16 * (i % kFT) + 4 * fk + r, a.N - 1);
      sc[i][r] = s[col];
      bs[i][r] = b != nullptr ? b[col] : 0.f;
    }
  }
  // Each 16-position tile is staged as rows of finished outputs in an area of
  // the wave's own and leaves in 16-byte pieces, whole rows of the wave's
  // features.
  using out_t = typename std::conditional<OUT == 0, float, __bf16>::type;
  constexpr int kElt = sizeof(out_t);
  constexpr int kPitch = kWFeat * kElt + 16;
  constexpr int kSegs = kWFeat * kElt / 16;  // pieces per row
  uint8_t* stage = smem + wid * 16 * kPitch;
  const bool full = n_wave + kWFeat <= a.N && a.vec_out;
#pragma unroll
  for (int f = 0; f < kPT; ++f) {
    if (f >= np) break;
    const int live = min(16, cnt - 16 * (2 * f + grp));  // positions of the tile
#pragma unroll
    for (int i = 0; i < kFT; ++i) {
      float y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = apply_act(a.act, fmaf(static_cast<float>(acc[i][f][r]), s_row[f] * sc[i][r], bs[i][r]));
        if constexpr (GATED)
          y[r] *= fmaf(static_cast<float>(acc[i + kFT][f][r]), s_row[f] * sc[i + kFT][r], bs[i + kFT][r]);
      }
      if (full) {
        uint8_t* to = stage + frow * kPitch + (16 * i + 4 * fk) * kElt;
        if constexpr (OUT == 0)
          *reinterpret_cast<f32x4*>(to) = f32x4{y[0], y[1], y[2], y[3]};
        else
          *reinterpret_cast<bf16x4*>(to) = bf16x4{static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                                                  static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
      } else if (frow < live) {
        store4<OUT>(a.C, out_row[f] * a.ldc, n_wave + 16 * i + 4 * fk, a.N, y);
      }
    }
    if (full) {
      // (a wave's LDS operations complete in order)
      i32x4 v[16 * kSegs / 64];
#pragma unroll
      for (int q = 0; q < 16 * kSegs / 64; ++q) {
        const int c = 64 * q + lane;
        v[q] = *reinterpret_cast<const i32x4*>(stage + c / kSegs * kPitch + c % kSegs * 16);
      }
#pragma unroll
      for (int q = 0; q < 16 * kSegs / 64; ++q) {
        const int c = 64 * q + lane, row = c / kSegs;
        const int64_t to = __shfl(out_row[f], row) * a.ldc + n_wave;
        if (row < live)
          *reinterpret_cast<i32x4*>(static_cast<uint8_t*>(a.C) + to * kElt + c % kSegs * 16) = v[q];
      }
    }
  }
}

}  // namespace tile
}  // namespace
}  // namespace convrot
