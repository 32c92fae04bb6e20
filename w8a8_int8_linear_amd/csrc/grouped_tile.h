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
//
// Bound by the matrix products inside a tile (a 128-byte slice of a tile with
// 205 positions in use takes 1.4 us, 1.0 us at the rate of a large library
// product) and by its ends, about 9.5 us per tile: the epilogue's arithmetic,
// its stores, and the first slices of the next tile.  128 groups with 65536
// pairs unevenly over them, bf16: gated K = 2048, N = 768 (412 GOP) 236-244
// us, 1.7 POPS; K = 768, N = 2048 (206 GOP) 190 us, 1.1 POPS.  Non-temporal
// stores were 1-2 % faster alone, but take from L2 what the next launch reads.
#pragma once
#include "grouped_lds.h"

namespace convrot {
namespace {
namespace tile {

constexpr int kThreads = 512;
constexpr int kRows = 256;       // weight rows, and most positions, of a tile
constexpr int kSlice = 128;      // bytes of K
constexpr int kBuf = kRows * kSlice;
constexpr int kXBase = 3 * kBuf;  // LDS: three weight slices, then two row slices
constexpr int kSmem = 5 * kBuf;
constexpr int kDma = kRows / 64;  // 1 KiB transfers per wave, slice and operand
constexpr int kPT = 8;            // 16-position tiles per wave
static_assert(kSmem <= 160 * 1024, "LDS budget");

// At most np * PER of this wave's operations outstanding (np uniform).
template <int PER, int NP>
__device__ __forceinline__ void wait_stores(int np) {
  if constexpr (NP == 0) {
    wait_vm<0>();
  } else {
    if (np >= NP) wait_vm<(PER * NP < 63 ? PER * NP : 63)>();
    else wait_stores<PER, NP - 1>(np);
  }
}

// OUT: 0 = fp32, 1 = bf16.  ACT: activation (the epilogue is unrolled over 128
// outputs per lane, and a run-time choice per output made it 13 us per tile
// longer).  KTAIL: K is no multiple of 128.
template <int OUT, int ACT, bool GATED, bool KTAIL>
__global__ __launch_bounds__(kThreads, 1) void grouped_tile_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int kFeat = GATED ? kRows / 2 : kRows;  // features per tile
  constexpr int kWFeat = kFeat / 4;                 // and per wave
  constexpr int kFT = kWFeat / 16;                  // 16-feature tiles per wave
  // The walk: each XCD (workgroup id mod 8) has a contiguous run of the tiles,
  // which its workgroups take in turn.
  const int total = *a.count * a.tiles_n;
  const int xcd = blockIdx.x % 8;
  const int stride = (gridDim.x - xcd + 7) / 8;
  const int run_end = (xcd + 1) * (total / 8) + min(xcd + 1, total % 8);
  int logical = xcd * (total / 8) + min(xcd, total % 8) + blockIdx.x / 8;
  if (logical >= run_end) return;

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
  struct Tile {
    int group, p0, cnt, n_blk;
    int x_pos[kDma];  // what names the lane's row of each transfer: position or pair
    int pair[2];      // the pairs of two of the wave's 128 positions
  };
  // Position within the tile of the wave's entry 64 h + lane.
  auto position = [&](int h) { return 16 * (2 * (4 * h + (lane >> 4)) + grp) + frow; };
  auto tile_at = [&](int id, Tile& t) {
    const int t_id = id / a.tiles_n;
    t.n_blk = id % a.tiles_n * kFeat;
    t.group = a.list[2 * t_id];
    t.p0 = a.list[2 * t_id + 1];
    t.cnt = tile_positions<4>(a.offsets, t.group, t.p0);
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int pos = t.p0 + min(8 * (wid + 8 * i) + (lane >> 3), t.cnt - 1);
      t.x_pos[i] = a.source == static_cast<int>(RowOrder::Sorted) ? pos : a.order[pos];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) t.pair[h] = a.order[t.p0 + min(position(h), t.cnt - 1)];
  };
  const uint8_t* w_base[kDma];
  uint32_t w_off[kDma];
  const uint8_t* x_ptr[kDma];
  int used = 0;  // positions of the current tile in whole 16
  auto enter = [&](const Tile& t) {
    used = (t.cnt + 15) & ~15;
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int row0 = 8 * (wid + 8 * i);  // uniform
      const bool up = GATED && row0 % 64 >= 32;
      const int feat = (GATED ? row0 / 64 * 32 + row0 % 32 : row0) + (lane >> 3);
      const int64_t ld = up ? a.ldb2 : a.ldb;
      w_base[i] = (up ? a.B2 : a.B) + (static_cast<int64_t>(t.group) * a.N + t.n_blk) * ld;
      w_off[i] = static_cast<uint32_t>(min(feat, a.N - t.n_blk - 1)) * static_cast<uint32_t>(ld);
      x_ptr[i] = a.A + static_cast<int64_t>(row_of(a.source, t.x_pos[i], t.x_pos[i], a.per_row)) * a.lda;
    }
  };
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

  i32x4 acc[4][kPT];
  int np = 0;  // position tiles of this wave
  // NP position tiles: those in use, rounded up to an even number (what the
  // last one multiplies then is not stored).
  auto read_step = [&](auto np_c, int st, int wbuf, int xbuf, i32x4(&fw)[4], i32x4(&fx)[kPT]) {
    const uint32_t aw = w_addr[st] + wbuf * kBuf, ax = x_addr[st] + xbuf * kBuf;
    static_for<4>([&](auto i_c) { lds_read16<16 * kSlice * decltype(i_c)::value>(fw[decltype(i_c)::value], aw); });
    static_for<decltype(np_c)::value>([&](auto f_c) {
      constexpr int f = decltype(f_c)::value;
      lds_read16<32 * kSlice * f>(fx[f], ax);
    });
  };
  auto compute_step = [&](auto np_c, int s, int st, i32x4(&fw)[4], i32x4(&fx)[kPT]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) landed(fw[i]);
    const bool dead = KTAIL && s * kSlice + 64 * st + 16 * fk >= a.K;
#pragma unroll
    for (int f = 0; f < decltype(np_c)::value; ++f) {
      landed(fx[f]);
      if constexpr (KTAIL) fx[f] = dead ? i32x4{} : fx[f];
    }
#pragma unroll
    for (int f = 0; f < decltype(np_c)::value; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fx[f], acc[i][f], 0, 0, 0);
  };

  Tile cur;
  tile_at(logical, cur);
  enter(cur);
  dma_w(0, 0);
  dma_x(0, 0);
  if (nk > 1) dma_w(1, 1);
  wait_vm<0>();

  while (true) {
    barrier();  // every wave's first slices have landed, and no wave stages outputs any more
    if (grp == 1) barrier();  // the second four run one phase behind
    const int p0 = cur.p0, cnt = cur.cnt, group = cur.group, n_blk = cur.n_blk;
    np = ((used >> 4) - grp + 1) >> 1;
    // Epilogue operands, one or two per lane: the wave's 64 weight rows'
    // scales and biases, and its 128 positions' scales and output rows.
    const int n_wave = n_blk + (wid & 3) * kWFeat;
    const bool up_lane = GATED && lane >= 32;
    const int64_t col = static_cast<int64_t>(group) * a.N + min(n_wave + (GATED ? lane & 31 : lane), a.N - 1);
    const float* bias = up_lane ? a.bias2 : a.bias;
    const float s_col = (up_lane ? a.sb2 : a.sb)[col];
    const float b_col = bias != nullptr ? bias[col] : 0.f;
    float s_pos[2];
    int out_row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pos = p0 + min(position(h), cnt - 1);
      s_pos[h] = a.sa[row_of(a.source, pos, cur.pair[h], a.per_row)];
      out_row[h] = row_of(a.dest, pos, cur.pair[h], a.per_row);
    }
    // The next tile's pairs are looked up now and used at this one's end: loads
    // return in order, so using them here would wait for the last tile's
    // stores, and waiting inside the slice loop would hold up every transfer.
    const int next = logical + stride;
    const bool more = next < run_end;
    if (more) tile_at(next, cur);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int f = 0; f < kPT; ++f) acc[i][f] = i32x4{};

    auto main_loop = [&](auto np_c) {
      int w_cur = 0;
      for (int s = 0; s < nk; ++s) {
        const int x_cur = s & 1;
        const int w_next = w_cur == 2 ? 0 : w_cur + 1;
        const int w_after = w_next == 2 ? 0 : w_next + 1;
        // Buffers: weights of slice s + 2 go where slice s - 1 was, rows of
        // s + 1 where s - 1 was; every wave's last read of those precedes the
        // barrier that opens slice s.
        i32x4 fw[4], fx[kPT];  // one step's fragments
        read_step(np_c, 0, w_cur, x_cur, fw, fx);
        if (s + 1 < nk) dma_x(s + 1, x_cur ^ 1);
        wait_lds();
        barrier();
        compute_step(np_c, s, 0, fw, fx);
        barrier();
        read_step(np_c, 1, w_cur, x_cur, fw, fx);
        if (s + 2 < nk) dma_w(s + 2, w_after);
        // all but the transfers just issued have landed; the barrier publishes them
        if (s + 2 < nk) wait_vm<kDma>(); else wait_vm<0>();
        wait_lds();
        barrier();
        compute_step(np_c, s, 1, fw, fx);
        if (grp == 0 || s + 1 < nk) barrier();
        w_cur = w_next;
      }
    };
    // (uniform per wave; every choice passes the same barriers)
    if (np > 6) main_loop(std::integral_constant<int, 8>{});
    else if (np > 4) main_loop(std::integral_constant<int, 6>{});
    else if (np > 2) main_loop(std::integral_constant<int, 4>{});
    else main_loop(std::integral_constant<int, 2>{});
    // (both halves have passed the same number of barriers, and every slice
    // read is done)

    // Epilogue: lane l holds, for tiles (i, f), position 16 (2 f + grp) +
    // l % 16 and features 16 i + 4 (l / 16) + r of the wave.  The next tile's
    // first slices are requested (weight buffers 0 and 1, row buffer 0) and
    // land while the outputs leave.
    // (the addresses below come from a copy of the lane number made here, so
    // that the compiler does not keep them in registers through the main loop)
    int lane_e = lane;
    opaque(lane_e);
    const int frow_e = lane_e & 15, fk_e = lane_e >> 4;
    if (more) {
      enter(cur);
      dma_w(0, 0);
      dma_x(0, 0);
      if (nk > 1) dma_w(1, 1);
    }
    sched_fence();
    // The wave's scales, biases and rows go to its own part of weight buffer
    // 2 or row buffer 1, and each 16-position tile is staged there as rows of
    // finished outputs, which leave in 16-byte pieces: whole rows of the
    // wave's features.
    using out_t = typename std::conditional<OUT == 0, float, __bf16>::type;
    constexpr int kElt = sizeof(out_t);
    constexpr int kPitch = kWFeat * kElt + 16;
    constexpr int kSegs = kWFeat * kElt / 16;  // pieces per row
    constexpr int kStores = 16 * kSegs / 64;   // store instructions per 16 positions
    constexpr int kMeta = 4 * (64 + 64 + 128 + 128);
    constexpr int kBufs = OUT == 0 && !GATED ? 1 : 2;
    constexpr int kArea = kMeta + kBufs * 16 * kPitch;
    static_assert(4 * kArea <= kBuf, "staging areas");
    uint8_t* area = smem + (wid < 4 ? 2 * kBuf : kXBase + kBuf) + (wid & 3) * kArea;
    float* m_scale = reinterpret_cast<float*>(area);       // [64] by weight row of the wave
    float* m_bias = m_scale + 64;                          // [64]
    float* m_pos = m_bias + 64;                            // [128] by position of the wave
    int* m_row = reinterpret_cast<int*>(m_pos + 128);      // [128]
    uint8_t* stage = area + kMeta;
    m_scale[lane_e] = s_col;
    m_bias[lane_e] = b_col;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m_pos[64 * h + lane_e] = s_pos[h];
      m_row[64 * h + lane_e] = out_row[h];
    }
    wave_sync();
    f32x4 sc[4], bs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sc[i] = *reinterpret_cast<const f32x4*>(m_scale + 16 * i + 4 * fk_e);
      bs[i] = *reinterpret_cast<const f32x4*>(m_bias + 16 * i + 4 * fk_e);
    }
    const bool full = n_wave + kWFeat <= a.N && a.vec_out;
    // Tile f is finished and staged, then tile f - 1 leaves (two areas in
    // turn, where they fit: its rows have long been written).
    auto finish = [&](auto f_c) {
      constexpr int f = decltype(f_c)::value;
      const float s_row = m_pos[16 * f + frow_e];
#pragma unroll
      for (int i = 0; i < kFT; ++i) {
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          y[r] = act_of<ACT>(fmaf(static_cast<float>(acc[i][f][r]), s_row * sc[i][r], bs[i][r]));
          if constexpr (GATED)
            y[r] *= fmaf(static_cast<float>(acc[i + kFT][f][r]), s_row * sc[i + kFT][r], bs[i + kFT][r]);
        }
        uint8_t* to = stage + f % kBufs * 16 * kPitch + frow_e * kPitch + (16 * i + 4 * fk_e) * kElt;
        if constexpr (OUT == 0)
          *reinterpret_cast<f32x4*>(to) = f32x4{y[0], y[1], y[2], y[3]};
        else
          *reinterpret_cast<bf16x4*>(to) = bf16x4{static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                                                  static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
      }
    };
    auto leave = [&](auto f_c) {
      constexpr int f = decltype(f_c)::value;
      const int live = min(16, cnt - 16 * (2 * f + grp));  // positions of the tile
      i32x4 v[kStores];
      int row[kStores];
#pragma unroll
      for (int q = 0; q < kStores; ++q) {
        const int c = 64 * q + lane_e;
        v[q] = *reinterpret_cast<const i32x4*>(stage + f % kBufs * 16 * kPitch + c / kSegs * kPitch + c % kSegs * 16);
        row[q] = m_row[16 * f + c / kSegs];
      }
#pragma unroll
      for (int q = 0; q < kStores; ++q) {
        const int c = 64 * q + lane_e, n = n_wave + c % kSegs * (16 / kElt);
        out_t* to = static_cast<out_t*>(a.C) + row[q] * a.ldc + n;
        if (c / kSegs >= live) continue;
        if (full) {
          *reinterpret_cast<i32x4*>(to) = v[q];
        } else {  // the ragged right edge, or rows that take no 16-byte stores
          const out_t* from =
              reinterpret_cast<const out_t*>(stage + f % kBufs * 16 * kPitch + c / kSegs * kPitch + c % kSegs * 16);
#pragma unroll 1
          for (int e = 0; e < 16 / kElt && n + e < a.N; ++e) to[e] = from[e];
        }
      }
    };
    static_for<kPT + 1>([&](auto f_c) {
      constexpr int f = decltype(f_c)::value;
      if constexpr (kBufs == 1) {
        if constexpr (f < kPT) {
          if (f < np) {
            finish(f_c);
            wave_sync();
            leave(f_c);
            wave_sync();
          }
        }
      } else {
        if constexpr (f < kPT) {
          if (f < np) finish(f_c);
        }
        if constexpr (f > 0) {
          if (f <= np) leave(std::integral_constant<int, f - 1>{});
        }
        wave_sync();
      }
    });
    if (!more) break;
    logical = next;
    // The first slices of the next tile have landed once no more operations
    // are outstanding than the stores issued behind them (a lower bound:
    // whole 16-position tiles only); the stores themselves may still fly.
    if (full) wait_stores<kStores, kPT>(np - 1);
    else wait_vm<0>();
  }
}

}  // namespace tile

template <int OUT, int ACT, bool GATED, bool KTAIL>
hipError_t launch_tile_typed(GroupedArgs a, const RowPlan& plan, hipStream_t stream) {
  auto kern = tile::grouped_tile_kernel<OUT, ACT, GATED, KTAIL>;
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
  // One workgroup fits a CU; each walks its XCD's run of tiles.
  const int64_t tiles = plan_max_tiles(plan.pairs, plan.groups, b) * a.tiles_n;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tiles, device_cus())));
  hipLaunchKernelGGL(kern, grid, dim3(tile::kThreads), tile::kSmem, stream, a);
  return hipGetLastError();
}

template <int ACT, bool GATED>
hipError_t launch_tile_act(const GroupedArgs& a, const RowPlan& plan, Elt out, hipStream_t stream) {
  if (a.K % tile::kSlice != 0)
    return out == Elt::F32 ? launch_tile_typed<0, ACT, GATED, true>(a, plan, stream)
                           : launch_tile_typed<1, ACT, GATED, true>(a, plan, stream);
  return out == Elt::F32 ? launch_tile_typed<0, ACT, GATED, false>(a, plan, stream)
                         : launch_tile_typed<1, ACT, GATED, false>(a, plan, stream);
}

}  // namespace
}  // namespace convrot
