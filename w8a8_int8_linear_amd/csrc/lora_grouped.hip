// Low-rank corrections of a batch whose rows use different adapters, for
// gfx950: with g the adapter of row m (a group of the plan),
//   T[m] = X[m] A_g^T                        A_g [r, K], fp32 sums
//   out[m, n] = Y[m, n] + scale_g sum_j T[m, j] B_g[n, j]
// and out[m] = Y[m] for rows without an adapter.
//
//  * down: a workgroup takes a tile of the plan (up to 16 or 64 rows of one
//    group), one block of K and up to 128 columns of r
//    (v_mfma_f32_16x16x32_bf16, A's rows as the row operand).  The fp32 sums
//    of every K block go to the workspace, one row per position of the plan:
//    few rows give few tiles, so K is split until the grid covers the CUs, and
//    the second product adds the blocks in order as it reads them (no third
//    launch).
//  * up: a wave takes 16 positions and runs along N in steps of 64 features.
//    It adds the K blocks' sums of its rows once and keeps them in registers
//    as bf16 terms: two (hi + lo, 16 bits of the fp32 sum) for a bf16 output,
//    three (24 bits, all of it) for an fp32 one, so that the correction is
//    not rounded before the output is (split_terms).  The sums are staged in LDS so that Y
//    is read and out written in whole 128-byte lines, and with 64-row tiles
//    B's rows pass through LDS once for the four waves.  Bound by Y and out.
//
// What the memory path moves per instruction decides here: with B's, T's and
// Y's pieces taken in the MFMA's own layout (16 rows x 64 bytes per load) the
// pair of launches took 75 us for 4099 rows (K = 2048, N = 6144, r = 64, 24
// adapters, bf16: 134 MB); whole lines, 50 us (2.7 TB/s).  48 rows of 64
// adapters (K = N = 4096, r = 16): 9.5 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grouped_lds.h"

namespace convrot {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kDownWaves = 8;
constexpr int kUpWaves = 4;
// Columns of r per down workgroup: a wave's fragments and accumulators of
// more would not fit its registers, so higher ranks read X again.
constexpr int kDownCols = 128;
// Down: K steps of fragments per register set (two sets), so that several
// workgroups fit a CU.
template <int RT>
constexpr int kSteps = RT <= 2 ? 2 : 1;

__device__ __forceinline__ f32x4 mma_bf16(const i32x4& a, const i32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// v as a sum of N bf16 terms of v's sign, none of them zero unless v is: an
// infinity of B then gives N infinities of one sign, and the sum is the
// formula's infinity (with a term of zero or of the other sign it would be a
// NaN).  All terms but the last are rounded towards zero, which also keeps
// what lies above bf16's largest number finite; the sum is off by at most 2^-16
// (N = 2) or 2^-24 (N = 3) of v.  Where nothing is left, 2^-32 of the first
// term stands in for zero (below |v| = 2^-94 it may be zero itself).  Every
// term of an infinity or a NaN is v.
template <int N>
__device__ __forceinline__ void split_terms(float v, __bf16 (&term)[N]) {
  auto cut = [](float x) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xFFFF0000u); };
  float t = cut(v);
  const float small = t * 2.3283064365386963e-10f;  // 2^-32
  term[0] = static_cast<__bf16>(t);
#pragma unroll
  for (int q = 1; q < N; ++q) {
    v -= t;
    v = fabsf(v) > 0.f ? v : small;  // (inf - inf: small is the infinity)
    t = q < N - 1 ? cut(v) : v;
    term[q] = static_cast<__bf16>(t);
  }
}

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
  int nb, spb;  // K blocks and steps per block
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

// Few rows per adapter.  A workgroup takes one 16-row tile, one block of K and
// up to 16 RT columns; its eight waves split the block's 32-wide steps, load
// fragments straight into registers and add their sums through LDS.
template <int RT>
__global__ __launch_bounds__(64 * kDownWaves) void lora_grouped_down_kernel(LoraArgs a) {
  constexpr int kAhead = kSteps<RT>;
  __shared__ f32x4 partial[kDownWaves][RT][64];
  const int tile = blockIdx.x / (a.nb * a.rb), kb = blockIdx.x / a.rb % a.nb;
  const int c0 = blockIdx.x % a.rb * kDownCols;
  if (tile >= *a.count) return;
  const int group = a.list[2 * tile], p0 = a.list[2 * tile + 1];
  const int cnt = tile_positions<0>(a.offsets, group, p0);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int row = lane & 15, ch = lane >> 4;
  const int steps = (a.K + 31) / 32;
  const int b0 = kb * a.spb, b1 = min(steps, b0 + a.spb);
  const int per = (b1 - b0 + kDownWaves - 1) / kDownWaves;
  const int s0 = b0 + wid * per, s1 = min(b1, s0 + per);
  const __bf16* x = a.X + static_cast<int64_t>(a.order[p0 + min(row, cnt - 1)]) * a.ldx + 8 * ch;
  const __bf16* w = a.A + group * a.stride_a + (c0 + row) * a.lda + 8 * ch;
  f32x4 acc[RT] = {};
  struct Frags {
    i32x4 x[kAhead], w[kAhead][RT];
  };
  auto load = [&](int st, Frags& f) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = 32 * (st + u);
      const bool live = st + u < s1 && k + 8 * ch < a.K;
#pragma unroll
      for (int j = 0; j < RT; ++j)
        f.w[u][j] = load8(w + static_cast<int64_t>(16 * j) * a.lda + k, live && c0 + 16 * j < a.r);
      f.x[u] = load8(x + k, live);
    }
  };
  auto mma = [&](const Frags& f) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = mma_bf16(f.w[u][j], f.x[u], acc[j]);
  };
  Frags fa, fb;
  load(s0, fa);
  for (int st = s0; st < s1; st += 2 * kAhead) {
    load(st + kAhead, fb);
    mma(fa);
    if (st + kAhead >= s1) break;
    load(st + 2 * kAhead, fa);
    mma(fb);
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) partial[wid][j][lane] = acc[j];
  __syncthreads();
  // Lane holds position p0 + row and columns c0 + 16 j + 4 ch + e; wave j
  // finishes column tile j.
  const int j = wid;
  if (j >= RT || row >= cnt || c0 + 16 * j >= a.r) return;
  f32x4 v = partial[0][j][lane];
#pragma unroll
  for (int q = 1; q < kDownWaves; ++q) v += partial[q][j][lane];
  *reinterpret_cast<f32x4*>(a.P + (static_cast<int64_t>(kb) * a.M + p0 + row) * a.r + c0 + 16 * j + 4 * ch) = v;
}

// Many rows per adapter.  A workgroup takes a tile of up to 64 positions, one
// block of K and up to 16 RT columns: slices of 64 K elements of those rows of
// X and A run through a ring in LDS (as the weight-streaming int8 kernel's),
// wave w multiplies its 16 positions with every column tile.  Fragments loaded
// straight into registers (16 rows x 64 bytes each) cost the vector-memory
// path about 97 clocks per load; the transfers move 1 KiB in whole lines.
template <int RT>
constexpr int kRingStages = RT <= 4 ? 4 : 3;
template <int RT>
constexpr int kRingBytes = (64 + 16 * RT) * 128;

template <int RT>
__global__ __launch_bounds__(256, 2) void lora_grouped_down_ring_kernel(LoraArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int kS = kRingStages<RT>, kBytes = kRingBytes<RT>;
  constexpr int kBlocks = kBytes / 1024;    // 1 KiB transfers per slice
  constexpr int kDma = (kBlocks + 3) / 4;   // and per wave (some load one twice)
  const int tile = blockIdx.x / (a.nb * a.rb), kb = blockIdx.x / a.rb % a.nb;
  const int c0 = blockIdx.x % a.rb * kDownCols;
  if (tile >= *a.count) return;
  const int group = a.list[2 * tile], p0 = a.list[2 * tile + 1];
  const int cnt = tile_positions<2>(a.offsets, group, p0);
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, ch = lane >> 4;
  const int first = kb * a.spb;
  const int nk = min((a.K + 63) / 64, first + a.spb) - first;  // slices of this block
  // Lane l of a transfer fills chunk l % 8 of row l / 8, which holds chunk
  // (l % 8) ^ (l / 8); rows past the tile's or the rank's last re-read it.
  const int ch16 = ((lane & 7) ^ (lane >> 3)) * 16;
  const uint8_t* from[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int r8 = 8 * min(wid + 4 * i, kBlocks - 1) + (lane >> 3);
    from[i] = reinterpret_cast<const uint8_t*>(
        r8 < 64 ? a.X + static_cast<int64_t>(a.order[p0 + min(r8, cnt - 1)]) * a.ldx
                : a.A + group * a.stride_a + static_cast<int64_t>(min(c0 + r8 - 64, a.r - 1)) * a.lda);
  }
  auto dma = [&](int s, int buf) {
    const int k = (first + s) * 128 + ch16;
    const uint32_t at = k < 2 * a.K ? k : 0;  // chunks past K re-read the row's first and are multiplied as zeros
#pragma unroll
    for (int i = 0; i < kDma; ++i) dma16(from[i] + at, smem + buf * kBytes + min(wid + 4 * i, kBlocks - 1) * 1024);
  };
#pragma unroll
  for (int s = 0; s < kS - 1; ++s)
    if (s < nk) dma(s, s);
  const uint32_t lds0 =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)(smem)));
  uint32_t f_off[2];
#pragma unroll
  for (int st = 0; st < 2; ++st) f_off[st] = lds0 + row * 128 + (((4 * st + ch) ^ (row & 7)) << 4);
  f32x4 acc[RT] = {};
  int buf = 0;
  for (int s = 0; s < nk; ++s) {
    // this wave's transfers of slice s have landed, those behind it may fly
    const int behind = min(kS - 2, nk - 1 - s);
    if (behind >= 2) wait_vm<(kS - 2) * kDma>();
    else if (behind == 1) wait_vm<kDma>();
    else wait_vm<0>();
    barrier();
    // the buffer of slice s - 1, which every wave has read
    if (s + kS - 1 < nk) dma(s + kS - 1, buf == 0 ? kS - 1 : buf - 1);
    i32x4 fx[2], fw[2][RT];
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const uint32_t at = f_off[st] + buf * kBytes;
      lds_read16<0>(fx[st], at + wid * 2048);
      static_for<RT>([&](auto j_c) {
        constexpr int j = decltype(j_c)::value;
        lds_read16<8192 + 2048 * j>(fw[st][j], at);
      });
    }
    wait_lds();
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const bool dead = (first + s) * 128 + 64 * st + 16 * ch >= 2 * a.K;
      landed(fx[st]);
      fx[st] = dead ? i32x4{} : fx[st];
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        landed(fw[st][j]);
        fw[st][j] = dead ? i32x4{} : fw[st][j];
        acc[j] = mma_bf16(fw[st][j], fx[st], acc[j]);
      }
    }
    buf = buf == kS - 1 ? 0 : buf + 1;
  }
  // Lane holds position p0 + 16 wid + row and columns c0 + 16 j + 4 ch + e.
  if (16 * wid + row >= cnt) return;
  float* out = a.P + (static_cast<int64_t>(kb) * a.M + p0 + 16 * wid + row) * a.r + c0 + 4 * ch;
#pragma unroll
  for (int j = 0; j < RT; ++j)
    if (c0 + 16 * j < a.r) *reinterpret_cast<f32x4*>(out + 16 * j) = acc[j];
}

// OUT: 0 = fp32, 1 = bf16.  KS: 32-wide steps of r.  MT: 16-position tiles per
// workgroup; its four waves are MT position tiles x 4 / MT column ranges.
// MT == 4: the waves share the features, whose rows of B pass through LDS.
template <int OUT, int KS, int MT>
__global__ __launch_bounds__(64 * kUpWaves) void lora_grouped_up_kernel(LoraArgs a) {
  using out_t = typename std::conditional<OUT == 0, float, __bf16>::type;
  constexpr int kTerms = OUT == 0 ? 3 : 2;
  constexpr int kVec = 16 / static_cast<int>(sizeof(out_t));
  constexpr int kSegs = 64 / kVec;           // 16-byte pieces per row of a step
  constexpr int kPieces = 16 * kSegs / 64;   // and per lane
  constexpr int kPitch = 64 + 4;             // fp32 per staged row (padded across banks)
  typedef out_t vec_t __attribute__((ext_vector_type(kVec)));
  constexpr bool kShare = MT == 4;
  constexpr int kBPitch = 32 * KS + 8;  // bf16 per staged row of B
  __shared__ float stage[kUpWaves][16 * kPitch];
  __shared__ __attribute__((aligned(16))) __bf16 b_lds[2][kShare ? 64 * kBPitch : 8];
  const int tile = blockIdx.x / a.col_blocks;
  if (tile >= *a.count) return;
  const int group = a.list[2 * tile], p0 = a.list[2 * tile + 1];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int row = lane & 15, ch = lane >> 4;
  const int sub = wid % MT;
  const bool adapted = group < a.groups;
  const int begin = a.offsets[group], last = adapted ? a.offsets[group + 1] : a.M;
  const int end = min(last, p0 + plan_tile_rows(last - begin, MT == 4 ? 2 : 0));
  const int cnt = min(16, end - p0 - 16 * sub);
  if ((!kShare && cnt <= 0) || (!adapted && !a.copy)) return;
  // the wave's first position (an idle wave of a sharing workgroup repeats
  // the tile's first row and stores nothing)
  const int w0 = cnt > 0 ? p0 + 16 * sub : p0;
  // Rows of the lane's pieces of Y and out: piece q is 16 bytes of row
  // (64 q + lane) / kSegs, so that an instruction covers whole 128-byte lines.
  const out_t* y[kPieces];
  out_t* o[kPieces];
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int64_t m = a.order[w0 + min((64 * q + lane) / kSegs, max(cnt, 1) - 1)];
    y[q] = static_cast<const out_t*>(a.Y) + m * a.ldy;
    o[q] = static_cast<out_t*>(a.out) + m * a.ldo;
  }
  const int col = lane % kSegs * kVec;

  bf16x8 t[KS][kTerms] = {};
  float scale = 0.f;
  const __bf16* bw = a.B;
  if (adapted) {
    scale = a.scales[group];
    bw += group * a.stride_b;
    // T, 64 columns at a time: lanes read along the rows and add the K blocks
    // in order, the sums are staged as rows, and every lane takes its
    // fragments' columns (32 s + 8 ch .. + 7 of row l % 16).
    constexpr int kChunk = KS >= 2 ? 2 : 1;  // k steps per pass
    constexpr int kRowPieces = 8 * kChunk;   // 16-byte pieces per row and pass
    constexpr int kPer = 16 * kRowPieces / 64;
    constexpr int kRun = 4;                  // K blocks requested at once
    float* st = stage[wid];
#pragma unroll
    for (int s0 = 0; s0 < KS; s0 += kChunk) {
      f32x4 v[kPer] = {};
      for (int b0 = 0; b0 < a.nb; b0 += kRun) {
        f32x4 w[kRun][kPer] = {};
#pragma unroll
        for (int b = 0; b < kRun; ++b)
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int piece = 64 * i + lane, c = 32 * s0 + piece % kRowPieces * 4;
            const int64_t at = (static_cast<int64_t>(b0 + b) * a.M + w0 + min(piece / kRowPieces, max(cnt, 1) - 1)) * a.r;
            if (b0 + b < a.nb && c < a.r) w[b][i] = *reinterpret_cast<const f32x4*>(a.P + at + c);
          }
#pragma unroll
        for (int b = 0; b < kRun; ++b)
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[i] += w[b][i];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = 64 * i + lane;
        *reinterpret_cast<f32x4*>(st + piece / kRowPieces * kPitch + piece % kRowPieces * 4) = v[i];
      }
      wave_sync();
#pragma unroll
      for (int s = s0; s < s0 + kChunk; ++s) {
        const f32x4* from = reinterpret_cast<const f32x4*>(st + row * kPitch + 32 * (s - s0) + 8 * ch);
        const f32x4 lo = from[0], hi = from[1];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          __bf16 term[kTerms];
          split_terms(e < 4 ? lo[e % 4] : hi[e % 4], term);
#pragma unroll
          for (int q = 0; q < kTerms; ++q) t[s][q][e] = term[q];
        }
      }
      wave_sync();
    }
  }

  const int first = (blockIdx.x % a.col_blocks * (kUpWaves / MT) + wid / MT) * a.col_steps * 64;
  float* st = stage[wid];
  // A step's pieces of Y and of B; the next step's are requested before this
  // one's are used.  B: fragments, or (kShare) the thread's 16-byte pieces of
  // the 64 rows, lane by lane along a row.
  constexpr int kB = kShare ? KS : 4 * KS;
  struct Step {
    vec_t old[kPieces];
    i32x4 b[kB];
  };
  auto load = [&](int n0, Step& f) {
    if (n0 >= a.N) return;
    const bool full = a.vec && n0 + col + kVec <= a.N;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      if (full) {
        f.old[q] = *reinterpret_cast<const vec_t*>(y[q] + n0 + col);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) f.old[q][e] = n0 + col + e < a.N ? y[q][n0 + col + e] : static_cast<out_t>(0.f);
      }
    }
    if (!adapted) return;
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int piece = 256 * i + static_cast<int>(threadIdx.x);  // of 64 rows x 4 KS pieces
      const int r = kShare ? piece / (4 * KS) : 16 * (i / KS) + row;
      const int c = kShare ? piece % (4 * KS) * 8 : 32 * (i % KS) + 8 * ch;
      f.b[i] = load8(bw + static_cast<int64_t>(min(n0 + r, a.N - 1)) * a.ldb + c, c < a.r);
    }
  };
  auto use = [&](int n0, const Step& f, int buf) {
    if (n0 >= a.N) return;
    f32x4 acc[4] = {};
    if (adapted) {
      if constexpr (kShare) {
        // One barrier per step: the buffer was last read two steps ago, and
        // every wave has passed the last step's barrier since.
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          const int piece = 256 * i + static_cast<int>(threadIdx.x);
          *reinterpret_cast<i32x4*>(&b_lds[buf][piece / (4 * KS) * kBPitch + piece % (4 * KS) * 8]) = f.b[i];
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          i32x4 b;
          if constexpr (kShare)
            b = *reinterpret_cast<const i32x4*>(&b_lds[buf][(16 * j + row) * kBPitch + 32 * s + 8 * ch]);
          else
            b = f.b[j * KS + s];
#pragma unroll
          for (int q = 0; q < kTerms; ++q) acc[j] = mma_bf16(b, __builtin_bit_cast(i32x4, t[s][q]), acc[j]);
        }
    }
    // Lane holds position w0 + row and features n0 + 16 j + 4 ch + e: staged
    // as rows in the wave's own area.
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4*>(st + row * kPitch + 16 * j + 4 * ch) = acc[j];
    wave_sync();
    const bool full = a.vec && n0 + col + kVec <= a.N;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int r = (64 * q + lane) / kSegs;
      float d[kVec];
#pragma unroll
      for (int e = 0; e < kVec; e += 4)
        *reinterpret_cast<f32x4*>(d + e) = *reinterpret_cast<const f32x4*>(st + r * kPitch + col + e);
      vec_t v;
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] = static_cast<out_t>(fmaf(scale, d[e], static_cast<float>(f.old[q][e])));
      if (!adapted) v = f.old[q];  // the same bits
      if (r >= cnt) continue;
      if (full) {
        *reinterpret_cast<vec_t*>(o[q] + n0 + col) = v;
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (n0 + col + e < a.N) o[q][n0 + col + e] = v[e];
      }
    }
    wave_sync();  // the next step overwrites the staged rows
  };
  Step fa, fb;
  load(first, fa);
  for (int it = 0; it < a.col_steps; it += 2) {
    const int n0 = first + 64 * it;
    if (it + 1 < a.col_steps) load(n0 + 64, fb);
    use(n0, fa, 0);
    if (it + 1 >= a.col_steps) break;
    if (it + 2 < a.col_steps) load(n0 + 128, fa);
    use(n0 + 64, fb, 1);
  }
}

// Rows per tile: tiles of 64 rows where groups hold that many on average
// (A and B are read by fewer workgroups), of 16 otherwise.
int tile_list(int64_t M, int64_t E) { return M / E >= 32 ? 2 : 0; }

// Blocks of K for the down product, counted in its steps (64-row tiles: 64
// elements, else 32): as many as give one workgroup per CU, with at least four
// steps per wave of a block (89 tiles, K = 2048, r = 64: the pair of launches
// took 57.0, 51.1, 55.1 and 60.7 us with 1, 2, 4 and 6 blocks; 51 tiles,
// K = 4096, r = 16: 12.5, 10.5, 9.9 and 10.8 us with 1, 2, 4 and 8).
int64_t down_steps(int64_t M, int64_t K, int64_t E) { return tile_list(M, E) == 2 ? (K + 63) / 64 : (K + 31) / 32; }
int down_blocks(int64_t M, int64_t K, int64_t r, int64_t E) {
  const int list = tile_list(M, E);
  const int64_t tiles = plan_max_tiles(M, E, list) * ((r + kDownCols - 1) / kDownCols);
  const int64_t steps = down_steps(M, K, E);
  int64_t nb = std::max<int64_t>(1, device_cus() / tiles);
  nb = std::min<int64_t>(nb, std::max<int64_t>(1, steps / (list == 2 ? 4 : 4 * kDownWaves)));
  nb = std::min<int64_t>(nb, 8);
  const int64_t spb = (steps + nb - 1) / nb;
  return static_cast<int>((steps + spb - 1) / spb);
}

template <int RT>
hipError_t launch_down(const LoraArgs& a, int list, dim3 grid, hipStream_t stream) {
  if (list != 2) {
    hipLaunchKernelGGL(lora_grouped_down_kernel<RT>, grid, dim3(64 * kDownWaves), 0, stream, a);
  } else {
    constexpr int kSmem = kRingStages<RT> * kRingBytes<RT>;
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t e =
        set_lds_limit(reinterpret_cast<const void*>(lora_grouped_down_ring_kernel<RT>), kSmem, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lora_grouped_down_ring_kernel<RT>, grid, dim3(256), kSmem, stream, a);
  }
  return hipGetLastError();
}

// Sets the second product's steps per wave and blocks of columns; its workgroups.
int64_t up_blocks(LoraArgs& a) {
  const int b = tile_list(a.M, a.groups);
  const int64_t tiles = plan_max_tiles(a.M, a.groups, b);
  const int ranges = b == 2 ? 1 : kUpWaves;  // column ranges per workgroup
  const int64_t steps = (a.N + 63) / 64;
  // Up to four steps per wave (a row's sums are read once for all of them)
  // while the grid still holds four workgroups per CU.
  int64_t per = 4;
  while (per > 1 && tiles * ((steps + per * ranges - 1) / (per * ranges)) < 4 * device_cus()) per /= 2;
  a.col_steps = static_cast<int>(per);
  a.col_blocks = static_cast<int>((steps + per * ranges - 1) / (per * ranges));
  return tiles * a.col_blocks;
}

template <int OUT, int KS>
void launch_up(LoraArgs a, const RowPlan& plan, hipStream_t stream) {
  const int b = tile_list(a.M, a.groups);
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + kPlanLists + b;  // with the tiles of rows without an adapter
  const dim3 grid(static_cast<unsigned>(up_blocks(a)));
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
  const int b = tile_list(M, plan.groups);
  a.list = plan.tiles + plan_list_at(plan.pairs, plan.groups, b);
  a.count = plan.tiles + b;
  a.nb = down_blocks(M, K, r, plan.groups);
  a.spb = static_cast<int>((down_steps(M, K, plan.groups) + a.nb - 1) / a.nb);
  a.rb = (a.r + kDownCols - 1) / kDownCols;
  const int64_t down = plan_max_tiles(plan.pairs, plan.groups, b) * a.nb * a.rb;
  if (down > kMaxLaunchThreads / (64 * kDownWaves) || up_blocks(a) > kMaxLaunchThreads / (64 * kUpWaves))
    return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(down));
  const hipError_t e = r <= 16   ? launch_down<1>(a, b, grid, stream)
                       : r <= 32 ? launch_down<2>(a, b, grid, stream)
                       : r <= 64 ? launch_down<4>(a, b, grid, stream)
                                 : launch_down<8>(a, b, grid, stream);
  if (e != hipSuccess) return e;
  if (dt == Elt::F32)
    launch_up_r<0>(a, plan, stream);
  else
    launch_up_r<1>(a, plan, stream);
  return hipGetLastError();
}

}  // namespace convrot
