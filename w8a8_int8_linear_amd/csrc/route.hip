// Rows that choose their weights: the router's choice of experts, the plan
// that groups (row, choice) pairs by the weight they chose, and the weighted
// sum that undoes the routing, for gfx950.
//
// Choice (convrot_route).  For a row of E logits l, scores
//   s_i = e^{l_i - max l} / sum_j e^{l_j - max l}   or   1 / (1 + e^{-l_i}),
// choice values c_i = s_i + b_i, the values of groups of experts (the sum of
// the two largest c), and the k largest c among the groups kept, ties to the
// lowest index.  One wavefront takes a row, E / 64 consecutive experts per
// lane, so that among equal values the lowest lane holds the lowest index and
// a maximum over the wavefront needs no index beside it: the owner is the
// first lane of a ballot.  Values are compared as unsigned keys whose order is
// that of the numbers; key 0 is an expert that cannot be chosen.
//   Without a bias and groups the score is a monotone function of the logit,
// and the choice is made on the fp32 logits themselves, exactly.  Otherwise
// two values of c may differ by less than fp32 resolves, so scores and choice
// are computed in fp64.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "device.h"
#include "lanes.h"
#include "launchers.h"

namespace convrot {
namespace {

constexpr int kRouteRows = 4;  // rows (wavefronts) per workgroup

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);  // -0 and 0 are equal
  return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return (b >> 63) != 0 ? ~b : b | 0x8000000000000000ull;
}

// x of the lane DPP control CTRL names (lanes outside ROW_MASK keep x).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_keep(uint32_t x) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), CTRL, ROW_MASK, 0xF, false));
}
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint64_t dpp_keep(uint64_t x) {
  const uint32_t lo = dpp_keep<CTRL, ROW_MASK>(static_cast<uint32_t>(x));
  const uint32_t hi = dpp_keep<CTRL, ROW_MASK>(static_cast<uint32_t>(x >> 32));
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint32_t read_lane(uint32_t x, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}
__device__ __forceinline__ uint64_t read_lane(uint64_t x, int lane) {
  return static_cast<uint64_t>(read_lane(static_cast<uint32_t>(x >> 32), lane)) << 32 |
         read_lane(static_cast<uint32_t>(x), lane);
}

// Largest key of the wavefront (uniform): rows of 16 lanes by rotations, then
// the row broadcasts that carry lane 15 / 31 into the following rows.
template <typename Key>
__device__ __forceinline__ Key wave_max(Key v) {
  v = max(v, dpp_keep<lanes::kQuadXor1, 0xF>(v));
  v = max(v, dpp_keep<lanes::kQuadXor2, 0xF>(v));
  v = max(v, dpp_keep<lanes::kRowRor4, 0xF>(v));
  v = max(v, dpp_keep<lanes::kRowRor8, 0xF>(v));
  v = max(v, dpp_keep<0x142, 0xA>(v));  // row_bcast:15 into rows 1 and 3
  v = max(v, dpp_keep<0x143, 0xC>(v));  // row_bcast:31 into rows 2 and 3
  return read_lane(v, 63);
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// A wavefront's own LDS writes are visible to its lanes past this point.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  // +inf counts as the largest finite value (the maximum's exponential is
  // 1); a NaN stays one
  const float x = static_cast<float>(*p);
  return x > 3.402823466e38f ? 3.402823466e38f : x;
}

// A logit an expert can be chosen by (-inf and NaN mark experts that cannot).
__device__ __forceinline__ bool open_logit(float x) { return x >= -3.402823466e38f; }

// Scores of a chosen expert in the precision T of the choice.
template <typename T>
__device__ __forceinline__ T score_of(float x, bool sigmoid, float mx, T inv_sum) {
  if (sigmoid) return T(1) / (T(1) + exp(-static_cast<T>(x)));
  return exp(static_cast<T>(x) - static_cast<T>(mx)) * inv_sum;
}

// NE: consecutive experts per lane.  WIDE: choice in fp64 with bias and
// groups; otherwise on the logits.
template <typename L, int NE, bool WIDE>
__global__ __launch_bounds__(64 * kRouteRows) void route_kernel(const L* __restrict__ logits, int64_t ldl, int M,
                                                                int E, const float* __restrict__ bias, RouteArgs ra,
                                                                int32_t* __restrict__ ids,
                                                                float* __restrict__ weights) {
  using T = typename std::conditional<WIDE, double, float>::type;
  using Key = typename std::conditional<WIDE, uint64_t, uint32_t>::type;
  extern __shared__ __attribute__((aligned(16))) double choice_values[];  // [kRouteRows][E], with groups
  const int lane = threadIdx.x & 63;
  const int wid = threadIdx.x >> 6;
  const int m = blockIdx.x * kRouteRows + wid;
  if (m >= M) return;  // (nothing below synchronises the workgroup)
  const L* row = logits + static_cast<int64_t>(m) * ldl;

  float x[NE];
  bool open[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int i = lane * NE + j;
    x[j] = i < E ? load_logit(row + i) : 0.f;
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    open[j] = lane * NE + j < E && open_logit(x[j]);
    if (open[j]) top = max(top, order_key(x[j]));
  }
  // The softmax's maximum; its sum only where it is used: with renormalised
  // weights it cancels, and without bias and groups it does not change the
  // choice.
  float mx = 0.f;
  T inv_sum = T(1);
  if (!ra.sigmoid) {
    const uint32_t t = wave_max(top);
    mx = __builtin_bit_cast(float, (t >> 31) != 0 ? t & 0x7FFFFFFFu : ~t);
    if (WIDE || !ra.renormalise) {
      T sum = T(0);
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (open[j]) sum += exp(static_cast<T>(x[j]) - static_cast<T>(mx));
      sum = wave_sum(sum);
      inv_sum = sum > T(0) ? T(1) / sum : T(0);
    }
  }

  Key key[NE];
  if constexpr (WIDE) {
    double c[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const int i = lane * NE + j;
      c[j] = open[j] ? score_of<double>(x[j], ra.sigmoid, mx, inv_sum) : 0.0;
      if (open[j] && bias != nullptr) c[j] += static_cast<double>(bias[i]);
      open[j] = open[j] && c[j] >= -1.7976931348623157e308;  // a bias of -inf or NaN closes its expert
    }
    if (ra.groups > 1) {
      // Group values: 64 / 2^ceil(log2 groups) lanes per group take every
      // such expert's choice value from LDS and merge their two largest.
      const double low = -__builtin_inf();
      double* cv = choice_values + wid * E;
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (lane * NE + j < E) cv[lane * NE + j] = open[j] ? c[j] : low;
      wave_sync();
      const int g = lane >> ra.log2_lanes, lanes_g = 1 << ra.log2_lanes, sub = lane & (lanes_g - 1);
      double a = low, b = low;  // a >= b
      if (g < ra.groups) {
        for (int i = sub; i < ra.per_group; i += lanes_g) {
          const double v = cv[g * ra.per_group + i];
          b = fmax(b, fmin(a, v));
          a = fmax(a, v);
        }
      }
      for (int s = 1; s < lanes_g; s <<= 1) {
        const double a2 = __shfl_xor(a, s), b2 = __shfl_xor(b, s);
        b = fmax(fmax(b, b2), fmin(a, a2));
        a = fmax(a, a2);
      }
      uint64_t gk = 0;
      if (g < ra.groups && sub == 0 && a > low) gk = order_key(b > low ? a + b : a);
      uint64_t kept = 0;  // (uniform) bit g: group g is kept
      for (int t = 0; t < ra.top_groups; ++t) {
        const uint64_t best = wave_max(gk);
        if (best == 0) break;
        const int owner = __ffsll(static_cast<unsigned long long>(__ballot(gk == best))) - 1;
        kept |= uint64_t{1} << (owner >> ra.log2_lanes);
        if (lane == owner) gk = 0;
      }
#pragma unroll
      for (int j = 0; j < NE; ++j) open[j] = open[j] && ((kept >> ((lane * NE + j) / ra.per_group)) & 1) != 0;
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) key[j] = open[j] ? order_key(c[j]) : 0;
  } else {
#pragma unroll
    for (int j = 0; j < NE; ++j) key[j] = open[j] ? order_key(x[j]) : 0;
  }

  // The k largest, one at a time; lane t keeps the t-th choice.
  int mine = -1;
  for (int t = 0; t < ra.k; ++t) {
    Key best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    }
    const Key top_key = wave_max(best);
    if (top_key == 0) break;
    const int owner = __ffsll(static_cast<unsigned long long>(__ballot(best == top_key))) - 1;
    const int chosen = owner * NE + __builtin_amdgcn_readlane(at, owner);
    if (lane == t) mine = chosen;
    if (lane == owner) {
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (j == at) key[j] = 0;
    }
  }
  // Weights of the chosen experts, their sum over the first k lanes in a fixed order.
  T s = T(0);
  if (mine >= 0) s = score_of<T>(load_logit(row + mine), ra.sigmoid, mx, inv_sum);
  if (ra.renormalise) {
    const T total = wave_sum(s);
    s = total > T(0) ? s / total : T(0);
  }
  if (lane < ra.k) {
    ids[static_cast<int64_t>(m) * ra.k + lane] = mine;
    weights[static_cast<int64_t>(m) * ra.k + lane] = static_cast<float>(s * static_cast<T>(ra.scale));
  }
}

template <typename L, bool WIDE>
hipError_t launch_route_typed(const L* logits, int64_t ldl, int64_t M, int64_t E, const float* bias,
                              const RouteArgs& ra, int32_t* ids, float* weights, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((M + kRouteRows - 1) / kRouteRows)), block(64 * kRouteRows);
  const size_t lds = ra.groups > 1 ? sizeof(double) * kRouteRows * E : 0;
  const int m = static_cast<int>(M), e = static_cast<int>(E);
#define CONVROT_ROUTE(NE_)                                                                                   \
  hipLaunchKernelGGL((route_kernel<L, NE_, WIDE>), grid, block, lds, stream, logits, ldl, m, e, bias, ra, ids, \
                     weights)
  if (E <= 64)
    CONVROT_ROUTE(1);
  else if (E <= 128)
    CONVROT_ROUTE(2);
  else if (E <= 256)
    CONVROT_ROUTE(4);
  else if (E <= 512)
    CONVROT_ROUTE(8);
  else
    CONVROT_ROUTE(16);
#undef CONVROT_ROUTE
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The plan: pairs in the order of their groups
// ---------------------------------------------------------------------------
//
// A stable counting sort of the pairs by id.  Every workgroup takes a chunk
// of consecutive pairs and needs, per group, how many pairs precede the chunk
// and how many there are in all.  Few pairs are counted by every workgroup
// anew (one launch); for more, a first launch leaves each chunk's counts in
// the plan and the second adds them up.  No count is added across workgroups
// by atomics, and pairs keep their order inside a group, so the plan is the
// same on every run.  Inside a chunk wavefronts take turns: a lane's place is
// the group's running count plus the lanes below it with the same id.
//   Bound by latency: the starts of the groups and of their tiles in all
// lists come from one scan (a run of consecutive groups per thread, six sums
// at once), which costs two barriers instead of three per sum.

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanSums = 1 + kPlanLists;  // pairs, and tiles of every list

__device__ __forceinline__ int group_of(int32_t id, int E) { return id < 0 || id >= E ? E : id; }

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                                  int chunk, int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];  // [E + 1]
  for (int i = threadIdx.x; i <= E; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int c0 = blockIdx.x * chunk, c1 = min(pairs, c0 + chunk);
  for (int i = c0 + threadIdx.x; i < c1; i += kPlanThreads) atomicAdd(&hist[group_of(ids[i], E)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i <= E; i += kPlanThreads) counts[static_cast<int64_t>(blockIdx.x) * (E + 1) + i] = hist[i];
}

// counts: the chunks' counts of plan_count_kernel, or NULL to count the ids.
__global__ __launch_bounds__(kPlanThreads) void plan_order_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                                  int chunk, const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ tiles) {
  extern __shared__ int32_t lds[];
  const int bins = E + 1;
  int32_t* place = lds;          // [bins]: pairs before this chunk, then this chunk's next place
  int32_t* sums = place + bins;  // [kPlanSums][bins + 1]: sums[0] first the pairs per group
  __shared__ int32_t part[kPlanSums][kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int c0 = blockIdx.x * chunk, c1 = min(pairs, c0 + chunk);
  for (int i = tid; i < bins; i += kPlanThreads) sums[i] = place[i] = 0;
  __syncthreads();
  if (counts == nullptr) {
    for (int i = tid; i < pairs; i += kPlanThreads) {
      const int g = group_of(ids[i], E);
      atomicAdd(&sums[g], 1);
      if (i < c0) atomicAdd(&place[g], 1);
    }
  } else {
    // Every group's counts of all chunks and of those before this one; with
    // few groups the threads share out the chunks too.
    const int chunks = gridDim.x, me = blockIdx.x;
    const int parts = max(1, kPlanThreads / bins);
    for (int i = tid; i < bins * parts; i += kPlanThreads) {
      const int g = i % bins;
      int all = 0, before = 0;
#pragma unroll 8
      for (int c = i / bins; c < chunks; c += parts) {
        const int n = counts[static_cast<int64_t>(c) * bins + g];
        all += n;
        before += c < me ? n : 0;
      }
      atomicAdd(&sums[g], all);
      atomicAdd(&place[g], before);
    }
  }
  __syncthreads();
  // Exclusive scans over the groups: thread t owns groups t per .. + per - 1.
  const int per = (bins + kPlanThreads - 1) / kPlanThreads;
  int own[kPlanSums] = {};
  for (int i = tid * per; i < min(bins, (tid + 1) * per); ++i) {
    const int n = sums[i];
    own[0] += n;
#pragma unroll
    for (int b = 0; b < kPlanLists; ++b) own[1 + b] += (n + (16 << b) - 1) >> (4 + b);
  }
  int upto[kPlanSums];
#pragma unroll
  for (int q = 0; q < kPlanSums; ++q) {
    int s = own[q];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    upto[q] = s;
    if (lane == 63) part[q][wid] = s;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPlanSums; ++q) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) before += w < wid ? part[q][w] : 0;
    upto[q] += before - own[q];
  }
  for (int i = tid * per; i < min(bins, (tid + 1) * per); ++i) {
    const int n = sums[i];
    sums[i] = upto[0];
    place[i] += upto[0];
    if (blockIdx.x == 0 && i <= E) offsets[i] = upto[0];
    upto[0] += n;
#pragma unroll
    for (int b = 0; b < kPlanLists; ++b) {
      sums[(1 + b) * (bins + 1) + i] = upto[1 + b];
      upto[1 + b] += (n + (16 << b) - 1) >> (4 + b);
    }
    if (i == E) {  // the totals
      sums[bins] = upto[0];
#pragma unroll
      for (int b = 0; b < kPlanLists; ++b) sums[(1 + b) * (bins + 1) + bins] = upto[1 + b];
    }
  }
  __syncthreads();

  // This chunk's pairs, 64 per wavefront and turn.
  for (int base = c0; base < c1; base += kPlanThreads) {
    const int i = base + tid;
    const bool live = i < c1;
    const int g = live ? group_of(ids[i], E) : bins;
    // lanes with the same group
    uint64_t same = __ballot(live);
    for (int b = 1; b <= E; b <<= 1) {
      const uint64_t set = __ballot((g & b) != 0);
      same &= (g & b) != 0 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
    const int turns = min(kPlanWaves, (c1 - base + 63) / 64);
    for (int w = 0; w < turns; ++w) {
      if (w == wid && live) {
        const int p = place[g];
        order[p + rank] = i;
        // the last lane of the group leaves the next place
        if (__popcll(same) == rank + 1) place[g] = p + rank + 1;
      }
      __syncthreads();
    }
  }

  // Tile lists: for rows-per-tile 16 << b, every group cut evenly into as few
  // tiles as hold it, the ungrouped positions (group E) last; entry {group,
  // first position}.  The lists are shared out over the workgroups.
  for (int b = 0; b < kPlanLists; ++b) {
    const int32_t* first = sums + (1 + b) * (bins + 1);
    const int total = first[bins];
    if (blockIdx.x == 0 && tid == 0) {
      tiles[b] = first[E];
      tiles[kPlanLists + b] = total;
    }
    int32_t* list = tiles + plan_list_at(pairs, E, b);
    for (int t = blockIdx.x * kPlanThreads + tid; t < total; t += gridDim.x * kPlanThreads) {
      int lo = 0, hi = bins - 1;  // the last group that starts at or before tile t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t) lo = mid; else hi = mid - 1;
      }
      list[2 * t] = lo;
      list[2 * t + 1] = sums[lo] + (t - first[lo]) * plan_tile_rows(sums[lo + 1] - sums[lo], b);
    }
  }
}

// ---------------------------------------------------------------------------
// The weighted sum of a row's k outputs
// ---------------------------------------------------------------------------
//
// out[m, n] = sum_j w[m, j] Y[m k + j, n], fp32, in the order of j.  Bound by
// the bytes of Y: a thread takes 16 bytes of columns and requests up to eight
// rows' pieces before it adds.  Rows of pairs without a group are not read
// (nothing was written there).
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(const T* __restrict__ Y, int64_t ldy,
                                                      const float* __restrict__ weights,
                                                      const int32_t* __restrict__ ids, int M, int k, int N, int E,
                                                      T* __restrict__ out, int64_t ldo) {
  constexpr int kVec = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  typedef T vec_t __attribute__((ext_vector_type(kVec)));
  const int segs = (N + kVec - 1) / kVec;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<int64_t>(M) * segs) return;
  const int m = static_cast<int>(at / segs), n = static_cast<int>(at % segs) * kVec;
  const T* y = Y + static_cast<int64_t>(m) * k * ldy + n;
  const int32_t* id = ids + static_cast<int64_t>(m) * k;
  const float* w = weights + static_cast<int64_t>(m) * k;
  float acc[kVec] = {};
  constexpr int kRun = 8;
  for (int j0 = 0; j0 < k; j0 += kRun) {
    vec_t v[kRun];
    float f[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const bool used = j0 + j < k && id[min(j0 + j, k - 1)] >= 0 && id[min(j0 + j, k - 1)] < E;
      f[j] = used ? w[j0 + j] : 0.f;
      v[j] = vec_t{};
      if (used) v[j] = *reinterpret_cast<const vec_t*>(y + static_cast<int64_t>(j0 + j) * ldy);
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j)
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[e] = fmaf(f[j], static_cast<float>(v[j][e]), acc[e]);
  }
  vec_t o;
#pragma unroll
  for (int e = 0; e < kVec; ++e) o[e] = static_cast<T>(acc[e]);
  *reinterpret_cast<vec_t*>(out + static_cast<int64_t>(m) * ldo + n) = o;
}

template <typename T>
hipError_t launch_combine_typed(const T* Y, int64_t ldy, const float* weights, const int32_t* ids, int64_t M,
                                int64_t k, int64_t N, int64_t E, T* out, int64_t ldo, hipStream_t stream) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  auto rows16 = [](const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * static_cast<int64_t>(sizeof(T))) % 16 == 0;
  };
  const bool vec = N % kVec == 0 && rows16(Y, ldy) && rows16(out, ldo);
  const int64_t work = M * (vec ? N / kVec : N);
  const dim3 grid(static_cast<unsigned>((work + 255) / 256));
  const int m = static_cast<int>(M), kk = static_cast<int>(k), n = static_cast<int>(N), e = static_cast<int>(E);
  if (vec)
    hipLaunchKernelGGL((combine_kernel<T, true>), grid, dim3(256), 0, stream, Y, ldy, weights, ids, m, kk, n, e, out,
                       ldo);
  else
    hipLaunchKernelGGL((combine_kernel<T, false>), grid, dim3(256), 0, stream, Y, ldy, weights, ids, m, kk, n, e, out,
                       ldo);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const void* logits, Elt dt, int64_t ldl, int64_t M, int64_t E, const float* bias,
                        RouteArgs ra, int32_t* ids, float* weights, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  ra.per_group = static_cast<int>(E) / ra.groups;
  ra.log2_lanes = 6;
  while ((64 >> ra.log2_lanes) < ra.groups) --ra.log2_lanes;
  const bool wide = bias != nullptr || ra.groups > 1;
  if (dt == Elt::F32) {
    const auto* l = static_cast<const float*>(logits);
    return wide ? launch_route_typed<float, true>(l, ldl, M, E, bias, ra, ids, weights, stream)
                : launch_route_typed<float, false>(l, ldl, M, E, bias, ra, ids, weights, stream);
  }
  const auto* l = static_cast<const __bf16*>(logits);
  return wide ? launch_route_typed<__bf16, true>(l, ldl, M, E, bias, ra, ids, weights, stream)
              : launch_route_typed<__bf16, false>(l, ldl, M, E, bias, ra, ids, weights, stream);
}

// Pairs counted by every workgroup anew, and pairs per chunk.  A chunk's
// turns are serial, and every workgroup reads all chunks' counts: 1024 pairs
// (16 turns) where the counts are added, 256 where each workgroup counts.
static constexpr int64_t kPlanRecount = 8192;
static int64_t plan_chunk(int64_t pairs) {
  const int64_t c = (pairs + kPlanMaxChunks - 1) / kPlanMaxChunks;
  return std::max<int64_t>(pairs > kPlanRecount ? 1024 : 256, (c + 63) / 64 * 64);
}

int64_t plan_ints(int64_t pairs, int64_t E) {
  return plan_list_at(pairs, E, kPlanLists) +
         (pairs > kPlanRecount ? (pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs) * (E + 1) : 0);
}

hipError_t launch_group_rows(const int32_t* ids, int64_t pairs, int64_t E, int32_t* order, int32_t* offsets,
                             int32_t* tiles, hipStream_t stream) {
  const int chunk = static_cast<int>(plan_chunk(pairs));
  const int p = static_cast<int>(pairs), e = static_cast<int>(E);
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, (pairs + chunk - 1) / chunk)));
  int32_t* counts = pairs > kPlanRecount ? tiles + plan_list_at(pairs, E, kPlanLists) : nullptr;
  if (counts != nullptr)
    hipLaunchKernelGGL(plan_count_kernel, grid, dim3(kPlanThreads), 4 * (E + 1), stream, ids, p, e, chunk, counts);
  const size_t lds = 4 * (E + 1 + kPlanSums * (E + 2));
  if (lds > 65536 - 1024) {  // more than about 2300 groups
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t err = set_lds_limit(reinterpret_cast<const void*>(plan_order_kernel),
                                         4 * (kPlanMaxGroups + 1 + kPlanSums * (kPlanMaxGroups + 2)), lds_set);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(plan_order_kernel, grid, dim3(kPlanThreads), lds, stream, ids, p, e, chunk, counts, order,
                     offsets, tiles);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const void* Y, Elt dt, int64_t ldy, const float* weights, const int32_t* ids,
                               int64_t M, int64_t k, int64_t N, int64_t E, void* out, int64_t ldo,
                               hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  if (dt == Elt::F32)
    return launch_combine_typed(static_cast<const float*>(Y), ldy, weights, ids, M, k, N, E, static_cast<float*>(out),
                                ldo, stream);
  return launch_combine_typed(static_cast<const __bf16*>(Y), ldy, weights, ids, M, k, N, E,
                              static_cast<__bf16*>(out), ldo, stream);
}

}  // namespace convrot
