// Rows that choose their weights: the router's choice of experts, the plan
// that groups (row, choice) pairs by the weight they chose, and the weighted
// sum that undoes the routing, for gfx950.
//
// Choice (convrot_route).  For a row of E logits l, scores
//   s_i = e^{l_i - max l} / sum_j e^{l_j - max l}   or   1 / (1 + e^{-l_i})
// choice values c_i = s_i + b_i, the values of groups of experts (the sum of
// the two largest c), and the k largest c among the groups kept, ties to the
// lowest index.  Values are compared as unsigned keys whose order is that of
// the numbers; key 0 is an expert that cannot be chosen.  Renormalised weights
// are fp32 too (a few units of 2^-24 off).
//   Without a bias the score is a monotone function of the logit, and experts
// are compared by their fp32 logits, exactly.  A bias and group values need c
// itself, and two of them may differ by less than fp32 resolves: they are
// computed in fp32 with a bound on their error, and where two values
// that the choice has to tell apart lie closer than their errors, the chosen
// ones are ordered again in fp64, or the whole row is done again.
//   Bound by a row's chain of dependent steps, not bytes (8192 rows of 256
// fp32 logits are 8 MB, 1.5 us): 16 lanes take a row where its k allows (four
// rows per wavefront), so that a maximum costs four lane exchanges for four
// rows.  For those rows (k = 8, logistic, 8 groups, bias) fp64 throughout with
// a wavefront per row took 23 us; this takes 11-13 us, and 15-16 us in launches
// where some row has to be done again.  In a graph, launch included: with a
// bias alone 12 (softmax) and 13 us (logistic), without bias and groups 7.6 us,
// one row of 128 4.6 us (4.0 on its own).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "grouped_lds.h"
#include "lanes.h"

namespace convrot {
namespace {

constexpr int kRouteWaves = 4;  // wavefronts per workgroup

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);  // -0 and 0 are equal
  return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return (b >> 63) != 0 ? ~b : b | 0x8000000000000000ull;
}

// The fp32 value of a key.
__device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, (k >> 31) != 0 ? k & 0x7FFFFFFFu : ~k);
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

// +inf counts as the largest finite value (the maximum's exponential is 1); a
// NaN stays one.
__device__ __forceinline__ float clamp_logit(float x) { return x > 3.402823466e38f ? 3.402823466e38f : x; }
template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  return clamp_logit(static_cast<float>(*p));
}

// A logit an expert can be chosen by (-inf and NaN mark experts that cannot).
__device__ __forceinline__ bool open_logit(float x) { return x >= -3.402823466e38f; }

// The score of logit x up to a factor common to a row's choices, most their
// largest logit: renormalised weights depend on the ratios alone, and where
// every chosen score underflows these still hold numbers (the largest's is 1, or
// for logistic scores at least 1/2).
//   e^x = e^most e^{x - most}
//   1 / (1 + e^{-x}) = e^m / (e^m + e^{m - x}),  m = min(most, 0)
// A score of zero in fp64 stays zero: e^{-x} past its largest number, or
// e^{x - max} below half its smallest.
template <typename T>
__device__ __forceinline__ T ratio_score(bool sigmoid, float logit, float max_logit, float most_logit) {
  if (sigmoid ? logit < -709.7827f : static_cast<double>(logit) - static_cast<double>(max_logit) < -745.1332191019412)
    return T(0);
  const T x = logit, most = most_logit;
  auto e = [](T v) {
    if constexpr (std::is_same_v<T, float>) return expf(v);
    else return exp(v);
  };
  if (!sigmoid) return e(x - most);
  const T m = most < T(0) ? most : T(0);
  return T(1) / (e(m) + e(m - x));
}

// One row in fp64 with a whole wavefront: E / 64 (rounded up, NE) consecutive
// experts per lane, so that among equal values the lowest lane holds the
// lowest index.  choice: E doubles of LDS of the wavefront's own (groups > 1).
template <int NE, typename L>
__device__ void route_row_exact(const L* row, int E, const float* bias, const RouteArgs& ra, double* choice,
                                int32_t* ids, float* weights) {
  const int lane = threadIdx.x & 63;
  auto score = [&](float x, float mx, double inv_sum) {
    if (ra.sigmoid) return 1.0 / (1.0 + exp(-static_cast<double>(x)));
    return exp(static_cast<double>(x) - static_cast<double>(mx)) * inv_sum;
  };
  float x[NE];
  bool open[NE];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int i = lane * NE + j;
    x[j] = i < E ? load_logit(row + i) : 0.f;
    open[j] = i < E && open_logit(x[j]);
    if (open[j]) top = max(top, order_key(x[j]));
  }
  float mx = 0.f;
  double inv_sum = 1.0;
  if (!ra.sigmoid) {
    mx = key_value(wave_max(top));
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (open[j]) sum += exp(static_cast<double>(x[j]) - static_cast<double>(mx));
    sum = wave_sum(sum);
    inv_sum = sum > 0.0 ? 1.0 / sum : 0.0;
  }
  uint64_t key[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int i = lane * NE + j;
    double c = open[j] ? score(x[j], mx, inv_sum) : 0.0;
    if (open[j] && bias != nullptr) c += static_cast<double>(bias[i]);
    open[j] = open[j] && c >= -1.7976931348623157e308;  // a bias of -inf or NaN closes its expert
    if (ra.groups > 1 && i < E) choice[i] = open[j] ? c : -__builtin_inf();
    key[j] = open[j] ? order_key(bias != nullptr ? c : static_cast<double>(x[j])) : 0;
  }
  if (ra.groups > 1) {
    // 64 / 2^ceil(log2 groups) lanes per group merge its two largest values.
    wave_sync();
    const double low = -__builtin_inf();
    int log2_lanes = 6;
    while ((64 >> log2_lanes) < ra.groups) --log2_lanes;
    const int g = lane >> log2_lanes, lanes_g = 1 << log2_lanes, sub = lane & (lanes_g - 1);
    const int per_group = E / ra.groups;
    double a = low, b = low;  // a >= b
    if (g < ra.groups) {
      for (int i = sub; i < per_group; i += lanes_g) {
        const double v = choice[g * per_group + i];
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
      kept |= uint64_t{1} << (owner >> log2_lanes);
      if (lane == owner) gk = 0;
    }
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (lane * NE + j >= E || ((kept >> ((lane * NE + j) / per_group)) & 1) == 0) key[j] = 0;
    wave_sync();  // the next row may overwrite the values
  }
  int mine = -1;
  for (int t = 0; t < ra.k; ++t) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    }
    const uint64_t top_key = wave_max(best);
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
  const float mine_x = mine >= 0 ? load_logit(row + mine) : 0.f;
  double s = mine >= 0 ? score(mine_x, mx, inv_sum) : 0.0;
  if (ra.renormalise) {
    const uint32_t most = wave_max(mine >= 0 ? order_key(mine_x) : 0u);
    if (mine >= 0) s = ratio_score<double>(ra.sigmoid, mine_x, mx, key_value(most));
    const double total = wave_sum(s);
    s = total > 0.0 ? s / total : 0.0;
  }
  if (lane < ra.k) {
    ids[lane] = mine;
    weights[lane] = static_cast<float>(s * static_cast<double>(ra.scale));
  }
}

// Reductions over the L lanes of a row (every lane gets the result).
template <int L, typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, F&& f) {
  auto as = [](uint32_t u) { return __builtin_bit_cast(T, u); };
  const auto bits = [](T t) { return __builtin_bit_cast(uint32_t, t); };
  v = f(v, as(lanes::dpp_u<lanes::kQuadXor1>(bits(v))));
  v = f(v, as(lanes::dpp_u<lanes::kQuadXor2>(bits(v))));
  v = f(v, as(lanes::dpp_u<lanes::kRowRor4>(bits(v))));
  v = f(v, as(lanes::dpp_u<lanes::kRowRor8>(bits(v))));
  if constexpr (L > 16) v = f(v, __shfl_xor(v, 16));
  if constexpr (L > 32) v = f(v, __shfl_xor(v, 32));
  return v;
}

// f over v[0 .. N) as a tree (N a power of two), so that the steps overlap.
template <int N, typename T, typename F>
__device__ __forceinline__ T tree(const T (&v)[N], F&& f) {
  if constexpr (N == 1) {
    return v[0];
  } else {
    T h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) h[i] = f(v[i], v[i + N / 2]);
    return tree<N / 2>(h, f);
  }
}

// L: lanes per row (at least k; k + 2 where there is a bias, or every row is
// done in fp64).
// NE: experts per lane, in runs of up to four consecutive ones that the lanes
// of a row take in turn.  WIDE: with a bias or groups; NX: experts per lane of
// the fp64 path.
template <typename Lg, int L, int NE, bool WIDE, int NX>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const Lg* __restrict__ logits, int64_t ldl, int M,
                                                                 int E, const float* __restrict__ bias, RouteArgs ra,
                                                                 int32_t* __restrict__ ids,
                                                                 float* __restrict__ weights) {
  constexpr int kRows = 64 / L;  // rows per wavefront
  constexpr int kRun = NE < 4 ? NE : 4;
  constexpr float kU = 5.9604645e-8f;  // 2^-24
  constexpr uint64_t kRowLanes = L == 64 ? ~uint64_t{0} : (uint64_t{1} << (L % 64)) - 1;
  extern __shared__ __attribute__((aligned(16))) double choice_lds[];  // per wavefront, RouteArgs::lds_doubles
  const int lane = threadIdx.x & 63;
  const int wid = threadIdx.x >> 6;
  const int l = lane % L, base = lane - l;  // lane within the row, the row's first lane
  const int m0 = (blockIdx.x * kRouteWaves + wid) * kRows;
  if (m0 >= M) return;  // (nothing below synchronises the workgroup)
  const int m = min(m0 + lane / L, M - 1);  // (rows past the last repeat it and store nothing)
  const Lg* row = logits + static_cast<int64_t>(m) * ldl;
  auto expert = [&](int j) { return (j / kRun * L + l) * kRun + j % kRun; };
  auto max_u = [](uint32_t a, uint32_t b) { return max(a, b); };
  auto min_i = [](int a, int b) { return min(a, b); };
  auto add_f = [](float a, float b) { return a + b; };
  auto max_f = [](float a, float b) { return fmaxf(a, b); };

  float x[NE];
  typedef Lg run_t __attribute__((ext_vector_type(kRun)));
#pragma unroll
  for (int j = 0; j < NE; j += kRun) {
    const int i = expert(j);
    if (ra.vec) {
      run_t v{};
      if (i < E) v = *reinterpret_cast<const run_t*>(row + i);
#pragma unroll
      for (int e = 0; e < kRun; ++e) x[j + e] = i < E ? clamp_logit(static_cast<float>(v[e])) : -__builtin_inff();
    } else {
#pragma unroll
      for (int e = 0; e < kRun; ++e) x[j + e] = i + e < E ? load_logit(row + i + e) : -__builtin_inff();
    }
  }
  uint32_t key[NE];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    key[j] = open_logit(x[j]) ? order_key(x[j]) : 0;
    top = max(top, key[j]);
  }
  // The softmax's maximum; its sum only where it is used: with renormalised
  // weights it cancels, and without bias and groups it does not change the
  // choice.
  float mx = 0.f, inv_sum = 1.f;
  if (!ra.sigmoid) {
    top = row_reduce<L>(top, max_u);
    mx = top != 0 ? key_value(top) : 0.f;
    if (WIDE || !ra.renormalise) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (key[j] != 0) sum += expf(x[j] - mx);
      sum = row_reduce<L>(sum, add_f);
      inv_sum = sum > 0.f ? 1.f / sum : 0.f;
    }
  }
  // Score in fp32, and its error in units of 2^-24.  Logistic: expf is good to
  // 2 units of e^-x, the sum and the quotient round once each, so s is off by
  // s (2 (1 - s) + 2) units, which is at most 2.  Softmax: the argument's
  // rounding moves e^-t by t units of itself, i.e. the score by less than one
  // unit of 1 (t e^-t < 0.4) and the sum by less than ln E units of itself; at
  // most 22 additions, expf and two roundings: 36 units of s.
  auto score = [&](float v) {
    return ra.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - mx) * inv_sum;
  };
  auto error = [&](float s, float c) { return kU * ((ra.sigmoid ? 2.1f : 36.f * s + 1.f) + fabsf(c)); };
  // The row's largest score.  Comparisons take the error it gives for every
  // value: with each one's own, a gap between two small scores would count
  // as settled although a value further down, of a large score, may truly lie
  // above both.  With one bound (c's own rounding moves by less than c does)
  // a gap between neighbours also separates all values above it from all below.
  const float s_max = ra.sigmoid ? 1.f : inv_sum;

  bool doubt = false;  // a choice the fp32 values do not settle
  if constexpr (WIDE) {
    // (without branches, so that the experts' chains overlap; what belongs to
    // no open expert is dropped by its key)
    float c[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) c[j] = score(x[j]);
    if (bias != nullptr) {
      typedef float bias_t __attribute__((ext_vector_type(kRun)));
#pragma unroll
      for (int j = 0; j < NE; j += kRun) {
        const int i = expert(j);
        if (ra.vec_bias) {
          const bias_t v = *reinterpret_cast<const bias_t*>(bias + min(i, E - kRun));
#pragma unroll
          for (int e = 0; e < kRun; ++e) c[j + e] += v[e];
        } else {
#pragma unroll
          for (int e = 0; e < kRun; ++e) c[j + e] += bias[min(i + e, E - 1)];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const bool open = key[j] != 0 && c[j] >= -3.402823466e38f;  // a bias of -inf or NaN closes its expert
      key[j] = !open ? 0 : bias != nullptr ? order_key(c[j]) : key[j];
    }
    if (ra.groups > 1) {
      // Group values: the row's choice values in LDS, lanes_g lanes per group
      // (rounds of L / lanes_g groups), then every group's rank by counting.
      const float low = -__builtin_inff();
      float* cv = reinterpret_cast<float*>(choice_lds + wid * ra.lds_doubles) + lane / L * (L * NE + 64);
      float* gv = cv + L * NE;
#pragma unroll
      for (int j = 0; j < NE; ++j) cv[expert(j)] = key[j] != 0 ? c[j] : low;
      wave_sync();
      const int per_group = E / ra.groups;
      int lanes_g = L;
      while (lanes_g > 1 && L / lanes_g < ra.groups) lanes_g >>= 1;
      float err = 0.f;  // of a group's value: two choice values and their sum
      bool past = false;  // a value that fp32 does not hold (biases next to its largest number)
      for (int g0 = 0; g0 < ra.groups; g0 += L / lanes_g) {
        const int g = g0 + l / lanes_g;
        float a = low, b = low;  // a >= b
        if (g < ra.groups) {
#pragma unroll 4
          for (int i = l % lanes_g; i < per_group; i += lanes_g) {
            const float v = cv[g * per_group + i];
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
        }
        for (int s = 1; s < lanes_g; s <<= 1) {
          const float a2 = __shfl_xor(a, s), b2 = __shfl_xor(b, s);
          b = fmaxf(fmaxf(b, b2), fminf(a, a2));
          a = fmaxf(a, a2);
        }
        if (g < ra.groups && l % lanes_g == 0) {
          gv[g] = b > low ? a + b : a;
          if (a > low) {
            err = fmaxf(err, 2.f * error(s_max, a) + kU * (b > low ? fabsf(b) + fabsf(a + b) : 0.f));
            past = past || fabsf(gv[g]) > 3.402823466e38f;
          }
        }
      }
      wave_sync();
      uint64_t kept = 0;
      float worst = -low, best_out = low;  // least kept value, largest one left out
      for (int g0 = 0; g0 < ra.groups; g0 += L) {
        const int g = g0 + l;
        const float v = g < ra.groups ? gv[g] : low;
        int rank = 0;
#pragma unroll 8
        for (int o = 0; o < ra.groups; ++o) {
          const float w = gv[o];
          rank += w > v || (w == v && o < g) ? 1 : 0;
        }
        const bool keep = v > low && rank < ra.top_groups;
        if (keep) worst = fminf(worst, v);
        else best_out = fmaxf(best_out, v);
        const uint64_t bits = __ballot(keep) >> base;
        kept |= (bits & kRowLanes) << g0;
      }
      worst = -row_reduce<L>(-worst, max_f);
      best_out = row_reduce<L>(best_out, max_f);
      err = row_reduce<L>(err, max_f);
      doubt = past || (best_out > low && worst - best_out <= 2.f * err);
      // the expert's group, i / per_group, by a product (half a group's width
      // away from the next integer, exact for these sizes)
      const float inv_group = 1.f / static_cast<float>(per_group);
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const int g = static_cast<int>((static_cast<float>(expert(j)) + 0.5f) * inv_group);
        if (((kept >> (g & 63)) & 1) == 0) key[j] = 0;
      }
    }
  }

  // The k largest, one at a time; lane t of the row keeps the t-th.  Where c
  // decides, two more are taken: neighbours must differ by more than their
  // errors (of the row's largest score), or the first k + 1 are ordered again
  // by their fp64 values.
  const bool check = WIDE && bias != nullptr;
  const int picks = ra.k + (check ? 2 : 0);
  int mine = -1;
  uint32_t mine_key = 0;
  for (int t = 0; t < picks; ++t) {
    uint32_t best = row_reduce<L>(tree<NE>(key, max_u), max_u);
    int at[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) at[j] = key[j] == best && best != 0 ? expert(j) : 0x7FFFFFFF;
    const int chosen = row_reduce<L>(tree<NE>(at, min_i), min_i);
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (expert(j) == chosen) key[j] = 0;
    if (l == t && best != 0) {
      mine = chosen;
      mine_key = best;
    }
  }
  float mine_x = mine >= 0 ? load_logit(row + mine) : 0.f;
  if (check) {
    const float c = mine >= 0 ? key_value(mine_key) : 0.f;
    const float err = error(s_max, c);
    const float c_next = __shfl(c, lane + 1), err_next = __shfl(err, lane + 1);
    const int next = __shfl(mine, lane + 1);
    // lane t: its choice and the next are not told apart
    const bool near = l <= ra.k && mine >= 0 && next >= 0 && c - c_next <= err + err_next;
    const uint64_t pairs = (__ballot(near) >> base) & kRowLanes;  // of this row
    const bool reorder = (pairs & ((uint64_t{1} << ra.k) - 1)) != 0;
    // the set of the first k + 1 is itself in doubt (or has no lane)
    doubt = doubt || ra.k + 2 > L || ((pairs >> (ra.k - 1)) & 3) == 3;
    if (__ballot(reorder) != 0) {  // (uniform)
      double inv = 1.0;
      if (!ra.sigmoid) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NE; ++j)
          if (open_logit(x[j])) sum += exp(static_cast<double>(x[j]) - static_cast<double>(mx));
#pragma unroll
        for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d);
        inv = sum > 0.0 ? 1.0 / sum : 0.0;
      }
      double cd = -__builtin_inf();
      if (mine >= 0 && l <= ra.k) {
        cd = ra.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(mine_x)))
                        : exp(static_cast<double>(mine_x) - static_cast<double>(mx)) * inv;
        cd += static_cast<double>(bias[mine]);
      }
      int rank = 0;
      for (int o = 0; o <= ra.k; ++o) {
        const double co = __shfl(cd, base + o);
        const int io = __shfl(mine, base + o);
        rank += io >= 0 && (co > cd || (co == cd && io < mine)) ? 1 : 0;
      }
      int sorted = -1;
      for (int o = 0; o <= ra.k; ++o) {
        const int ro = __shfl(rank, base + o), io = __shfl(mine, base + o);
        if (io >= 0 && ro == l) sorted = io;
      }
      if (reorder) {
        mine = sorted;
        mine_x = mine >= 0 ? load_logit(row + mine) : 0.f;
      }
    }
  }
  // Weights of the first k lanes, summed in a fixed order.
  float s = 0.f;
  if (mine >= 0 && l < ra.k) s = score(mine_x);
  if (ra.renormalise) {
    // e^-60 times 1 / E is an ordinary fp32 number; scores below that are
    // taken relative to the row's largest choice (for softmax without a bias
    // or groups that is the largest logit, which they are relative to already)
    const bool chosen = mine >= 0 && l < ra.k;
    const bool far = chosen && (ra.sigmoid ? mine_x : mine_x - mx) < -60.f;
    if ((WIDE || ra.sigmoid) && __ballot(far) != 0) {  // (uniform)
      const uint32_t most = row_reduce<L>(chosen ? order_key(mine_x) : 0u, max_u);
      const bool row_far = ((__ballot(far) >> base) & kRowLanes) != 0;
      if (chosen && row_far) s = ratio_score<float>(ra.sigmoid, mine_x, mx, key_value(most));
    }
    const float total = row_reduce<L>(s, add_f);
    s = total > 0.f ? s / total : 0.f;
  }
  uint64_t again = 0;  // (uniform) lanes in doubt
  bool settled = true;
  if constexpr (WIDE) {
    again = __ballot(doubt);
    settled = ((again >> base) & kRowLanes) == 0;
  }
  if (l < ra.k && settled && m0 + lane / L < M) {
    ids[static_cast<int64_t>(m) * ra.k + l] = mine;
    weights[static_cast<int64_t>(m) * ra.k + l] = s * ra.scale;
  }
  if constexpr (WIDE) {
    if (again != 0) {
      wave_sync();
      for (int r = 0; r < kRows && m0 + r < M; ++r) {
        if (((again >> (r * L)) & kRowLanes) == 0) continue;
        const int64_t mr = m0 + r;
        route_row_exact<NX>(logits + mr * ldl, E, bias, ra, choice_lds + wid * ra.lds_doubles, ids + mr * ra.k,
                            weights + mr * ra.k);
      }
    }
  }
}

template <typename Lg, bool WIDE, int L, int NE, int NX>
hipError_t launch_route_typed(const Lg* logits, int64_t ldl, int64_t M, int64_t E, const float* bias, RouteArgs ra,
                              int32_t* ids, float* weights, hipStream_t stream) {
  constexpr int64_t rows = kRouteWaves * (64 / L);
  constexpr int kRun = NE < 4 ? NE : 4;
  ra.vec = E % kRun == 0 && ldl % kRun == 0 && (reinterpret_cast<uintptr_t>(logits) % (kRun * sizeof(Lg))) == 0;
  ra.vec_bias = E % kRun == 0 && (reinterpret_cast<uintptr_t>(bias) % (kRun * sizeof(float))) == 0;
  // fp32 choice and group values of the wavefront's rows, or one row in fp64
  ra.lds_doubles = ra.groups > 1 ? static_cast<int>(std::max<int64_t>(E, (64 / L * (L * NE + 64) + 1) / 2)) : 0;
  const size_t lds = sizeof(double) * kRouteWaves * ra.lds_doubles;  // at most 32 KiB
  // (a launch holds 2^32 / 256 workgroups less one; more rows take several)
  constexpr int64_t step = kMaxLaunchThreads / (64 * kRouteWaves) * rows;
  for (int64_t m0 = 0; m0 < M; m0 += step) {
    const int64_t m = std::min(step, M - m0);
    hipLaunchKernelGGL((route_kernel<Lg, L, NE, WIDE, NX>), dim3(static_cast<unsigned>((m + rows - 1) / rows)),
                       dim3(64 * kRouteWaves), lds, stream, logits + m0 * ldl, ldl, static_cast<int>(m),
                       static_cast<int>(E), bias, ra, ids + m0 * ra.k, weights + m0 * ra.k);
  }
  return hipGetLastError();
}

// Sixteen lanes per row up to 14 choices and 256 experts (at most 16 per lane),
// more lanes above.
template <typename Lg, bool WIDE>
hipError_t launch_route_lanes(const Lg* l, int64_t ldl, int64_t M, int64_t E, const float* bias, const RouteArgs& ra,
                              int32_t* ids, float* weights, hipStream_t s) {
#define CONVROT_ROUTE(L_, NE_, NX_) return launch_route_typed<Lg, WIDE, L_, NE_, NX_>(l, ldl, M, E, bias, ra, ids, weights, s)
  if (ra.k <= 14 && E <= 256) {
    if (E <= 16) CONVROT_ROUTE(16, 1, 1);
    if (E <= 64) CONVROT_ROUTE(16, 4, 1);
    if (E <= 128) CONVROT_ROUTE(16, 8, 2);
    CONVROT_ROUTE(16, 16, 4);
  }
  if (ra.k <= 30 && E <= 512) CONVROT_ROUTE(32, 16, 8);
  CONVROT_ROUTE(64, 16, 16);
#undef CONVROT_ROUTE
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
// same on every run.
//   Bound by latency: the starts of the groups and of their tiles in all
// lists come from one scan (a run of consecutive groups per thread, six sums
// at once), which costs two barriers instead of three per sum.  65536 pairs of
// 256 groups: 2.7 us to count, 11.1 us to order (13 us with the wavefronts of
// a chunk in turn); one token's eight pairs: 5.4 us (9.2 us with 1024 threads
// and the tile lists one after the other).

constexpr int kPlanThreads = 1024;
constexpr int kPlanSums = 1 + kPlanLists;  // pairs, and tiles of every list
constexpr int kPlanWaveBins = 1024;

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

// T: threads.  counts: the chunks' counts of plan_count_kernel, or NULL to
// count the ids.
template <int T>
__global__ __launch_bounds__(T) void plan_order_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                                  int chunk, const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ tiles) {
  constexpr int kWaves = T / 64;
  extern __shared__ int32_t lds[];
  const int bins = E + 1;
  int32_t* place = lds;          // [bins]: pairs before this chunk, then this chunk's next place
  int32_t* sums = place + bins;  // [kPlanSums][bins + 1]: sums[0] first the pairs per group
  __shared__ int32_t part[kPlanSums][kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int c0 = blockIdx.x * chunk, c1 = min(pairs, c0 + chunk);
  for (int i = tid; i < bins; i += T) sums[i] = place[i] = 0;
  __syncthreads();
  // (requested with the counts; used when the places are known)
  const int first_group = c0 + tid < c1 ? group_of(ids[c0 + tid], E) : bins;
  if (counts == nullptr) {
#pragma unroll 4
    for (int i = tid; i < pairs; i += T) {
      const int g = group_of(ids[i], E);
      atomicAdd(&sums[g], 1);
      if (i < c0) atomicAdd(&place[g], 1);
    }
  } else {
    // Every group's counts of all chunks and of those before this one; with
    // few groups the threads share out the chunks too.
    const int chunks = gridDim.x, me = blockIdx.x;
    const int parts = max(1, T / bins);
    for (int i = tid; i < bins * parts; i += T) {
      const int g = i % bins;
      int all = 0, before = 0;
#pragma unroll 16
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
  const int per = (bins + T - 1) / T;
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
    for (int w = 0; w < kWaves; ++w) before += w < wid ? part[q][w] : 0;
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

  // This chunk's pairs, 64 per wavefront at a time: a lane's place is the
  // group's next place, plus the pairs of the wavefronts before it, plus the
  // lanes below it with the same group.  With up to kPlanWaveBins groups the
  // wavefronts leave their counts in LDS and add those before them; with more
  // they take turns.
  const bool counted = bins <= kPlanWaveBins;
  uint16_t* wave_counts = reinterpret_cast<uint16_t*>(sums + kPlanSums * (bins + 1));  // [kWaves][bins]
  for (int base = c0; base < c1; base += T) {
    const int i = base + tid;
    const bool live = i < c1;
    const int g = base == c0 ? first_group : live ? group_of(ids[i], E) : bins;
    // lanes with the same group
    uint64_t same = __ballot(live);
    for (int b = 1; b <= E; b <<= 1) {
      const uint64_t set = __ballot((g & b) != 0);
      same &= (g & b) != 0 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
    const bool lead = live && rank == 0;  // the first lane of its group
    const int turns = min(kWaves, (c1 - base + 63) / 64);
    if (counted) {
      for (int q = tid; q < kWaves * bins; q += T) wave_counts[q] = 0;
      __syncthreads();
      if (lead) wave_counts[wid * bins + g] = static_cast<uint16_t>(__popcll(same));
      __syncthreads();
      if (live) {
        int p = place[g] + rank;
#pragma unroll 4
        for (int w = 0; w < wid; ++w) p += wave_counts[w * bins + g];
        order[p] = i;
      }
      if (base + T < c1) {  // (uniform) the next 1024 pairs' places
        __syncthreads();
        if (lead) atomicAdd(&place[g], static_cast<int>(__popcll(same)));
        __syncthreads();
      }
    } else {
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
  }

  // Tile lists: for rows-per-tile 16 << b, every group cut evenly into as few
  // tiles as hold it, the ungrouped positions (group E) last; entry {group,
  // first position}.  Sixteen lanes take sixteen entries; they are shared out
  // over the lists, which are written side by side.
  constexpr int kUnits = T / 16 / kPlanLists;  // per list and workgroup
  const int unit = tid / 16;
  if (blockIdx.x == 0 && tid < kPlanLists) {
    tiles[tid] = sums[(1 + tid) * (bins + 1) + E];
    tiles[kPlanLists + tid] = sums[(1 + tid) * (bins + 1) + bins];
  }
  if (unit >= kUnits * kPlanLists) return;
  const int b = unit % kPlanLists;
  const int32_t* first = sums + (1 + b) * (bins + 1);
  int64_t at = 0;  // (by constants: a division by 16 << b would take longer than the search)
#pragma unroll
  for (int q = 0; q < kPlanLists; ++q) at = b == q ? plan_list_at(pairs, E, q) : at;
  int32_t* list = tiles + at;
  const int total = first[bins], stride = gridDim.x * kUnits * 16;
  for (int t = (static_cast<int>(blockIdx.x) * kUnits + unit / kPlanLists) * 16 + tid % 16; t < total; t += stride) {
    int lo = 0, hi = bins - 1;  // the last group that starts at or before tile t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= t) lo = mid; else hi = mid - 1;
    }
    list[2 * t] = lo;
    list[2 * t + 1] = sums[lo] + (t - first[lo]) * plan_tile_rows(sums[lo + 1] - sums[lo], b);
  }
}

// ---------------------------------------------------------------------------
// The weighted sum of a row's k outputs
// ---------------------------------------------------------------------------
//
// out[m, n] = sum_j w[m, j] Y[m k + j, n], fp32, in the order of j.  Bound by
// the bytes of Y: a thread takes 16 bytes of columns and requests up to eight
// rows' pieces before it adds.  Rows of pairs without a group are not read
// (nothing was written there).  65536 bf16 rows of 2048 added to 8192 (302
// MB): 59 us, 5.1 TB/s, what a copy of 1 GiB reaches.
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
  // A launch holds fewer than 2^32 threads; more outputs take several.
  const int64_t segs = vec ? N / kVec : N;
  const int64_t step = std::max<int64_t>(1, (int64_t{1} << 31) / std::max<int64_t>(segs, 1));
  const int kk = static_cast<int>(k), n = static_cast<int>(N), e = static_cast<int>(E);
  for (int64_t m0 = 0; m0 < M; m0 += step) {
    const int m = static_cast<int>(std::min(step, M - m0));
    const dim3 grid(static_cast<unsigned>((m * segs + 255) / 256));
    auto* kern = vec ? combine_kernel<T, true> : combine_kernel<T, false>;
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream, Y + m0 * k * ldy, ldy, weights + m0 * k, ids + m0 * k, m, kk, n,
                       e, out + m0 * ldo, ldo);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const void* logits, Elt dt, int64_t ldl, int64_t M, int64_t E, const float* bias,
                        RouteArgs ra, int32_t* ids, float* weights, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const bool wide = bias != nullptr || ra.groups > 1;
  if (dt == Elt::F32) {
    const auto* l = static_cast<const float*>(logits);
    return wide ? launch_route_lanes<float, true>(l, ldl, M, E, bias, ra, ids, weights, stream)
                : launch_route_lanes<float, false>(l, ldl, M, E, bias, ra, ids, weights, stream);
  }
  const auto* l = static_cast<const __bf16*>(logits);
  return wide ? launch_route_lanes<__bf16, true>(l, ldl, M, E, bias, ra, ids, weights, stream)
              : launch_route_lanes<__bf16, false>(l, ldl, M, E, bias, ra, ids, weights, stream);
}

// Pairs counted by every workgroup anew, and pairs per chunk.  Where the counts
// are added, every workgroup reads those of all chunks, so a chunk is 1024
// pairs: one pass of a workgroup's threads (beyond 1023 groups its sixteen
// wavefronts take turns).  Where every workgroup counts all pairs anyway, 256,
// so that more workgroups share the placing and the tile lists.
static constexpr int64_t kPlanRecount = 8192;
// 256 threads where the pairs and the groups are few (barriers and the scan over
// wavefronts are what costs), 1024 otherwise (us, 256 and 1024 threads): 8 pairs
// of 128 groups 5.4, 6.8; 512 of 256 7.3, 7.7; 2048 of 128 6.7, 7.7; 4096 of 128
// 7.8, 8.0; 2048 of 1023 9.4, 9.2; 8192 of 256 10.3, 9.1.
static constexpr int64_t kPlanSmall = 4096, kPlanSmallGroups = 512;
static int64_t plan_chunk(int64_t pairs) {
  const int64_t c = (pairs + kPlanMaxChunks - 1) / kPlanMaxChunks;
  return std::max<int64_t>(pairs > kPlanRecount ? 1024 : 256, (c + 63) / 64 * 64);
}

int64_t plan_ints(int64_t pairs, int64_t E) {
  return plan_list_at(pairs, E, kPlanLists) +
         (pairs > kPlanRecount ? (pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs) * (E + 1) : 0);
}

template <int T>
static hipError_t launch_plan_order(dim3 grid, const int32_t* ids, int pairs, int E, int chunk, const int32_t* counts,
                                    int32_t* order, int32_t* offsets, int32_t* tiles, hipStream_t stream) {
  auto lds_bytes = [](int groups) {
    const int bins = groups + 1;
    return 4 * (bins + kPlanSums * (bins + 1)) + (bins <= kPlanWaveBins ? 2 * (T / 64) * bins : 0);
  };
  const int lds = lds_bytes(E);
  if (lds > 65536 - 1024) {  // more than about 2300 groups
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t err = set_lds_limit(reinterpret_cast<const void*>(plan_order_kernel<T>),
                                         lds_bytes(static_cast<int>(kPlanMaxGroups)), lds_set);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(plan_order_kernel<T>, grid, dim3(T), lds, stream, ids, pairs, E, chunk, counts, order, offsets,
                     tiles);
  return hipGetLastError();
}

hipError_t launch_group_rows(const int32_t* ids, int64_t pairs, int64_t E, int32_t* order, int32_t* offsets,
                             int32_t* tiles, hipStream_t stream) {
  const int chunk = static_cast<int>(plan_chunk(pairs));
  const int p = static_cast<int>(pairs), e = static_cast<int>(E);
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, (pairs + chunk - 1) / chunk)));
  int32_t* counts = pairs > kPlanRecount ? tiles + plan_list_at(pairs, E, kPlanLists) : nullptr;
  if (counts != nullptr)
    hipLaunchKernelGGL(plan_count_kernel, grid, dim3(kPlanThreads), 4 * (E + 1), stream, ids, p, e, chunk, counts);
  if (pairs <= kPlanSmall && E <= kPlanSmallGroups)
    return launch_plan_order<256>(grid, ids, p, e, chunk, counts, order, offsets, tiles, stream);
  return launch_plan_order<kPlanThreads>(grid, ids, p, e, chunk, counts, order, offsets, tiles, stream);
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
