// Internal launcher declarations shared by the C-ABI layer (api.cpp) and the
// kernel translation units.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

enum class Elt : int { F32 = 0, BF16 = 1, I32 = 2 };
enum class RotKind : int { Regular = 0, Randomized = 1 };
// Activation of a fused epilogue (values of convrot_act).
enum class Act : int { None = 0, GeluErf = 1, GeluTanh = 2, Silu = 3 };

// Fused group rotation + whole-row absmax + int8 quantisation of `rows` rows
// of X.  When `q` is null the kernel writes the fp32 rotated rows to `xrot`
// instead (checking mode).  t16: the codes in the TILE16 layout (ldq == K,
// K % 64 == 0, q holding whole tiles of 16 rows).  Shapes were validated by
// the caller.
hipError_t launch_pack_rows(const void* X, Elt xdt, int64_t rows, int64_t K, int64_t ldx,
                            int log2G, RotKind kind, const int8_t* signs,
                            int8_t* q, int64_t ldq, float* scale,
                            float* xrot, int64_t ldr, hipStream_t stream, bool t16 = false);

// The same kernel in int4 weight mode: codes clamped to [-7, 7], scale =
// row max / 7, written as nibble pairs (K / 2 bytes per row of q).
hipError_t launch_pack_rows_w4(const void* X, Elt xdt, int64_t rows, int64_t K, int64_t ldx, int log2G,
                               RotKind kind, const int8_t* signs, uint8_t* q, int64_t ldq, float* scale,
                               hipStream_t stream);

// int4 nibble pairs [rows, ldq bytes] -> int8 codes [rows, ldd].
hipError_t launch_unpack_w4(const uint8_t* q, int64_t ldq, int64_t rows, int64_t K, int8_t* dst, int64_t ldd,
                            hipStream_t stream);

// Tiled matrix-core GEMM, C = A B^T with both operands K-contiguous.
//   int8 mode : A = Qx [M, K] int8, B = Qw [N, K] int8, exact int32
//               accumulation, epilogue acc * sa[m] * sb[n] + bias[n]
//               (or the raw accumulator when out == I32).
//   bf16 mode : A = X [M, K] bf16, B = W [N, K] bf16, fp32 accumulation,
//               epilogue acc + bias[n].
// lda/ldb/ldc in elements.
hipError_t launch_gemm_i8(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                          const float* sa, const float* sb, const float* bias,
                          int64_t M, int64_t N, int64_t K,
                          void* C, Elt out, int64_t ldc, hipStream_t stream);

hipError_t launch_gemm_bf16(const void* A, int64_t lda, const void* B, int64_t ldb,
                            const float* bias, int64_t M, int64_t N, int64_t K,
                            void* C, Elt out, int64_t ldc, hipStream_t stream);

// int8 mode with a fused activation, Y = act(A sa sb + bias); `act` is
// GeluErf or GeluTanh and `out` F32 or BF16.
hipError_t launch_gemm_i8_act(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                              const float* sa, const float* sb, const float* bias, Act act,
                              int64_t M, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                              hipStream_t stream);

// launch_gemm_i8_act that also writes, for the next layer's pack, the
// largest magnitude of every G-group (G = 2^log2g, log2g in {2, 4, 6, 8}) of
// each output row (as stored) after the regular rotation R_G:
// rowmax [M, ldm] fp32.  Needs N % 256 == 0, K % 128 == 0, C aligned for
// 4-element stores (ldc % 4 == 0).
hipError_t launch_gemm_i8_act_rowmax(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* sa,
                                     const float* sb, const float* bias, Act act, int64_t M, int64_t N, int64_t K,
                                     void* C, Elt out, int64_t ldc, float* rowmax, int64_t ldm, int log2g,
                                     hipStream_t stream);

// The pack of rows of X whose per-group maxima of the rotated values are
// given (pmax [rows, ldp], as launch_gemm_i8_act_rowmax writes them): int8
// codes and scales, regular kind, log2G in {2, 4, 6, 8}.  The same bits as
// launch_pack_rows for maxima computed with the same operations.
hipError_t launch_pack_rows_prescaled(const void* X, Elt xdt, int64_t rows, int64_t K, int64_t ldx, int log2G,
                                      const float* pmax, int64_t ldp, int8_t* q, int64_t ldq, float* scale,
                                      hipStream_t stream);

// Gated pair sharing the packed activation A:
//   Y = act(A Bg^T sa sbg + biasg) * (A Bu^T sa sbu + biasu)
// `act` is GeluErf or GeluTanh and `out` F32 or BF16.
hipError_t launch_gemm_i8_gated(const int8_t* A, int64_t lda, const int8_t* Bg, int64_t ldbg,
                                const float* sbg, const float* biasg, const int8_t* Bu, int64_t ldbu,
                                const float* sbu, const float* biasu, const float* sa, Act act,
                                int64_t M, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                                hipStream_t stream);

// Weight-streaming kernels for small M (M <= kGemvMaxRows).  The int8 one
// gives the same result bits as launch_gemm_i8; the bf16 one computes the
// same as launch_gemm_bf16 up to fp32 summation order.  `ws` is NULL (no
// split over K) or a 16-byte aligned buffer of at least
// gemv_workspace_bytes(...) bytes for the split's partial sums.
constexpr int64_t kGemvMaxRows = 16;
// Partial-sum bytes a small-M launch over M rows, N outputs and K inputs
// splits into on the current device (0: that shape does not split).  bf16:
// the unquantised mode; w4: int4 weights; gated: two weights per launch.
int64_t gemv_workspace_bytes(int64_t M, int64_t N, int64_t K, bool bf16, bool w4, bool gated);
hipError_t launch_gemv_i8(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                          const float* sa, const float* sb, const float* bias,
                          int64_t M, int64_t N, int64_t K,
                          void* C, Elt out, int64_t ldc, void* ws, hipStream_t stream, bool tiled = false,
                          bool xtiled = false);

// Small-M linears that pack their own activation rows: bf16 X [M, ldx
// elements], M <= kPackinMaxRows, K <= packin_max_k(gated), rotated with
// G = 2^log2g of `kind` and quantised exactly as launch_pack_rows does, then
// the same products and epilogue as launch_gemv_i8 / _i8_gated on those
// codes (the same result bits as packing first).
constexpr int64_t kPackinMaxRows = 4;
int64_t packin_max_k(bool gated);
hipError_t launch_gemv_i8_packin(const void* X, int64_t ldx, int log2g, RotKind kind, const int8_t* signs,
                                 const int8_t* B, int64_t ldb, const float* sb, const float* bias, Act act, int64_t M,
                                 int64_t N, int64_t K, void* C, Elt out, int64_t ldc, hipStream_t stream, bool tiled);
hipError_t launch_gemv_i8_gated_packin(const void* X, int64_t ldx, int log2g, RotKind kind, const int8_t* signs,
                                       const int8_t* Bg, int64_t ldbg, const float* sbg, const float* biasg,
                                       const int8_t* Bu, int64_t ldbu, const float* sbu, const float* biasu, Act act,
                                       int64_t M, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                                       hipStream_t stream, bool tiled);

hipError_t launch_gemv_bf16(const void* A, int64_t lda, const void* B, int64_t ldb,
                            const float* bias, int64_t M, int64_t N, int64_t K,
                            void* C, Elt out, int64_t ldc, void* ws, hipStream_t stream);
hipError_t launch_gemv_i8_act(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                              const float* sa, const float* sb, const float* bias, Act act,
                              int64_t M, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                              void* ws, hipStream_t stream, bool tiled = false, bool xtiled = false);
hipError_t launch_gemv_i8_gated(const int8_t* A, int64_t lda, const int8_t* Bg, int64_t ldbg,
                                const float* sbg, const float* biasg, const int8_t* Bu, int64_t ldbu,
                                const float* sbu, const float* biasu, const float* sa, Act act,
                                int64_t M, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                                void* ws, hipStream_t stream, bool tiled = false, bool xtiled = false);

// The weight of a small-M launch in the TILE16 layout (`tiled`): tiles of
// 16 rows, each 64-byte K unit of a tile 1 KiB of consecutive memory; ldb is
// then the bytes of one row.  Needs N % 16 == 0 and whole units.  The int8
// launches above also read the activation A in that layout (`xtiled`: M <=
// 16 rows in one tile, lda == K, K % 64 == 0), whose fragment loads then
// cover whole lines.
//
// TILE16 copy of rows of row_bytes bytes (row_bytes % 64 == 0, rows % 16 ==
// 0): dst receives rows * row_bytes bytes, s_out a copy of s_in [rows].
hipError_t launch_tile_rows(const uint8_t* src, int64_t lds, uint8_t* dst, int64_t rows, int64_t row_bytes,
                            const float* s_in, float* s_out, hipStream_t stream);

// Data-free smoothing of an FFN's intermediate channels (offline): s [F]
// and, where the outputs are non-null, the scaled fp32 weights
// W_up / s (rows) and W_down * s (columns).
hipError_t launch_smooth_ffn(const void* up, Elt up_dt, int64_t ldu, const void* dn, Elt dn_dt, int64_t ldd, int64_t F,
                             int64_t K, int64_t K_out, bool max_norm, float* s, float* up_out, int64_t ldu_out,
                             float* dn_out, int64_t ldd_out, hipStream_t stream);

// Number of K blocks the down product splits K into on the current device
// (1: no split).  With nb > 1 it needs nb * M * r fp32 partials.
int lora_down_blocks(int64_t M, int64_t K, int64_t r);
// T = X A^T rounded to bf16: X bf16 [M, K], A bf16 [r, K] (r % 16 == 0,
// r <= 256), T bf16 [M, ldt]; `partials` (16-byte aligned) holds
// lora_down_blocks(M, K, r) * M * r floats when that count is above 1.
hipError_t launch_lora_down(const void* X, int64_t ldx, const void* A, int64_t lda, int64_t M, int64_t K, int64_t r,
                            void* T, int64_t ldt, float* partials, hipStream_t stream);
// Y[m, n] += scale * sum_j T[m, j] B[n, j]: T bf16 [M, r], B bf16 [N, r]
// (r % 16 == 0, rows 16-byte aligned), Y fp32 or bf16 [M, ldy], in place.
hipError_t launch_lora_up(const void* T, int64_t ldt, const void* B, int64_t ldb, int64_t M, int64_t N, int64_t r,
                          float scale, void* Y, Elt out, int64_t ldy, hipStream_t stream);

// Small-M kernels with int4 weights (nibble pairs, ldb in bytes): the same
// accumulators as the int8 kernels on the expanded codes.  `act` may be
// None (then `out` may be I32) for the plain linear.
hipError_t launch_gemv_w4(const int8_t* A, int64_t lda, const uint8_t* B, int64_t ldb, const float* sa,
                          const float* sb, const float* bias, Act act, int64_t M, int64_t N, int64_t K, void* C,
                          Elt out, int64_t ldc, void* ws, hipStream_t stream, bool tiled = false);
hipError_t launch_gemv_w4_gated(const int8_t* A, int64_t lda, const uint8_t* Bg, int64_t ldbg, const float* sbg,
                                const float* biasg, const uint8_t* Bu, int64_t ldbu, const float* sbu,
                                const float* biasu, const float* sa, Act act, int64_t M, int64_t N, int64_t K,
                                void* C, Elt out, int64_t ldc, void* ws, hipStream_t stream, bool tiled = false);

// ---------------------------------------------------------------------------
// Rows that choose their weights
// ---------------------------------------------------------------------------

// The router's rule (convrot_routing); vec, vec_bias and lds_doubles are set by
// the launcher.
struct RouteArgs {
  int k;
  int groups;
  int top_groups;
  bool sigmoid;
  bool renormalise;
  float scale;
  bool vec;         // runs of logits are loaded as vectors
  bool vec_bias;    // and runs of the bias
  int lds_doubles;  // LDS of a wavefront for choice values
};
constexpr int64_t kRouteMaxExperts = 1024;
constexpr int64_t kRouteMaxChoices = 64;  // one lane keeps each choice
hipError_t launch_route(const void* logits, Elt dt, int64_t ldl, int64_t M, int64_t E, const float* bias,
                        RouteArgs ra, int32_t* ids, float* weights, hipStream_t stream);

// The plan of pairs grouped by id.  `tiles` starts with kPlanLists counts of
// grouped tiles and kPlanLists counts of all tiles, then list b (tiles of at
// most 16 << b positions, {group, first position} each) at plan_list_at(.., b);
// the ungrouped positions are group E.
constexpr int kPlanLists = 5;
constexpr int64_t kPlanMaxChunks = 256;
constexpr int64_t kPlanMaxPairs = int64_t{1} << 22;
constexpr int64_t kPlanMaxGroups = 4096;
// Most tiles of 16 << b positions: every non-empty group adds at most one
// that is not full.
__host__ __device__ inline int64_t plan_max_tiles(int64_t pairs, int64_t E, int b) {
  return pairs / (16 << b) + (E + 1 < pairs ? E + 1 : pairs);
}
__host__ __device__ inline int64_t plan_list_at(int64_t pairs, int64_t E, int b) {
  int64_t at = 2 * kPlanLists;
  for (int i = 0; i < b; ++i) at += 2 * plan_max_tiles(pairs, E, i);
  return at;
}
// Rows of a group's tiles in the list of 16 << b: the group is cut evenly into
// as few tiles as it needs (in whole 16 rows; the last may be shorter), so
// that their work differs little.
__host__ __device__ inline int plan_tile_rows(int rows, int b) {
  const int n = (rows + (16 << b) - 1) >> (4 + b);
  return n <= 1 ? 16 << b : ((rows + n - 1) / n + 15) & ~15;
}
int64_t plan_ints(int64_t pairs, int64_t E);  // int32 values of `tiles`
hipError_t launch_group_rows(const int32_t* ids, int64_t pairs, int64_t E, int32_t* order, int32_t* offsets,
                             int32_t* tiles, hipStream_t stream);

// out[m] = sum_j weights[m, j] Y[m k + j] over pairs whose id is in [0, E).
hipError_t launch_combine_rows(const void* Y, Elt dt, int64_t ldy, const float* weights, const int32_t* ids,
                               int64_t M, int64_t k, int64_t N, int64_t E, void* out, int64_t ldo,
                               hipStream_t stream);

// Threads of a launch in one dimension: fewer than 2^32 (the runtime drops what
// is above without an error).  Launchers split their rows, or return
// hipErrorInvalidConfiguration before they launch anything.
constexpr int64_t kMaxLaunchThreads = (int64_t{1} << 32) - 1;

// A plan as the products read it: pair p of row p / per_row sits at position
// i with order[i] = p.
struct RowPlan {
  const int32_t* order;
  const int32_t* offsets;
  const int32_t* tiles;
  int64_t pairs;
  int groups;
  int per_row;
};
// Which row of an operand belongs to a position (convrot_row_order).
enum class RowOrder : int { Row = 0, Pair = 1, Sorted = 2 };

// Grouped linears over stacked weights [groups * N, K]: the rows of group e
// meet weight rows e N .. (e + 1) N - 1.
//   plain  Y = act(A sa sb + bias)            (act None; Gelu; Silu)
//   gated  Y = act(A sa sb + bias) * (A sa sb2 + bias2), the second product with B2
hipError_t launch_linear_grouped(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* sa,
                                 const float* sb, const float* bias, const int8_t* B2, int64_t ldb2, const float* sb2,
                                 const float* bias2, bool gated, Act act, const RowPlan& plan, RowOrder source,
                                 RowOrder dest, int64_t N, int64_t K, void* C, Elt out, int64_t ldc,
                                 hipStream_t stream);

// Low-rank corrections of rows in different groups: T = X A_g^T into the
// workspace, then out = Y + scale_g T B_g^T.
int64_t lora_grouped_ws_bytes(int64_t M, int64_t K, int64_t r, int64_t E);
hipError_t launch_lora_grouped(const void* X, int64_t ldx, const void* A, int64_t lda, int64_t stride_a,
                               const void* B, int64_t ldb, int64_t stride_b, const float* scales, int64_t M,
                               int64_t K, int64_t N, int64_t r, const RowPlan& plan, const void* Y, int64_t ldy,
                               void* out, int64_t ldo, Elt dt, void* ws, hipStream_t stream);

}  // namespace convrot
