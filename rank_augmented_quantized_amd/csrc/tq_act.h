// Shared by the kernels of the fused-epilogue layer and of the experts'
// products (tq_act.hip, tq_expert.hip): their arguments, the tiles of ragged
// expert segments and the activations.
#pragma once

#include "tq_kernels.h"

namespace tq {

// Activation codes of the C ABI (tq_act).
enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

constexpr int kMaxExperts = 1024;
constexpr int kRowsTile = 16;  // rows per tile of the rows kernel

// Sorted rows of E experts: expert e holds rows [offsets[e], offsets[e + 1])
// of P; row p reads token order[p] / topk (order null: token p itself).
struct Segments {
  const int32_t* offsets;  // E + 1, on the device
  const int32_t* order;    // P pair indices, or null
  int E, P, topk;
  int ntok;  // rows of X
};

// One layer (or E of them, stacked) with its epilogue:
//   v = s_x s_w (C_x C_w^T) + T L2 + bias,  Y = act(v) [x v of the other half] + residual.
// T, L1 and L2 as in the rank-augmented layer, but T is not rounded to one
// bf16 value: the fp32 sum is split into tparts of them, each the rounded
// rest (error 2^-8 |t|, 2^-16 |t|, 2^-24 |t| with 1, 2, 3), and every part
// multiplies L2 on the MFMA.  An fp32 Y takes 3 (fp32 accuracy), a bf16 Y 2
// (one part's error would reach the size of Y's own rounding where the
// low-rank term is as large as Y); a part costs r_pad of the d + tparts r_pad
// steps of the product.
struct ActArgs {
  const uint8_t* A;  // activation codes, one row per token (lda bytes)
  const float* sx;   // one per token
  const uint8_t* B;  // weight codes: N rows of ldb bytes per expert
  const float* sw;
  int64_t lda, ldb;
  int M;             // rows: tokens, or P sorted rows
  int N;             // weight channels (gated: 2 x the output channels)
  int Kb;            // packed code bytes per weight row (d / 2)
  const uint8_t* lowrank;  // packed factors per expert (L1^T, then L2^T), or null
  int64_t lr_stride;       // bytes per expert
  int64_t l2_off;          // bytes from a blob's start to its L2^T
  int r_pad;
  int tparts;
  const float* Tp;   // rows kernel: nchunk fp32 partials of T, each M x r_pad
  int nchunk;
  const bf16_t* T;   // tile kernel: M rows of tparts r_pad
  const float* bias; // N per expert, or null
  const void* res;   // M x output channels, or null
  int res_bf16;
  int act;
  void* Y;
  int y_bf16;
  Segments seg;
  const int4* map;  // experts: table of row tiles, written by the prologue
};

// The tile of up to TM consecutive rows of one expert that has index t among
// all the experts' tiles in order; rows = 0: there are fewer tiles.  Called by
// whole waves (each finds it for itself; no barrier).  Offsets are clamped to
// 0 .. P and to be non-decreasing, so no row index leaves the buffers.
struct RowTile {
  int e, row0, rows;
};
template <int TM>
__device__ __forceinline__ RowTile expert_tile(const Segments& s, int t) {
  constexpr int R = 4;  // offsets of 4 x 64 experts in flight
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < s.E; e0 += 64 * R) {
    int a[R], b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = min(e0 + 64 * r + lane, s.E - 1);
      a[r] = s.offsets[e];
      b[r] = s.offsets[e + 1];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      a[r] = min(max(a[r], 0), s.P);
      b[r] = min(max(b[r], a[r]), s.P);
      const int tiles = e0 + 64 * r + lane < s.E ? (b[r] - a[r] + TM - 1) / TM : 0;
      int inc = tiles;  // inclusive sum over the lanes
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(inc, d);
        if (lane >= d) inc += y;
      }
      const int total = __builtin_amdgcn_readlane(inc, 63);
      if (t < base + total) {
        const uint64_t past = __ballot(base + inc > t);  // lanes whose tiles end behind t
        const int l = __builtin_amdgcn_readfirstlane((int)__builtin_ctzll(past));
        const int j = t - base - (__builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(tiles, l));
        const int ra = __builtin_amdgcn_readlane(a[r], l), rb = __builtin_amdgcn_readlane(b[r], l);
        return RowTile{e0 + 64 * r + l, ra + j * TM, min(TM, rb - ra - j * TM)};
      }
      base += total;
    }
  }
  return RowTile{0, 0, 0};
}
// Most such tiles: every expert with rows has at most one that is not full.
__host__ __device__ inline int64_t max_expert_tiles(int64_t P, int64_t E, int64_t TM) { return P / TM + (E < P ? E : P); }

// Token of sorted row p (p inside 0 .. P - 1).
__device__ __forceinline__ int row_token(const Segments& s, int p) {
  if (!s.order) return p;
  return (int)min((uint32_t)s.order[p] / (uint32_t)s.topk, (uint32_t)(s.ntok - 1));
}

constexpr int kMaxTParts = 3;

// gelu(x) = x Phi(x) with Phi from the complementary error function:
// erfc(z) = P(t) exp(-z^2), t = 1 / (1 + 0.3275911 z), z = |x| / sqrt(2)
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26: absolute
// error at most 1.5e-7 for every z >= 0).  x < 0 uses it directly and x > 0
// its complement, so neither side cancels; the error in gelu is at most
// 0.75e-7 |x|.
__device__ __forceinline__ float gelu_erf(float x) {
  const float z = fabsf(x) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, z, 1.0f));
  float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  p = __builtin_fmaf(p, t, 1.421413741f);
  p = __builtin_fmaf(p, t, -0.284496736f);
  p = __builtin_fmaf(p, t, 0.254829592f);
  const float c = 0.5f * p * t * __expf(-z * z);  // Phi(-|x|)
  return x * (x < 0.0f ? c : 1.0f - c);
}
// x / (1 + exp(-k x)): silu (k = 1), and gelu_tanh, whose tanh form is
// x sigmoid(2 sqrt(2 / pi) (x + 0.044715 x^3)).  exp overflows to inf for
// very negative arguments and the quotient is then -0, as the limit.
__device__ __forceinline__ float x_sigmoid(float x, float u) { return x * __builtin_amdgcn_rcpf(1.0f + __expf(-u)); }

// The activation of four values (one branch for the four).
__device__ __forceinline__ void activate4(float (&v)[4], int act) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = v[q] < 0.0f ? 0.0f : v[q];
      break;
    case ACT_SILU:
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = x_sigmoid(v[q], v[q]);
      break;
    case ACT_GELU:
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = gelu_erf(v[q]);
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = x_sigmoid(v[q], 1.5957691216057308f * __builtin_fmaf(0.044715f * v[q] * v[q], v[q], v[q]));
      break;
    default: break;
  }
}

// Work split of the experts' first low-rank stage.
struct ExpertTPlan {
  int rt;      // 16-row groups per block: 1 (rows product, k-chunk partials), 2 or 4 (tile product)
  int qs;      // 16-column slices per block
  int ncg;     // column groups of 16 qs
  int ksteps;  // 32-k steps per chunk
  int nchunk;
  int tiles;   // row tiles (upper bound)
};
ExpertTPlan plan_expert_t(int64_t P, int E, int d, int r_pad, bool partial);
struct ExpertPrologue {
  const void* X;
  int d;
  uint8_t* xc;  // per token: codes and scale
  float* sx;
  const uint8_t* lowrank;
  int64_t lr_stride;
  int r_pad, tparts;
  Segments seg;
  ExpertTPlan t;
  float* Tp;  // partials of T
  unsigned* counters;  // tile product with k split: one per tile and column group, zero between calls
  bf16_t* T;  // tile product: T in bf16 parts
  int4* map;  // table of row tiles of map_rows rows
  int map_rows;
  int nqb;    // set by the launcher
};
hipError_t launch_expert_prologue(const ExpertPrologue& p, bool bf16, bool packed, hipStream_t st);
// The product and its epilogue: up to 16 rows per tile, bound by the weights
// (codes nibble-packed), or 256 channels by up to 256 rows (int8-order codes).
hipError_t launch_rows_act(const ActArgs& a, bool gated, bool experts, hipStream_t st);
hipError_t launch_tile_act(const ActArgs& a, bool gated, bool experts, hipStream_t st);
// Rows per tile of launch_tile_act for M rows of E experts (E = 0: one layer) and N weight channels.
int tile_act_rows(int64_t M, int64_t E);
// Routing plan and combination (tq_expert.hip).
size_t expert_plan_ws_bytes(int64_t P, int E);
hipError_t launch_expert_plan(const void* ids, bool i64, int64_t P, int E, int32_t* offsets, int32_t* order,
                              int32_t* pos, void* ws, hipStream_t st);
hipError_t launch_expert_combine(const void* Z, bool z_bf16, int n, int topk, int m, int64_t P, const int32_t* pos,
                                 const void* w, bool w_bf16, const void* res, bool res_bf16, void* Y, bool y_bf16,
                                 hipStream_t st);

}  // namespace tq
