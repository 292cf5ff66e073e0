// The rank-augmented W4A4 layer with its epilogue -- bias, activation, the
// product of two halves, residual -- for one layer and for rows sorted by
// expert (gfx950).
//
//   v = s_x s_w (C_x C_w^T) + T L2 + bias,   Y = act(v) + residual,
//   gated (N = 2 h channels):  Y[:, j] = act(v[:, j]) v[:, h + j] + residual[:, j]
//
// with the exact int32 product on the int8 MFMA and T = X L1 in
// two or three bf16 parts
// (TwinQuant notes, "TwinQuant: Learnable Subspace Decomposition for W4A4 LLM
// Quantization", section 02 and section 04.C: both components and what follows
// them in one epilogue, one store of Y).

#include "tq_act.h"

namespace tq {
namespace {

// ---------------------------------------------------------------------------
// Rows kernel: up to 16 rows per tile, bound by reading the weight codes.
//   Block: GB groups of 16 output channels (gated: GB groups of each half)
//   of one row tile; its WAVES waves split K into contiguous ranges of
//   64-byte steps, U steps of every group in flight, and take each activation
//   fragment for all groups.  v_mfma_i32_16x16x64_i8 on codes expanded by
//   unpack16 (lane l: row or channel l % 16, code bytes 16 (l / 16) ..); the
//   waves' int32 sums meet exactly in LDS and wave g finishes group g, for
//   gated layers both halves, so the product of the halves needs no exchange.
//   Blocks of one channel group over the row tiles are 8 apart, on the same
//   XCD: an expert's weights come from HBM once, later tiles from its L2.
// ---------------------------------------------------------------------------
template <int WAVES, int GB, bool GATED, bool EX>
__global__ __launch_bounds__(WAVES * 64, WAVES == 4 ? 4 : 2) void k_rows_act(ActArgs g) {
  constexpr int NG = GATED ? 2 * GB : GB;  // 16-channel weight groups
  constexpr int U = 8 / NG > 1 ? 8 / NG : 1;
  constexpr int NT = WAVES * 64;
  __shared__ __attribute__((aligned(16))) int red[WAVES][NG][4][64];
  extern __shared__ __attribute__((aligned(16))) bf16_t sT[];  // [16][tparts r_pad]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, lg = lane >> 4;
  const int NO = GATED ? g.N / 2 : g.N;  // output channels
  const int ncb = (NO + 16 * GB - 1) / (16 * GB);
  // channel blocks in eights, row tiles inside
  const int rtiles = gridDim.x / ((ncb + 7) / 8 * 8);
  const int cb = (blockIdx.x / (8 * rtiles)) * 8 + (blockIdx.x & 7);
  if (cb >= ncb) return;
  const int t = (blockIdx.x >> 3) % rtiles;
  RowTile rt;
  if (EX) {
    rt = expert_tile<16>(g.seg, t);
    if (rt.rows == 0) return;
  } else {
    rt = RowTile{0, 16 * t, min(16, g.M - 16 * t)};
  }
  const int o0 = 16 * GB * cb;  // first output channel
  const uint8_t* W = g.B + (size_t)rt.e * g.N * g.ldb;
  // weight row of group q, lane channel l (clamped to the last)
  auto wrow = [&](int q, int l) { return (q >= GB ? NO : 0) + min(o0 + 16 * (q % GB) + l, NO - 1); };
  const uint8_t* bp[NG];
#pragma unroll
  for (int q = 0; q < NG; ++q) bp[q] = W + (size_t)wrow(q, l16) * g.ldb + 16 * lg;
  const int arow = rt.row0 + min(l16, rt.rows - 1);
  const uint8_t* ap = g.A + (size_t)(EX ? row_token(g.seg, arow) : arow) * g.lda + 16 * lg;

  const int KS = (g.Kb + 63) / 64;
  const int per = (KS + WAVES - 1) / WAVES;
  const int sbeg = wave * per, send = min(KS, sbeg + per);
  // loads from clamped addresses (the row's last 16 bytes, so the offset from
  // this lane group's start is negative for rows shorter than a step), masked
  // where used
  const int kb_last = min((max(send, sbeg + 1) - 1) * 64, g.Kb - 16 - 16 * lg);

  // ---- T: the fp32 partials of the tile's rows summed in chunk order and
  // split into bf16 parts (rows behind the tile's are zero) ----
  const int rp = g.r_pad, tw = g.tparts * rp;
  for (int i = tid; i < 16 * (rp >> 2); i += NT) {
    const int row = i / (rp >> 2), q = i % (rp >> 2);
    float4 v = float4{0.f, 0.f, 0.f, 0.f};
    if (row < rt.rows) {
      const float* p = g.Tp + (size_t)(rt.row0 + row) * rp + 4 * q;
      const size_t stride = (size_t)g.M * rp;
      for (int c = 0; c < g.nchunk; ++c) {
        const float4 x = *reinterpret_cast<const float4*>(p + c * stride);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
    }
    for (int part = 0; part < g.tparts; ++part) {
      const uint2 b = uint2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      *reinterpret_cast<uint2*>(sT + row * tw + part * rp + 4 * q) = b;
      v = float4{v.x - bf16_lo(b.x), v.y - bf16_hi(b.x), v.z - bf16_lo(b.y), v.w - bf16_hi(b.y)};
    }
  }

  // ---- integer product ----
  i32x4 acc[NG];
#pragma unroll
  for (int q = 0; q < NG; ++q) acc[q] = i32x4{0, 0, 0, 0};
  for (int s0 = sbeg; s0 < send; s0 += U) {
    uint4 bv[NG][U], av[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min((s0 + u) * 64, kb_last);
#pragma unroll
      for (int q = 0; q < NG; ++q) bv[q][u] = *reinterpret_cast<const uint4*>(bp[q] + kb);
      av[u] = *reinterpret_cast<const uint4*>(ap + kb);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u >= send) continue;
      if ((s0 + u) * 64 + 16 * lg >= g.Kb) av[u] = uint4{0, 0, 0, 0};  // past the row: zero codes
      const i32x4 a0 = unpack16(av[u].x, av[u].y), a1 = unpack16(av[u].z, av[u].w);
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, unpack16(bv[q][u].x, bv[q][u].y), acc[q], 0, 0, 0);
        acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, unpack16(bv[q][u].z, bv[q][u].w), acc[q], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][q][i][lane] = acc[q][i];
  __syncthreads();
  if (wave >= GB) return;

  // ---- epilogue of group `wave`: lane l, element i -> row 4 (l / 16) + i, channel l % 16 ----
  const int oc = o0 + 16 * wave + l16;
  float sx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = rt.row0 + min(4 * lg + i, rt.rows - 1);
    sx[i] = g.sx[EX ? row_token(g.seg, p) : p];
  }
  const bf16_t* L2 = g.lowrank ? reinterpret_cast<const bf16_t*>(g.lowrank + rt.e * g.lr_stride + g.l2_off) : nullptr;
  float v[GATED ? 2 : 1][4];
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    const int q = wave + h * GB, ch = wrow(q, l16);
    const float sw = g.sw[(size_t)rt.e * g.N + ch];
    const float bias = g.bias ? g.bias[(size_t)rt.e * g.N + ch] : 0.0f;
    f32x4 lr = {0.f, 0.f, 0.f, 0.f};
    for (int t0 = 0; t0 < rp; t0 += 32) {
      const uint4 l2 = *reinterpret_cast<const uint4*>(L2 + (size_t)ch * rp + t0 + 8 * lg);
      for (int part = g.tparts - 1; part >= 0; --part) {
        const uint4 tv = *reinterpret_cast<const uint4*>(sT + l16 * tw + part * rp + t0 + 8 * lg);
        lr = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(tv), as_bf16x8(l2), lr, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s += red[w][q][i][lane];
      v[h][i] = (float)(s >> 8) * (sx[i] * sw) + lr[i] + bias;
    }
  }
  activate4(v[0], g.act);
  if (oc >= NO) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * lg + i;
    if (row >= rt.rows) break;
    const size_t o = (size_t)(rt.row0 + row) * NO + oc;
    float y = v[0][i];
    if (GATED) y *= v[GATED ? 1 : 0][i];
    if (g.res) y += g.res_bf16 ? bf16_to_f32(((const bf16_t*)g.res)[o]) : ((const float*)g.res)[o];
    if (g.y_bf16)
      ((bf16_t*)g.Y)[o] = (bf16_t)(pack_bf16x2(y, y) & 0xFFFFu);
    else
      ((float*)g.Y)[o] = y;
  }
}

template <int WAVES, int GB, bool GATED, bool EX>
hipError_t rows_t(const ActArgs& a, hipStream_t st) {
  const int64_t no = GATED ? a.N / 2 : a.N, ncb = (no + 16 * GB - 1) / (16 * GB);
  const int64_t tiles = EX ? max_expert_tiles(a.M, a.seg.E, 16) : (a.M + 15) / 16;
  const int64_t blocks = (ncb + 7) / 8 * 8 * tiles;
  if (blocks <= 0 || blocks > INT32_MAX) return hipErrorInvalidValue;
  launch_kernel(k_rows_act<WAVES, GB, GATED, EX>, dim3((unsigned)blocks), dim3(WAVES * 64), (unsigned)(32 * a.tparts * a.r_pad), st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_act(const ActArgs& a, bool gated, bool experts, hipStream_t st) {
  if (gated) return experts ? rows_t<4, 1, true, true>(a, st) : rows_t<4, 1, true, false>(a, st);
  return experts ? rows_t<4, 2, false, true>(a, st) : rows_t<4, 2, false, false>(a, st);
}

}  // namespace tq
