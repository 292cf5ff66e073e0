// Tile product of the layer with its epilogue, for one layer and for experts'
// rows (gfx950): exact int32 sums of weight and activation codes on
// v_mfma_i32_32x32x32_i8 (TwinQuant notes, "TwinQuant: Learnable Subspace
// Decomposition for W4A4 LLM Quantization", section 04.C and Figure 4), then
// low-rank term, bias, activation, product of a gated layer's halves and
// residual in registers, and one store.
//
// A block is 4 waves and its LDS at most 80 KB, so that two blocks share a
// compute unit: one's epilogue, barriers and load waits run under the other's
// MFMAs.  (The rank-augmented layer's kernel, tq_gemm8.hip, has one block of
// 8 waves per unit; with this epilogue, which is longer, every tile would
// pay it in full.)
//
// Direct loads (buffer_load ... lds) bring packed weight codes, 128 k of the
// block's channels at a time into a ring of three slots, and int8-order
// activation codes, 64 k of its rows at a time into a ring of four; both
// planes have 64-byte LDS rows.  One loop step is half a weight slot, 64 k:
//   wait for the loads issued three steps ago or earlier, barrier, multiply
//   (the weights expanded to 16 x code at fragment read), and meanwhile issue
//   the activations of step h + 3 and half of the weights of slot h / 2 + 2
//   into what step h - 1 freed.
// Gated layers: a wave's 64 channels are 32 of the gate half and the same 32
// of the other half, so their product is taken in registers; the weight stays
// in its stacked layout, the rows are picked by the loads' addresses (a wave's
// loads lie all in one half).  Experts: a tile's rows belong to one expert,
// found in a table of row tiles that the prologue wrote; token rows are
// gathered by the loads' addresses, which costs nothing in the loop.

#include <type_traits>

#include "tq_act.h"

namespace tq {
namespace {

__device__ __forceinline__ void stage_barrier() { asm volatile("s_barrier" ::: "memory"); }
// LDS rows of 64 bytes: chunk c (16 bytes) of row r sits at slot c ^ psw(r).
// A 16-byte LDS read serves 16 lanes at a time, measured to be lanes 0-3,
// 12-15, 20-23 and 24-27 together and 4-11, 16-19 and 28-31 together (and the
// same in the upper half): row quads {0, 3, 5, 6} and {1, 2, 4, 7}.  Rows
// share their place modulo 256 bytes with every fourth row, so the quads of
// each set need four different slots, which r / 4 modulo 4 gives.  (With slots
// distinct over consecutive rows instead, every read took two passes: 5.5 M
// of 11.1 M read cycles at 4096 x 4096 x 4096 were conflicts.)
__device__ __forceinline__ int psw(int r) { return (r >> 2) & 3; }

// vectors at any element's address (odd channel counts put rows off 16 bytes)
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));

// KF: code rows are whole slots (d % 128 == 0), so no load needs the
// end-of-row test.
template <int BM, int BN, bool GATED, bool EX, bool KF>
__global__ __launch_bounds__(256, 2) void k_tile_act(ActArgs g) {
  constexpr int WGM = BM / 64, WGN = 4 / WGM;  // wave grid: channels x rows
  constexpr int WM = 64, WN = BN / WGN;
  constexpr int FM = 2, FN = WN / 32;
  static_assert((BM == 256 || BM == 128) && WN >= 32, "tile shapes");
  constexpr int WPL = BM * 64, XPL = BN * 64;  // one slot of each ring
  constexpr int NWS = 3, NXS = 4, XBASE = NWS * WPL;
  constexpr int WI = WPL / 2 / 1024 / 4, XI = XPL / 1024 / 4;  // direct loads per wave per step
  constexpr int NL = WI + XI;
  constexpr int OC = GATED ? BM / 2 : BM;  // output channels per tile
  constexpr int OW = GATED ? 32 : 64;      // per wave
  constexpr int LDS = NWS * WPL + NXS * XPL;
  static_assert(WI >= 1 && XI >= 1, "each wave fills whole 1 KB pieces");
  static_assert(4 * WN * OW * 2 <= LDS && 2 * LDS <= 160 * 1024, "Y staging fits in the rings; two blocks per unit");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  const int l32 = lane & 31, lg = lane >> 5;
  const int NO = GATED ? g.N / 2 : g.N;
  const int tiles_m = (NO + OC - 1) / OC;
  int tm, tn;
  RowTile rt;
  {
    // experts: the number of row tiles is known on the device only, and
    // blocks behind the last tile leave
    const int tiles_n = EX ? g.map[0].x : (g.M + BN - 1) / BN;
    const int T = tiles_n * tiles_m;
    if ((int)blockIdx.x >= T) return;
    // consecutive blocks go round-robin over the 8 XCDs: regroup so that each
    // XCD has consecutive tiles, walked in groups of 4 channel tiles
    const int x = blockIdx.x & 7;
    const int b = x * (T >> 3) + min(x, T & 7) + (blockIdx.x >> 3);
    const int gsz = 4 * tiles_n, first = (b / gsz) * 4, gm = min(tiles_m - first, 4), r = b % gsz;
    tm = first + r % gm;
    tn = r / gm;
  }
  if (EX) {
    const int4 e = g.map[1 + tn];
    rt = RowTile{e.x, e.y, e.z};
  } else {
    rt = RowTile{0, tn * BN, min(BN, g.M - tn * BN)};
  }
  const int o0 = tm * OC;  // first output channel
  const int Kb = g.Kb, Kx = 2 * Kb;
  const size_t wrow0 = (size_t)rt.e * g.N;

  // ---- direct loads: load i of a wave fills 1 KB, 16 rows of 64 bytes, rows
  // 16 (wave + 4 i) + lane / 4 of the plane; the XOR swizzle of the LDS rows
  // is applied to the fetched chunk.  Gated: LDS weight row r holds half
  // (r / 32) % 2, output channel 32 (r / 64) + r % 32.
  const int half = GATED ? (wave >> 1) & 1 : 0;
  const int wrows = min(OC, NO - o0);  // weight rows of the half (or tile) that exist
  const i32x4 rw = buffer_rsrc(g.B + (wrow0 + (size_t)half * NO + o0) * g.ldb, (uint32_t)(wrows * g.ldb));
  const bool gather = EX && g.seg.order != nullptr;
  const i32x4 rx = gather ? buffer_rsrc(g.A, (uint32_t)((int64_t)g.seg.ntok * g.lda))
                          : buffer_rsrc(g.A + (size_t)rt.row0 * g.lda, (uint32_t)(rt.rows * g.lda));
  const int cpk = (lane & 3) ^ psw(16 * wave + (lane >> 2));  // 16-row pieces are 64 rows apart: one swizzle
  int vw[2 * WI], vx[XI];
#pragma unroll
  for (int i = 0; i < 2 * WI; ++i) {
    const int r = 16 * (wave + 4 * i) + (lane >> 2);
    const int c = GATED ? 32 * (r >> 6) + (r & 31) : r;
    vw[i] = c < wrows ? (int)(c * g.ldb) + 16 * cpk : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int r = 16 * (wave + 4 * i) + (lane >> 2);
    const int row = gather ? row_token(g.seg, rt.row0 + min(r, rt.rows - 1)) : r;
    vx[i] = r < rt.rows ? (int)(row * g.lda) + 16 * cpk : kOutOfRange;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int KH = (Kx + 63) / 64, KT = (Kb + 63) / 64;
  // part p (0, 1) of weight slot kt, and the activations of step h
  auto issue_w = [&](int kt, int p, int slot) {
    const int so = 64 * kt;
    const bool ok = KF || so + 16 * cpk < Kb;
#pragma unroll
    for (int i = 0; i < WI; ++i)
      load_lds16(rw, lds0 + slot * WPL + 1024 * (wave + 4 * (WI * p + i)), ok ? vw[WI * p + i] : kOutOfRange, so);
  };
  auto issue_x = [&](int h, int slot) {
    const int so = 64 * h;
    const bool ok = KF || so + 16 * cpk < Kx;
#pragma unroll
    for (int i = 0; i < XI; ++i)
      load_lds16(rx, lds0 + XBASE + slot * XPL + 1024 * (wave + 4 * i), ok ? vx[i] : kOutOfRange, so);
  };

  // ---- fragments: MFMA s (0, 1) of step h takes, for lane group lg, the 16
  // codes of half s of packed chunk 2 (h % 2) + lg, which is int8 chunk 2 lg
  // + s of the step's activations
  int fa[2], fb[2];
  {
    const int ra = wm * WM + l32, rb = wn * WN + l32;
#pragma unroll
    for (int p = 0; p < 2; ++p) fa[p] = ra * 64 + 16 * ((2 * p + lg) ^ psw(ra));
#pragma unroll
    for (int s = 0; s < 2; ++s) fb[s] = XBASE + rb * 64 + 16 * ((2 * lg + s) ^ psw(rb));
  }
  i32x16 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0;

  int ws = 0, xs = 0;  // ring slots of the current step
  auto step = [&](int h, auto pc) {
    constexpr int p = decltype(pc)::value;
    // the loads of the last two steps (NL each while there are weights and
    // activations left to fetch) may stay in flight
    if (h + 3 < KH)
      wait_vmcnt<2 * NL>();
    else
      wait_vmcnt<0>();
    stage_barrier();
    const uint8_t* sw = smem + ws * WPL;
    const uint8_t* sx = smem + xs * XPL;
    uint4 pa[FM];
    i32x4 xb[2][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) pa[f] = *reinterpret_cast<const uint4*>(sw + fa[p] + 2048 * f);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int f = 0; f < FN; ++f) xb[s][f] = *reinterpret_cast<const i32x4*>(sx + fb[s] + 2048 * f);
    if (h + 3 < KH) issue_x(h + 3, xs == 0 ? NXS - 1 : xs - 1);
    if ((h >> 1) + 2 < KT) issue_w((h >> 1) + 2, p, ws == 0 ? NWS - 1 : ws - 1);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      i32x4 av[FM];
#pragma unroll
      for (int f = 0; f < FM; ++f) av[f] = s ? unpack16(pa[f].z, pa[f].w) : unpack16(pa[f].x, pa[f].y);
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[a], xb[s][b], acc[a][b], 0, 0, 0);
    }
    xs = xs == NXS - 1 ? 0 : xs + 1;
    if (p == 1) ws = ws == NWS - 1 ? 0 : ws + 1;
  };
  // what steps -4 .. -1 would have issued, in their order
  issue_w(0, 0, 0);
  issue_w(0, 1, 0);
  issue_x(0, 0);
  if (KH > 1) issue_x(1, 1);
  if (KT > 1) issue_w(1, 0, 1);
  if (KH > 2) issue_x(2, 2);
  if (KT > 1) issue_w(1, 1, 1);
  for (int h = 0; h < KH; h += 2) {
    step(h, std::integral_constant<int, 0>{});
    if (h + 1 < KH) step(h + 1, std::integral_constant<int, 1>{});
  }

  // ---- epilogue.  32x32 result layout: lane l, element e -> channel 8 (e / 4)
  // + 4 (l / 32) + e % 4 of block a, row l % 32 of block b.  Block a is the
  // wave's 32 channels 32 a .., or, gated, its 32 channels of half a.
  // oc(a, e4): first of the four output channels of group e4.
  const int ow = o0 + wm * OW;
  auto oc = [&](int a, int e4) { return ow + (GATED ? 0 : 32 * a) + 8 * e4 + 4 * lg; };
  auto lrow = [&](int b) { return wn * WN + 32 * b + l32; };  // row within the tile
  // four consecutive fp32 of a per-channel vector, from output channel c in half h (clamped at its end)
  auto load4 = [&](const float* p, int h, int c) -> f32x4 {
    const float* q = p + wrow0 + (size_t)h * NO;
    if (c + 3 < NO) return *reinterpret_cast<const f32x4u*>(q + c);
    return f32x4{q[min(c, NO - 1)], q[min(c + 1, NO - 1)], q[min(c + 2, NO - 1)], q[min(c + 3, NO - 1)]};
  };
  f32x16 y[FM][FN];
  {
    f32x4 sw[FM][4];
    float sx[FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) sw[a][e4] = load4(g.sw, GATED ? a : 0, oc(a, e4));
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      const int p = rt.row0 + min(lrow(b), rt.rows - 1);
      sx[b] = g.sx[EX ? row_token(g.seg, p) : p] * (1.0f / 16);  // the weights carry 16 x code
    }
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) y[a][b][e] = (float)acc[a][b][e] * (sw[a][e >> 2][e & 3] * sx[b]);
  }
  if (g.r_pad > 0) {
    // y[channel][row] += sum_t L2^T[channel][t] T[row][t] on the bf16 MFMA, 16
    // t per step, the small parts of T first
    const int rp = g.r_pad;
    const bf16_t* L2 = reinterpret_cast<const bf16_t*>(g.lowrank + rt.e * g.lr_stride + g.l2_off);
    const bf16_t* lp[FM];
    const bf16_t* tp[FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
      lp[a] = L2 + ((size_t)(GATED ? a * NO : 0) + min(ow + (GATED ? 0 : 32 * a) + l32, NO - 1)) * rp + 8 * lg;
#pragma unroll
    for (int b = 0; b < FN; ++b)
      tp[b] = g.T + ((size_t)rt.row0 + min(lrow(b), rt.rows - 1)) * g.tparts * rp + 8 * lg;
    // step j: part j % tparts of t-range 16 (j / tparts), the last part first;
    // DEPTH steps of operands in flight
    constexpr int DEPTH = 3;
    uint4 la[DEPTH][FM], tb[DEPTH][FN];
    const int J = rp / 16 * g.tparts;
    int lt = 0, lpart = g.tparts;  // of the next step to load
    auto load_step = [&](uint4 (&l)[FM], uint4 (&t)[FN]) {
      if (--lpart < 0) {
        lpart = g.tparts - 1;
        lt += 16;
      }
#pragma unroll
      for (int a = 0; a < FM; ++a) l[a] = *reinterpret_cast<const uint4*>(lp[a] + lt);
#pragma unroll
      for (int b = 0; b < FN; ++b) t[b] = *reinterpret_cast<const uint4*>(tp[b] + lpart * rp + lt);
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load_step(la[d], tb[d]);  // J >= 4
    for (int j = 0; j < J; j += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (j + d < J) {
#pragma unroll
          for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
              y[a][b] =
                  __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(la[d][a]), as_bf16x8(tb[d][b]), y[a][b], 0, 0, 0);
          if (j + d + DEPTH < J) load_step(la[d], tb[d]);
        }
      }
    }
  }

  // bf16 Y is staged per wave in LDS (WN rows of OW channels, chunk j of row r
  // swizzled, and the 8-byte halves of a chunk swapped where bit 4 of r is
  // set, so that the 32 rows a store touches fall on distinct banks) and
  // leaves as whole 64- or 128-byte row pieces; fp32 Y is stored directly.
  __syncthreads();  // every wave is done with the rings
  uint8_t* sY = smem + wave * (WN * OW * 2);
  auto ychunk = [&](int row, int j) { return row * (OW * 2) + 16 * (GATED ? j ^ ((row >> 2) & 3) : j ^ ((row >> 1) & 7)); };
#pragma unroll
  for (int a = 0; a < (GATED ? 1 : FM); ++a) {
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const int c = oc(a, e4);
      f32x4 b0, b1;
      if (g.bias) {
        b0 = load4(g.bias, 0, c);
        b1 = GATED ? load4(g.bias, 1, c) : b0;
      }
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        const int row = lrow(b);
        float v[4], u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = y[a][b][4 * e4 + q];
          u[q] = GATED ? y[1][b][4 * e4 + q] : 1.0f;
        }
        if (g.bias) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q] += b0[q];
            u[q] += GATED ? b1[q] : 0.0f;
          }
        }
        activate4(v, g.act);
        if (GATED) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] *= u[q];
        }
        const size_t o = ((size_t)rt.row0 + row) * NO + c;
        if (g.res && row < rt.rows) {
          if (g.res_bf16) {
            const bf16_t* rp = (const bf16_t*)g.res + o;
            if (c + 3 < NO) {
              const u32x2u w = *reinterpret_cast<const u32x2u*>(rp);
              v[0] += bf16_lo(w[0]); v[1] += bf16_hi(w[0]); v[2] += bf16_lo(w[1]); v[3] += bf16_hi(w[1]);
            } else {
              for (int q = 0; q < 4; ++q)
                if (c + q < NO) v[q] += bf16_to_f32(rp[q]);
            }
          } else {
            const float* rp = (const float*)g.res + o;
            if (c + 3 < NO) {
              const f32x4 w = *reinterpret_cast<const f32x4u*>(rp);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] += w[q];
            } else {
              for (int q = 0; q < 4; ++q)
                if (c + q < NO) v[q] += rp[q];
            }
          }
        }
        if (g.y_bf16) {
          const int r = 32 * b + l32;
          *reinterpret_cast<uint2*>(sY + ychunk(r, 4 * a + e4) + 8 * (lg ^ ((r >> 4) & 1))) =
              uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else if (row < rt.rows) {
          float* yp = (float*)g.Y + o;
          if (c + 3 < NO) {
            *reinterpret_cast<f32x4u*>(yp) = f32x4u{v[0], v[1], v[2], v[3]};
          } else {
            for (int q = 0; q < 4; ++q)
              if (c + q < NO) yp[q] = v[q];
          }
        }
      }
    }
  }
  if (g.y_bf16) {
    // 16 bytes per lane; a wave reads only its own staging area
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_wave_barrier();
    constexpr int LPR = OW / 8, RPI = 64 / LPR;  // lanes per row, rows per step
    const int jc = lane % LPR, c = ow + 8 * jc;
#pragma unroll 4
    for (int r0 = 0; r0 < WN; r0 += RPI) {
      const int r = r0 + lane / LPR, row = wn * WN + r;
      uint4 v = *reinterpret_cast<const uint4*>(sY + ychunk(r, jc));
      if ((r >> 4) & 1) v = uint4{v.z, v.w, v.x, v.y};
      if (row < rt.rows) {
        bf16_t* yp = (bf16_t*)g.Y + ((size_t)rt.row0 + row) * NO + c;
        if (c + 7 < NO) {
          *reinterpret_cast<u32x4u*>(yp) = u32x4u{v.x, v.y, v.z, v.w};
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          for (int q = 0; q < 8; ++q)
            if (c + q < NO) yp[q] = (bf16_t)((q & 1) ? (w[q >> 1] >> 16) : (w[q >> 1] & 0xFFFFu));
        }
      }
    }
  }
}

template <int BM, int BN, bool GATED, bool EX>
hipError_t tile_t(const ActArgs& a, hipStream_t st) {
  constexpr int OC = GATED ? BM / 2 : BM;
  const int64_t no = GATED ? a.N / 2 : a.N;
  const int64_t blocks = (no + OC - 1) / OC * (EX ? max_expert_tiles(a.M, a.seg.E, BN) : (a.M + BN - 1) / BN);
  if (blocks <= 0 || blocks > INT32_MAX || 256 * a.ldb >= ((int64_t)1 << 31) || 256 * a.lda >= ((int64_t)1 << 31))
    return hipErrorInvalidValue;
  if (a.Kb % 64 == 0)
    launch_kernel(k_tile_act<BM, BN, GATED, EX, true>, dim3((unsigned)blocks), dim3(256), 0, st, a);
  else
    launch_kernel(k_tile_act<BM, BN, GATED, EX, false>, dim3((unsigned)blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <bool GATED>
hipError_t tile_one(const ActArgs& a, hipStream_t st) {
  constexpr int OC = GATED ? 128 : 256;
  const int64_t no = GATED ? a.N / 2 : a.N, cols = (no + OC - 1) / OC;
  // too few tiles for two blocks on each of the 256 compute units: half as
  // many rows, then half as many channels per tile
  if (cols * ((a.M + 127) / 128) >= 448) return tile_t<256, 128, GATED, false>(a, st);
  if (cols * ((a.M + 63) / 64) >= 448) return tile_t<256, 64, GATED, false>(a, st);
  return tile_t<128, 64, GATED, false>(a, st);
}

template <bool GATED>
hipError_t tile_experts(const ActArgs& a, hipStream_t st) {
  return tile_act_rows(a.M, a.seg.E) == 128 ? tile_t<256, 128, GATED, true>(a, st) : tile_t<256, 64, GATED, true>(a, st);
}

}  // namespace

// By the average rows of an expert: a tile of twice as many rows would be
// half empty, and one of half as many would read the weights twice.
int tile_act_rows(int64_t M, int64_t E) { return M / E > 96 ? 128 : 64; }

hipError_t launch_tile_act(const ActArgs& a, bool gated, bool experts, hipStream_t st) {
  if (experts) return gated ? tile_experts<true>(a, st) : tile_experts<false>(a, st);
  return gated ? tile_one<true>(a, st) : tile_one<false>(a, st);
}

}  // namespace tq
