// Tile product of the layer with its epilogue, for one layer and for experts'
// rows (gfx950).  The main loop is the rank-augmented layer's (tq_gemm8.hip):
// packed weight codes and int8-order activation codes go from HBM into LDS
// by direct loads, three stages of 128 k, weights are expanded to int8 at
// fragment read, v_mfma_i32_32x32x32_i8 accumulates exactly in int32
// (TwinQuant notes, "TwinQuant: Learnable Subspace Decomposition for W4A4 LLM
// Quantization", section 04.C and Figure 4).  What differs:
//  * gated layers: a wave's 64 channels are 32 of the gate half and the same
//    32 of the other half, so the product of the halves is taken in registers
//    (the weight stays in its stacked layout: the rows are picked by the
//    direct loads' addresses, a wave's loads lying all in one half);
//  * experts: a tile's rows belong to one expert, found in a table of row
//    tiles that the prologue wrote; token rows are gathered by the loads'
//    addresses, which cost nothing in the loop;
//  * the epilogue: low-rank term in two or three bf16 parts of T, bias,
//    activation, product of the halves, residual, one store.

#include "tq_act.h"

namespace tq {
namespace {

__device__ __forceinline__ void stage_barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ int psw(int r) { return ((r >> 1) ^ (r >> 3)) & 3; }

// vectors at any element's address (odd channel counts put rows off 16 bytes)
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));

// KF: code rows are whole stages, so no load needs the end-of-row test.
template <int BM, int BN, bool GATED, bool EX, bool KF>
__global__ __launch_bounds__(512) void k_tile_act(ActArgs g) {
  constexpr int WGM = BM / 64, WGN = 8 / WGM;  // wave grid: channels x rows
  constexpr int WM = 64, WN = BN / WGN;
  constexpr int FM = 2, FN = WN / 32;
  static_assert(WN >= 32 && (BM == 256 || BM == 128), "tile shapes");
  constexpr int WPL = BM * 64, XPL = BN * 128, SPL = WPL + XPL;
  constexpr int NST = 3, AHEAD = 2;
  constexpr int WI = WPL / 1024 / 8, XI = XPL / 1024 / 8;  // direct loads per wave per stage
  constexpr int NL = WI + XI;
  constexpr int OC = GATED ? BM / 2 : BM;  // output channels per tile
  constexpr int OW = GATED ? 32 : 64;      // per wave
  static_assert(WI >= 1 && XI >= 1, "each wave fills whole 1 KB pieces");
  static_assert(8 * WN * OW * 2 <= NST * SPL, "Y staging fits in the stage buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NST * SPL];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  const int l32 = lane & 31, lg = lane >> 5;
  const int NO = GATED ? g.N / 2 : g.N;
  const int tiles_m = (NO + OC - 1) / OC;
  int tm, tn;
  RowTile rt;
  if (EX) {
    // the number of row tiles is known on the device only: blocks behind the
    // last tile leave
    const int T = g.map[0].x * tiles_m;
    if ((int)blockIdx.x >= T) return;
    const int tiles_n = g.map[0].x;
    // regroup per XCD (any T), then walk groups of 4 channel tiles
    const int x = blockIdx.x & 7;
    const int b = x * (T >> 3) + min(x, T & 7) + (blockIdx.x >> 3);
    const int gsz = 4 * tiles_n, first = (b / gsz) * 4, gm = min(tiles_m - first, 4), r = b % gsz;
    tm = first + r % gm;
    tn = r / gm;
    const int4 e = g.map[1 + tn];
    rt = RowTile{e.x, e.y, e.z};
  } else {
    tile_of_block(blockIdx.x, tiles_m, (g.M + BN - 1) / BN, tm, tn);
    rt = RowTile{0, tn * BN, min(BN, g.M - tn * BN)};
  }
  const int o0 = tm * OC;  // first output channel
  const int Kb = g.Kb, Kx = 2 * Kb;
  const size_t wrow0 = (size_t)rt.e * g.N;

  // ---- direct loads.  Load i of a wave fills 1 KB: 16 packed weight rows of
  // 64 bytes, rows 16 (wave + 8 i) + lane / 4, or 8 activation rows of 128
  // bytes; the XOR swizzles are applied to the fetched chunk.  Gated: LDS
  // weight row r holds half (r / 32) % 2, output channel 32 (r / 64) + r % 32.
  const int half = GATED ? (wave >> 1) & 1 : 0;
  const int wrows = min(OC, NO - o0);  // weight rows of the half (or tile) that exist
  const i32x4 rw = buffer_rsrc(g.B + (wrow0 + (size_t)half * NO + o0) * g.ldb, (uint32_t)(wrows * g.ldb));
  const bool gather = EX && g.seg.order != nullptr;
  const i32x4 rx = gather ? buffer_rsrc(g.A, (uint32_t)((int64_t)g.seg.ntok * g.lda))
                          : buffer_rsrc(g.A + (size_t)rt.row0 * g.lda, (uint32_t)(rt.rows * g.lda));
  const int cpk = (lane & 3) ^ (((lane >> 3) ^ (2 * (wave & 1) + (lane >> 5))) & 3);
  const int c8 = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
  int vw[WI], vx[XI];
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    const int r = 16 * (wave + 8 * i) + (lane >> 2);
    const int c = GATED ? 32 * (r >> 6) + (r & 31) : r;
    vw[i] = c < wrows ? (int)(c * g.ldb) + 16 * cpk : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int r = 8 * (wave + 8 * i) + (lane >> 3);
    int row = r;
    if (gather) row = row_token(g.seg, rt.row0 + min(r, rt.rows - 1));
    vx[i] = r < rt.rows ? (int)(row * g.lda) + 16 * c8 : kOutOfRange;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  auto issue_one = [&](int i, int kt, int buf) {
    const uint32_t base = lds0 + buf * SPL;
    if (i < WI) {
      const int sw = 64 * kt;
      load_lds16(rw, base + 1024 * (wave + 8 * i), (KF || sw + 16 * cpk < Kb) ? vw[i] : kOutOfRange, sw);
    } else {
      const int sx = 128 * kt;
      load_lds16(rx, base + WPL + 1024 * (wave + 8 * (i - WI)), (KF || sx + 16 * c8 < Kx) ? vx[i - WI] : kOutOfRange,
                 sx);
    }
  };

  // ---- fragments: step s of a stage covers, for lane group lg, the codes of
  // packed chunk 2 (s / 2) + lg, half s % 2, which is int8 chunk 4 (s / 2) +
  // 2 lg + s % 2
  int fa[2], fb[4];
  {
    const int ra = wm * WM + l32, rb = wn * WN + l32;
#pragma unroll
    for (int p = 0; p < 2; ++p) fa[p] = ra * 64 + 16 * ((2 * p + lg) ^ psw(ra));
#pragma unroll
    for (int s = 0; s < 4; ++s) fb[s] = WPL + rb * 128 + 16 * swz(4 * (s >> 1) + 2 * lg + (s & 1), rb);
  }
  i32x16 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0;

  // multiply the stage in buffer buf; the loads of stage kn (>= 0) into
  // buffer nb are spread over the k-steps
  auto compute = [&](int buf, int kn, int nb) {
    const uint8_t* s0 = smem + buf * SPL;
    uint4 pa[2][FM];
    i32x4 xb[2][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) pa[0][f] = *reinterpret_cast<const uint4*>(s0 + fa[0] + 2048 * f);
#pragma unroll
    for (int f = 0; f < FN; ++f) xb[0][f] = *reinterpret_cast<const i32x4*>(s0 + fb[0] + 4096 * f);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int p = s >> 1, h = s & 1;
      if (s == 0) {
#pragma unroll
        for (int f = 0; f < FM; ++f) pa[1][f] = *reinterpret_cast<const uint4*>(s0 + fa[1] + 2048 * f);
      }
      if (s + 1 < 4) {
#pragma unroll
        for (int f = 0; f < FN; ++f) xb[(s + 1) & 1][f] = *reinterpret_cast<const i32x4*>(s0 + fb[s + 1] + 4096 * f);
      }
      i32x4 av[FM];
#pragma unroll
      for (int f = 0; f < FM; ++f)
        av[f] = h ? unpack16(pa[p][f].z, pa[p][f].w) : unpack16(pa[p][f].x, pa[p][f].y);
#pragma unroll
      for (int a = 0; a < FM; ++a) {
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[a], xb[s & 1][b], acc[a][b], 0, 0, 0);
        if (a == 0 && kn >= 0) {
#pragma unroll
          for (int i = NL * s / 4; i < NL * (s + 1) / 4; ++i) issue_one(i, kn, nb);
        }
      }
    }
  };

  const int KT = (Kb + 63) / 64;
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (j < KT) issue_one(i, j, j);
  }
  int buf = 0;
  for (int kt = 0; kt < KT; ++kt) {
    if (kt + AHEAD - 1 < KT)
      wait_vmcnt<(AHEAD - 1) * NL>();
    else
      wait_vmcnt<0>();
    stage_barrier();
    compute(buf, kt + AHEAD < KT ? kt + AHEAD : -1, buf == 0 ? NST - 1 : buf - 1);
    buf = buf == NST - 1 ? 0 : buf + 1;
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
    for (int t0 = 0; t0 < rp; t0 += 16) {
      uint4 la[FM];
#pragma unroll
      for (int a = 0; a < FM; ++a) la[a] = *reinterpret_cast<const uint4*>(lp[a] + t0);
      for (int part = g.tparts - 1; part >= 0; --part) {
        uint4 tb[FN];
#pragma unroll
        for (int b = 0; b < FN; ++b) tb[b] = *reinterpret_cast<const uint4*>(tp[b] + part * rp + t0);
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
          for (int b = 0; b < FN; ++b)
            y[a][b] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(la[a]), as_bf16x8(tb[b]), y[a][b], 0, 0, 0);
      }
    }
  }

  // bf16 Y is staged per wave in LDS (WN rows of OW channels, chunk j of row r
  // swizzled, and the 8-byte halves of a chunk swapped where bit 4 of r is
  // set, so that the 32 rows a store touches fall on distinct banks) and
  // leaves as whole 64- or 128-byte row pieces; fp32 Y is stored directly.
  __syncthreads();  // every wave is done with the stage buffers
  uint8_t* sY = smem + wave * (WN * OW * 2);
  auto ychunk = [&](int row, int j) { return row * (OW * 2) + 16 * (GATED ? j ^ ((row >> 2) & 3) : j ^ ((row >> 1) & 7)); };
#pragma unroll
  for (int a = 0; a < (GATED ? 1 : FM); ++a) {
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const int c = oc(a, e4);
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      const f32x4 b0 = g.bias ? load4(g.bias, 0, c) : zero;
      const f32x4 b1 = GATED && g.bias ? load4(g.bias, 1, c) : zero;
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        const int row = lrow(b);
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = y[a][b][4 * e4 + q] + b0[q];
        activate4(v, g.act);
        if (GATED) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] *= y[1][b][4 * e4 + q] + b1[q];
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
    launch_kernel(k_tile_act<BM, BN, GATED, EX, true>, dim3((unsigned)blocks), dim3(512), 0, st, a);
  else
    launch_kernel(k_tile_act<BM, BN, GATED, EX, false>, dim3((unsigned)blocks), dim3(512), 0, st, a);
  return hipGetLastError();
}

template <bool GATED>
hipError_t tile_one(const ActArgs& a, hipStream_t st) {
  constexpr int OC = GATED ? 128 : 256;
  const int64_t no = GATED ? a.N / 2 : a.N, cols = (no + OC - 1) / OC;
  // fewer 256 x 256 tiles than compute units: half as many rows, then half as
  // many channels per tile
  if (cols * ((a.M + 255) / 256) >= 224) return tile_t<256, 256, GATED, false>(a, st);
  if (cols * ((a.M + 127) / 128) >= 224) return tile_t<256, 128, GATED, false>(a, st);
  return tile_t<128, 128, GATED, false>(a, st);
}

template <bool GATED>
hipError_t tile_experts(const ActArgs& a, hipStream_t st) {
  switch (tile_act_rows(a.M, a.seg.E)) {
    case 256: return tile_t<256, 256, GATED, true>(a, st);
    case 128: return tile_t<256, 128, GATED, true>(a, st);
    default: return tile_t<256, 64, GATED, true>(a, st);
  }
}

}  // namespace

// By the average rows of an expert: a tile of twice as many rows would be
// half empty, and one of half as many would read the weights twice.
int tile_act_rows(int64_t M, int64_t E) {
  const int64_t avg = M / E;
  return avg > 192 ? 256 : (avg > 96 ? 128 : 64);
}

hipError_t launch_tile_act(const ActArgs& a, bool gated, bool experts, hipStream_t st) {
  if (experts) return gated ? tile_experts<true>(a, st) : tile_experts<false>(a, st);
  return gated ? tile_one<true>(a, st) : tile_one<false>(a, st);
}

}  // namespace tq
