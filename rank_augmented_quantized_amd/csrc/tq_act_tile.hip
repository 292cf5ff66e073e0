// Tile product of the layer with its epilogue, for one layer and for experts'
// rows (gfx950): exact int32 sums of weight and activation codes on
// v_mfma_i32_32x32x32_i8 (TwinQuant notes, "TwinQuant: Learnable Subspace
// Decomposition for W4A4 LLM Quantization", section 04.C and Figure 4), then
// low-rank term, bias, activation, product of a gated layer's halves and
// residual in registers, and one store.
//
// What bounds it: MFMA issue, and next to it the vector cache, which takes
// about four cycles per cache line that a load touches, whatever it takes of
// the line.  Every operand therefore comes by direct loads (buffer_load ...
// lds) of whole 128-byte lines where its rows are that long:
//   * packed weight codes, 256 k (128 bytes) of the block's channels per slot,
//     a ring of two slots;
//   * int8-order activation codes, 128 k (128 bytes) of its rows per slot, a
//     ring of three or four;
//   * for the low-rank term, 32 ranks at a time of L2^T and of the parts of T
//     (read straight from memory by the MFMA's lanes, 16 bytes of each of 32
//     rows, they cost as much as a quarter of the main loop).
// One stage is 128 k: wait for the loads issued two (activations of a ring of
// four: three) stages ago, barrier, multiply, and meanwhile issue the
// activations of a later stage and, in even stages, the next weight slot into
// what the last stage freed.
// Gated layers: a wave's 64 channels are 32 of the gate half and the same 32
// of the other half, so their product is taken in registers; the weight stays
// in its stacked layout, the rows are picked by the loads' addresses.
// Measured, int8 operations: 4096 x 4096 x 4096, r = 32, 58 us, 2.4 POP/s
// (67 us with a bf16 residual, 33.5 MB more); 2047 tokens of 4096 -> 14336
// gated, r = 64, 211 us, 2.3 POP/s; 4096 tokens x 2 of 8 such experts 867 us,
// 2.2 POP/s; a pure MFMA loop reaches 4.1 to 4.4 POP/s.  1111 tokens x 8 of
// 128 experts of 2048 -> 768 gated, 64-row tiles: 88 us, bound by feeding LDS
// (256 KB per tile of 16 stages, 6.7 TB/s over all units).
// Experts: a tile's rows belong to one expert, found in a table of row tiles
// that the prologue wrote; token rows are gathered by the loads' addresses,
// which costs nothing in the loop.

#include <type_traits>

#include "tq_act.h"

namespace tq {
namespace {

__device__ __forceinline__ void stage_barrier() { asm volatile("s_barrier" ::: "memory"); }
// A 16-byte LDS read serves 16 lanes at a time, measured to be lanes 0-3,
// 12-15, 20-23 and 24-27 together and 4-11, 16-19 and 28-31 together (and the
// same in the upper half): row quads {0, 3, 5, 6} and {1, 2, 4, 7}.  LDS rows
// of 128 bytes share their place modulo 256 with every second row, rows of
// 64 bytes with every fourth; chunk c (16 bytes) of row r sits at slot c ^
// rsw(r) or c ^ psw(r), distinct over such a group.
__device__ __forceinline__ int rsw(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int psw(int r) { return (r >> 2) & 3; }

// vectors at any element's address (odd channel counts put rows off 16 bytes)
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));

// KF: code rows are whole weight slots (d % 256 == 0), so no load needs the
// end-of-row test.
template <int BM, int BN, int NW, bool GATED, bool EX, bool KF>
__global__ __launch_bounds__(64 * NW, 2) void k_tile_act(ActArgs g) {
  constexpr int WGM = BM / 64, WGN = NW / WGM;  // wave grid: channels x rows
  constexpr int WM = 64, WN = BN / WGN;
  constexpr int FM = 2, FN = WN / 32;
  static_assert((BM == 256 || BM == 128) && (NW == 8 || NW == 4) && WN >= 32, "tile shapes");
  constexpr int WPL = BM * 128, XPL = BN * 128;  // one slot of each ring
  constexpr int NWS = 2, NXS = NW == 8 ? 3 : 4, AH = NXS - 1, XBASE = NWS * WPL;
  constexpr int WL = WPL / 1024 / NW, XL = XPL / 1024 / NW;  // direct loads per wave per slot
  constexpr int OC = GATED ? BM / 2 : BM;                    // output channels per tile
  constexpr int OW = GATED ? 32 : 64;                        // per wave
  constexpr int LDS = NWS * WPL + NXS * XPL;
  // low-rank panels: 32 ranks of L2^T (BM rows) and of each part of T (BN rows)
  constexpr int PPL = BM * 64, TPL = BN * 64, PANEL = PPL + kMaxTParts * TPL;
  constexpr int PL = PPL / 1024 / NW, TL = TPL / 1024 / NW;  // direct loads per wave per panel and part
  static_assert(WL >= 1 && XL >= 1 && PL >= 1 && TL >= 1, "each wave fills whole 1 KB pieces");
  static_assert(LDS <= 160 * 1024 && NW * WN * OW * 2 <= LDS && 2 * PANEL <= LDS, "the epilogue fits in the rings");
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
  const int wrows = min(OC, NO - o0);  // weight rows of a half (or of the tile) that exist
  // gated: LDS row r of the channels holds half (r / 32) % 2, output channel
  // 32 (r / 64) + r % 32
  auto chan_row = [&](int r) { return GATED ? 32 * (r >> 6) + (r & 31) : r; };

  // ---- direct loads: load i of a wave fills 1 KB, rows 8 (wave + NW i) +
  // lane / 8 of the plane; the XOR swizzle of the LDS rows is applied to the
  // fetched chunk.  A load's weight rows lie all in one half.
  i32x4 rw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int half = !GATED ? 0 : (NW == 8 ? (wave >> 2) & 1 : h);
    rw[h] = buffer_rsrc(g.B + (wrow0 + (size_t)half * NO + o0) * g.ldb, (uint32_t)(wrows * g.ldb));
  }
  const bool gather = EX && g.seg.order != nullptr;
  const i32x4 rx = gather ? buffer_rsrc(g.A, (uint32_t)((int64_t)g.seg.ntok * g.lda))
                          : buffer_rsrc(g.A + (size_t)rt.row0 * g.lda, (uint32_t)(rt.rows * g.lda));
  const int c8 = (lane & 7) ^ rsw(8 * wave + (lane >> 3));  // the planes' 8-row pieces are 8 NW rows apart: one swizzle
  int vw[WL], vx[XL];
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int c = chan_row(8 * (wave + NW * i) + (lane >> 3));
    vw[i] = c < wrows ? (int)(c * g.ldb) + 16 * c8 : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = 8 * (wave + NW * i) + (lane >> 3);
    const int row = gather ? row_token(g.seg, rt.row0 + min(r, rt.rows - 1)) : r;
    vx[i] = r < rt.rows ? (int)(row * g.lda) + 16 * c8 : kOutOfRange;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int KT = (Kx + 127) / 128, KW = (Kb + 127) / 128;  // stages, weight slots
  auto issue_w = [&](int i, int s) {                        // load i of weight slot s
    const int so = 128 * s;
    load_lds16(rw[i & 1], lds0 + (s & 1) * WPL + 1024 * (wave + NW * i),
               (KF || so + 16 * c8 < Kb) ? vw[i] : kOutOfRange, so);
  };
  auto issue_x = [&](int i, int kt, int slot) {  // load i of the activations of stage kt
    const int so = 128 * kt;
    load_lds16(rx, lds0 + XBASE + slot * XPL + 1024 * (wave + NW * i),
               (KF || so + 16 * c8 < Kx) ? vx[i] : kOutOfRange, so);
  };

  // ---- fragments: step s (0..3) of stage kt takes, for lane group lg, the 16
  // codes of half s % 2 of packed chunk 4 (kt % 2) + 2 (s / 2) + lg, which is
  // int8 chunk 4 (s / 2) + 2 lg + s % 2 of the stage's activations
  const int ra = wm * WM + l32, rb = wn * WN + l32;
  i32x16 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0;

  int xs = 0;  // activation slot of the current stage
  auto stage = [&](int kt, auto hc) {
    constexpr int hf = decltype(hc)::value;  // kt % 2
    // may stay in flight (loads go out in the order weights, activations):
    // the activations of the last AH - 1 stages, and the weights of the last
    // even stage if this one is odd
    if (kt + AH < KT)
      wait_vmcnt<(AH - 1) * XL + (hf ? WL : 0)>();
    else
      wait_vmcnt<0>();
    stage_barrier();
    const uint8_t* sw = smem + ((kt >> 1) & 1) * WPL + ra * 128;
    const uint8_t* sx = smem + XBASE + xs * XPL + rb * 128;
    const bool more_x = kt + AH < KT, more_w = hf == 0 && kt / 2 + 1 < KW;
    const int xn = xs == 0 ? NXS - 1 : xs - 1;  // the last stage's slot
    uint4 pa[2][FM];
    i32x4 xb[2][FN];
    auto read_w = [&](int p) {
#pragma unroll
      for (int f = 0; f < FM; ++f)
        pa[p][f] = *reinterpret_cast<const uint4*>(sw + 4096 * f + 16 * ((4 * hf + 2 * p + lg) ^ rsw(ra)));
    };
    auto read_x = [&](int s) {
#pragma unroll
      for (int f = 0; f < FN; ++f)
        xb[s & 1][f] =
            *reinterpret_cast<const i32x4*>(sx + 4096 * f + 16 * ((4 * (s >> 1) + 2 * lg + (s & 1)) ^ rsw(rb)));
    };
    read_w(0);
    read_x(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int p = s >> 1, h = s & 1;
      if (s == 0) read_w(1);
      if (s + 1 < 4) read_x(s + 1);
      i32x4 av[FM];
#pragma unroll
      for (int f = 0; f < FM; ++f)
        av[f] = h ? unpack16(pa[p][f].z, pa[p][f].w) : unpack16(pa[p][f].x, pa[p][f].y);
#pragma unroll
      for (int a = 0; a < FM; ++a) {
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[a], xb[s & 1][b], acc[a][b], 0, 0, 0);
        if (a == 0) {  // loads spread over the steps: weights first
          if (hf == 0) {
#pragma unroll
            for (int i = (WL + XL) * s / 4; i < (WL + XL) * (s + 1) / 4; ++i) {
              if (i < WL) {
                if (more_w) issue_w(i, kt / 2 + 1);
              } else if (more_x) {
                issue_x(i - WL, kt + AH, xn);
              }
            }
          } else if (more_x) {
#pragma unroll
            for (int i = XL * s / 4; i < XL * (s + 1) / 4; ++i) issue_x(i, kt + AH, xn);
          }
        }
      }
    }
    xs = xs == NXS - 1 ? 0 : xs + 1;
  };
#pragma unroll
  for (int i = 0; i < WL; ++i) issue_w(i, 0);
#pragma unroll
  for (int j = 0; j < AH; ++j)
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (j < KT) issue_x(i, j, j);
  for (int kt = 0; kt < KT; kt += 2) {
    stage(kt, std::integral_constant<int, 0>{});
    if (kt + 1 < KT) stage(kt + 1, std::integral_constant<int, 1>{});
  }

  // ---- epilogue.  32x32 result layout: lane l, element e -> channel 8 (e / 4)
  // + 4 (l / 32) + e % 4 of block a, row l % 32 of block b.  Block a is the
  // wave's 32 channels 32 a .., or, gated, its 32 channels of half a.
  // oc(a, e4): first of the four output channels of group e4.
  const int ow = o0 + wm * OW;
  auto oc = [&](int a, int e4) { return ow + (GATED ? 0 : 32 * a) + 8 * e4 + 4 * lg; };
  auto lrow = [&](int b) { return wn * WN + 32 * b + l32; };  // row within the tile

  // low-rank panels: panel t (32 ranks) into buffer t % 2, LDS rows of 64
  // bytes; load i of a wave fills rows 16 (wave + NW i) + lane / 4
  const int rp = g.r_pad, tw = g.tparts * rp;
  const int cpk = (lane & 3) ^ psw(16 * wave + (lane >> 2));
  auto issue_panel = [&](int t) {
    const uint32_t base = lds0 + (t & 1) * PANEL;
    const int half = GATED ? (wave >> 1) & 1 : 0;  // a load's 16 rows lie all in one half
    const i32x4 rl = buffer_rsrc(g.lowrank + rt.e * g.lr_stride + g.l2_off + ((size_t)half * NO + o0) * rp * 2,
                                 (uint32_t)(wrows * rp * 2));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int c = chan_row(16 * (wave + NW * i) + (lane >> 2));
      load_lds16(rl, base + 1024 * (wave + NW * i), c < wrows ? c * rp * 2 + 16 * cpk : kOutOfRange, 64 * t);
    }
    const i32x4 rt_ = buffer_rsrc(g.T + (size_t)rt.row0 * tw, (uint32_t)(rt.rows * tw * 2));
    for (int part = 0; part < g.tparts; ++part)
#pragma unroll
      for (int i = 0; i < TL; ++i) {
        const int r = 16 * (wave + NW * i) + (lane >> 2);
        load_lds16(rt_, base + PPL + part * TPL + 1024 * (wave + NW * i),
                   r < rt.rows ? r * tw * 2 + 16 * cpk : kOutOfRange, 64 * t + part * rp * 2);
      }
  };
  // four consecutive fp32 of a per-channel vector, from output channel c in half h (clamped at its end)
  auto load4 = [&](const float* p, int h, int c) -> f32x4 {
    const float* q = p + wrow0 + (size_t)h * NO;
    if (c + 3 < NO) return *reinterpret_cast<const f32x4u*>(q + c);
    return f32x4{q[min(c, NO - 1)], q[min(c + 1, NO - 1)], q[min(c + 2, NO - 1)], q[min(c + 3, NO - 1)]};
  };
  stage_barrier();  // every wave is done with the rings
  if (rp > 0) {
    issue_panel(0);
    if (rp > 32) issue_panel(1);
  }
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
  // y[channel][row] += sum_t L2^T[channel][t] T[row][t] on the bf16 MFMA, 16 t
  // per step, the small parts of T first
  for (int t = 0; t < rp / 32; ++t) {
    wait_vmcnt<0>();
    stage_barrier();  // panels up to t + 1 are there
    const uint8_t* pl = smem + (t & 1) * PANEL + ra * 64;
    const uint8_t* pt = smem + (t & 1) * PANEL + PPL + rb * 64;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 la[FM];
#pragma unroll
      for (int a = 0; a < FM; ++a) la[a] = *reinterpret_cast<const uint4*>(pl + 2048 * a + 16 * ((2 * s + lg) ^ psw(ra)));
      for (int part = g.tparts - 1; part >= 0; --part) {
        uint4 tb[FN];
#pragma unroll
        for (int b = 0; b < FN; ++b)
          tb[b] = *reinterpret_cast<const uint4*>(pt + part * TPL + 2048 * b + 16 * ((2 * s + lg) ^ psw(rb)));
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
          for (int b = 0; b < FN; ++b)
            y[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(la[a]), as_bf16x8(tb[b]), y[a][b], 0, 0, 0);
      }
    }
    if (t + 2 < rp / 32) {
      stage_barrier();  // every wave is done with panel t
      issue_panel(t + 2);
    }
  }

  // bf16 Y is staged per wave in LDS (WN rows of OW channels, chunk j of row r
  // swizzled, and the 8-byte halves of a chunk swapped where bit 4 of r is
  // set, so that the 32 rows a store touches fall on distinct banks) and
  // leaves as whole 64- or 128-byte row pieces; fp32 Y is stored directly.
  stage_barrier();  // every wave is done with the panels
  uint8_t* sY = smem + wave * (WN * OW * 2);
  auto ychunk = [&](int row, int j) { return row * (OW * 2) + 16 * (GATED ? j ^ ((row >> 2) & 3) : j ^ ((row >> 1) & 7)); };
  constexpr int LPR = OW / 8, RPI = 64 / LPR;  // lanes per row piece, rows per 64 lanes
  // A bf16 residual comes the same way, as whole row pieces into the places
  // that Y takes (without the swap of halves), 8 bytes of it are read there
  // just before Y's replace them, by the same lanes.  (The same 8 bytes of 32
  // rows per load, straight from memory: 13 us of 80 at 4096 x 4096 x 4096.)
  // Direct loads want 4-byte addresses, so odd channel counts and fp32
  // residuals are read from memory.
  const bool has_res = !EX && g.res;
  const bool res_lds = has_res && g.res_bf16 && g.y_bf16 && (NO & 1) == 0 && (int64_t)BN * NO < (1 << 29);
  if (res_lds) {
    const i32x4 rr = buffer_rsrc((const bf16_t*)g.res + (size_t)rt.row0 * NO, (uint32_t)(rt.rows * NO * 2));
    const uint32_t at = lds0 + wave * (WN * OW * 2);
#pragma unroll
    for (int r0 = 0; r0 < WN; r0 += RPI) {
      const int r = r0 + lane / LPR, row = wn * WN + r;
      const int j = GATED ? (lane % LPR) ^ ((r >> 2) & 3) : (lane % LPR) ^ ((r >> 1) & 7);
      const int c = ow + 8 * j;
      load_lds16(rr, at + r0 * (OW * 2), row < rt.rows && c < NO ? (row * NO + c) * 2 : kOutOfRange, 0);
    }
    wait_vmcnt<0>();
    asm volatile("" ::: "memory");
  }
  // Four values of group (a, e4) and row block b, from the activation on:
  // bias, activation, the other half.
  auto value4 = [&](int a, int e4, int b, const f32x4& b0, const f32x4& b1, auto act, float (&v)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = y[a][b][4 * e4 + q];
    if (g.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += b0[q];
    }
    activate4(v, act);
    if (GATED) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= g.bias ? y[1][b][4 * e4 + q] + b1[q] : y[1][b][4 * e4 + q];
    }
  };
  auto stage4 = [&](int a, int e4, int b, const float (&v)[4]) {
    const int r = 32 * b + l32;
    *reinterpret_cast<uint2*>(sY + ychunk(r, 4 * a + e4) + 8 * (lg ^ ((r >> 4) & 1))) =
        uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  };
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
  // bf16 Y of a tile whose channels all exist: one straight run of code per
  // activation (the general path's branches, unrolled over the tile, span more
  // code than the instruction cache holds)
  auto finish = [&](auto act) {
#pragma unroll
    for (int a = 0; a < (GATED ? 1 : FM); ++a)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4 b0 = g.bias ? load4(g.bias, 0, oc(a, e4)) : zero4;
        const f32x4 b1 = GATED && g.bias ? load4(g.bias, 1, oc(a, e4)) : zero4;
        float v[FN][4];
#pragma unroll
        for (int b = 0; b < FN; ++b) value4(a, e4, b, b0, b1, act, v[b]);
        if (res_lds) {
#pragma unroll
          for (int b = 0; b < FN; ++b) {
            const uint2 w = *reinterpret_cast<const uint2*>(sY + ychunk(32 * b + l32, 4 * a + e4) + 8 * lg);
            v[b][0] += bf16_lo(w.x); v[b][1] += bf16_hi(w.x); v[b][2] += bf16_lo(w.y); v[b][3] += bf16_hi(w.y);
          }
          // both halves of the chunks have been read before Y's are written
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
#pragma unroll
        for (int b = 0; b < FN; ++b) stage4(a, e4, b, v[b]);
      }
  };
  const bool straight = g.y_bf16 && o0 + OC <= NO && (!has_res || res_lds);
  if (straight) {
    switch (g.act) {
      case ACT_RELU: finish(std::integral_constant<int, ACT_RELU>{}); break;
      case ACT_SILU: finish(std::integral_constant<int, ACT_SILU>{}); break;
      case ACT_GELU: finish(std::integral_constant<int, ACT_GELU>{}); break;
      case ACT_GELU_TANH: finish(std::integral_constant<int, ACT_GELU_TANH>{}); break;
      default: finish(std::integral_constant<int, ACT_NONE>{}); break;
    }
  } else {
#pragma unroll
    for (int a = 0; a < (GATED ? 1 : FM); ++a)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const int c = oc(a, e4);
        const f32x4 b0 = g.bias ? load4(g.bias, 0, c) : zero4;
        const f32x4 b1 = GATED && g.bias ? load4(g.bias, 1, c) : zero4;
#pragma unroll
        for (int b = 0; b < FN; ++b) {
          const int row = lrow(b);
          float v[4];
          value4(a, e4, b, b0, b1, g.act, v);
          const size_t o = ((size_t)rt.row0 + row) * NO + c;
          const int nc = row < rt.rows ? min(4, NO - c) : 0;  // values of this lane that exist
          if (res_lds) {
            const uint2 w = *reinterpret_cast<const uint2*>(sY + ychunk(32 * b + l32, 4 * a + e4) + 8 * lg);
            v[0] += bf16_lo(w.x); v[1] += bf16_hi(w.x); v[2] += bf16_lo(w.y); v[3] += bf16_hi(w.y);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          } else if (has_res && !g.res_bf16 && nc == 4) {
            const f32x4 w = *reinterpret_cast<const f32x4u*>((const float*)g.res + o);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += w[q];
          } else if (has_res) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q < nc) v[q] += g.res_bf16 ? bf16_to_f32(((const bf16_t*)g.res)[o + q]) : ((const float*)g.res)[o + q];
          }
          if (g.y_bf16) {
            stage4(a, e4, b, v);
          } else if (nc == 4) {
            *reinterpret_cast<f32x4u*>((float*)g.Y + o) = f32x4u{v[0], v[1], v[2], v[3]};
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q < nc) ((float*)g.Y)[o + q] = v[q];
          }
        }
      }
  }
  if (g.y_bf16) {
    // 16 bytes per lane; a wave reads only its own staging area
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_wave_barrier();
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

template <int BM, int BN, int NW, bool GATED, bool EX>
hipError_t tile_t(const ActArgs& a, hipStream_t st) {
  constexpr int OC = GATED ? BM / 2 : BM;
  const int64_t no = GATED ? a.N / 2 : a.N;
  const int64_t blocks = (no + OC - 1) / OC * (EX ? max_expert_tiles(a.M, a.seg.E, BN) : (a.M + BN - 1) / BN);
  if (blocks <= 0 || blocks > INT32_MAX || 256 * a.ldb >= ((int64_t)1 << 31) || 256 * a.lda >= ((int64_t)1 << 31))
    return hipErrorInvalidValue;
  if (a.Kb % 128 == 0)
    launch_kernel(k_tile_act<BM, BN, NW, GATED, EX, true>, dim3((unsigned)blocks), dim3(64 * NW), 0, st, a);
  else
    launch_kernel(k_tile_act<BM, BN, NW, GATED, EX, false>, dim3((unsigned)blocks), dim3(64 * NW), 0, st, a);
  return hipGetLastError();
}

template <bool GATED>
hipError_t tile_one(const ActArgs& a, hipStream_t st) {
  constexpr int OC = GATED ? 128 : 256;
  const int64_t no = GATED ? a.N / 2 : a.N, cols = (no + OC - 1) / OC;
  // three quarters of the compute units must have a tile: else half as many
  // rows, then small tiles, two blocks per unit.  d = 4096, gated, 256- against
  // 128-row tiles: 512 tokens x 12288 (192 tiles of 256) 59.6 and 69.1 us;
  // 2048 x 4096 ungated (128 tiles) 55.7 and 39.1.  128-row against small tiles:
  // 256 x 14336 (224 tiles) 37.0 and 47.7; 1024 x 4096 ungated (128) 33.1 and
  // 25.8; 128 x 14336 (112) 50.6 and 25.8.
  if (cols * ((a.M + 255) / 256) >= 192) return tile_t<256, 256, 8, GATED, false>(a, st);
  if (cols * ((a.M + 127) / 128) >= 192) return tile_t<256, 128, 8, GATED, false>(a, st);
  return tile_t<128, 64, 4, GATED, false>(a, st);
}

template <bool GATED>
hipError_t tile_experts(const ActArgs& a, hipStream_t st) {
  switch (tile_act_rows(a.M, a.seg.E)) {
    case 256: return tile_t<256, 256, 8, GATED, true>(a, st);
    case 128: return tile_t<256, 128, 8, GATED, true>(a, st);
    default: return tile_t<128, 64, 4, GATED, true>(a, st);
  }
}

}  // namespace

// By the average rows of an expert: a tile of twice as many rows would be half
// empty more often than not, and one of half as many reads the weights twice.
// 8 experts, 4096 -> 14336 gated: 125 rows each, 221 us with 64-row tiles and
// 208 with 128; 250 rows, 310 with 128 and 323 with 256; 500 rows, 536 with 128
// and 506 with 256; 1024 rows, 1013 and 901.  128 experts, 2048 -> 768 gated:
// 128 rows, 120 us with 64 and 108 with 128.
int tile_act_rows(int64_t M, int64_t E) {
  const int64_t avg = M / E;
  return avg > 384 ? 256 : (avg > 96 ? 128 : 64);
}

hipError_t launch_tile_act(const ActArgs& a, bool gated, bool experts, hipStream_t st) {
  if (experts) return gated ? tile_experts<true>(a, st) : tile_experts<false>(a, st);
  return gated ? tile_one<true>(a, st) : tile_one<false>(a, st);
}

}  // namespace tq
