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
//   of one row tile; its 4 waves split K into contiguous ranges of 64-byte
//   steps, U steps of every group in flight, and take each activation
//   fragment for all groups.  v_mfma_i32_16x16x64_i8 on codes expanded by
//   unpack16 (lane l: row or channel l % 16, code bytes 16 (l / 16) ..); the
//   waves' int32 sums meet exactly in LDS and wave g finishes group g, for
//   gated layers both halves, so the product of the halves needs no exchange.
//   A block's life is one chain of memory round trips (row tile; weights;
//   nothing else, because everything the epilogue reads is requested right
//   behind the first weights), and several blocks per unit cover each other.
//   Blocks of one channel group over the row tiles are 8 apart, on the same
//   XCD: an expert's weights come from HBM once, later tiles from its L2.
//   24 tokens x 6 of 64 experts of 1408 -> 2048, r = 32: 15.7 us, 66 MB of the
//   active experts' weights at 4.2 TB/s.  (Non-temporal weight loads were
//   slower, and so were deeper register prefetches: they spill or thrash L1.)
// ---------------------------------------------------------------------------
template <int GB, bool GATED, bool EX, int U>
__global__ __launch_bounds__(256, 4) void k_rows_act(ActArgs g) {
  constexpr int WAVES = 4, NT = 256;
  constexpr int H = GATED ? 2 : 1, NG = H * GB;  // halves, 16-channel weight groups
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
    const int4 e = g.map[1 + t];  // unspecified behind the last tile, inside the table
    if (t >= g.map[0].x) return;
    rt = RowTile{e.x, e.y, e.z};
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

  const int KS = (g.Kb + 63) / 64;
  const int per = (KS + WAVES - 1) / WAVES;
  const int sbeg = wave * per, send = min(KS, sbeg + per);
  // loads from clamped addresses (the row's last 16 bytes, so the offset from
  // this lane group's start is negative for rows shorter than a step), masked
  // where used
  const int kb_last = min((max(send, sbeg + 1) - 1) * 64, g.Kb - 16 - 16 * lg);
  uint4 bv[NG][U], av[U];
  const int arow = rt.row0 + min(l16, rt.rows - 1);
  auto load_w = [&](int s0) {
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int u = 0; u < U; ++u) bv[q][u] = *reinterpret_cast<const uint4*>(bp[q] + min((s0 + u) * 64, kb_last));
  };
  load_w(sbeg);
  const uint8_t* ap = g.A + (size_t)(EX ? row_token(g.seg, arow) : arow) * g.lda + 16 * lg;
  auto load_a = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u) av[u] = *reinterpret_cast<const uint4*>(ap + min((s0 + u) * 64, kb_last));
  };
  load_a(sbeg);

  // ---- what the epilogue reads, requested behind the first weights: scales
  // and bias of this wave's group, its first 64 ranks of L2, and the thread's
  // first piece (4 columns of a row) of the partials of T ----
  const int rp = g.r_pad, tw = g.tparts * rp, rq = rp >> 2;
  const int gw = min(wave, GB - 1);
  float sw[H], bias[H], sx[4];
  uint4 l2[H][2];
  const bf16_t* L2 = reinterpret_cast<const bf16_t*>(g.lowrank + rt.e * g.lr_stride + g.l2_off);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int ch = wrow(gw + h * GB, l16);
    sw[h] = g.sw[(size_t)rt.e * g.N + ch];
    bias[h] = g.bias ? g.bias[(size_t)rt.e * g.N + ch] : 0.0f;
    if (rp > 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        l2[h][i] = *reinterpret_cast<const uint4*>(L2 + (size_t)ch * rp + min(32 * i, rp - 32) + 8 * lg);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = rt.row0 + min(4 * lg + i, rt.rows - 1);
    sx[i] = g.sx[EX ? row_token(g.seg, p) : p];
  }
  constexpr int C = 4;  // partials in flight
  float4 tv = float4{0.f, 0.f, 0.f, 0.f};
  auto load_t = [&](int i) {  // piece i, summed in chunk order
    float4 v = float4{0.f, 0.f, 0.f, 0.f};
    if (i < rt.rows * rq) {
      const float* p = g.Tp + (size_t)(rt.row0 + i / rq) * rp + 4 * (i % rq);
      const size_t stride = (size_t)g.M * rp;
      for (int c0 = 0; c0 < g.nchunk; c0 += C) {
        float4 x[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
          x[c] = *reinterpret_cast<const float4*>(p + min(c0 + c, g.nchunk - 1) * stride);
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c0 + c < g.nchunk) {
            v.x += x[c].x; v.y += x[c].y; v.z += x[c].z; v.w += x[c].w;
          }
      }
    }
    return v;
  };

  // ---- integer product ----
  i32x4 acc[NG];
#pragma unroll
  for (int q = 0; q < NG; ++q) acc[q] = i32x4{0, 0, 0, 0};
  auto mma = [&](int s0) {
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
  };
  mma(sbeg);
  for (int s0 = sbeg + U; s0 < send; s0 += U) {
    load_w(s0);
    load_a(s0);
    mma(s0);
  }
#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][q][i][lane] = acc[q][i];

  // ---- T in bf16 parts (rows behind the tile's are zero) ----
  for (int i = tid; i < 16 * rq; i += NT) {
    tv = load_t(i);
    for (int part = 0; part < g.tparts; ++part) {
      const uint2 b = uint2{pack_bf16x2(tv.x, tv.y), pack_bf16x2(tv.z, tv.w)};
      *reinterpret_cast<uint2*>(sT + (i / rq) * tw + part * rp + 4 * (i % rq)) = b;
      tv = float4{tv.x - bf16_lo(b.x), tv.y - bf16_hi(b.x), tv.z - bf16_lo(b.y), tv.w - bf16_hi(b.y)};
    }
  }
  __syncthreads();
  if (wave >= GB) return;

  // ---- epilogue of group `wave`: lane l, element i -> row 4 (l / 16) + i, channel l % 16 ----
  const int oc = o0 + 16 * wave + l16;
  float v[H][4];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int q = wave + h * GB;
    f32x4 lr = {0.f, 0.f, 0.f, 0.f};
    auto lr_step = [&](int t0, const uint4& l) {
      for (int part = g.tparts - 1; part >= 0; --part) {
        const uint4 tv = *reinterpret_cast<const uint4*>(sT + l16 * tw + part * rp + t0 + 8 * lg);
        lr = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(tv), as_bf16x8(l), lr, 0, 0, 0);
      }
    };
    if (rp > 0) lr_step(0, l2[h][0]);
    if (rp > 32) lr_step(32, l2[h][1]);
    for (int t0 = 64; t0 < rp; t0 += 32)
      lr_step(t0, *reinterpret_cast<const uint4*>(L2 + (size_t)wrow(q, l16) * rp + t0 + 8 * lg));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s += red[w][q][i][lane];
      v[h][i] = (float)(s >> 8) * (sx[i] * sw[h]) + lr[i] + bias[h];
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
    if (GATED) y *= v[H - 1][i];
    if (g.res) y += g.res_bf16 ? bf16_to_f32(((const bf16_t*)g.res)[o]) : ((const float*)g.res)[o];
    if (g.y_bf16)
      ((bf16_t*)g.Y)[o] = (bf16_t)(pack_bf16x2(y, y) & 0xFFFFu);
    else
      ((float*)g.Y)[o] = y;
  }
}

// ---------------------------------------------------------------------------
// Stream kernel: the rows kernel's work for rows of d = 2048 .. 16384, as a
// stream that never drains.  One item is 16 GB output channels (gated: of each
// half) of one row tile; a block takes a contiguous range of the items.
//   * NS stream waves take 128-byte pieces of K in turn (neighbouring waves on
//     neighbouring lines).  A wave keeps the tile's activation codes of its
//     pieces in registers and streams the weights
//     through its own LDS ring by direct loads, R units (one piece of all the
//     item's rows, 8 rows of 128 contiguous bytes per load) ahead, across item
//     and tile boundaries; it waits for its own loads only.
//   * One loader wave brings what the epilogue reads per item -- rows of L2^T,
//     scales, bias -- into another ring by direct loads, D items ahead: with
//     the stream waves keeping the memory queues full a round trip takes
//     several microseconds, longer than an item.
//   * One epilogue wave sums the stream waves' int32 partials of the last
//     item, adds the low-rank term, applies the epilogue and stores, while
//     the next item streams.
// Per item two barriers: partials and item data are there; they have been read.
// Bound by HBM: 4 tokens x 2 of 8 experts of 4096 -> 14336 gated, r = 64, 5
// experts active: 54 us, 312 MB at 5.7 TB/s, the rate of a large read; without
// the loader wave about a tenth more.  One layer of that shape, one token, is
// 63 MB in 16.5 us, 3.8 TB/s: starting and draining the rings is a third of it.
// ---------------------------------------------------------------------------
constexpr int kPiece = 128;  // bytes of a weight row per unit
// chunk c (16 bytes) of LDS row r sits at slot c ^ (r / 2 modulo 8): a fragment
// read's 16 simultaneous lanes (rows 0-3 and 12-15 with one chunk, rows 4-11
// with its neighbour) then hit different banks
__device__ __forceinline__ int ssw(int r) { return (r >> 1) & 7; }
constexpr int kItemsAhead = 3;
// item data: NG groups of 16 rows of L2^T (2 rp bytes each), then NG x 16
// scales, then NG x 16 biases, each padded to 256 bytes
__host__ __device__ constexpr int item_bytes(int ng, int rp) { return ng * 32 * rp + 512; }

// wait until at most n (uniform, at most 2 (NG 8 + 2)) of the wave's loads are outstanding
template <int N>
__device__ __forceinline__ void wait_vmcnt_upto(int n) {
  if constexpr (N > 0) {
    if (n < N) return wait_vmcnt_upto<N - 1>(n);
  }
  wait_vmcnt<N>();
}
// load_lds16 with the non-temporal hint, for weights that one launch reads once
__device__ __forceinline__ void load_lds16_nt(i32x4 rsrc, uint32_t lds, int voff, int soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen nt lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0");
}
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ONCE: weights loaded with the non-temporal hint.
template <int NS, int PW, int GB, bool GATED, bool EX, int R, bool ONCE>
__global__ __launch_bounds__(64 * (NS + 2), NS == 4 ? 2 : 1) void k_stream_act(ActArgs g) {
  constexpr int H = GATED ? 2 : 1, NG = H * GB;
  constexpr int UNIT = NG * 16 * kPiece, LPU = 2 * NG;  // bytes and direct loads per unit
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  auto red = reinterpret_cast<int (*)[NG][4][64]>(smem + NS * R * UNIT);
  uint8_t* items = smem + NS * R * UNIT + NS * NG * 1024;
  const int rp = g.r_pad, IB = item_bytes(NG, rp);
  bf16_t* sT = reinterpret_cast<bf16_t*>(items + kItemsAhead * IB);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int NO = GATED ? g.N / 2 : g.N;
  const int ngi = (NO + 16 * GB - 1) / (16 * GB);  // items per row tile
  const int64_t total = (int64_t)(EX ? g.map[0].x : (g.M + 15) / 16) * ngi;
  const int64_t i0 = total * blockIdx.x / gridDim.x, i1 = total * (blockIdx.x + 1) / gridDim.x;
  if (i0 >= i1) return;
  const int n = (int)(i1 - i0);
  auto tile_of = [&](int t) {
    if (!EX) return RowTile{0, 16 * t, min(16, g.M - 16 * t)};
    const int4 e = g.map[1 + t];
    return RowTile{__builtin_amdgcn_readfirstlane(e.x), __builtin_amdgcn_readfirstlane(e.y),
                   __builtin_amdgcn_readfirstlane(e.z)};
  };
  auto lds_of = [&](const uint8_t* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
  };
  const int t_first = (int)(i0 / ngi), c_first = (int)(i0 % ngi);

  if (wave < NS) {
    // ---- stream wave: np pieces, every NS-th from its own number on ----
    const int KP = (g.Kb + kPiece - 1) / kPiece;
    const int np = max(0, (KP - wave + NS - 1) / NS);
    const int units = n * np;
    const uint8_t* ringp = smem + wave * R * UNIT;
    const uint32_t ring = lds_of(ringp);
    // load cursor: item (tile lt of expert le, channel group lc) and piece;
    // the expert is looked up only where the tile changes (that load waits
    // behind the ring's)
    int lt = t_first, lc = c_first, lp = 0, issued = 0;
    int le = tile_of(lt).e;
    i32x4 rsrc[H];
    int vo[2];  // rows 8 h + lane / 8 of a 16-row group; chunk lane % 8 of the LDS row
    auto set_item = [&]() {
      const int o0 = 16 * GB * lc, rows = min(16 * GB, NO - o0);
#pragma unroll
      for (int h = 0; h < H; ++h)
        rsrc[h] = buffer_rsrc(g.B + ((size_t)le * g.N + (size_t)h * NO + o0) * g.ldb, (uint32_t)(rows * g.ldb));
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + (lane >> 3);
      vo[h] = (int)(r * g.ldb) + 16 * ((lane & 7) ^ ssw(r));
    }
    auto issue = [&](int slot) {
      const int so = kPiece * (wave + NS * lp);
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 8 * h + (lane >> 3);
          const bool ok = so + 16 * ((lane & 7) ^ ssw(r)) < g.Kb;  // rows past the channels end past the resource
          const uint32_t at = ring + slot * UNIT + q * (16 * kPiece) + h * 1024;
          const int off = ok ? vo[h] + (int)(16 * (q % GB) * g.ldb) : kOutOfRange;
          if constexpr (ONCE)
            load_lds16_nt(rsrc[q / GB], at, off, so);
          else
            load_lds16(rsrc[q / GB], at, off, so);
        }
      ++issued;
      if (++lp == np) {
        lp = 0;
        if (++lc == ngi) {
          lc = 0;
          ++lt;
          if (issued < units) le = tile_of(lt).e;
        }
        if (issued < units) set_item();
      }
    };
    uint4 av[PW][2];  // activation codes of the wave's pieces: lane row l % 16, bytes 64 s + 16 (l / 16) of a piece
    auto load_a = [&](int t) {
      const RowTile rt = tile_of(t);
      const int row = rt.row0 + min(l16, rt.rows - 1);
      const uint8_t* ap = g.A + (size_t)(EX ? row_token(g.seg, row) : row) * g.lda;
#pragma unroll
      for (int p = 0; p < PW; ++p)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int k = kPiece * (wave + NS * p) + 64 * s + 16 * lg;
          av[p][s] = *reinterpret_cast<const uint4*>(ap + min(k, g.Kb - 16));
          if (p >= np || k >= g.Kb) av[p][s] = uint4{0, 0, 0, 0};
        }
    };
    load_a(t_first);
    set_item();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (issued < units) issue(r);
    int tile = t_first, c = c_first, done = 0, slot = 0;
    for (int it = 0; it < n; ++it) {
      i32x4 acc[NG];
#pragma unroll
      for (int q = 0; q < NG; ++q) acc[q] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < PW; ++p) {
        if (p < np) {
          if (units - done >= R)
            wait_vmcnt<(R - 1) * LPU>();
          else
            wait_vmcnt<0>();
          asm volatile("" ::: "memory");
          const uint8_t* u = ringp + slot * UNIT + l16 * kPiece;
          uint4 bv[2][NG];
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int q = 0; q < NG; ++q)
              bv[s][q] = *reinterpret_cast<const uint4*>(u + q * (16 * kPiece) + 16 * ((4 * s + lg) ^ ssw(l16)));
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before the slot is loaded again
          if (issued < units) issue(slot);
          slot = slot == R - 1 ? 0 : slot + 1;
          ++done;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const i32x4 a0 = unpack16(av[p][s].x, av[p][s].y), a1 = unpack16(av[p][s].z, av[p][s].w);
#pragma unroll
            for (int q = 0; q < NG; ++q) {
              acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, unpack16(bv[s][q].x, bv[s][q].y), acc[q], 0, 0, 0);
              acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, unpack16(bv[s][q].z, bv[s][q].w), acc[q], 0, 0, 0);
            }
          }
        }
      }
      if (it > 0) asm volatile("s_barrier" ::: "memory");  // the last item's partials have been read
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][q][i][lane] = acc[q][i];
      lds_barrier();
      if (++c == ngi) {
        c = 0;
        ++tile;
        if (it + 1 < n) load_a(tile);
      }
    }
    return;
  }

  if (wave == NS) {
    // ---- loader wave: item data, kItemsAhead items ahead ----
    const int pieces = rp >> 5;  // 1 KB pieces of a group's 16 rows of L2^T (32 rp bytes, contiguous)
    const int loads = NG * pieces + (g.bias ? 2 : 1);
    const uint32_t at = lds_of(items);
    int lt = t_first, lc = c_first, e = tile_of(lt).e;
    auto issue = [&](int i) {
      const uint32_t slot = at + (i % kItemsAhead) * IB;
      const int o0 = 16 * GB * lc;
      for (int h = 0; h < H; ++h) {
        const size_t ch = (size_t)h * NO + o0;  // first of the item's channels in this half
        const int rows = min(16 * GB, NO - o0);
        const i32x4 rl = buffer_rsrc(g.lowrank + e * g.lr_stride + g.l2_off + ch * rp * 2, (uint32_t)(rows * rp * 2));
        for (int p = 0; p < GB * pieces; ++p) load_lds16(rl, slot + (h * GB * pieces + p) * 1024, 1024 * p + 16 * lane, 0);
      }
      // lane 16 q + j: channel j of group q
      const int q = lane >> 4, o = o0 + 16 * (q % GB) + l16;
      const int off = q < NG && o < NO ? 4 * (int)((q / GB) * NO + o) : kOutOfRange;
      load_lds4(buffer_rsrc(g.sw + (size_t)e * g.N, (uint32_t)g.N * 4), slot + NG * 32 * rp, off);
      if (g.bias) load_lds4(buffer_rsrc(g.bias + (size_t)e * g.N, (uint32_t)g.N * 4), slot + NG * 32 * rp + 256, off);
      if (++lc == ngi) {
        lc = 0;
        ++lt;
        if (i + 1 < n) e = tile_of(lt).e;
      }
    };
    for (int i = 0; i < min(n, kItemsAhead); ++i) issue(i);
    for (int it = 0; it < n; ++it) {
      // item it has arrived: only later items' loads are outstanding
      wait_vmcnt_upto<(kItemsAhead - 1) * (NG * 8 + 2)>(min(kItemsAhead - 1, n - 1 - it) * loads);
      asm volatile("s_barrier" ::: "memory");
      if (it + 1 < n) asm volatile("s_barrier" ::: "memory");
      if (it + kItemsAhead < n) issue(it + kItemsAhead);
    }
    return;
  }

  // ---- epilogue wave: lane l, element i -> row 4 (l / 16) + i, channel l % 16 ----
  const int tw = g.tparts * rp, rq = rp >> 2;
  int tile = t_first, c = c_first;
  RowTile rt = RowTile{0, 0, 0};
  float sx[4];
  for (int it = 0; it < n; ++it) {
    if (it == 0 || c == 0) {  // a new tile: its scales, and T in bf16 parts (rows behind the tile's are zero)
      rt = tile_of(tile);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = rt.row0 + min(4 * lg + i, rt.rows - 1);
        sx[i] = g.sx[EX ? row_token(g.seg, p) : p];
      }
      for (int i = lane; i < 16 * rq; i += 64) {
        float4 v = float4{0.f, 0.f, 0.f, 0.f};
        if (i < rt.rows * rq) {
          const float* p = g.Tp + (size_t)(rt.row0 + i / rq) * rp + 4 * (i % rq);
          const size_t stride = (size_t)g.M * rp;
#pragma unroll 8
          for (int k = 0; k < g.nchunk; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(p + k * stride);
            v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
          }
        }
        for (int part = 0; part < g.tparts; ++part) {
          const uint2 b = uint2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
          *reinterpret_cast<uint2*>(sT + (i / rq) * tw + part * rp + 4 * (i % rq)) = b;
          v = float4{v.x - bf16_lo(b.x), v.y - bf16_hi(b.x), v.z - bf16_lo(b.y), v.w - bf16_hi(b.y)};
        }
      }
    }
    asm volatile("s_barrier" ::: "memory");  // the item's partials and data are there
    const uint8_t* item = items + (it % kItemsAhead) * IB;
    float v[NG][4];
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      const float sw = reinterpret_cast<const float*>(item + NG * 32 * rp)[16 * q + l16];
      const float bias = g.bias ? reinterpret_cast<const float*>(item + NG * 32 * rp + 256)[16 * q + l16] : 0.0f;
      f32x4 lr = {0.f, 0.f, 0.f, 0.f};
      for (int t0 = 0; t0 < rp; t0 += 32) {
        const uint4 l2 = *reinterpret_cast<const uint4*>(item + q * 32 * rp + l16 * 2 * rp + 2 * t0 + 16 * lg);
        for (int part = g.tparts - 1; part >= 0; --part) {
          const uint4 tv = *reinterpret_cast<const uint4*>(sT + l16 * tw + part * rp + t0 + 8 * lg);
          lr = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(tv), as_bf16x8(l2), lr, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < NS; ++w) s += red[w][q][i][lane];
        v[q][i] = (float)(s >> 8) * (sx[i] * sw) + lr[i] + bias;
      }
    }
    if (it + 1 < n) lds_barrier();  // read
#pragma unroll
    for (int b = 0; b < GB; ++b) {
      activate4(v[b], g.act);
      const int oc = 16 * GB * c + 16 * b + l16;
      if (oc < NO) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 4 * lg + i;
          if (row >= rt.rows) break;
          const size_t o = (size_t)(rt.row0 + row) * NO + oc;
          float y = v[b][i];
          if (GATED) y *= v[NG - GB + b][i];
          if (g.res) y += g.res_bf16 ? bf16_to_f32(((const bf16_t*)g.res)[o]) : ((const float*)g.res)[o];
          if (g.y_bf16)
            ((bf16_t*)g.Y)[o] = (bf16_t)(pack_bf16x2(y, y) & 0xFFFFu);
          else
            ((float*)g.Y)[o] = y;
        }
      }
    }
    if (++c == ngi) {
      c = 0;
      ++tile;
    }
  }
}

template <int NS, int GB, bool GATED, int R>
unsigned stream_lds(const ActArgs& a) {
  constexpr int NG = GATED ? 2 * GB : GB;
  return NS * R * NG * 16 * kPiece + NS * NG * 1024 + kItemsAhead * item_bytes(NG, a.r_pad) + 32 * a.tparts * a.r_pad;
}

template <int NS, int PW, int GB, bool GATED, bool EX, int R, bool ONCE>
hipError_t stream_t(const ActArgs& a, hipStream_t st) {
  const unsigned lds = stream_lds<NS, GB, GATED, R>(a);
  if (a.Kb > kPiece * NS * PW || lds > 160 * 1024) return hipErrorInvalidValue;
  const int64_t no = GATED ? a.N / 2 : a.N, ngi = (no + 16 * GB - 1) / (16 * GB);
  const int64_t items = ngi * (EX ? max_expert_tiles(a.M, a.seg.E, kRowsTile) : (a.M + 15) / 16);
  const unsigned blocks = (unsigned)std::min<int64_t>(items, NS == 4 ? 512 : 256);  // two or one per compute unit
  launch_kernel(k_stream_act<NS, PW, GB, GATED, EX, R, ONCE>, dim3(blocks), dim3(64 * (NS + 2)), lds, st, a);
  return hipGetLastError();
}

template <int GB, bool GATED, bool EX, int U>
hipError_t rows_t(const ActArgs& a, hipStream_t st) {
  const int64_t no = GATED ? a.N / 2 : a.N, ncb = (no + 16 * GB - 1) / (16 * GB);
  const int64_t tiles = EX ? max_expert_tiles(a.M, a.seg.E, kRowsTile) : (a.M + 15) / 16;
  const int64_t blocks = (ncb + 7) / 8 * 8 * tiles;
  if (blocks <= 0 || blocks > INT32_MAX) return hipErrorInvalidValue;
  launch_kernel(k_rows_act<GB, GATED, EX, U>, dim3((unsigned)blocks), dim3(256), (unsigned)(32 * a.tparts * a.r_pad), st, a);
  return hipGetLastError();
}

// The stream's weight loads are non-temporal where a launch reads the weights
// once: one row tile, and experts, most of which have one (without
// the hint and with it 67.7 and 59.5 us for the 5 experts of d = 4096, 129 and 116 for 32 tokens x 2 of 8, 57.6 and
// 49.6 for one layer of 8192 -> 28672 gated; one layer of 4096 -> 14336 gated,
// out of the last-level cache, 22.1 and 21.7).  Two row tiles find each
// other's weights in the caches: 29.0 us, with the hint 31.7.
template <bool GATED, bool EX, int NS, int PW>
hipError_t stream_e(const ActArgs& a, hipStream_t st) {
  constexpr int SGB = GATED ? 1 : 2;
  if constexpr (!EX) {
    if (a.M > kRowsTile) return stream_t<NS, PW, SGB, GATED, EX, 3, false>(a, st);
  }
  return stream_t<NS, PW, SGB, GATED, EX, 3, true>(a, st);
}

// The stream from d = 2048 on: below, an item is over before a round trip
// (64 experts of d = 1408, 24 tokens: 20 us against the rows kernel's 15.5;
// d = 2048 equal; 5 experts of d = 4096: 54 against 71; one layer of d =
// 14336, 8 tokens: 12.3 against 19.4), and up to 16384, whose codes a wave
// still holds in registers.
template <bool GATED, bool EX>
hipError_t rows_e(const ActArgs& a, hipStream_t st) {
  constexpr int SGB = GATED ? 1 : 2, RGB = GATED ? 2 : 4;
  if (a.Kb >= 1024 && a.Kb <= 2048) return stream_e<GATED, EX, 4, 4>(a, st);
  // (ranks above 128 leave no room for 8 waves' rings)
  if (a.Kb > 2048 && a.Kb <= 8192 && stream_lds<8, SGB, GATED, 3>(a) <= 160 * 1024)
    return stream_e<GATED, EX, 8, 8>(a, st);
  return rows_t<RGB, GATED, EX, 2>(a, st);
}

}  // namespace

hipError_t launch_rows_act(const ActArgs& a, bool gated, bool experts, hipStream_t st) {
  if (experts) return gated ? rows_e<true, true>(a, st) : rows_e<false, true>(a, st);
  return gated ? rows_e<true, false>(a, st) : rows_e<false, false>(a, st);
}

}  // namespace tq
