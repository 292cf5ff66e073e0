// Kernels around the experts' products (gfx950): the routing plan (pairs
// sorted by expert), the first low-rank stage of the sorted rows and the
// weighted combination of the experts' outputs.

#include <type_traits>

#include "tq_act.h"

namespace tq {
namespace {

// ---------------------------------------------------------------------------
// Routing plan: a stable counting sort of P = n topk pairs by expert id.
//   offsets[e] = number of kept pairs with an expert below e, and a pair's
//   position = offsets[its expert] + its rank among the pairs of that expert
//   in pair order.  Pairs whose id lies outside 0 .. E - 1 are dropped.
// Ranks come from counts alone, never from the order in which atomics land,
// so the plan is the same on every run.  A wave ranks 64 consecutive pairs by
// ballots over the id's bits (lanes with an equal id); its counts per expert
// in LDS carry the rank across its rounds, and sums over the waves in wave
// order carry it across the block.
// A block of 16 waves takes 2048 to 16384 pairs.  Up to kPlanOne pairs the
// whole plan is one block and one launch; more take two launches: the blocks'
// histograms, then each block sums the histograms of the blocks before it.
// Bound by latency: 16 tokens x 8 of 128 experts 7.4 us a call, 32768 x 8 of
// 256 11.4 us for 4.2 MB.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
// one block against two launches: 4096 pairs of 128 experts 6.8 and 7.3 us, 8192 pairs 11.3 and 7.6
constexpr int kPlanOne = 4096;
// Pairs per block beyond that.  A wave ranks its pairs one round after the
// other, so few per block are fastest until every block's reading of all
// blocks' histograms weighs more (2048, 4096 and 16384 pairs per block, 256
// experts: 2^18 pairs 11.8, 14.4 and 28.3 us; 2^19 16.1, 18.1 and 29.8; 2^20
// 37, 26 and 33; 2^22 364, 131 and 49; 2^24 5131, 1593 and 243).
constexpr int plan_rounds(int64_t P) { return P <= (1 << 19) ? 2 : (P <= (1 << 20) ? 4 : 16); }
constexpr int plan_chunk(int64_t P) { return plan_rounds(P) * kPlanThreads; }

// id of pair i as an expert index, or E when dropped
template <typename I>
__device__ __forceinline__ int plan_id(const I* ids, int64_t i, int64_t P, int E) {
  if (i >= P) return E;
  const I v = ids[i];
  return (v >= 0 && v < (I)E) ? (int)v : E;
}

// lanes of the wave with the same id (0 .. E) as this lane
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool on = (id >> b) & 1;
    const uint64_t s = __ballot(on);
    m &= on ? s : ~s;
  }
  return m;
}

// orders a wave's LDS accesses on either side, across its lanes
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename I>
__global__ __launch_bounds__(kPlanThreads) void k_plan_hist(const I* ids, int64_t P, int E, int chunk, int32_t* hist) {
  __shared__ int cnt[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= E; e += kPlanThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * chunk;
  for (int j = threadIdx.x; j < chunk; j += kPlanThreads) atomicAdd(&cnt[plan_id(ids, i0 + j, P, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlanThreads) hist[(size_t)blockIdx.x * E + e] = cnt[e];
}

// ONE: the whole plan in one block.  R: rounds of 64 pairs per wave, whose ids
// (requested at once) and matching lanes stay in registers between the two passes.
template <typename I, bool ONE, int R>
__global__ __launch_bounds__(kPlanThreads) void k_plan(const I* ids, int64_t P, int E, int bits, const int32_t* hist,
                                                       int32_t* offsets, int32_t* order, int32_t* pos) {
  extern __shared__ int cnt[];  // [waves][E + 1]: counts, then next positions
  __shared__ int wsum[kPlanWaves];
  __shared__ int part[2][kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int stride = E + 1;
  // this wave's consecutive pairs
  const int64_t b0 = ONE ? 0 : (int64_t)blockIdx.x * (R * kPlanThreads);
  const int64_t iend = ONE ? P : min(P, b0 + R * kPlanThreads);
  const int64_t i0 = b0 + (int64_t)w * R * 64 + lane;
  int id[R];
#pragma unroll
  for (int r = 0; r < R; ++r) id[r] = plan_id(ids, i0 + 64 * r, iend, E);
  // the blocks' histograms: thread (e, g) sums every G-th block's count of expert e, all and before this block
  const int Er = (E + 63) & ~63, G = kPlanThreads / Er, g = tid / Er, eg = tid % Er;
  if (!ONE) {
    int total = 0, before = 0;
    if (g < G && eg < E) {
#pragma unroll 16
      for (int b = g; b < (int)gridDim.x; b += G) {
        const int h = hist[(size_t)b * E + eg];
        total += h;
        before += b < (int)blockIdx.x ? h : 0;
      }
    }
    part[0][tid] = total;
    part[1][tid] = before;
  }
  for (int i = tid; i < kPlanWaves * stride; i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  int* my = cnt + w * stride;
  uint64_t m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = same_id(id[r], bits);
    if ((m[r] & ((1ull << lane) - 1)) == 0) my[id[r]] += __popcll(m[r]);  // one lane per id
    wave_sync();
  }
  __syncthreads();
  // thread e: expert e's pairs in this block's waves, in all blocks, and before this block
  int total = 0, before = 0;
  if (tid < E) {
    if (ONE) {
      for (int v = 0; v < kPlanWaves; ++v) total += cnt[v * stride + tid];
    } else {
      for (int v = 0; v < G; ++v) {
        total += part[0][v * Er + tid];
        before += part[1][v * Er + tid];
      }
    }
  }
  int inc = total;  // inclusive sum over the experts: in the wave, then across the waves
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 63) wsum[w] = inc;
  __syncthreads();
  for (int v = 0; v < w; ++v) inc += wsum[v];
  if (tid < E) {
    if (blockIdx.x == 0) {
      if (tid == 0) offsets[0] = 0;
      offsets[tid + 1] = inc;
    }
    int next = inc - total + before;
    for (int v = 0; v < kPlanWaves; ++v) {
      const int c = cnt[v * stride + tid];
      cnt[v * stride + tid] = next;
      next += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = i0 + 64 * r;
    const uint64_t below = m[r] & ((1ull << lane) - 1);
    const int at = my[id[r]] + __popcll(below);
    wave_sync();
    if (below == 0) my[id[r]] = at + __popcll(m[r]);
    wave_sync();
    if (i < iend) {
      pos[i] = id[r] < E ? at : -1;
      if (id[r] < E) order[at] = (int32_t)i;
    }
  }
}

// The table of row tiles of TM rows: map[0].x = their number, map[1 + t] =
// {expert, first row, rows, 0}.  One block of 256 threads; lds: kMaxExperts + 5 words.
__device__ __forceinline__ void write_tile_map(const Segments& s, int TM, int4* map, int* lds) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int* wsum = lds + kMaxExperts + 1;
  int base = 0;
  if (tid == 0) lds[0] = 0;
  for (int e0 = 0; e0 < s.E; e0 += 256) {  // lds[e] = tiles of the experts below e
    const int e = e0 + tid;
    int n = 0;
    if (e < s.E) {
      const int a = min(max(s.offsets[e], 0), s.P), b = min(max(s.offsets[e + 1], a), s.P);
      n = (b - a + TM - 1) / TM;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(n, d);
      if (lane >= d) n += y;
    }
    if (lane == 63) wsum[w] = n;
    __syncthreads();
    for (int v = 0; v < w; ++v) n += wsum[v];
    if (e < s.E) lds[e + 1] = base + n;
    base += wsum[0] + wsum[1] + wsum[2] + wsum[3];
    __syncthreads();
  }
  const int total = min(base, (int)max_expert_tiles(s.P, s.E, TM));  // the table's size, whatever the offsets
  if (tid == 0) map[0] = int4{total, 0, 0, 0};
  for (int t = tid; t < total; t += 256) {
    int lo = 0, hi = s.E - 1;  // the last expert with lds[e] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (lds[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int a = min(max(s.offsets[lo], 0), s.P), b = min(max(s.offsets[lo + 1], a), s.P);
    const int row0 = a + (t - lds[lo]) * TM;
    map[1 + t] = int4{lo, row0, min(TM, b - row0), 0};
  }
}

// ---------------------------------------------------------------------------
// Prologue of the experts' layers, one launch of three kinds of blocks:
//  * block 0: the table of row tiles -- how many there are, then expert,
//    first row and row count of each -- so that the product's blocks find
//    their rows with one load;
//  * then T[p] = X[token(p)] L1_e for 16 RT rows of one expert, QS 16-column
//    slices and one k-chunk, on v_mfma_f32_16x16x32_bf16 (lane l: row or
//    column l % 16, the 8 k at 8 (l / 16)).  The four waves take pairs
//    of 32-k steps round-robin, U steps in flight; their partials are summed
//    through LDS in wave order, 32 columns at a time;
//  * the rest: codes and s_x of four tokens, one per wave (int8 order for the
//    tile product, PK: nibble-packed for the rows product); a token is
//    quantised once, whatever the number of its experts.  These blocks are
//    short and fill the units beside the T blocks.
// Few rows per expert (PK, RT = 1): L1_e is what is read (r_pad d values per
// tile), so k is split over blocks and the partials are summed by the product
// kernel.  Many rows (RT = 2 or 4): 32 or 64 rows share each read of L1_e and
// T leaves as bf16 parts, summed by the last block of a tile where k is split.
// Bound by the vector cache: a fragment load takes 64 bytes from each of 16
// rows, about 5.5 TB/s over all units whatever is in flight.  4096 tokens x 2
// of 8 experts, d = 4096, r = 64: 40 us; 4 tokens of them 6 us.
// ---------------------------------------------------------------------------
template <typename XT, int CH, int RT, int QS, bool PK>
__global__ __launch_bounds__(256) void k_expert_prologue(ExpertPrologue a) {
  constexpr int U = 2, COLS = 16 * QS;
  __shared__ __attribute__((aligned(16))) float sP[4][16 * RT][33];
  static_assert(sizeof(sP) >= 4 * (kMaxExperts + 5), "the table's scratch");
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const Segments& s = a.seg;
  const ExpertTPlan& pl = a.t;
  const int d = a.d;
  int b = blockIdx.x;
  if (b == 0) {
    write_tile_map(s, a.map_rows, a.map, reinterpret_cast<int*>(sP));
    return;
  }
  --b;
  const int ntb = a.r_pad ? pl.tiles * pl.nchunk * pl.ncg : 0;
  if (b >= ntb) {
    const int row = 4 * (b - ntb) + w;
    if (row >= s.ntok) return;
    const float sx = quant_row_i8_wave<XT, CH, PK>((const XT*)a.X + (size_t)row * d, d >> 3, lane,
                                                   a.xc + (size_t)row * (PK ? d >> 1 : d), nullptr);
    if (lane == 0) a.sx[row] = sx;
    return;
  }
  const int lr = lane & 15, lg = lane >> 4;
  const int cg = b % pl.ncg;
  b /= pl.ncg;
  const int c = b % pl.nchunk, t = b / pl.nchunk;
  const RowTile rt = expert_tile<16 * RT>(s, t);
  if (rt.rows == 0) return;
  const XT* xr[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    xr[i] = (const XT*)a.X + (size_t)row_token(s, rt.row0 + min(16 * i + lr, rt.rows - 1)) * d + 8 * lg;
  const bf16_t* lp =
      reinterpret_cast<const bf16_t*>(a.lowrank + rt.e * a.lr_stride) + (size_t)(COLS * cg + lr) * d + 8 * lg;
  const int s0 = c * pl.ksteps, s1 = min(d >> 5, s0 + pl.ksteps);

  f32x4 acc[RT][QS];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int q = 0; q < QS; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a wave takes pairs of steps (128 bytes of each row: whole lines); the next
  // pairs are requested before the MFMAs of these
  uint4 xa[2][U][RT], lb[2][U][QS];
  auto load = [&](int sb, uint4 (&x)[U][RT], uint4 (&l)[U][QS]) {
    auto k_of = [&](int u) { return 32 * min(sb + 8 * (u >> 1) + (u & 1), s1 - 1); };  // clamped: masked below
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        Load8<XT>::load(xr[i] + k_of(u), v, x[u][i]);
      }
#pragma unroll
    for (int q = 0; q < QS; ++q)
#pragma unroll
      for (int u = 0; u < U; ++u) l[u][q] = *reinterpret_cast<const uint4*>(lp + (size_t)16 * q * d + k_of(u));
  };
  auto mma = [&](int sb, const uint4 (&x)[U][RT], const uint4 (&l)[U][QS]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (sb + 8 * (u >> 1) + (u & 1) < s1) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < QS; ++q)
            acc[i][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x[u][i]), as_bf16x8(l[u][q]), acc[i][q], 0, 0, 0);
      }
  };
  const int sb0 = s0 + 2 * w;
  if (sb0 < s1) load(sb0, xa[0], lb[0]);
  for (int sb = sb0; sb < s1; sb += 8 * U) {
    if (sb + 4 * U < s1) load(sb + 4 * U, xa[1], lb[1]);
    mma(sb, xa[0], lb[0]);
    if (sb + 8 * U < s1) load(sb + 8 * U, xa[0], lb[0]);
    if (sb + 4 * U < s1) mma(sb + 4 * U, xa[1], lb[1]);
  }
#pragma unroll
  for (int q0 = 0; q0 < QS; q0 += 2) {
    if (q0 > 0) __syncthreads();
    // 16x16 result layout: lane l, element i -> row 4 (l / 16) + i, column l % 16
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sP[w][16 * i + 4 * lg + e][16 * q + lr] = acc[i][q0 + q][e];
    __syncthreads();
    for (int e = tid; e < rt.rows * 32; e += 256) {
      const int rr = e >> 5, cc = e & 31;
      const float v = sP[0][rr][cc] + sP[1][rr][cc] + sP[2][rr][cc] + sP[3][rr][cc];
      const size_t p = (size_t)rt.row0 + rr;
      const int col = COLS * cg + 16 * q0 + cc;
      if (PK)
        a.Tp[((size_t)c * s.P + p) * a.r_pad + col] = v;
      else if (pl.nchunk == 1)
        store_t(a.T, p, a.r_pad, a.tparts, col, v);
      else  // at the device's point of coherence, for the block that sums
        __hip_atomic_store(&a.Tp[((size_t)c * s.P + p) * a.r_pad + col], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (PK || pl.nchunk == 1) return;
  // the last chunk's block of a tile and column group sums the partials in
  // chunk order (every block's stores complete before it counts itself)
  __shared__ int s_last;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  unsigned* ctr = a.counters + t * pl.ncg + cg;
  if (tid == 0)
    s_last = __hip_atomic_fetch_add(ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)pl.nchunk - 1;
  __syncthreads();
  if (!s_last) return;
  for (int e = tid; e < rt.rows * COLS; e += 256) {
    const int rr = e / COLS, col = COLS * cg + e % COLS;
    const size_t p = (size_t)rt.row0 + rr, stride = (size_t)s.P * a.r_pad;
    const float* pp = a.Tp + p * a.r_pad + col;
    float sum = 0.0f;
    for (int k0 = 0; k0 < pl.nchunk; k0 += 8) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = __hip_atomic_load(pp + min(k0 + k, pl.nchunk - 1) * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < pl.nchunk) sum += x[k];
    }
    store_t(a.T, p, a.r_pad, a.tparts, col, sum);
  }
  if (tid == 0) __hip_atomic_store(ctr, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// Combination: Y[t] = residual[t] + sum_j w[t][j] Z[pos[t][j]], fp32 in order
// of j and one rounding.  Dropped pairs (pos outside 0 .. P - 1) add nothing,
// whatever their weight or the rows of Z hold.  Bound by reading Z: VEC
// columns (16 bytes of bf16) per thread and up to 8 rows in flight; the
// token's positions and weights are the same for the whole block.  4095 tokens
// x 8 of a prefill batch in bf16, 322 MB: 65 us, 4.9 TB/s, the rate of a copy.
// ---------------------------------------------------------------------------
constexpr int kCombineTokens = 1 << 20;  // per grid layer: a launch takes fewer than 2^32 threads along x
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    uint4 raw;
    Load8<T>::load(p, v, raw);
  } else if constexpr (sizeof(T) == 2) {
    v[0] = bf16_to_f32(*p);
  } else {
    v[0] = *p;
  }
}

template <typename ZT, typename WT, int VEC>
__global__ __launch_bounds__(256) void k_combine(const ZT* __restrict__ Z, int n, int topk, int m, int P,
                                                 const int32_t* __restrict__ pos, const WT* __restrict__ wt,
                                                 const void* res, int res_bf16, void* Y, int y_bf16) {
  const int t = blockIdx.z * kCombineTokens + blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * VEC;
  if (c >= m || t >= n) return;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  const size_t o = (size_t)t * m + c;
  if (res) {
    if (res_bf16)
      load_vec<bf16_t, VEC>((const bf16_t*)res + o, acc);
    else
      load_vec<float, VEC>((const float*)res + o, acc);
  }
  constexpr int J = 8;
  for (int j0 = 0; j0 < topk; j0 += J) {
    float z[J][VEC], w[J];
    bool on[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int jj = min(j0 + j, topk - 1);
      const int p = pos[(size_t)t * topk + jj];
      on[j] = j0 + j < topk && p >= 0 && p < P;
      float wv[1];
      load_vec<WT, 1>(wt + (size_t)t * topk + jj, wv);
      w[j] = wv[0];
      if (on[j]) load_vec<ZT, VEC>(Z + (size_t)p * m + c, z[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (on[j]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = __builtin_fmaf(w[j], z[j][i], acc[i]);
      }
  }
  if (y_bf16) {
    bf16_t* y = (bf16_t*)Y + o;
    if constexpr (VEC == 8)
      *reinterpret_cast<uint4*>(y) = uint4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                           pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])};
    else
      *y = (bf16_t)(pack_bf16x2(acc[0], acc[0]) & 0xFFFFu);
  } else {
    float* y = (float*)Y + o;
    if constexpr (VEC == 8) {
      reinterpret_cast<float4*>(y)[0] = float4{acc[0], acc[1], acc[2], acc[3]};
      reinterpret_cast<float4*>(y)[1] = float4{acc[4], acc[5], acc[6], acc[7]};
    } else {
      *y = acc[0];
    }
  }
}


template <typename I>
hipError_t plan_t(const I* ids, int64_t P, int E, int32_t* offsets, int32_t* order, int32_t* pos, void* ws,
                  hipStream_t st) {
  int bits = 1;
  while ((1 << bits) <= E) ++bits;  // ids 0 .. E
  const unsigned lds = (unsigned)(kPlanWaves * (E + 1) * 4);
  auto one = [&](auto rc) {
    launch_kernel(k_plan<I, true, decltype(rc)::value>, dim3(1), dim3(kPlanThreads), lds, st, ids, P, E, bits,
                  (const int32_t*)nullptr, offsets, order, pos);
    return hipGetLastError();
  };
  if (P <= kPlanThreads) return one(std::integral_constant<int, 1>{});
  if (P <= 2 * kPlanThreads) return one(std::integral_constant<int, 2>{});
  if (P <= kPlanOne) return one(std::integral_constant<int, kPlanOne / kPlanThreads>{});
  const int chunk = plan_chunk(P);
  const unsigned blocks = (unsigned)((P + chunk - 1) / chunk);
  launch_kernel(k_plan_hist<I>, dim3(blocks), dim3(kPlanThreads), 0, st, ids, P, E, chunk, (int32_t*)ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  auto many = [&](auto rc) {
    launch_kernel(k_plan<I, false, decltype(rc)::value>, dim3(blocks), dim3(kPlanThreads), lds, st, ids, P, E, bits,
                  (const int32_t*)ws, offsets, order, pos);
    return hipGetLastError();
  };
  switch (plan_rounds(P)) {
    case 2: return many(std::integral_constant<int, 2>{});
    case 4: return many(std::integral_constant<int, 4>{});
    default: return many(std::integral_constant<int, 16>{});
  }
}

template <typename XT, int CH, bool PK>
hipError_t prologue_t(const ExpertPrologue& a, hipStream_t st) {
  const int64_t blocks = 1 + (int64_t)a.nqb + (a.r_pad ? (int64_t)a.t.tiles * a.t.nchunk * a.t.ncg : 0);
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(256);
  if constexpr (PK) {
    if (a.t.qs == 4)
      launch_kernel(k_expert_prologue<XT, CH, 1, 4, PK>, grid, block, 0, st, a);
    else
      launch_kernel(k_expert_prologue<XT, CH, 1, 2, PK>, grid, block, 0, st, a);
  } else if (a.t.rt == 4) {
    if (a.t.qs == 4)
      launch_kernel(k_expert_prologue<XT, CH, 4, 4, PK>, grid, block, 0, st, a);
    else
      launch_kernel(k_expert_prologue<XT, CH, 4, 2, PK>, grid, block, 0, st, a);
  } else {
    if (a.t.qs == 4)
      launch_kernel(k_expert_prologue<XT, CH, 2, 4, PK>, grid, block, 0, st, a);
    else
      launch_kernel(k_expert_prologue<XT, CH, 2, 2, PK>, grid, block, 0, st, a);
  }
  return hipGetLastError();
}

// rows of up to 2048, 4096 or 16384 values in a wave's registers
template <typename XT, bool PK>
hipError_t prologue_d(const ExpertPrologue& a, hipStream_t st) {
  if (a.d <= 2048) return prologue_t<XT, 4, PK>(a, st);
  if (a.d <= 4096) return prologue_t<XT, 8, PK>(a, st);
  return prologue_t<XT, 32, PK>(a, st);
}

template <typename ZT, typename WT>
hipError_t combine_t(const void* Z, int n, int topk, int m, int P, const int32_t* pos, const void* w, const void* res,
                     bool res_bf16, void* Y, bool y_bf16, hipStream_t st) {
  const unsigned x = (unsigned)std::min(n, kCombineTokens), z = (unsigned)((n - 1) / kCombineTokens + 1);
  if (m % 8 == 0)
    launch_kernel(k_combine<ZT, WT, 8>, dim3(x, (unsigned)((m + 2047) / 2048), z), dim3(256), 0, st, (const ZT*)Z, n, topk,
                  m, P, pos, (const WT*)w, res, res_bf16 ? 1 : 0, Y, y_bf16 ? 1 : 0);
  else
    launch_kernel(k_combine<ZT, WT, 1>, dim3(x, (unsigned)((m + 255) / 256), z), dim3(256), 0, st, (const ZT*)Z, n, topk, m,
                  P, pos, (const WT*)w, res, res_bf16 ? 1 : 0, Y, y_bf16 ? 1 : 0);
  return hipGetLastError();
}

}  // namespace

// grows with P, so that a workspace for the most pairs serves fewer
size_t expert_plan_ws_bytes(int64_t P, int E) {
  if (P <= kPlanOne) return 0;
  const int64_t blocks = (P + plan_chunk(P) - 1) / plan_chunk(P);
  return (size_t)std::max<int64_t>(blocks, P > (1 << 19) ? 256 : 0) * (size_t)E * 4;
}

hipError_t launch_expert_plan(const void* ids, bool i64, int64_t P, int E, int32_t* offsets, int32_t* order,
                              int32_t* pos, void* ws, hipStream_t st) {
  return i64 ? plan_t((const int64_t*)ids, P, E, offsets, order, pos, ws, st)
             : plan_t((const int32_t*)ids, P, E, offsets, order, pos, ws, st);
}

ExpertTPlan plan_expert_t(int64_t P, int E, int d, int r_pad, bool partial) {
  ExpertTPlan p{};
  if (r_pad == 0) return p;
  const int nq = r_pad / 16, steps = d / 32;
  p.qs = std::min(nq, 4);
  p.ncg = nq / p.qs;
  // 64 rows per read of L1 where experts have that many (8192 rows over 8
  // experts of d = 4096, r = 64: 39 us against 48 with 32 rows), else 32
  p.rt = partial ? 1 : (P / E >= 48 ? 4 : 2);
  p.tiles = (int)max_expert_tiles(P, E, 16 * p.rt);
  // partial: chunks of 16 steps (512 k), at most 16 of them for the product
  // kernel to sum.  Otherwise k is split only where there are fewer blocks
  // than two per compute unit (64 tokens over 8 experts of d = 4096: 12 blocks
  // of all of k took 32 us), into chunks of at least 8 steps, one per wave and
  // batch of loads.
  const int blocks = std::max(1, p.tiles * p.ncg);
  p.nchunk = partial ? std::max(1, std::min((steps + 15) / 16, 16))
                     : (blocks >= 256 ? 1 : std::max(1, std::min((steps + 7) / 8, 512 / blocks)));
  p.ksteps = ((steps + p.nchunk - 1) / p.nchunk + 1) & ~1;  // whole pairs
  p.nchunk = (steps + p.ksteps - 1) / p.ksteps;
  return p;
}

hipError_t launch_expert_prologue(const ExpertPrologue& p, bool bf16, bool packed, hipStream_t st) {
  ExpertPrologue a = p;
  a.nqb = (a.seg.ntok + 3) / 4;
  if (a.d > 16384) {  // longer rows than a wave holds: a block per row
    a.nqb = 0;
    const hipError_t e = packed ? launch_quant_rows_fast(a.X, bf16, a.seg.ntok, a.d, a.d, 4, 4, a.xc, a.sx, nullptr, nullptr, st)
                                : launch_quant_rows_i8(a.X, bf16, a.seg.ntok, a.d, a.d, 4, a.xc, a.sx, nullptr, nullptr, st);
    if (e != hipSuccess) return e;
  }
  if (bf16) return packed ? prologue_d<bf16_t, true>(a, st) : prologue_d<bf16_t, false>(a, st);
  return packed ? prologue_d<float, true>(a, st) : prologue_d<float, false>(a, st);
}

hipError_t launch_expert_combine(const void* Z, bool z_bf16, int n, int topk, int m, int64_t P, const int32_t* pos,
                                 const void* w, bool w_bf16, const void* res, bool res_bf16, void* Y, bool y_bf16,
                                 hipStream_t st) {
  const int p = (int)P;
  if (z_bf16)
    return w_bf16 ? combine_t<bf16_t, bf16_t>(Z, n, topk, m, p, pos, w, res, res_bf16, Y, y_bf16, st)
                  : combine_t<bf16_t, float>(Z, n, topk, m, p, pos, w, res, res_bf16, Y, y_bf16, st);
  return w_bf16 ? combine_t<float, bf16_t>(Z, n, topk, m, p, pos, w, res, res_bf16, Y, y_bf16, st)
                : combine_t<float, float>(Z, n, topk, m, p, pos, w, res, res_bf16, Y, y_bf16, st);
}

}  // namespace tq
