// Parameters shared by the kernels of the many-token paged attention.
#pragma once

#include "paged.cuh"

namespace echo {

struct PrefillParams {
  echo_paged_kv_t C;
  echo_paged_scales_t X;             // of a cache in 8 bits
  const void *q;
  int64_t q_stride;
  const int32_t *q_start, *seq_len;
  int N, B, Hq, G;
  FastDiv page, group;               // by page_tokens and by G
  const float *slopes;
  int window;
  const int32_t *first_tok, *prefix_len;
  ScoreForm f;
  void *out;
  float *lse;
  float *po, *pml;                   // partials [2 CTAs][rows][d], [2 CTAs][rows][2]
  int32_t *rec;                      // [CTAs][8]: the split row tile that ends in the CTA
  int prows;                         // rows of a partial
  int wide;                          // out is 32-byte aligned
  // SOME: sequences of no more packed rows than `above` are left out, and where *some is 0 there are no others
  int above;
  const int32_t *some;
};

// Rows of sequence b: [s0, s0 + n).
struct SeqRows {
  int s0, n;
};
__device__ __forceinline__ SeqRows seq_rows(const PrefillParams &P, int b) {
  SeqRows r;
  r.s0 = min(max(P.q_start[b], 0), P.N);
  r.n = max(min(max(P.q_start[b + 1], 0), P.N) - r.s0, 0);
  return r;
}

constexpr int PF_MAX_CTAS = 320;     // partial slots: two a CTA
constexpr int PF_MAX_ROWS = 256;     // packed rows of a row tile: 256 in bf16, 64 in float32
constexpr int PF_MAX_B = 2048;       // sequences of a call
static_assert(kPgRecords == 8 * PF_MAX_CTAS && kPgSomeAt >= 8 * (PF_MAX_CTAS / 2), "the bf16 kernel's records end ahead of the note");
constexpr int PF_ITEM_WEIGHT = 1;    // of a row tile besides its tiles of the cache, in units

// A row tile of one KV head, and its part in a CTA's run of units.
struct RowTile {
  int b, kvh, s0, n, len, pre, r0, nr;
  int first, lo, hi;                 // over its rows: smallest first token and lower end, past the last position
  int holes;                         // some row's first token lies behind it: [lo, hi) may hold tokens that no row sees
  TileSpan span;
  int i0, i1;                        // tiles of the span in this run; i1 < 0: the run is over
  int elsewhere;                     // 1: begun in another CTA, 2: goes on in another
  int c0;                            // CTA of its first unit
};

// What the rows of row tile rt of sequence b see.  Groups of `lanes` lanes (1, 8 or 32) share the
// rows of a tile; with more than one, every lane of the warp calls.
template <int ROWS, int KEYS>
__device__ __forceinline__ void row_tile_range(const PrefillParams &P, int b, int rt, RowTile &I, int lanes) {
  const SeqRows R = seq_rows(P, b);
  const int G = P.G;
  I.b = b;
  I.s0 = R.s0;
  I.n = R.n;
  I.len = paged_len(P.C, P.seq_len, b);
  I.pre = P.prefix_len ? min(P.prefix_len[b], I.len) : 0;
  I.r0 = rt * ROWS;
  I.nr = (int)min((int64_t)ROWS, (int64_t)R.n * G - I.r0);
  // tokens of the tile at positions >= 0
  const int i0 = max(div_by(P.group, I.r0), I.n - I.len), i1 = div_by(P.group, I.r0 + I.nr - 1);
  const int p0 = I.len - I.n;
  int first = 0, lo = 0;
  bool behind = false;
  if (i1 < i0) {                                          // no row of the tile is there
    first = lo = 0x7fffffff;
    I.pre = 0;
  } else if (P.first_tok) {
    first = lo = 0x7fffffff;
    for (int i = i0 + ((int)threadIdx.x & (lanes - 1)); i <= i1; i += 8 * lanes) {
      int f[8];                                           // eight loads under way at a time
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = i + k * lanes <= i1 ? __ldg(P.first_tok + R.s0 + i + k * lanes) : 0x7fffffff;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int g = max(f[k], 0);
        first = min(first, g);
        lo = min(lo, P.window ? max(g, p0 + i + k * lanes - P.window + 1) : g);
        behind |= i + k * lanes <= i1 && g > p0 + i + k * lanes;
      }
    }
  }
  if (P.first_tok && lanes > 1) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < lanes) {
        first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
  }
  if (!P.first_tok && i1 >= i0 && P.window) lo = max(0, p0 + i0 - P.window + 1);
  I.holes = P.first_tok && lanes == 32 ? __any_sync(0xffffffffu, behind) : 0;     // (the walk's; the plan has no use for it)
  I.first = first;
  I.lo = lo;
  I.hi = i1 < i0 ? 0 : p0 + i1 + 1;
  I.span = tile_span(first, I.pre, lo, I.hi, KEYS);
  if (I.span.nA + I.span.nB == 0) I.span.nA = 1;          // nothing seen: one tile of zeros writes the empty rows
}

// Whether one of rows i0 .. i1 (row i at position p0 + i) sees token t = tw + lane otherwise than by
// its prefix; a whole warp calls.  Row i sees [lower(i), position(i)], so t is seen if, of the rows at
// t or behind it, the smallest lower end is not behind t (an empty row's lies behind its own
// position: it never is the one).
// A function of its own: inlined into the tensor-core kernel's walk, where row tiles with holes are
// rare, it cost every prompt 1 % (8192 tokens: 918 against 907 us, and 1014 unrolled over a tile).
static __device__ __noinline__ bool seen_from(const int32_t *first_tok, int window, int p0, int i0, int i1, int tw) {
  const int lane = threadIdx.x & 31;
  auto lower = [&](int i) {
    if (i < i0 || i > i1) return 0x7fffffff;
    const int g = max(__ldg(first_tok + i), 0);
    return window ? max(g, p0 + i - window + 1) : g;
  };
  int later = 0x7fffffff, own = lower(tw - p0 + lane);
#pragma unroll 1
  for (int i = max(tw - p0 + 32, i0) + lane; i <= i1; i += 32) later = min(later, lower(i));
  later = __reduce_min_sync(0xffffffffu, later);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_down_sync(0xffffffffu, own, o);
    if (lane + o < 32) own = min(own, y);
  }
  return min(own, later) <= tw + lane;
}
// That for the rows of a row tile.
__device__ __forceinline__ bool seen_by_some(const PrefillParams &P, const RowTile &I, int tw) {
  const int p0 = I.len - I.n;
  return seen_from(P.first_tok + I.s0, P.window, p0, max(div_by(P.group, I.r0), -p0), div_by(P.group, I.r0 + I.nr - 1), tw);
}

// Deals the units out: unit = one KEYS-token tile of the cache for one row tile of ROWS packed
// rows of one KV head, ordered by (sequence, row tile, KV head, tile); a row tile begins with
// PF_ITEM_WEIGHT units' worth of weight (its queries, its epilogue).  CTA c gets the weights
// [per c, per (c + 1)): a tile belongs to the CTA that holds its last one.
struct PlanShared {
  uint32_t sum[32];
  uint32_t before;                   // weight before row tile `found`
  int found;                         // row tile in which the run begins, -1: no run
  int tiles[PF_MAX_B + 1];           // row tiles before each sequence
};
struct RunPlan {
  uint32_t per, u0, u1;              // below 2^31: the call refuses more
  int ntiles;
};
// Last sequence whose row tiles begin at or before x.
__device__ __forceinline__ int plan_seq(const PlanShared &S, int B, int x) {
  int a = 0, c = B - 1;
  while (a < c) {
    const int m = (a + c + 1) >> 1;
    if (S.tiles[m] <= x) a = m; else c = m - 1;
  }
  return a;
}
// Inclusive sum over the block of v, and the block's total; the whole block calls it.
template <int THREADS>
__device__ __forceinline__ uint32_t plan_scan(PlanShared &S, uint32_t v, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) S.sum[warp] = v;
  __syncthreads();
  const uint32_t w = lane < THREADS / 32 ? S.sum[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, w);
  return v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}
// `wt`: shared memory for the weights of PLAN_TILES row tiles, free again when the call ends.
constexpr int PLAN_TILES = 8192;
template <int ROWS, int KEYS, int THREADS, bool SOME = false>
__device__ __forceinline__ RunPlan prefill_plan(const PrefillParams &P, PlanShared &S, uint32_t *wt) {
  const int tid = threadIdx.x;
  RunPlan pl;
  if (tid == 0) S.found = -1;
  uint32_t base = 0, sum;
  bool bad = false;                                       // q_start descends
#pragma unroll 1
  for (int b0 = 0; b0 < P.B; b0 += THREADS) {
    const int b = b0 + tid;
    const int64_t rows = b < P.B ? (int64_t)seq_rows(P, b).n * P.G : 0;
    const uint32_t n = SOME && rows <= P.above ? 0 : (uint32_t)((rows + ROWS - 1) / ROWS);
    bad |= b < P.B && min(P.q_start[b], P.N) > max(P.q_start[b + 1], 0);
    const uint32_t end = base + plan_scan<THREADS>(S, n, sum);
    if (b < P.B) S.tiles[b] = (int)(end - n);
    base += sum;
  }
  if (tid == 0) S.tiles[P.B] = (int)base;
  // sequences that overlap: nothing bounds their row tiles' number, no work is done
  if (bad) paged_fail(P.C.status, ECHO_ERR_INVALID_ARG);
  pl.ntiles = __syncthreads_or(bad) ? 0 : (int)base;
  // PLAN_TILES row tiles at a time: their weights, then a scan in which a thread takes a run of
  // them.  The first pass gives the total, the second (the same values, where they all fit) the
  // row tile that holds the CTA's first weight.  First tokens are read by up to eight lanes a
  // tile, as many as there are threads for.
  int grp = 1;
  while (P.first_tok && grp < 8 && 2 * grp * pl.ntiles <= THREADS) grp *= 2;
  uint32_t n = 0, end = 0;
  pl.per = pl.u0 = pl.u1 = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t at = 0;
#pragma unroll 1
    for (int x0 = 0; x0 < pl.ntiles; x0 += PLAN_TILES) {
      const int nx = min(PLAN_TILES, pl.ntiles - x0);
      if (pass == 0 || pl.ntiles > PLAN_TILES) {
        __syncthreads();
#pragma unroll 1
        for (int i = tid / grp; i < ((nx + 31) & ~31); i += THREADS / grp) {
          RowTile I;
          const int x = x0 + min(i, nx - 1), b = plan_seq(S, P.B, x);
          row_tile_range<ROWS, KEYS>(P, b, x - S.tiles[b], I, grp);
          if (i < nx && (tid & (grp - 1)) == 0)
            wt[i] = (uint32_t)(I.span.nA + I.span.nB + PF_ITEM_WEIGHT) * (uint32_t)P.C.n_kv_heads;
        }
        __syncthreads();
      }
      const int c = (nx + THREADS - 1) / THREADS, i0 = min(tid * c, nx), i1 = min(i0 + c, nx);
      if (pass == 0 || pl.ntiles > PLAN_TILES) {
        n = 0;
        for (int i = i0; i < i1; ++i) n += wt[i];
        end = at + plan_scan<THREADS>(S, n, sum);
      }
      at += sum;
      if (pass == 1) {
        if (end - n <= pl.u0 && pl.u0 < end) {
          uint32_t u = end - n;
          int i = i0;
          while (u + wt[i] <= pl.u0) u += wt[i++];
          S.found = x0 + i;
          S.before = u;
        }
        if (pl.u0 < at) break;                            // the same in every thread
      }
    }
    if (pass == 0) {
      pl.per = max((at + gridDim.x - 1) / gridDim.x, 1u);
      pl.u0 = pl.per * blockIdx.x;
      pl.u1 = min(at, pl.u0 + pl.per);
      if (pl.u0 >= at) break;
    }
  }
  fence_proxy_async_smem();                               // the loads take wt's place
  __syncthreads();
  return pl;
}

// The walk over the row tiles of a CTA's run.  A whole warp moves it together.
template <int ROWS, int KEYS>
struct RowTileWalk {
  const PrefillParams &P;
  const PlanShared &S;
  const RunPlan pl;
  RowTile I;
  int xt, b;
  uint32_t ws;                       // weight before the row tile

  __device__ __forceinline__ void enter() {
    while (b + 1 < P.B && S.tiles[b + 1] <= xt) ++b;
    row_tile_range<ROWS, KEYS>(P, b, xt - S.tiles[b], I, 32);
    if ((threadIdx.x & 31) == 0 && I.len < I.n) paged_fail(P.C.status, ECHO_ERR_INVALID_ARG);
  }
  __device__ __forceinline__ void part(int i0) {          // its tiles in this run; none: the run is over
    const int nt = I.span.nA + I.span.nB;
    I.i0 = i0;
    I.i1 = min(nt, (int)(pl.u1 - ws) - PF_ITEM_WEIGHT);
    I.elsewhere = (I.i0 > 0 ? 1 : 0) | (I.i1 < nt ? 2 : 0);
    I.c0 = (int)((ws + PF_ITEM_WEIGHT) / pl.per);
    if (I.i1 <= I.i0) I.i1 = -1;
  }
  __device__ __forceinline__ RowTileWalk(const PrefillParams &p, const PlanShared &s, const RunPlan &r)
      : P(p), S(s), pl(r), I(), xt(s.found), b(0), ws(0) {
    I.i1 = -1;
    if (xt < 0) return;
    b = plan_seq(S, P.B, xt);
    enter();
    const int nt = I.span.nA + I.span.nB + PF_ITEM_WEIGHT;
    I.kvh = (int)((pl.u0 - S.before) / nt);
    ws = S.before + (uint32_t)I.kvh * nt;
    part(max(0, (int)(pl.u0 - ws) - PF_ITEM_WEIGHT));
  }
  __device__ __forceinline__ void next() {
    ws += I.span.nA + I.span.nB + PF_ITEM_WEIGHT;
    if (I.kvh + 1 < P.C.n_kv_heads) {
      ++I.kvh;
    } else if (++xt < pl.ntiles) {
      I.kvh = 0;
      enter();
    } else {
      I.i1 = -1;
      return;
    }
    part(0);
  }
};

// Leaves word that a split row tile ends in this CTA.
__device__ __forceinline__ void join_record(const PrefillParams &P, int c0, int s0, int r0, int nr, int kvh) {
  int32_t *rec = P.rec + blockIdx.x * 8;
  rec[1] = c0;
  rec[2] = s0;
  rec[3] = r0;
  rec[4] = nr;
  rec[5] = kvh;
  rec[0] = 1;
}

// Joins the partials of the row tile that ends in CTA blockIdx.x, in the order of their units:
// slot 1 of its first CTA, then slot 0 of the following ones.  A warp takes a row: the maximum
// of all first, so that the weighted sums are independent loads.
template <typename T, int D, bool SOME = false>
__global__ void __launch_bounds__(128) paged_prefill_join_kernel(const __grid_constant__ PrefillParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (SOME && *P.some == 0) return;
  const int c1 = blockIdx.x;
  const int4 ra = *reinterpret_cast<const int4 *>(P.rec + c1 * 8), rb = *reinterpret_cast<const int4 *>(P.rec + c1 * 8 + 4);
  if (ra.x == 0) return;
  const int c0 = ra.y, s0 = ra.z, r0 = ra.w, nr = rb.x, kvh = rb.y, np = c1 - c0 + 1;
  const int lane = threadIdx.x & 31;
  constexpr int VL = D / 32;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < nr; r += gridDim.y * 4) {
    auto row = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * P.prows + r; };
    float M = -INFINITY, L = 0.f, v[VL];
    for (int i = lane; i < np; i += 32) M = fmaxf(M, P.pml[row(i) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int i = 0; i < VL; ++i) v[i] = 0.f;
    const float z = M == -INFINITY ? 0.f : M;
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      const float2 ml = *reinterpret_cast<const float2 *>(P.pml + row(i) * 2);
      const float *o = P.po + row(i) * D + lane * VL;
      float x[VL];
      if constexpr (VL == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(o);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2 *>(o);
        x[0] = f.x; x[1] = f.y;
      }
      const float w = ex2(ml.x - z);
      L += w * ml.y;
#pragma unroll
      for (int e = 0; e < VL; ++e) v[e] = fmaf(w, x[e], v[e]);
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const int tk = div_by(P.group, r0 + r), hd = kvh * P.G + (r0 + r) - tk * P.G;
    const int64_t orow = (int64_t)(s0 + tk) * P.Hq + hd;
    T *dst = (T *)P.out + orow * D + lane * VL;
#pragma unroll
    for (int i = 0; i < VL; i += 2) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<__nv_bfloat162 *>(dst + i) = __floats2bfloat162_rn(v[i] * inv, v[i + 1] * inv);
      else
        *reinterpret_cast<float2 *>(dst + i) = make_float2(v[i] * inv, v[i + 1] * inv);
    }
    if (lane == 0) P.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPgLn2;
  }
}

echo_status_t launch_prefill_tc(PrefillParams &P, cudaStream_t st);   // bf16
echo_status_t launch_prefill_q8(PrefillParams &P, cudaStream_t st);   // e4m3 codes, bf16 queries
echo_status_t launch_prefill_some(PrefillParams &P, cudaStream_t st); // that, of sequences of more than P.above packed rows
echo_status_t launch_prefill_rows(PrefillParams &P, cudaStream_t st); // rows that were codes

}  // namespace echo
