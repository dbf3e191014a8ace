// Attention of many new tokens over a paged key/value cache: prompts, chunks of prompts,
// drafted tokens.  Scores, masks and results as in the single-token call, per row.
//
// The query heads of one KV head are packed with the tokens: packed row r of a sequence is
// token r / G, head r % G of the group, so that every tile of rows reads its keys and values
// once whatever G is, and a few drafted tokens still fill a tile.
//
// The work is dealt out evenly over the GPU (prefill_plan in paged_prefill.cuh), split row tiles
// are joined by a second kernel.  bf16 runs on the tensor cores (paged_prefill_tc.cu).
// Float32 (below), two CTAs an SM: row tiles of 64 packed rows, 64-token tiles of the cache, a
// running maximum and sum; 256 threads hold 4 x 4 scores and 4 x d/16 results each.  Float32
// arithmetic throughout: 4 d operations for each pair of query head and seen token on the FMA
// units, which bound it together with shared memory (eight 16-byte loads to 64 FMAs).
//
// Measured on a GB300: two sequences of 600-1100 tokens, 8 heads of 64 over 4, two-way prefix,
// 59 us (1.2 GFLOP; FMA issue 42 %, shared memory 52 %, one wave of 304 CTAs); 129 us with a CTA a row
// tile, which leaves the last rows of a causal mask to few of them.

#include <cuda_fp16.h>

#include "paged_prefill.cuh"

namespace echo {

constexpr int PS_THREADS = 256, PS_ROWS = 64, PS_KEYS = 64;

struct PsShared {
  int pos[PS_ROWS], lo[PS_ROWS], first[PS_ROWS];
  float slope[PS_ROWS];
  int64_t row[PS_KEYS];
  PlanShared plan;
};

template <int D>
constexpr size_t ps_smem() {
  return sizeof(float) * (size_t)(PS_ROWS + 2 * PS_KEYS) * D + sizeof(PsShared);
}

// Float offset of 16-byte chunk c of row r in a tile of D-value rows: chunks are permuted by
// the row, so that sixteen rows read at one chunk take two wavefronts, the least there is.
template <int D>
__device__ __forceinline__ int ps_at(int r, int c) { return r * D + ((c ^ (r & 7)) << 2); }

template <int D>
__global__ void __launch_bounds__(PS_THREADS, 2) paged_prefill_simt_kernel(const __grid_constant__ PrefillParams P) {
  extern __shared__ __align__(16) float ps_sm[];
  float *qs = ps_sm;                                     // [64][D]
  float *ks = qs + PS_ROWS * D;                          // [64][D] keys, chunks permuted; then [64][64] weights
  float *vs = ks + PS_KEYS * D;                          // [64][D] values
  float *pp = ks;
  PsShared &S = *reinterpret_cast<PsShared *>(vs + PS_KEYS * D);
  constexpr int KC = D / 4, OC = D / 64;                 // chunks of a row; float4 columns of a thread's results
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = P.G;
  if (tid == 0) P.rec[blockIdx.x * 8] = 0;
  const RunPlan pl = prefill_plan<PS_ROWS, PS_KEYS, PS_THREADS>(P, S.plan, reinterpret_cast<uint32_t *>(ps_sm));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (RowTileWalk<PS_ROWS, PS_KEYS> W(P, S.plan, pl); W.I.i1 >= 0; W.next()) {
    const RowTile &I = W.I;
    __syncthreads();                                     // the last row tile's shared values are read
    if (tid < PS_ROWS) {
      int pos = -1, lo = 0x7fffffff, first = 0x7fffffff; // a row that is not there sees nothing
      float sl = 0.f;
      if (tid < I.nr) {
        const int i = div_by(P.group, I.r0 + tid), g = I.r0 + tid - i * G;
        pos = I.len - I.n + i;
        first = P.first_tok ? max(P.first_tok[I.s0 + i], 0) : 0;
        lo = P.window ? max(first, pos - P.window + 1) : first;
        if (pos < 0) { first = lo = 0x7fffffff; }
        if (P.slopes) sl = P.slopes[I.kvh * G + g] * kPgLog2e;
      }
      S.pos[tid] = pos;
      S.lo[tid] = lo;
      S.first[tid] = first;
      S.slope[tid] = sl;
    }
    for (int i = tid; i < PS_ROWS * KC; i += PS_THREADS) {
      const int r = i / KC, c = i % KC;
      const bool there = r < I.nr;
      const int t = there ? div_by(P.group, I.r0 + r) : 0, g = there ? I.r0 + r - t * G : 0;
      cp_async_16(qs + r * D + 4 * c, (const float *)P.q + (int64_t)(I.s0 + t) * P.q_stride + (int64_t)(I.kvh * G + g) * D + 4 * c,
                  there ? 16u : 0u);
    }
    float o[4][OC][4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < OC; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    }
    const float *kb = (const float *)P.C.k + (int64_t)I.kvh * P.C.head_stride, *vb = (const float *)P.C.v + (int64_t)I.kvh * P.C.head_stride;
    for (int it = I.i0; it < I.i1; ++it) {
      const int t0 = I.span.tile(it) * PS_KEYS;
      if (tid < PS_KEYS) {
        const int t = t0 + tid;
        const bool own = I.holes ? seen_by_some(P, I, t0 + (tid & 32)) : t >= I.lo && t < I.hi;
        const bool some = t < I.len && t >= I.first && (own || t < I.pre);
        S.row[tid] = some ? paged_row(P.C, I.b, t) : -1;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < PS_KEYS * KC / PS_THREADS; ++i) {
        const int r = (i * PS_THREADS + tid) / KC, c = (i * PS_THREADS + tid) % KC;
        const int64_t g = S.row[r];
        cp_async_16(ks + ps_at<D>(r, c), kb + (g >= 0 ? g : 0) + 4 * c, g >= 0 ? 16u : 0u);
      }
      cp_async_commit();
#pragma unroll
      for (int i = 0; i < PS_KEYS * KC / PS_THREADS; ++i) {
        const int r = (i * PS_THREADS + tid) / KC, c = (i * PS_THREADS + tid) % KC;
        const int64_t g = S.row[r];
        cp_async_16(vs + r * D + 4 * c, vb + (g >= 0 ? g : 0) + 4 * c, g >= 0 ? 16u : 0u);
      }
      cp_async_commit();
      cp_async_wait<1>();                                // the queries and the keys
      __syncthreads();
      float s[4][4] = {};
#pragma unroll 8
      for (int c = 0; c < KC; ++c) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qv[i] = *reinterpret_cast<const float4 *>(qs + (ty * 4 + i) * D + 4 * c);
          kv[i] = *reinterpret_cast<const float4 *>(ks + ps_at<D>(tx + 16 * i, c));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(qv[i].x, kv[j].x, fmaf(qv[i].y, kv[j].y, fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, s[i][j]))));
      }
      bool there[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) there[j] = S.row[tx + 16 * j] >= 0;
      __syncthreads();                                   // the keys are read: the weights take their place
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i, pos = S.pos[r], lo = S.lo[r], first = S.first[r];
        const float slope = S.slope[r];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + tx + 16 * j;
          const bool seen = there[j] && t >= first && ((t <= pos && t >= lo) || t < I.pre);
          float a = score_log2(P.f, s[i][j]);
          if (P.slopes) a -= slope * fabsf((float)(pos - t));
          s[i][j] = seen ? a : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float nm = fmaxf(m[i], mx), z = nm == -INFINITY ? 0.f : nm;
        const float corr = ex2(m[i] - z);
        m[i] = nm;
        l[i] *= corr;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = ex2(s[i][j] - z);
          l[i] += p;
          pp[r * PS_KEYS + tx + 16 * j] = p;
        }
#pragma unroll
        for (int j = 0; j < OC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][j][e] *= corr;
      }
      cp_async_wait<0>();                                // the values
      __syncthreads();
#pragma unroll 4
      for (int t = 0; t < PS_KEYS; t += 4) {
        float4 pv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4 *>(pp + (ty * 4 + i) * PS_KEYS + t);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < OC; ++j) {
            const float4 vv = *reinterpret_cast<const float4 *>(vs + (t + u) * D + 64 * j + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = u == 0 ? pv[i].x : u == 1 ? pv[i].y : u == 2 ? pv[i].z : pv[i].w;
              o[i][j][0] = fmaf(p, vv.x, o[i][j][0]);
              o[i][j][1] = fmaf(p, vv.y, o[i][j][1]);
              o[i][j][2] = fmaf(p, vv.z, o[i][j][2]);
              o[i][j][3] = fmaf(p, vv.w, o[i][j][3]);
            }
          }
      }
      __syncthreads();                                   // weights and values are read
    }
    const bool whole = I.elsewhere == 0;
    const int64_t slot = 2 * blockIdx.x + ((I.elsewhere & 1) ? 0 : 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      float L = l[i];
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
      if (r >= I.nr) continue;
      const int t = div_by(P.group, I.r0 + r), g = I.r0 + r - t * G;
      const float f = !whole ? 1.f : L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
      const int64_t row = (int64_t)(I.s0 + t) * P.Hq + I.kvh * G + g, prow = slot * P.prows + r;
      float *dst = (whole ? (float *)P.out + row * D : P.po + prow * D) + 4 * tx;
#pragma unroll
      for (int j = 0; j < OC; ++j)
        *reinterpret_cast<float4 *>(dst + 64 * j) = make_float4(o[i][j][0] * f, o[i][j][1] * f, o[i][j][2] * f, o[i][j][3] * f);
      if (tx == 0) {
        if (whole) P.lse[row] = L == 0.f ? -INFINITY : (m[i] + log2f(L)) * kPgLn2;
        else *reinterpret_cast<float2 *>(P.pml + prow * 2) = make_float2(m[i], L);
      }
    }
    if (tid == 0 && I.elsewhere == 1) join_record(P, I.c0, I.s0, I.r0, I.nr, I.kvh);
  }
}

// A cache in 8 bits in 16 bits, page by page of the sequences' tables: each code times its power of two, keys in
// bf16, for products with bf16 queries, values in float16, for products with float16 weights; either holds it
// exactly.  One byte read and two written a value: HBM.  A CTA takes pages in turn, a thread 16 codes at a time.
// Of a sequence the tokens that its rows see are written, [first, pre) by a prefix and [lo, len) from the smallest
// lower end on; the others' places are left alone (256 tokens, 32 heads over 8, under a window of 512 at 128K: 178 us
// with every row, 43 so).  Entries that are no page stay none in the new table.
constexpr int PQ_THREADS = 256;
struct SeenTokens {
  int first, pre, lo, len;           // (pre <= lo: what a prefix adds)
};
// The whole block calls it.
__device__ __forceinline__ SeenTokens seen_tokens(const PrefillParams &P, int b) {
  __shared__ int red[2][PQ_THREADS / 32];
  const SeqRows R = seq_rows(P, b);
  SeenTokens s;
  s.len = min(max(__ldg(P.seq_len + b), 0), P.C.max_pages * P.C.page_tokens);
  const int p0 = s.len - R.n, i0 = max(0, -p0);           // rows at positions >= 0
  if (i0 >= R.n) return {0, 0, 0, 0};
  s.first = 0;
  s.lo = P.window ? max(0, p0 + i0 - P.window + 1) : 0;
  if (P.first_tok) {
    int f = 0x7fffffff, l = 0x7fffffff;
#pragma unroll 4
    for (int i = i0 + (int)threadIdx.x; i < R.n; i += PQ_THREADS) {
      const int g = max(__ldg(P.first_tok + R.s0 + i), 0);
      f = min(f, g);
      l = min(l, P.window ? max(g, p0 + i - P.window + 1) : g);
    }
    f = __reduce_min_sync(0xffffffffu, f);
    l = __reduce_min_sync(0xffffffffu, l);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = f, red[1][threadIdx.x >> 5] = l;
    __syncthreads();
    s.first = __reduce_min_sync(0xffffffffu, red[0][threadIdx.x & (PQ_THREADS / 32 - 1)]);
    s.lo = __reduce_min_sync(0xffffffffu, red[1][threadIdx.x & (PQ_THREADS / 32 - 1)]);
  }
  s.pre = P.prefix_len ? min(min(__ldg(P.prefix_len + b), s.len), s.lo) : 0;
  return s;
}
template <int D>
__global__ void __launch_bounds__(PQ_THREADS) paged_q8_rows_kernel(const __grid_constant__ PrefillParams P, int n, uint16_t *k,
                                                                   uint16_t *v, int32_t *table) {
  constexpr int CH = D / 16;
  const echo_paged_kv_t &C = P.C;
  const echo_paged_scales_t &X = P.X;
  const int T = C.page_tokens, H = C.n_kv_heads;
  SeenTokens S = {};
  int of = -1;                                            // the sequence that S is of
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int b = i / C.max_pages, p0 = (i - b * C.max_pages) * T;
    const int32_t e = __ldg(C.page_table + i);            // (on its way under the look at first tokens)
    if (b != of) S = seen_tokens(P, of = b);
    const int a0 = max(p0, S.first), a1 = min(p0 + T, S.pre), b0 = max(p0, S.lo), b1 = min(p0 + T, S.len);
    if (a0 >= a1 && b0 >= b1) continue;
    const bool page = e >= 0 && e < C.n_pages;
    if (threadIdx.x == 0) table[i] = page ? i : -1;
    if (!page) continue;
    const int64_t to = (int64_t)i * T * H * D;
    const int na = max(a1 - a0, 0), nr = na + max(b1 - b0, 0);
    for (int64_t x = threadIdx.x; x < (int64_t)nr * H * CH; x += PQ_THREADS) {
      const int c = (int)(x % CH), h = (int)(x / CH % H), y = (int)(x / CH / H), t = (y < na ? a0 + y : b0 + (y - na)) - p0;
      const int64_t from = (int64_t)e * C.page_stride + (int64_t)t * C.row_stride + (int64_t)h * C.head_stride + c * 16;
      const int64_t s = (int64_t)e * X.page_stride + (int64_t)t * X.row_stride + (int64_t)h * X.head_stride;
      const uint4 a[2] = {__ldg(reinterpret_cast<const uint4 *>((const uint8_t *)C.k + from)),
                          __ldg(reinterpret_cast<const uint4 *>((const uint8_t *)C.v + from))};
      const float kf = exp2i(q8_exp(__ldg(X.k + s)));
      const uint32_t vf = q8_half_pow(q8_exp(__ldg(X.v + s)));
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t u[4] = {a[w].x, a[w].y, a[w].z, a[w].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          q8_halves(u[q], o[2 * q], o[2 * q + 1]);
#pragma unroll
          for (int z = 2 * q; z < 2 * q + 2; ++z) {
            if (w) {
              o[z] = q8_hmul2(o[z], vf);
            } else {
              const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&o[z]));
              const __nv_bfloat162 b = __floats2bfloat162_rn(y.x * kf, y.y * kf);
              o[z] = *reinterpret_cast<const uint32_t *>(&b);
            }
          }
        }
        uint4 *dst = reinterpret_cast<uint4 *>((w ? v : k) + to + ((int64_t)h * T + t) * D + c * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

template <int D>
static echo_status_t launch_simt(const PrefillParams &P, cudaStream_t st) {
  static_assert(2 * (ps_smem<D>() + 1024) <= 228 * 1024, "two CTAs an SM");
  ECHO_CUDA_OK(allow_smem<paged_prefill_simt_kernel<D>>(ps_smem<D>()));
  const int grid = std::min(2 * sm_count(), PF_MAX_CTAS);
  paged_prefill_simt_kernel<D><<<grid, PS_THREADS, ps_smem<D>(), st>>>(P);
  ECHO_LAUNCH_OK();
  ECHO_CUDA_OK(launch_after(paged_prefill_join_kernel<float, D>, dim3(grid, (P.prows + 3) / 4), dim3(128), 0, st, P));
  return ECHO_OK;
}

}  // namespace echo

using namespace echo;

// Two partials a CTA, of the rows of a row tile at most, and a record each.  Float32 has twice the
// CTAs of bf16 and a quarter of the rows at most: the larger of the two holds both (with 64 packed
// rows or fewer that is float32's).
static int prefill_prows(int64_t N, int64_t G, int rows) { return (int)std::min<int64_t>(rows, N * G); }

extern "C" size_t echo_paged_prefill_workspace_bytes(int32_t N, int32_t B, int32_t Hq, int32_t n_kv_heads, int32_t d) {
  if (N <= 0 || B <= 0 || Hq <= 0 || n_kv_heads <= 0 || d <= 0 || Hq % n_kv_heads) return 0;
  const int64_t G = Hq / n_kv_heads;
  const size_t a = (size_t)(PF_MAX_CTAS / 2) * 2 * prefill_prows(N, G, PF_MAX_ROWS), b = (size_t)PF_MAX_CTAS * 2 * prefill_prows(N, G, PS_ROWS);
  return (std::max(a, b) * (d + 2) + (size_t)PF_MAX_CTAS * 8) * sizeof(float);
}

// Where a cache in 8 bits is written out in 16 bits first.  Turning a tile's codes costs the tensor-core kernel
// some 0.7 us each time that a row tile reads it; writing them out and reading them back, 3 bytes a
// value of HBM, is 2.5 us a tile, once.  A prompt of 8192, 64 heads over 8: 1430 us on the codes, 932 written
// out first; 512 tokens over 32K, capped: 500 and 448 (424 since).  The rule goes by averages, and mixtures bear it: 4096
// tokens beside 30 single ones of 1K 481 on the codes, 351 written out, of 8K 708 and 751; 1024 beside 7 of 32K 375 both.
// A GiB holds 256K tokens of 8 heads of 128: some 0.3 ms of HBM at most where few rows read them.
static bool q8_rows_first(int64_t N, int64_t B, int64_t G, int64_t bytes) {
  return N * G >= 4 * PF_MAX_ROWS * B && bytes <= (1ll << 30);
}
static size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
// Keys (or values) of every page-table entry in 16 bits, and the table of where they lie.
static int64_t q8_rows_bytes(int64_t B, int64_t n_kv_heads, int64_t d, int64_t max_pages, int64_t page_tokens) {
  const double n = (double)B * max_pages * page_tokens * n_kv_heads * d * 2;
  return n < 1e15 ? (int64_t)n : (int64_t)1e15;
}

extern "C" size_t echo_paged_prefill_q8_workspace_bytes(int32_t N, int32_t B, int32_t Hq, int32_t n_kv_heads, int32_t d,
                                                        int32_t max_pages, int32_t page_tokens) {
  const size_t base = echo_paged_prefill_workspace_bytes(N, B, Hq, n_kv_heads, d);
  if (!base || max_pages <= 0 || page_tokens <= 0) return 0;
  const int64_t rows = q8_rows_bytes(B, n_kv_heads, d, max_pages, page_tokens);
  if (!q8_rows_first(N, B, Hq / n_kv_heads, 2 * rows)) return base;
  return round256(base) + 2 * round256((size_t)rows) + round256((size_t)B * max_pages * 4);
}

// Writes the cache's rows out and points P at them: pages of the same tokens, heads first, entry (b, p) at
// b * max_pages + p.
static echo_status_t launch_q8_rows(PrefillParams &P, unsigned char *at, cudaStream_t st) {
  const PrefillParams R = P;
  const echo_paged_kv_t &C = R.C;
  const size_t rows = round256((size_t)q8_rows_bytes(P.B, C.n_kv_heads, C.head_dim, C.max_pages, C.page_tokens));
  echo_paged_kv_t &W = P.C;
  W.k = at;
  W.v = at + rows;
  W.row_stride = C.head_dim;
  W.head_stride = (int64_t)C.page_tokens * C.head_dim;
  W.page_stride = W.head_stride * C.n_kv_heads;
  W.n_pages = P.B * C.max_pages;
  W.dtype = ECHO_BF16;                                    // (16 bits a value)
  int32_t *table = reinterpret_cast<int32_t *>(at + 2 * rows);
  W.page_table = table;
  const dim3 grid(std::min(W.n_pages, 8 * sm_count()));
  if (C.head_dim == 128) paged_q8_rows_kernel<128><<<grid, PQ_THREADS, 0, st>>>(R, W.n_pages, (uint16_t *)W.k, (uint16_t *)W.v, table);
  else paged_q8_rows_kernel<64><<<grid, PQ_THREADS, 0, st>>>(R, W.n_pages, (uint16_t *)W.k, (uint16_t *)W.v, table);
  ECHO_LAUNCH_OK();
  return ECHO_OK;
}

// Calls of a few new tokens a sequence on average (few_tokens_q8) over codes.  Up to FEW_ALL_ROWS packed rows go the
// way of single tokens as they are; of more, sequences of more than FEW_ROWS (the rows that its units hold, and read
// the cache for) go to the tensor cores, found from q_start on the device: a batch's average tells nothing of its longest
// sequence.  Measured with 8 KV heads of 128: 255 single tokens of 1K-4K beside 700 tokens of a prompt of 8K 1235 us by the
// average, 638 so; 2048 rows of one of 1024 sequences (the others empty) 507 and 89 us.  Where no sequence
// has more the second kernel and its join cost 9 us: 64 x 4 tokens over 2K-6K 201 and 210 us, 256 x 1 over 1K-4K 331 and
// 340.  Of 1024 rows 31 single tokens beside 97 over 8K take 189 us here and 146 so; 16 x 4 over 17K-20K 208 and 217.
constexpr int FEW_ROWS = 32, FEW_ALL_ROWS = 1024;

// scales: of a cache in 8 bits, and else NULL.
static echo_status_t attn_prefill(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales, const void *q,
                                  int64_t q_stride, const int32_t *q_start, const int32_t *seq_len, int32_t N,
                                  int32_t B, int32_t Hq, const echo_attn_scores_t *scores_of, void *out, float *lse,
                                  void *workspace, size_t workspace_bytes, cudaStream_t cs) {
  const echo_status_t st = paged_scores_check(scores_of);
  if (st != ECHO_OK) return st;
  if (!q || !q_start || !seq_len || !out || !lse || N <= 0 || B <= 0 || Hq <= 0) return ECHO_ERR_INVALID_ARG;
  if (Hq % cache->n_kv_heads || Hq / cache->n_kv_heads > 128 || cache->n_kv_heads > 65535 || B > PF_MAX_B)
    return ECHO_ERR_UNSUPPORTED;
  const int act = paged_act_type(cache->dtype);
  if (!paged_rows_ok(q, q_stride, act) || !paged_rows_ok(out, 0, act)) return ECHO_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) ||
      workspace_bytes < echo_paged_prefill_workspace_bytes(N, B, Hq, cache->n_kv_heads, cache->head_dim))
    return ECHO_ERR_INVALID_ARG;
  PrefillParams P;
  P.C = *cache;
  P.X = scales ? *scales : echo_paged_scales_t{};
  P.q = q; P.q_stride = q_stride; P.q_start = q_start; P.seq_len = seq_len;
  P.N = N; P.B = B; P.Hq = Hq; P.G = Hq / cache->n_kv_heads;
  P.page = fast_div(cache->page_tokens); P.group = fast_div(P.G);
  if ((int64_t)N * P.G > 0x7fff0000ll) return ECHO_ERR_UNSUPPORTED;
  P.slopes = scores_of->slopes; P.window = scores_of->window;
  P.first_tok = scores_of->first_tok; P.prefix_len = scores_of->prefix_len;
  P.f = score_form(scores_of);
  P.out = out; P.lse = lse;
  const bool bf = act == ECHO_BF16;
  P.prows = prefill_prows(N, P.G, bf ? PF_MAX_ROWS : PS_ROWS);
  // the units are counted in 32 bits: row tiles x (tiles of the longest sequence) x KV heads
  const double tiles = (double)N * P.G / (scales ? PF_MAX_ROWS / 2 : bf ? PF_MAX_ROWS : PS_ROWS) + B;
  const double deep = (double)cache->max_pages * cache->page_tokens / (bf ? 2 * PS_KEYS : PS_KEYS) + 4;
  if (tiles * deep * cache->n_kv_heads > 2147483647.0) return ECHO_ERR_UNSUPPORTED;
  P.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  P.rec = reinterpret_cast<int32_t *>(workspace);
  P.po = reinterpret_cast<float *>(P.rec + 8 * PF_MAX_CTAS);
  P.pml = P.po + (size_t)(bf ? PF_MAX_CTAS : 2 * PF_MAX_CTAS) * P.prows * cache->head_dim;
  P.above = 0;
  P.some = nullptr;
  if (scales && few_tokens_q8(N, B, P.G, scores_of)) {
    const bool all = (int64_t)N * P.G <= FEW_ALL_ROWS;    // (no sequence has more)
    const echo_status_t few = launch_few_tokens_q8(cache, scales, q, q_stride, q_start, seq_len, N, B, Hq, scores_of,
                                                   all ? FEW_ALL_ROWS : FEW_ROWS, out, lse, workspace, cs);
    if (all || few != ECHO_OK) return few;
    P.above = FEW_ROWS;
    P.some = P.rec + kPgSomeAt;
    return launch_prefill_some(P, cs);
  }
  if (scales) {
    const size_t base = echo_paged_prefill_workspace_bytes(N, B, Hq, cache->n_kv_heads, cache->head_dim);
    const size_t all = echo_paged_prefill_q8_workspace_bytes(N, B, Hq, cache->n_kv_heads, cache->head_dim, cache->max_pages,
                                                             cache->page_tokens);
    if (all > base && workspace_bytes >= all) {
      const echo_status_t w = launch_q8_rows(P, (unsigned char *)workspace + round256(base), cs);
      return w == ECHO_OK ? launch_prefill_rows(P, cs) : w;
    }
    return launch_prefill_q8(P, cs);
  }
  if (bf) return launch_prefill_tc(P, cs);
  return cache->head_dim == 128 ? launch_simt<128>(P, cs) : launch_simt<64>(P, cs);
}

extern "C" echo_status_t echo_paged_attn_prefill(const echo_paged_kv_t *cache, const void *q, int64_t q_stride,
                                                 const int32_t *q_start, const int32_t *seq_len, int32_t N, int32_t B,
                                                 int32_t Hq, const echo_attn_scores_t *scores, void *out, float *lse,
                                                 void *workspace, size_t workspace_bytes, echo_stream_t stream) {
  const echo_status_t st = paged_check(cache);
  if (st != ECHO_OK) return st;
  return attn_prefill(cache, nullptr, q, q_stride, q_start, seq_len, N, B, Hq, scores, out, lse, workspace,
                      workspace_bytes, (cudaStream_t)stream);
}

extern "C" echo_status_t echo_paged_attn_prefill_q8(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales,
                                                    const void *q, int64_t q_stride, const int32_t *q_start,
                                                    const int32_t *seq_len, int32_t N, int32_t B, int32_t Hq,
                                                    const echo_attn_scores_t *scores_of, void *out, float *lse,
                                                    void *workspace, size_t workspace_bytes, echo_stream_t stream) {
  echo_status_t st = paged_check(cache, true);
  if (st == ECHO_OK) st = paged_scales_check(scales);
  if (st != ECHO_OK) return st;
  return attn_prefill(cache, scales, q, q_stride, q_start, seq_len, N, B, Hq, scores_of, out, lse, workspace,
                      workspace_bytes, (cudaStream_t)stream);
}
