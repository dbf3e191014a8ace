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

template <int D>
static echo_status_t launch_simt(const PrefillParams &P, cudaStream_t st) {
  static_assert(2 * (ps_smem<D>() + 1024) <= 228 * 1024, "two CTAs an SM");
  ECHO_CUDA_OK(allow_smem<paged_prefill_simt_kernel<D>>(ps_smem<D>()));
  const int grid = std::min(2 * sm_count(), PF_MAX_CTAS);
  paged_prefill_simt_kernel<D><<<grid, PS_THREADS, ps_smem<D>(), st>>>(P);
  ECHO_LAUNCH_OK();
  ECHO_CUDA_OK(launch_after(paged_prefill_join_kernel<float, D>, dim3(grid, (P.prows + 3) / 4), dim3(128), st, P));
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

extern "C" echo_status_t echo_paged_attn_prefill(const echo_paged_kv_t *cache, const void *q, int64_t q_stride,
                                                 const int32_t *q_start, const int32_t *seq_len, int32_t N, int32_t B,
                                                 int32_t Hq, const echo_attn_scores_t *scores, void *out, float *lse,
                                                 void *workspace, size_t workspace_bytes, echo_stream_t stream) {
  echo_status_t st = paged_check(cache);
  if (st == ECHO_OK) st = paged_scores_check(scores);
  if (st != ECHO_OK) return st;
  if (!q || !q_start || !seq_len || !out || !lse || N <= 0 || B <= 0 || Hq <= 0) return ECHO_ERR_INVALID_ARG;
  if (Hq % cache->n_kv_heads || Hq / cache->n_kv_heads > 128 || cache->n_kv_heads > 65535 || B > PF_MAX_B)
    return ECHO_ERR_UNSUPPORTED;
  if (!paged_rows_ok(q, q_stride, cache->dtype) || !paged_rows_ok(out, 0, cache->dtype)) return ECHO_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) ||
      workspace_bytes < echo_paged_prefill_workspace_bytes(N, B, Hq, cache->n_kv_heads, cache->head_dim))
    return ECHO_ERR_INVALID_ARG;
  PrefillParams P;
  P.C = *cache;
  P.q = q; P.q_stride = q_stride; P.q_start = q_start; P.seq_len = seq_len;
  P.N = N; P.B = B; P.Hq = Hq; P.G = Hq / cache->n_kv_heads;
  P.page = fast_div(cache->page_tokens); P.group = fast_div(P.G);
  if ((int64_t)N * P.G > 0x7fff0000ll) return ECHO_ERR_UNSUPPORTED;
  P.slopes = scores->slopes; P.window = scores->window;
  P.first_tok = scores->first_tok; P.prefix_len = scores->prefix_len;
  P.f = score_form(scores);
  P.out = out; P.lse = lse;
  cudaStream_t cs = (cudaStream_t)stream;
  const bool bf = cache->dtype == ECHO_BF16;
  P.prows = prefill_prows(N, P.G, bf ? PF_MAX_ROWS : PS_ROWS);
  // the units are counted in 32 bits: row tiles x (tiles of the longest sequence) x KV heads
  const double tiles = (double)N * P.G / (bf ? PF_MAX_ROWS : PS_ROWS) + B;
  const double deep = (double)cache->max_pages * cache->page_tokens / (bf ? 2 * PS_KEYS : PS_KEYS) + 4;
  if (tiles * deep * cache->n_kv_heads > 2147483647.0) return ECHO_ERR_UNSUPPORTED;
  P.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  P.rec = reinterpret_cast<int32_t *>(workspace);
  P.po = reinterpret_cast<float *>(P.rec + 8 * PF_MAX_CTAS);
  P.pml = P.po + (size_t)(bf ? PF_MAX_CTAS : 2 * PF_MAX_CTAS) * P.prows * cache->head_dim;
  if (bf) return launch_prefill_tc(P, cs);
  return cache->head_dim == 128 ? launch_simt<128>(P, cs) : launch_simt<64>(P, cs);
}
