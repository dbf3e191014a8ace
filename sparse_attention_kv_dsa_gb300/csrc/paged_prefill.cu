// Attention of many new tokens over a paged key/value cache: prompts, chunks of prompts,
// drafted tokens.  Scores, masks and results as in the single-token call, per row.
//
// The query heads of one KV head are packed with the tokens: packed row r of a sequence is
// token r / G, head r % G of the group, so that every tile of rows reads its keys and values
// once whatever G is, and a few drafted tokens still fill a tile.
//
// bf16 runs on the tensor cores (paged_prefill_tc.cu).  Float32 (below): one CTA takes 64 packed rows of one (sequence, KV head) and walks the
// 64-token tiles that some row sees, with a running maximum and sum; 256 threads hold 4 x 4
// scores and 4 x d/16 results each.  Float32 arithmetic throughout: 4 d operations for each
// pair of query head and seen token on the FMA units.

#include "paged_prefill.cuh"

namespace echo {

// The sequence and row tile of tile index x: the x-th tile of `rows` packed rows, sequences in
// order; false past the last one.  Every thread of the block calls it (128 or more).
template <int THREADS>
__device__ __forceinline__ bool find_tile(const PrefillParams &P, int x, int rows, int &b, int &tile) {
  __shared__ int ft_warp[THREADS / 32], ft_seq, ft_tile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) ft_seq = -1;
  int base = 0;
  for (int b0 = 0; b0 < P.B; b0 += THREADS) {
    int n = 0;
    if (b0 + tid < P.B) n = (int)(((int64_t)seq_rows(P, b0 + tid).n * P.G + rows - 1) / rows);
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) ft_warp[warp] = v;
    __syncthreads();
    int end = base + v;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) end += ft_warp[w];
      base += ft_warp[w];
    }
    if (end - n <= x && x < end) {
      ft_seq = b0 + tid;
      ft_tile = x - (end - n);
    }
    __syncthreads();
    if (ft_seq >= 0) break;
  }
  b = ft_seq;
  tile = ft_tile;
  return b >= 0;
}

constexpr int PS_THREADS = 256, PS_ROWS = 64, PS_KEYS = 64;
constexpr int PS_PS = PS_KEYS + 4;                       // row stride of the probabilities

template <int D>
constexpr size_t ps_smem() {
  return sizeof(float) * ((size_t)PS_ROWS * D + (size_t)PS_KEYS * (D + 4) + (size_t)PS_ROWS * PS_PS);
}

__device__ __forceinline__ float4 ps_load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <int D>
__global__ void __launch_bounds__(PS_THREADS) paged_prefill_simt_kernel(const __grid_constant__ PrefillParams P) {
  extern __shared__ __align__(16) float ps_sm[];
  float *qs = ps_sm;                                     // [64][D]
  float *ks = qs + PS_ROWS * D;                          // [64][D + 4] keys, then [64][D] values
  float *pp = ks + PS_KEYS * (D + 4);                    // [64][68]
  __shared__ int s_pos[PS_ROWS], s_lo[PS_ROWS], s_first[PS_ROWS];
  __shared__ float s_slope[PS_ROWS];
  __shared__ int64_t s_row[PS_KEYS];
  __shared__ int s_min[3];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  int b, rt;
  if (!find_tile<PS_THREADS>(P, (int)(gridDim.x - 1 - blockIdx.x), PS_ROWS, b, rt)) return;   // long rows first
  const int kvh = blockIdx.y, G = P.G;
  const SeqRows R = seq_rows(P, b);
  const int len = paged_len(P.C, P.seq_len, b);
  if (len < R.n && tid == 0) paged_fail(P.C.status, ECHO_ERR_INVALID_ARG);
  const int pre = P.prefix_len ? min(P.prefix_len[b], len) : 0;
  const int r0 = rt * PS_ROWS, nr = (int)min((int64_t)PS_ROWS, (int64_t)R.n * G - r0);
  if (tid == 0) { s_min[0] = 0x7fffffff; s_min[1] = 0x7fffffff; s_min[2] = 0; }
  __syncthreads();
  if (tid < PS_ROWS) {
    int pos = -1, lo = 0x7fffffff, first = 0x7fffffff;   // a row that is not there sees nothing
    float sl = 0.f;
    if (tid < nr) {
      const int i = (r0 + tid) / G, g = (r0 + tid) % G;
      pos = len - R.n + i;
      first = P.first_tok ? max(P.first_tok[R.s0 + i], 0) : 0;
      lo = P.window ? max(first, pos - P.window + 1) : first;
      if (pos < 0) { first = lo = 0x7fffffff; }
      if (P.slopes) sl = P.slopes[kvh * G + g] * kPgLog2e;
    }
    s_pos[tid] = pos;
    s_lo[tid] = lo;
    s_first[tid] = first;
    s_slope[tid] = sl;
    atomicMin(&s_min[0], first);
    atomicMin(&s_min[1], lo);
    atomicMax(&s_min[2], pos + 1);
  }
  for (int i = tid; i < PS_ROWS * (D / 4); i += PS_THREADS) {
    const int r = i / (D / 4), c = i % (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nr) {
      const int t = (r0 + r) / G, g = (r0 + r) % G;
      v = ps_load4((const float *)P.q + (int64_t)(R.s0 + t) * P.q_stride + (int64_t)(kvh * G + g) * D + 4 * c);
    }
    *reinterpret_cast<float4 *>(qs + r * D + 4 * c) = v;
  }
  __syncthreads();
  const int first_min = s_min[0], lo_min = s_min[1], hi = s_min[2];
  const TileSpan span = tile_span(first_min, pre, lo_min, hi, PS_KEYS);

  constexpr int OC = D / 64;                             // float4 columns of a thread
  float o[4][OC][4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < OC; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
  }
  const float *kb = (const float *)P.C.k + (int64_t)kvh * P.C.head_stride, *vb = (const float *)P.C.v + (int64_t)kvh * P.C.head_stride;
  const int nt = span.nA + span.nB;
  for (int it = 0; it < nt; ++it) {
    const int t0 = span.tile(it) * PS_KEYS;
    __syncthreads();
    if (tid < PS_KEYS) {
      const int t = t0 + tid;
      const bool some = t < len && t >= first_min && ((t >= lo_min && t < hi) || t < pre);
      s_row[tid] = some ? paged_row(P.C, b, t) : -1;
    }
    __syncthreads();
    for (int i = tid; i < PS_KEYS * (D / 4); i += PS_THREADS) {
      const int r = i / (D / 4), c = i % (D / 4);
      const int64_t g = s_row[r];
      *reinterpret_cast<float4 *>(ks + r * (D + 4) + 4 * c) =
          g >= 0 ? ps_load4(kb + g + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    float s[4][4] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qv[i] = *reinterpret_cast<const float4 *>(qs + (ty * 4 + i) * D + c);
        kv[i] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * i) * (D + 4) + c);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(qv[i].x, kv[j].x, fmaf(qv[i].y, kv[j].y, fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, s[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i, pos = s_pos[r], lo = s_lo[r], first = s_first[r];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + tx + 16 * j;
        const bool seen = s_row[tx + 16 * j] >= 0 && t >= first && ((t <= pos && t >= lo) || t < pre);
        float a = score_log2(P.f, s[i][j]);
        if (P.slopes) a -= s_slope[r] * fabsf((float)(pos - t));
        s[i][j] = seen ? a : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float nm = fmaxf(m[i], mx), z = nm == -INFINITY ? 0.f : nm;
      const float corr = exp2f(m[i] - z);
      m[i] = nm;
      l[i] *= corr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - z);
        l[i] += p;
        pp[r * PS_PS + tx + 16 * j] = p;
      }
#pragma unroll
      for (int j = 0; j < OC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] *= corr;
    }
    __syncthreads();
    for (int i = tid; i < PS_KEYS * (D / 4); i += PS_THREADS) {
      const int r = i / (D / 4), c = i % (D / 4);
      const int64_t g = s_row[r];
      *reinterpret_cast<float4 *>(ks + r * D + 4 * c) =
          g >= 0 ? ps_load4(vb + g + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
#pragma unroll 2
    for (int t = 0; t < PS_KEYS; t += 4) {
      float4 pv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4 *>(pp + (ty * 4 + i) * PS_PS + t);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < OC; ++j) {
          const float4 vv = *reinterpret_cast<const float4 *>(ks + (t + u) * D + 64 * j + 4 * tx);
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
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    float L = l[i];
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
    if (r >= nr) continue;
    const int t = (r0 + r) / G, g = (r0 + r) % G;
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const int64_t row = (int64_t)(R.s0 + t) * P.Hq + kvh * G + g;
    float *dst = (float *)P.out + row * D + 4 * tx;
#pragma unroll
    for (int j = 0; j < OC; ++j)
      *reinterpret_cast<float4 *>(dst + 64 * j) =
          make_float4(o[i][j][0] * inv, o[i][j][1] * inv, o[i][j][2] * inv, o[i][j][3] * inv);
    if (tx == 0) P.lse[row] = L == 0.f ? -INFINITY : (m[i] + log2f(L)) * kPgLn2;
  }
}

template <int D>
static echo_status_t launch_simt(const PrefillParams &P, cudaStream_t st) {
  const int64_t tiles = ((int64_t)P.N * P.G + PS_ROWS - 1) / PS_ROWS + P.B;
  if (tiles > 0x7fffffff) return ECHO_ERR_UNSUPPORTED;
  ECHO_CUDA_OK(allow_smem<paged_prefill_simt_kernel<D>>(ps_smem<D>()));
  paged_prefill_simt_kernel<D><<<dim3((unsigned)tiles, P.C.n_kv_heads), PS_THREADS, ps_smem<D>(), st>>>(P);
  ECHO_LAUNCH_OK();
  return ECHO_OK;
}

}  // namespace echo

using namespace echo;

// bf16: two partials a CTA, of the rows of a row tile at most, and a record each; float32: none
// is needed, but the size does not ask for the type.
static int prefill_prows(int64_t N, int64_t G) { return (int)std::min<int64_t>(PF_ROWS, N * G); }

extern "C" size_t echo_paged_prefill_workspace_bytes(int32_t N, int32_t B, int32_t Hq, int32_t n_kv_heads, int32_t d) {
  if (N <= 0 || B <= 0 || Hq <= 0 || n_kv_heads <= 0 || d <= 0 || Hq % n_kv_heads) return 0;
  return (size_t)PF_MAX_CTAS * (2 * (size_t)prefill_prows(N, Hq / n_kv_heads) * (d + 2) + 8) * sizeof(float);
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
  if (cache->dtype == ECHO_BF16) {
    P.prows = prefill_prows(N, P.G);
    P.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    P.po = reinterpret_cast<float *>(workspace);
    P.pml = P.po + (size_t)2 * PF_MAX_CTAS * P.prows * cache->head_dim;
    P.rec = reinterpret_cast<int32_t *>(P.pml + (size_t)2 * PF_MAX_CTAS * P.prows * 2);
    return launch_prefill_tc(P, cs);
  }
  return cache->head_dim == 128 ? launch_simt<128>(P, cs) : launch_simt<64>(P, cs);
}
