// Append of new tokens to a paged key/value cache with the rotation of their positions.
//
// For a row at position p, pair j of the first r values of every query and key head:
//   a' = a cos(p, j) - b sin(p, j),  b' = b cos(p, j) + a sin(p, j),
// pairs (j, j + r/2) or (2j, 2j + 1); keys and values go to the page row of token p,
// queries to q_out.  Each value is read and written once and costs three operations, so the
// call is bound by HBM for prompts and by the latency of one launch and of its dependent
// look-ups (sequence, length, page) for single tokens.
//
// One CTA takes one row.  A thread handles one pair of 16-byte chunks, the same pair in
// every head that it visits, so its cosines and sines stay in registers; with half-split
// pairs the two chunks are the two halves of the pairs, otherwise they are neighbours.
//
// Measured on a GB300: 8512 bf16 rows of 64 + 8 + 8 heads of 128 (353 MB) 58 us, 6.1 TB/s, 89 %
// of the copy rate (CTAs of 256 threads: 67 us); 1568 float32 rows of 12 + 4 + 4 heads of 64
// (16 MB) 11.5 us and 8 single tokens 10.5 us, which are the caller's: a call in a captured graph
// takes 4.8 and 3.4 us.

#include "paged.cuh"

namespace echo {

constexpr int PA_THREADS = 128;

struct AppendParams {
  echo_paged_kv_t C;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  void *q_out;
  const int32_t *q_start, *seq_len;
  int N, B, Hq;
  const float *cos_sin;
  int max_pos, rot, interleaved;
};

template <typename T>
struct Chunk;                                     // 16 bytes as floats
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4 &u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T>
__global__ void __launch_bounds__(PA_THREADS) paged_append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int CN = Chunk<T>::N;
  const int n = blockIdx.x, tid = threadIdx.x;
  const echo_paged_kv_t &C = P.C;
  const int d = C.head_dim, Hkv = C.n_kv_heads;
  // the row's sequence: entries q_start[1..B] not above n
  int b = n, i = 0, nb = 1;
  if (P.q_start) {
    int cnt = 0;
    for (int base = 1; base <= P.B; base += PA_THREADS) {
      const int j = base + tid;
      cnt += __syncthreads_count(j <= P.B && P.q_start[j] <= n);
    }
    if (cnt >= P.B) return;                       // behind the last sequence
    b = cnt;
    const int s0 = min(max(P.q_start[b], 0), P.N), s1 = min(max(P.q_start[b + 1], 0), P.N);
    i = n - s0;
    nb = s1 - s0;
    if (i < 0) return;
  }
  const int64_t cap = (int64_t)C.max_pages * C.page_tokens;
  const int64_t pos = (int64_t)P.seq_len[b] - nb + i;
  if (pos < 0 || pos >= cap || (P.rot && pos >= P.max_pos)) {
    if (tid == 0) paged_fail(C.status, ECHO_ERR_INVALID_ARG);
    return;
  }
  const int64_t row = paged_row(C, b, (int)pos);

  // this thread's pair of chunks
  const int U = d / (2 * CN), u = tid % U, h0 = tid / U, hstep = PA_THREADS / U;
  const int rc = P.rot / CN;                      // rotated chunks of a head
  int ca = 2 * u, cb = 2 * u + 1;
  if (!P.interleaved && u < rc / 2) { ca = u; cb = u + rc / 2; }
  const bool turn = ca < rc;
  float cs[CN], sn[CN];                           // of the CN pairs of the two chunks
  if (turn) {
    // half-split: pairs ca*CN ..; neighbours: pairs ca*CN/2 .. (both chunks, CN pairs in all)
    const float *t = P.cos_sin + pos * P.rot + (P.interleaved ? ca * (CN / 2) : ca * CN);
#pragma unroll
    for (int e = 0; e < CN; ++e) {
      cs[e] = __ldg(t + e);
      sn[e] = __ldg(t + P.rot / 2 + e);
    }
  }
  const int H = P.Hq + 2 * Hkv;
  for (int h = h0; h < H; h += hstep) {
    const T *src;
    T *dst;
    bool rotate = turn;
    if (h < P.Hq) {
      src = (const T *)P.q + (int64_t)n * P.q_stride + (int64_t)h * d;
      dst = (T *)P.q_out + ((int64_t)n * P.Hq + h) * d;
    } else if (h < P.Hq + Hkv) {
      if (row < 0) continue;
      src = (const T *)P.k + (int64_t)n * P.k_stride + (int64_t)(h - P.Hq) * d;
      dst = (T *)C.k + row + (int64_t)(h - P.Hq) * C.head_stride;
    } else {
      if (row < 0) continue;
      src = (const T *)P.v + (int64_t)n * P.v_stride + (int64_t)(h - P.Hq - Hkv) * d;
      dst = (T *)C.v + row + (int64_t)(h - P.Hq - Hkv) * C.head_stride;
      rotate = false;
    }
    uint4 a = reinterpret_cast<const uint4 *>(src)[ca], c = reinterpret_cast<const uint4 *>(src)[cb];
    if (rotate) {
      float x[CN], y[CN];
      Chunk<T>::get(a, x);
      Chunk<T>::get(c, y);
      if (P.interleaved) {
#pragma unroll
        for (int e = 0; e < CN; e += 2) {
          const float x0 = x[e], x1 = x[e + 1], y0 = y[e], y1 = y[e + 1];
          x[e] = x0 * cs[e / 2] - x1 * sn[e / 2];
          x[e + 1] = x1 * cs[e / 2] + x0 * sn[e / 2];
          y[e] = y0 * cs[CN / 2 + e / 2] - y1 * sn[CN / 2 + e / 2];
          y[e + 1] = y1 * cs[CN / 2 + e / 2] + y0 * sn[CN / 2 + e / 2];
        }
      } else {
#pragma unroll
        for (int e = 0; e < CN; ++e) {
          const float x0 = x[e], y0 = y[e];
          x[e] = x0 * cs[e] - y0 * sn[e];
          y[e] = y0 * cs[e] + x0 * sn[e];
        }
      }
      a = Chunk<T>::put(x);
      c = Chunk<T>::put(y);
    }
    reinterpret_cast<uint4 *>(dst)[ca] = a;
    reinterpret_cast<uint4 *>(dst)[cb] = c;
  }
}

}  // namespace echo

using namespace echo;

extern "C" void echo_paged_struct_sizes(size_t out[2]) {
  out[0] = sizeof(echo_paged_kv_t);
  out[1] = sizeof(echo_attn_scores_t);
}

extern "C" echo_status_t echo_paged_append(const echo_paged_kv_t *cache, const void *q, int64_t q_stride,
                                           const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                           void *q_out, const int32_t *q_start, const int32_t *seq_len, int32_t N,
                                           int32_t B, int32_t Hq, const float *cos_sin, int32_t max_pos,
                                           int32_t rot_dim, int32_t interleaved, echo_stream_t stream) {
  const echo_status_t st = paged_check(cache);
  if (st != ECHO_OK) return st;
  if (!k || !v || !seq_len || N <= 0 || B <= 0 || Hq < 0 || rot_dim < 0) return ECHO_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (q != nullptr) != (Hq > 0)) return ECHO_ERR_INVALID_ARG;
  if (!q_start && N != B) return ECHO_ERR_INVALID_ARG;
  if (rot_dim && (!cos_sin || max_pos <= 0)) return ECHO_ERR_INVALID_ARG;
  if (rot_dim % 16 || rot_dim > cache->head_dim) return ECHO_ERR_UNSUPPORTED;
  if (!paged_rows_ok(k, k_stride, cache->dtype) || !paged_rows_ok(v, v_stride, cache->dtype) ||
      (q && (!paged_rows_ok(q, q_stride, cache->dtype) || !paged_rows_ok(q_out, 0, cache->dtype))))
    return ECHO_ERR_INVALID_ARG;
  AppendParams P;
  P.C = *cache;
  P.q = q; P.k = k; P.v = v;
  P.q_stride = q_stride; P.k_stride = k_stride; P.v_stride = v_stride;
  P.q_out = q_out;
  P.q_start = q_start; P.seq_len = seq_len;
  P.N = N; P.B = B; P.Hq = Hq;
  P.cos_sin = cos_sin; P.max_pos = max_pos; P.rot = rot_dim; P.interleaved = interleaved != 0;
  if (cache->dtype == ECHO_BF16)
    paged_append_kernel<__nv_bfloat16><<<N, PA_THREADS, 0, (cudaStream_t)stream>>>(P);
  else
    paged_append_kernel<float><<<N, PA_THREADS, 0, (cudaStream_t)stream>>>(P);
  ECHO_LAUNCH_OK();
  return ECHO_OK;
}
