// Shared parts of the paged-cache calls: argument checks, page-table look-ups, the range
// of tokens that a query sees, and the base-2 form of its scores.
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"

namespace echo {

constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ host checks --
inline int paged_elem_size(int dtype) { return dtype == ECHO_F32 ? 4 : dtype == ECHO_E4M3 ? 1 : 2; }

// q8: a cache in 8 bits is wanted, and else none.
inline echo_status_t paged_check(const echo_paged_kv_t *c, bool q8 = false) {
  if (!c || !c->k || !c->v || !c->page_table || c->n_pages <= 0 || c->page_tokens <= 0 || c->n_kv_heads <= 0 ||
      c->max_pages <= 0)
    return ECHO_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return ECHO_ERR_UNSUPPORTED;
  if (q8 ? c->dtype != ECHO_E4M3 : c->dtype != ECHO_BF16 && c->dtype != ECHO_F32) return ECHO_ERR_UNSUPPORTED;
  // positions, and positions rounded up to a tile, stay below 2^31
  if ((int64_t)c->max_pages * c->page_tokens > 0x7fff0000ll) return ECHO_ERR_UNSUPPORTED;
  const int64_t es = paged_elem_size(c->dtype);
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15) return ECHO_ERR_INVALID_ARG;
  if ((c->page_stride * es | c->row_stride * es | c->head_stride * es) & 15) return ECHO_ERR_INVALID_ARG;
  return ECHO_OK;
}

inline echo_status_t paged_scales_check(const echo_paged_scales_t *s) {
  return s && s->k && s->v ? ECHO_OK : ECHO_ERR_INVALID_ARG;
}
// The type of a cache's activations.
inline int paged_act_type(int dtype) { return dtype == ECHO_F32 ? ECHO_F32 : ECHO_BF16; }

// Rows of packed heads: 16-byte aligned, a whole number of 16-byte chunks apart.
inline bool paged_rows_ok(const void *p, int64_t stride, int dtype) {
  return !((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * paged_elem_size(dtype))) & 15);
}

// Division of 0 <= t < 2^31 by a fixed d: the high word of t * (floor(2^64 / d) + 1), whose
// excess t * (1 - frac) / 2^64 stays below 1 / d.
struct FastDiv {
  uint64_t m;
  int d;
};
inline FastDiv fast_div(int d) { return {d > 1 ? ~0ull / (uint64_t)d + 1 : 0ull, d}; }

// ----------------------------------------------------------------- device parts --
__device__ __forceinline__ int div_by(const FastDiv &f, int t) {
  return f.d == 1 ? t : (int)__umul64hi((uint64_t)t, f.m);
}

__device__ __forceinline__ void paged_fail(int32_t *status, int32_t code) {
  if (status) atomicCAS(status, 0, code);
}

// Tokens of sequence b, cut to what its page-table row can hold.
__device__ __forceinline__ int paged_len(const echo_paged_kv_t &C, const int32_t *seq_len, int b) {
  const int cap = C.max_pages * C.page_tokens;
  const int n = seq_len[b];
  if (n < 0 || n > cap) paged_fail(C.status, ECHO_ERR_INVALID_ARG);
  return min(max(n, 0), cap);
}

// Offset (in values) of head 0 of token t's row, or -1 when its page-table entry is not a page.
__device__ __forceinline__ int64_t paged_row(const echo_paged_kv_t &C, int b, int t) {
  const int pg = t / C.page_tokens;
  const int32_t e = __ldg(C.page_table + (int64_t)b * C.max_pages + pg);
  if (e < 0 || e >= C.n_pages) {
    paged_fail(C.status, ECHO_ERR_PAGE);
    return -1;
  }
  return (int64_t)e * C.page_stride + (int64_t)(t - pg * C.page_tokens) * C.row_stride;
}

// Offset (in bytes) of head 0 of the exponents of token t in page e (paged_row's).
__device__ __forceinline__ int64_t paged_scale_row(const echo_paged_scales_t &X, int page_tokens, int e, int t, int pg) {
  return (int64_t)e * X.page_stride + (int64_t)(t - pg * page_tokens) * X.row_stride;
}
constexpr int kQ8MinExp = -15, kQ8MaxExp = 7;             // exponents of rows in 8 bits: code * 2^e is a float16
// The exponent that a byte holds.
__device__ __forceinline__ int q8_exp(uint32_t byte) {
  return min(max((int)byte - 127, kQ8MinExp), kQ8MaxExp);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // -126 .. 127
// The smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8): past 1.75 the sum carries into the exponent.
__device__ __forceinline__ int q8_row_exp(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 135;
  return min(max(e, kQ8MinExp), kQ8MaxExp);
}
// The power of two that brings a query's largest value into [2^13, 2^14), as float16 holds it: products
// with codes stay below 2^23, and what is 2^-30 of the largest value or more keeps its bits (eight of them, down to
// float16's step of 2^-24).  Heads below 2^-87 stay smaller.
__device__ __forceinline__ int q8_query_exp(float amax) {
  const int e = 13 + 127 - (int)(__float_as_uint(amax) >> 23);
  return amax == 0.f ? 0 : min(max(e, -114), 100);
}
// Four floats to e4m3 codes, the first lowest; to nearest even, saturating.
__device__ __forceinline__ uint32_t q8_codes(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Codes 0, 1 and codes 2, 3 of a word as float16 pairs (exact).
__device__ __forceinline__ void q8_halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 2^e, e an exponent of a row in 8 bits, as a pair of float16.
__device__ __forceinline__ uint32_t q8_half_pow(int e) {
  static_assert(kQ8MinExp == -15, "one exponent below float16's normal numbers");
  const uint32_t h = e >= -14 ? (uint32_t)(15 + e) << 10 : 1u << 9;
  return h | (h << 16);
}
__device__ __forceinline__ uint32_t q8_hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Scores in base-2 units: log2(e) * x of a raw product s = q . k.
//   no cap:  s * a             with a = scale log2(e)
//   cap:     c tanh(s a)       with a = scale / cap, c = cap log2(e)
// tanh(u) is a polynomial for small u (a few roundings of u itself) and else
// 1 - 2 / (2^(2 u log2 e) + 1), off by some 1e-7, where the approximate tanh instruction is off
// by 5e-4 of the cap.
struct ScoreForm {
  float a, c;
  int capped;
};
inline ScoreForm score_form(const echo_attn_scores_t *s) {
  ScoreForm f;
  f.capped = s->softcap > 0.f;
  f.a = f.capped ? (float)((double)s->scale / (double)s->softcap) : s->scale * kPgLog2e;
  f.c = s->softcap * kPgLog2e;
  return f;
}

// The form's factors have to be numbers that float32 holds: a finite (0 * inf is no score), c far
// enough from both ends that a product flushed to 0 below 2^-126 is nothing beside it and that c
// times a masked -inf stays one (c in the denormals reads as 0).
inline echo_status_t paged_scores_check(const echo_attn_scores_t *s) {
  if (!s || !std::isfinite(s->scale) || !std::isfinite(s->softcap) || s->window < 0) return ECHO_ERR_INVALID_ARG;
  if (s->softcap != 0.f && !(s->softcap >= 1e-30f && s->softcap <= 1e30f)) return ECHO_ERR_INVALID_ARG;
  return std::isfinite(score_form(s).a) ? ECHO_OK : ECHO_ERR_INVALID_ARG;
}

// 2^x, denormals as 0 (two units in the last place; half the cost of exp2f's full range).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tanh_ex2(float u) { return 1.f - __fdividef(2.f, ex2(2.f * kPgLog2e * u) + 1.f); }
// tanh(u) = u (1 + w (c1 + w (c2 + ...))), w = u^2 <= 1/2: minimax in relative error, found by an
// exchange of extrema; with the coefficients as float32 holds them 3.6e-8 off (at u = 0.683).
constexpr float kTanhW = 0.5f;
constexpr float kTanh1 = -0.3333311080932617f, kTanh2 = 0.13328056037425995f, kTanh3 = -0.05350292846560478f,
                kTanh4 = 0.01996474526822567f, kTanh5 = -0.005034889094531536f;
__device__ __forceinline__ float tanh_small(float u) {    // u^2 <= kTanhW
  const float w = u * u;
  return fmaf(u * w, fmaf(w, fmaf(w, fmaf(w, fmaf(w, kTanh5, kTanh4), kTanh3), kTanh2), kTanh1), u);
}
__device__ __forceinline__ float score_tanh(float u) { return u * u <= kTanhW ? tanh_small(u) : tanh_ex2(u); }
__device__ __forceinline__ float score_log2(const ScoreForm &f, float s) {
  const float u = s * f.a;
  return f.capped ? f.c * score_tanh(u) : u;
}

// Allows kernel K its dynamic shared memory: once for each device, not with every launch (the
// call costs several microseconds of host time).
template <auto K>
inline cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches K so that it may start up while the kernel before it in the stream ends; K itself
// waits for it (griddepcontrol.wait) before it reads what that kernel wrote.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_after(void (*K)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, K, args...);
}

// The tiles of `tile` tokens that hold [first, pre) or [lo, hi): tiles tA .. tA + nA - 1, then
// tB .. tB + nB - 1, in ascending order and without a tile twice.
struct TileSpan {
  int tA, nA, tB, nB;
  __device__ __forceinline__ int tile(int i) const { return i < nA ? tA + i : tB + (i - nA); }
};
__device__ __forceinline__ TileSpan tile_span(int first, int pre, int lo, int hi, int tile) {
  TileSpan s = {0, 0, 0, 0};
  int eA = 0, eB = 0;
  const bool a = first < pre, b = lo < hi;
  if (a) { s.tA = first / tile; eA = (pre + tile - 1) / tile; }
  if (b) { s.tB = lo / tile; eB = (hi + tile - 1) / tile; }
  if (a && b && s.tB <= eA) {                    // they touch: one run (lo >= first)
    s.tA = min(s.tA, s.tB);
    eA = max(eA, eB);
  } else if (b) {
    s.nB = eB - s.tB;
  }
  s.nA = a ? eA - s.tA : 0;
  return s;
}

// The many-token call's workspace: records of split row tiles (PF_MAX_CTAS of 8 int32), then partials.  Of a call
// over codes the last record, which no CTA has, tells whether some sequence has more than a few rows.
constexpr int kPgRecords = 8 * 320, kPgSomeAt = kPgRecords - 8;

// Attention of a few new tokens a sequence over a cache in 8 bits (paged_decode.cu): whether a many-token
// call is one, and the call (its arguments checked), which leaves out sequences of more than `most` packed rows
// and notes in the workspace whether there are any (not if q_start descends, which it reports).
bool few_tokens_q8(int64_t N, int64_t B, int64_t G, const echo_attn_scores_t *scores);
echo_status_t launch_few_tokens_q8(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales, const void *q, int64_t q_stride,
                                   const int32_t *q_start, const int32_t *seq_len, int32_t N, int32_t B, int32_t Hq,
                                   const echo_attn_scores_t *scores_of, int most, void *out, float *lse, void *workspace, cudaStream_t st);

}  // namespace echo
