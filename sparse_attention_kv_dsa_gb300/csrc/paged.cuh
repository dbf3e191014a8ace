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
inline int paged_elem_size(int dtype) { return dtype == ECHO_F32 ? 4 : 2; }

inline echo_status_t paged_check(const echo_paged_kv_t *c) {
  if (!c || !c->k || !c->v || !c->page_table || c->n_pages <= 0 || c->page_tokens <= 0 || c->n_kv_heads <= 0 ||
      c->max_pages <= 0)
    return ECHO_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || (c->dtype != ECHO_BF16 && c->dtype != ECHO_F32))
    return ECHO_ERR_UNSUPPORTED;
  // positions, and positions rounded up to a tile, stay below 2^31
  if ((int64_t)c->max_pages * c->page_tokens > 0x7fff0000ll) return ECHO_ERR_UNSUPPORTED;
  const int64_t es = paged_elem_size(c->dtype);
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15) return ECHO_ERR_INVALID_ARG;
  if ((c->page_stride * es | c->row_stride * es | c->head_stride * es) & 15) return ECHO_ERR_INVALID_ARG;
  return ECHO_OK;
}

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
__device__ __forceinline__ float score_tanh(float u) {
  const float w = u * u;
  if (!(w <= kTanhW)) return tanh_ex2(u);
  return fmaf(u * w, fmaf(w, fmaf(w, fmaf(w, fmaf(w, kTanh5, kTanh4), kTanh3), kTanh2), kTanh1), u);
}
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
inline cudaError_t launch_after(void (*K)(KArgs...), dim3 grid, dim3 block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
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

}  // namespace echo
