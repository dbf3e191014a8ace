// Parameters shared by the kernels of the many-token paged attention.
#pragma once

#include "paged.cuh"

namespace echo {

struct PrefillParams {
  echo_paged_kv_t C;
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

constexpr int PF_MAX_CTAS = 160;     // partial slots: two a CTA
constexpr int PF_ROWS = 256;         // packed rows of a row tile of the tensor-core kernel
constexpr int PF_MAX_B = 4096;       // sequences of a call

echo_status_t launch_prefill_tc(PrefillParams &P, cudaStream_t st);

}  // namespace echo
