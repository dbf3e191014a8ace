// Many-token attention over a paged cache in 8 bits.

#include "paged_prefill_tc.cuh"

namespace echo {

echo_status_t launch_prefill_q8(PrefillParams &P, cudaStream_t st) {
  return P.C.head_dim == 128 ? launch_mod<128, PT_CODES>(P, st) : launch_mod<64, PT_CODES>(P, st);
}

// The sequences that a call of a few tokens each has left.  They may be chunks of prompts: row tiles of 256 that do not
// alternate.
template <int D>
static echo_status_t launch_some(PrefillParams &P, cudaStream_t st) {
  switch ((P.f.capped ? 1 : 0) | (P.slopes || P.f.a < 0.f ? 2 : 0)) {
    case 0: return launch_tc<D, 0, false, PT_CODES, true>(P, st);
    case 1: return launch_tc<D, 1, false, PT_CODES, true>(P, st);
    case 2: return launch_tc<D, 2, false, PT_CODES, true>(P, st);
    default: return launch_tc<D, 3, false, PT_CODES, true>(P, st);
  }
}
echo_status_t launch_prefill_some(PrefillParams &P, cudaStream_t st) {
  return P.C.head_dim == 128 ? launch_some<128>(P, st) : launch_some<64>(P, st);
}

// (Rows are written out for 1024 rows a sequence or more: row tiles do not alternate.)
template <int D>
static echo_status_t launch_rows(PrefillParams &P, cudaStream_t st) {
  switch ((P.f.capped ? 1 : 0) | (P.slopes || P.f.a < 0.f ? 2 : 0)) {
    case 0: return launch_tc<D, 0, false, PT_WRITTEN>(P, st);
    case 1: return launch_tc<D, 1, false, PT_WRITTEN>(P, st);
    case 2: return launch_tc<D, 2, false, PT_WRITTEN>(P, st);
    default: return launch_tc<D, 3, false, PT_WRITTEN>(P, st);
  }
}
echo_status_t launch_prefill_rows(PrefillParams &P, cudaStream_t st) {
  return P.C.head_dim == 128 ? launch_rows<128>(P, st) : launch_rows<64>(P, st);
}

}  // namespace echo
