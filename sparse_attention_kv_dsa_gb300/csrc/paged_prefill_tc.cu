// Many-token attention over a paged cache in bf16.

#include "paged_prefill_tc.cuh"

namespace echo {

echo_status_t launch_prefill_tc(PrefillParams &P, cudaStream_t st) {
  return P.C.head_dim == 128 ? launch_mod<128, PT_BF16>(P, st) : launch_mod<64, PT_BF16>(P, st);
}

}  // namespace echo
