// Attention of many new tokens over the 4-bit cache: the kernel's instances (a file of
// their own, so that they compile beside the others).

#include "paged_many.cuh"

namespace sage {

cudaError_t launch_paged_many_q4(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st) {
  return bf16 ? launch_many_dim<kKindQ4, true>(p, sms, st)
              : launch_many_dim<kKindQ4, false>(p, sms, st);
}

}  // namespace sage
