// Attention of few new tokens over caches of 16 and 8 bits: the kernel's instances.

#include "paged_few.cuh"

namespace sage {

int paged_few_rows(int Dp) { return Dp == 64 ? 32 : 16; }

size_t paged_few_bytes() { return 2 * static_cast<size_t>(kMaxCtas) * kPartBytes; }

cudaError_t launch_paged_few(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st) {
  if (p.c.kind == kKindQ4) return launch_paged_few_q4(p, bf16, sms, st);
  if (p.c.kind == kKindQ8)
    return bf16 ? launch_kind<kKindQ8, true>(p, sms, st) : launch_kind<kKindQ8, false>(p, sms, st);
  return bf16 ? launch_kind<kKindBF16, true>(p, sms, st)
              : launch_kind<kKindF16, false>(p, sms, st);
}

}  // namespace sage
