// Attention of many new tokens over caches of 16 and 8 bits: the kernel's instances.

#include "paged_many.cuh"

namespace sage {

size_t paged_many_bytes() { return 2 * static_cast<size_t>(kMaxManyCtas) * kManyPartBytes; }

// 16-bit pages are copied as boxes of whole pages or 128 slots, by tensor maps;
// codes need not be.
bool paged_many_serves(const PagedGeo& c, int group) {
  if (group > 16384) return false;
  return c.kind == kKindQ8 || c.kind == kKindQ4 || page_boxes(c);
}

cudaError_t launch_paged_many(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st) {
  if (p.c.kind == kKindQ4) return launch_paged_many_q4(p, bf16, sms, st);
  if (p.c.kind == kKindQ8)
    return bf16 ? launch_many_dim<kKindQ8, true>(p, sms, st)
                : launch_many_dim<kKindQ8, false>(p, sms, st);
  return bf16 ? launch_many_dim<kKindBF16, true>(p, sms, st)
              : launch_many_dim<kKindF16, false>(p, sms, st);
}

}  // namespace sage
