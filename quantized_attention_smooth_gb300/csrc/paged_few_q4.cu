// Attention of few new tokens over the 4-bit cache: the kernel's instances (a file of
// their own, so that they compile beside the others).

#include "paged_few.cuh"

namespace sage {

bool paged_maps4(const PagedGeo& c, int rows, CUtensorMap* codes, CUtensorMap* scales) {
  const uint64_t row = 16 * ((static_cast<uint64_t>(c.D) + 31) / 32);     // bytes of a row
  const uint64_t words = static_cast<uint64_t>(c.Dp) / 64;                // of a row's scales
  const uint64_t slots = static_cast<uint64_t>(c.page_size), heads = static_cast<uint64_t>(c.Hkv),
                 pages = static_cast<uint64_t>(c.num_pages);
  const uint64_t dims[4] = {row, slots, heads, pages};
  const uint64_t strides[3] = {static_cast<uint64_t>(c.token_stride),
                               static_cast<uint64_t>(c.head_stride),
                               static_cast<uint64_t>(c.page_stride)};
  const uint32_t box[4] = {static_cast<uint32_t>(c.Dp) / 2, static_cast<uint32_t>(rows), 1, 1};
  // all of a head's scales in a page are one row
  const uint64_t sdims[4] = {slots * words, 1, heads, pages};
  const uint64_t sstrides[3] = {slots * words * 4, slots * words * 4, slots * words * 4 * heads};
  const uint32_t sbox[4] = {static_cast<uint32_t>(rows * words), 1, 1, 1};
  // rows of 64 or 32 bytes, turned so that eight of one vector hit every bank once
  const CUtensorMapSwizzle turn =
      c.Dp == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  if (!encode_tiled(&codes[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.k, dims, strides, box, turn) ||
      !encode_tiled(&codes[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.v, dims, strides, box, turn))
    return false;
  return scales == nullptr ||
         (encode_tiled(&scales[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, c.k_groups, sdims, sstrides,
                       sbox, CU_TENSOR_MAP_SWIZZLE_NONE) &&
          encode_tiled(&scales[1], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, c.v_groups, sdims, sstrides,
                       sbox, CU_TENSOR_MAP_SWIZZLE_NONE));
}

cudaError_t launch_paged_few_q4(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st) {
  return bf16 ? launch_kind<kKindQ4, true>(p, sms, st) : launch_kind<kKindQ4, false>(p, sms, st);
}

}  // namespace sage
