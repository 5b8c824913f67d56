// Device helpers shared by the two kernels that read the paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sage_device.cuh"
#include "sage_paged.h"

namespace sage {

// What a sequence's rows can see, in blocks of kBlock keys: `sink` blocks from key
// 0, then the blocks from `from` on, `count` in all.
struct Span {
  int sink, from, count;
};
template <int kBlock>
__device__ __forceinline__ Span span_of(int p_lo, int p_hi, int window, int sinks) {
  Span r{0, 0, 0};
  if (p_hi < 0) return r;
  int lo = 0;
  if (window > 0 && p_lo - window + 1 > 0) lo = p_lo - window + 1;
  r.from = lo / kBlock;
  if (lo > 0) {
    const int s = min(sinks, lo);
    r.sink = min((s + kBlock - 1) / kBlock, r.from);
  }
  r.count = r.sink + p_hi / kBlock + 1 - r.from;
  return r;
}

template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// A row's reference, from which P = 2^(x - reference) is taken, moves only when a
// logit has outgrown it by 2^kLazy; any reference gives the same result.  In fp16
// the reference is 2^7 below the maximum at which it is taken: P reaches 2^15, within
// fp16's 65504, and a weight of 2^-31 of the largest is still a step of fp16.  (With
// P up to 2^8 weights of 2^-25 and less went missing in O, but not in l.)
constexpr float kLazy = 8.0f;
template <bool kBF16>
constexpr float kBelow = kBF16 ? 0.0f : 7.0f;

// The exponent of |x|, within -126..126 (zero and subnormal numbers: -126), so
// that 2^e and 2^-e are both normal; and 2^e.
__device__ __forceinline__ int exponent_of(float x) {
  const int e = static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127;
  return e < -126 ? -126 : e > 126 ? 126 : e;
}
__device__ __forceinline__ float power_of_2(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four int8 codes of a word as two fp16 pairs, exactly: the byte n + 128 under
// 0x64 is the fp16 number 1024 + n + 128.
__device__ __forceinline__ void int8_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  lo = __byte_perm(w, 0x64646464u, 0x4140);
  hi = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 bias = __floats2half2_rn(1152.0f, 1152.0f);
  __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), bias);
  __half2 b = __hsub2(*reinterpret_cast<__half2*>(&hi), bias);
  lo = *reinterpret_cast<uint32_t*>(&a);
  hi = *reinterpret_cast<uint32_t*>(&b);
}

// (v & mask) | 0x64006400 in one instruction; written out, the compiler takes two.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t masked_under(uint32_t v) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "n"(kMask), "r"(0x64006400u));
  return r;
}

// Eight codes u of four bits as numbers u - 8, exactly: pairs of nibbles j and j + 4.
// Under 0x64 a nibble is the fp16 number 1024 + u, four bits higher 1024 + 16 u.
__device__ __forceinline__ void nibbles_to_half(uint32_t w, uint32_t (&h)[4]) {
  const __half2 bias = __floats2half2_rn(-1032.0f, -1032.0f);
  const __half2 part = __floats2half2_rn(0.0625f, 0.0625f), bias16 = __floats2half2_rn(-72.0f, -72.0f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i == 0 ? w : w >> 8;
    const uint32_t lo = masked_under<0x000F000Fu>(v), hi = masked_under<0x00F000F0u>(v);
    const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&lo), bias);
    const __half2 b = __hfma2(*reinterpret_cast<const __half2*>(&hi), part, bias16);
    h[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
    h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// Asynchronous copies to shared memory of 16 or 8 bytes; `bytes` of them are read,
// the rest is zero.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;"
               :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8, %2;"
               :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
         "r"(smem_u32(bar))
      : "memory");
}

// A vector of a row that ends after `left` more elements (untouched where none
// are left), zero unless `see`.  kForm 0: all are there; 2: rows of 8-bit codes
// that start or end on 8 bytes only.
template <int kForm>
__device__ __forceinline__ void copy_part(uint32_t dst, const uint8_t* src, bool see, int left) {
  if constexpr (kForm == 2) {
    if (left > 0) copy8(dst, src, see ? 8 : 0);
    if (left > 8) copy8(dst + 8, see ? src + 8 : src, see ? 8 : 0);
  } else {
    if (kForm == 0 || left > 0) copy16(dst, src, see ? 16 : 0);
  }
}

// The page slot of a key: a shift where the page size is a power of two.
__device__ __forceinline__ int page_of(const PagedGeo& c, int key) {
  return c.page_shift >= 0 ? key >> c.page_shift : key / c.page_size;
}

}  // namespace sage
