// Geometry of the paged cache and of a batch of new tokens, shared by the
// host launchers and the kernels that write and read the cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sage_geom.h"

namespace sage {

constexpr int kKindF16 = 0, kKindBF16 = 1, kKindQ8 = 2;   // as in sage.h

struct PagedGeo {
  uint8_t* k;                // pages; elements of 2 bytes, or 1 (kKindQ8)
  uint8_t* v;
  float* k_scale;            // [num_pages][Hkv][page_size]
  const float* k_mean;       // [Hkv][Dp]
  const float* v_scale;      // [Hkv][Dp]
  int64_t num_pages;
  int64_t page_stride, token_stride, head_stride;   // elements
  int32_t Hkv, D, Dp, page_size, kind;
  int32_t page_shift;        // log2(page_size), or -1
  int32_t wide;              // every row is whole 16-byte vectors that start on 16 bytes
  const int32_t* cu_q;
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t total_q, table_stride;
  int32_t nseq, max_q, max_kv;
  uint32_t* status;
};

// Rotation and row strides of sage_rope and sage_kv_append.
struct RowsParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_out;           // sage_rope only
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, qo_tok, qo_head, ko_tok, ko_head;
  int64_t T;
  int32_t Hq, Hkv, D;        // Hq = 0: no q rows
  const void* pos;           // sage_rope only
  int32_t pos64;
  const double* inv_freq;    // NULL: no rotation
  int32_t R, interleaved;
  float mscale, sign;        // sign -1: the inverse rotation
  int32_t vec;               // 16-byte rows: base, strides and D in whole vectors
  int32_t toks;              // tokens per CTA (set by the launcher)
  PagedGeo c;                // sage_kv_append only
};

// mode 0: sage_rope; 1: append to a 16-bit cache; 2: append to a Q8 cache.
cudaError_t launch_rows(const RowsParams& p, int mode, bool bf16, int sms, cudaStream_t st);

constexpr int kArrivalBytes = 8192 - 256;

struct PagedAttnParams {
  PagedGeo c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_tok, q_head;     // elements
  int32_t Hq, group;         // group = Hq / Hkv
  uint32_t magic;            // floor(2^32 / group) + 1: divides small numbers by the group
  int32_t window, sinks;     // window 0: every earlier key
  float scale_log2;          // sm_scale * log2(e)
  int32_t q_vec;             // q rows in whole 16-byte vectors
  int32_t tensor_copies;     // the 8-bit cache's pages go by tensor copies (set by the launcher)
  int32_t min_rows, max_rows;  // rows (tokens x group) of the sequences a launch serves
  uint8_t* parts;            // split results (workspace)
  uint32_t* arrivals;        // kArrivalBytes of the workspace, zero between calls
  int32_t join_inside;       // parts joined by the kernel itself (set by the launcher)
  uint64_t timeout_ns;
};

cudaError_t launch_paged_few(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st);
size_t paged_few_bytes();
int paged_few_rows(int Dp);   // rows (new tokens x group) that one of its tiles holds
cudaError_t launch_paged_many(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st);
size_t paged_many_bytes();
bool paged_many_serves(const PagedGeo& c, int group);

#ifdef __CUDACC__
// A sequence's first row, new tokens and cached length; false (and the status
// bit) if an entry breaks the call's bounds.
__device__ __forceinline__ bool paged_seq(const PagedGeo& c, int s, int* start, int* n, int* len) {
  const int a = c.cu_q[s], b = c.cu_q[s + 1], l = c.kv_lens[s];
  if (a < 0 || b < a || b > c.total_q || b - a > c.max_q || l < 0 || l > c.max_kv) {
    atomicOr(c.status, kStatusBadSeqlens);
    return false;
  }
  *start = a;
  *n = b - a;
  *len = l;
  return true;
}

// The page of a sequence's page slot, or -1 (and the status bit) if the
// table's entry lies outside the cache.
__device__ __forceinline__ int paged_page(const PagedGeo& c, int s, int slot) {
  const int p = c.table[s * c.table_stride + slot];
  if (p < 0 || p >= c.num_pages) {
    atomicOr(c.status, kStatusBadPage);
    return -1;
  }
  return p;
}
#endif

}  // namespace sage
