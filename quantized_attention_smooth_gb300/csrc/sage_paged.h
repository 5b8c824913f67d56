// Geometry of the paged cache and of a batch of new tokens, shared by the
// host launchers and the kernels that write and read the cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sage_geom.h"

namespace sage {

constexpr int kKindF16 = 0, kKindBF16 = 1, kKindQ8 = 2,   // as in sage.h
              kKindQ4 = 3;

struct PagedGeo {
  uint8_t* k;                // pages; elements of 2 bytes, or 1 (kKindQ8; kKindQ4: two codes)
  uint8_t* v;
  float* k_scale;            // [num_pages][Hkv][page_size], kKindQ8
  uint16_t* k_groups;        // [num_pages][Hkv][page_size][Dp/32] fp16, kKindQ4
  uint16_t* v_groups;
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
  const void* pos;           // sage_rope, and rotations at given positions
  int32_t pos64;
  int32_t naxes;             // 0: one position a token, of pos (sage_rope) or the cache's place
  const double* inv_freq;    // NULL: no rotation
  int32_t R, interleaved;
  float mscale, sign;        // sign -1: the inverse rotation
  int32_t vec;               // 16-byte rows: base, strides and D in whole vectors
  int32_t toks;              // tokens per CTA (set by the launcher)
  PagedGeo c;                // sage_kv_append only
  // behind the rest: what every call reads stays together
  int64_t axis_stride;       // elements between the axes' positions
  const uint8_t* axis_of;    // each pair's axis; NULL: the first
};

// mode 0: sage_rope; 1: append to a 16-bit cache; 2, 3: append to a Q8 or Q4 cache.
cudaError_t launch_rows(const RowsParams& p, int mode, bool bf16, int sms, cudaStream_t st);

// sage_kv_gather: k_out and v_out with their strides in k and v's fields of RowsParams.
cudaError_t launch_gather(const RowsParams& p, bool bf16, int sms, cudaStream_t st);

// A pool's tables and a step's (sage_paged_step, sage_paged_trim).
struct PoolParams {
  int32_t* free_pages;
  int32_t* left;
  int32_t* table;
  int32_t* lens;
  uint32_t* marks;
  int64_t table_stride, width;         // of the pool's table
  int32_t num_pages, page_size, max_requests, n;
  int32_t page_shift;                  // log2(page_size), or -1
  const int32_t* requests;
  const int32_t* new_lens;             // trim: lengths to keep, or NULL
  int32_t* cu_q;                       // step only, down to max_kv
  int32_t* kv_lens;
  int32_t* block_table;
  int64_t* positions;
  int64_t* slots;
  int32_t* denied;
  int64_t rows, plan_stride;
  int32_t plan_width, max_q, max_kv;
  int4* seqs;                          // workspace: one per sequence
  uint32_t* status;
};
constexpr int kMaxStepSeqs = 65536;
cudaError_t launch_paged_step(const PoolParams& p, cudaStream_t st);
cudaError_t launch_paged_trim(const PoolParams& p, cudaStream_t st);

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
  int32_t team;              // CTAs that read neighbouring heads side by side (likewise)
  uint64_t timeout_ns;
};

cudaError_t launch_paged_few(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st);
// Tensor maps of a 4-bit cache in boxes of `rows` slots: codes of K and V, and their scales
// (NULL: none).
bool paged_maps4(const PagedGeo& c, int rows, CUtensorMap* codes, CUtensorMap* scales);
cudaError_t launch_paged_few_q4(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st);
size_t paged_few_bytes();
int paged_few_rows(int Dp);   // rows (new tokens x group) that one of its tiles holds
cudaError_t launch_paged_many(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st);
cudaError_t launch_paged_many_q4(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st);
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
