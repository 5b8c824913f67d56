// C entry points of rotary positions, the paged cache's writer and the
// attention over it: argument checks and launches.

#include <climits>
#include <cmath>

#include "sage.h"
#include "sage_host.h"
#include "sage_paged.h"

using namespace sage;

namespace {

bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 39;
constexpr size_t kStatusBytes = 256;   // then the arrival counters
constexpr size_t kClearBytes = kStatusBytes + kArrivalBytes;
static_assert(kClearBytes == SAGE_PAGED_CLEAR_BYTES, "the header says what the caller clears");
// Mean rows of a sequence from which on the tensor-core kernel takes them all.
// Both sides measured (us, single tokens over 4000 keys beside chunks over as many):
//   heads, channels   chunks     single tokens   mean rows   two kernels   one
//   32 on 8, 128      1 x 1500   0               6000        132           123
//   32 on 8, 128      4 x 1500   16              1203        458           440
//   32 on 8, 128      4 x 400    16              323         200           179
//   32 on 8, 128      4 x 400    64              98          319           329
//   16 on 16, 80      16 x 1500  16              750         847           855
//   16 on 16, 80      4 x 1500   64              89          566           642
//   8 on 2, 64        4 x 400    4               802         74            49
//   8 on 2, 64        1 x 100    4               83          65            32
// The one kernel wins with few single tokens (about 4, or 16 with a group of 4) and
// the two with many, by a quarter at most.  The mean, which is all that the host
// knows, tells them apart only roughly: batches of many single tokens are on their
// faster side, small ones with few of them pay up to twice (the last row).
constexpr int64_t kAllMany = 512;
size_t few_bytes() { return (paged_few_bytes() + 255) / 256 * 256; }

// {token, head} strides of a (T, H, D) tensor; NULL: dense.  A dimension of
// one entry has no stride worth checking.
sage_status row_strides(const char* what, const int64_t* s, int64_t T, int64_t H, int64_t D,
                        int64_t* tok, int64_t* head) {
  *tok = H * D;
  *head = D;
  if (s == nullptr) return SAGE_OK;
  if (T > 1) *tok = s[0];
  if (H > 1) *head = s[1];
  if (*tok <= 0 || *head <= 0 || *tok >= kMaxStride || *head >= kMaxStride)
    return refuse(SAGE_ERR_UNSUPPORTED,
                  "%s strides {%lld, %lld} must be positive and below 2^39 (zero, broadcast or "
                  "negative strides are not served)",
                  what, (long long)*tok, (long long)*head);
  return SAGE_OK;
}

sage_status check_dtype(int dtype) {
  if (dtype != SAGE_F16 && dtype != SAGE_BF16)
    return refuse(SAGE_ERR_INVALID_ARG, "dtype %d is neither SAGE_F16 nor SAGE_BF16", dtype);
  return SAGE_OK;
}

sage_status check_rotation(const double* inv_freq, int64_t R, int64_t D) {
  if (inv_freq == nullptr || !on(inv_freq, 8))
    return refuse(SAGE_ERR_INVALID_ARG, "inv_freq must be an 8-byte aligned device pointer");
  if (R < 2 || R > D || R % 2 != 0)
    return refuse(SAGE_ERR_INVALID_ARG, "rotary dimension R=%lld must be even, 2..D (D=%lld)",
                  (long long)R, (long long)D);
  return SAGE_OK;
}

bool vec_rows(const void* p, int64_t tok, int64_t head) {
  return on(p, 16) && tok % 8 == 0 && head % 8 == 0;
}

sage_status paged_geo(const sage_paged_cache* cache, const sage_paged_batch* b, void* ws,
                      size_t ws_bytes, PagedGeo* g) {
  if (cache == nullptr || b == nullptr)
    return refuse(SAGE_ERR_INVALID_ARG, "cache and batch must not be null");
  const int kind = cache->kind;
  if (kind != SAGE_F16 && kind != SAGE_BF16 && kind != SAGE_Q8)
    return refuse(SAGE_ERR_INVALID_ARG, "cache kind %d is none of SAGE_F16, SAGE_BF16, SAGE_Q8",
                  kind);
  if (cache->D < 8 || cache->D > 128 || cache->D % 8 != 0)
    return refuse(SAGE_ERR_UNSUPPORTED, "a paged cache needs head_dim D=%lld in 8..128, a "
                  "multiple of 8", (long long)cache->D);
  if (cache->page_size < 16 || cache->page_size > 65536 || cache->page_size % 16 != 0)
    return refuse(SAGE_ERR_UNSUPPORTED, "page_size=%lld must be a multiple of 16, up to 65536",
                  (long long)cache->page_size);
  if (cache->Hkv < 1 || cache->Hkv > 65535 || cache->num_pages < 1 || cache->num_pages > INT_MAX)
    return refuse(SAGE_ERR_INVALID_ARG, "Hkv=%lld or num_pages=%lld out of range",
                  (long long)cache->Hkv, (long long)cache->num_pages);
  if (cache->k == nullptr || cache->v == nullptr || !on(cache->k, 16) || !on(cache->v, 16))
    return refuse(SAGE_ERR_INVALID_ARG, "cache k and v must be 16-byte aligned device pointers");
  const int64_t ps = cache->num_pages > 1 ? cache->page_stride : cache->D;
  const int64_t ts = cache->token_stride;
  const int64_t hs = cache->Hkv > 1 ? cache->head_stride : cache->D;
  if (ps < cache->D || ts < cache->D || hs < cache->D || ps >= kMaxStride || ts >= kMaxStride ||
      hs >= kMaxStride || ps % 8 != 0 || ts % 8 != 0 || hs % 8 != 0)
    return refuse(SAGE_ERR_UNSUPPORTED, "cache strides {page %lld, token %lld, head %lld} must be "
                  "multiples of 8 elements, at least D and below 2^39",
                  (long long)ps, (long long)ts, (long long)hs);
  if (static_cast<__int128>(cache->num_pages) * ps +
          static_cast<__int128>(cache->page_size) * ts + static_cast<__int128>(cache->Hkv) * hs >
      (static_cast<__int128>(1) << 60))
    return refuse(SAGE_ERR_UNSUPPORTED, "the cache's extent exceeds 2^60 elements");
  if (kind == SAGE_Q8) {
    if (cache->k_scale == nullptr || cache->k_mean == nullptr || cache->v_scale == nullptr ||
        !on(cache->k_scale, 16) || !on(cache->k_mean, 16) || !on(cache->v_scale, 16))
      return refuse(SAGE_ERR_INVALID_ARG, "a SAGE_Q8 cache needs k_scale, k_mean and v_scale, "
                    "16-byte aligned device pointers");
  }
  if (b->nseq < 0 || b->total_q < 0 || b->max_q < 0 || b->max_kv < 0 || b->table_width < 0)
    return refuse(SAGE_ERR_INVALID_ARG, "negative batch size (nseq=%lld total_q=%lld max_q=%d "
                  "max_kv=%d table_width=%lld)", (long long)b->nseq, (long long)b->total_q,
                  b->max_q, b->max_kv, (long long)b->table_width);
  if (b->nseq > (1 << 20) || b->total_q > INT_MAX)
    return refuse(SAGE_ERR_UNSUPPORTED, "more than 2^20 sequences or 2^31-1 tokens");
  if (b->table_width > INT_MAX ||
      static_cast<__int128>(b->table_width) * cache->page_size < b->max_kv)
    return refuse(SAGE_ERR_INVALID_ARG, "max_kv=%d exceeds the block table's %lld pages of %lld",
                  b->max_kv, (long long)b->table_width, (long long)cache->page_size);
  if (b->nseq > 0 && b->total_q > 0) {
    if (b->cu_q == nullptr || b->kv_lens == nullptr || !on(b->cu_q, 4) || !on(b->kv_lens, 4) ||
        (b->max_kv > 0 && (b->block_table == nullptr || !on(b->block_table, 4))))
      return refuse(SAGE_ERR_INVALID_ARG,
                    "cu_q, kv_lens and block_table must be aligned device pointers");
    if (b->nseq > 1 && (b->table_stride < b->table_width || b->table_stride >= kMaxStride))
      return refuse(SAGE_ERR_INVALID_ARG, "table_stride=%lld is below table_width=%lld or beyond "
                    "2^39", (long long)b->table_stride, (long long)b->table_width);
  }
  if (ws == nullptr || !on(ws, 256))
    return refuse(SAGE_ERR_WORKSPACE, "workspace must be a 256-byte aligned device pointer");
  if (ws_bytes < sage_workspace_bytes_paged())
    return refuse(SAGE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes,
                  sage_workspace_bytes_paged());
  *g = PagedGeo{};
  g->k = static_cast<uint8_t*>(cache->k);
  g->v = static_cast<uint8_t*>(cache->v);
  g->k_scale = cache->k_scale;
  g->k_mean = cache->k_mean;
  g->v_scale = cache->v_scale;
  g->num_pages = cache->num_pages;
  g->page_stride = ps;
  g->token_stride = ts;
  g->head_stride = hs;
  g->Hkv = static_cast<int32_t>(cache->Hkv);
  g->D = static_cast<int32_t>(cache->D);
  g->Dp = cache->D <= 64 ? 64 : 128;
  g->page_size = static_cast<int32_t>(cache->page_size);
  g->kind = kind;
  g->page_shift = (g->page_size & (g->page_size - 1)) == 0 ? __builtin_ctz(g->page_size) : -1;
  // strides are multiples of 8 elements: 16 bytes, or 8 of an 8-bit cache
  const int64_t vec = kind == SAGE_Q8 ? 16 : 8;
  g->wide = cache->D % vec == 0 && ps % vec == 0 && ts % vec == 0 && hs % vec == 0;
  g->cu_q = b->cu_q;
  g->kv_lens = b->kv_lens;
  g->table = b->block_table;
  g->total_q = b->total_q;
  g->table_stride = b->nseq > 1 ? b->table_stride : 0;
  g->nseq = static_cast<int32_t>(b->nseq);
  g->max_q = b->max_q;
  g->max_kv = b->max_kv;
  g->status = static_cast<uint32_t*>(ws);
  return SAGE_OK;
}

}  // namespace

extern "C" {

size_t sage_workspace_bytes_paged(void) {
  return kClearBytes + few_bytes() + paged_many_bytes();
}

sage_status sage_rope(const void* q, const void* k, void* q_out, void* k_out, int dtype, int64_t T,
                      int64_t Hq, int64_t Hkv, int64_t D, const int64_t* q_strides,
                      const int64_t* k_strides, const int64_t* qo_strides,
                      const int64_t* ko_strides, const void* pos, int pos_bits,
                      const double* inv_freq, int64_t R, int interleaved, float mscale,
                      int inverse, sage_stream_t stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  if (D < 1 || D > 128)
    return refuse(SAGE_ERR_UNSUPPORTED, "head_dim D=%lld outside 1..128", (long long)D);
  if (k == nullptr && Hkv != 0)
    return refuse(SAGE_ERR_INVALID_ARG, "k is null but Hkv=%lld", (long long)Hkv);
  if (T < 0 || Hq < 1 || Hkv < 0 || Hq > 65535 || Hkv > 65535)
    return refuse(SAGE_ERR_INVALID_ARG, "T=%lld, Hq=%lld or Hkv=%lld out of range", (long long)T,
                  (long long)Hq, (long long)Hkv);
  if (T == 0) return succeeded();
  if (q == nullptr || q_out == nullptr || (Hkv > 0 && k_out == nullptr) || !on(q, 2) ||
      !on(k, 2) || !on(q_out, 2) || !on(k_out, 2))
    return refuse(SAGE_ERR_INVALID_ARG, "q, k and their outputs must be 2-byte aligned device "
                  "pointers");
  if (pos_bits != 32 && pos_bits != 64)
    return refuse(SAGE_ERR_INVALID_ARG, "pos_bits=%d is neither 32 nor 64", pos_bits);
  if (pos == nullptr || !on(pos, pos_bits / 8))
    return refuse(SAGE_ERR_INVALID_ARG, "pos must be an aligned device pointer");
  if ((s = check_rotation(inv_freq, R, D)) != SAGE_OK) return s;
  RowsParams p{};
  if ((s = row_strides("q", q_strides, T, Hq, D, &p.q_tok, &p.q_head)) != SAGE_OK) return s;
  if ((s = row_strides("q_out", qo_strides, T, Hq, D, &p.qo_tok, &p.qo_head)) != SAGE_OK) return s;
  if (Hkv > 0) {
    if ((s = row_strides("k", k_strides, T, Hkv, D, &p.k_tok, &p.k_head)) != SAGE_OK) return s;
    if ((s = row_strides("k_out", ko_strides, T, Hkv, D, &p.ko_tok, &p.ko_head)) != SAGE_OK)
      return s;
  }
  if ((q == q_out && (p.q_tok != p.qo_tok || p.q_head != p.qo_head)) ||
      (Hkv > 0 && k == k_out && (p.k_tok != p.ko_tok || p.k_head != p.ko_head)))
    return refuse(SAGE_ERR_INVALID_ARG, "an output in place needs its input's strides");
  int sms = 0;
  if ((s = require_device(&sms)) != SAGE_OK) return s;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.T = T;
  p.Hq = static_cast<int32_t>(Hq);
  p.Hkv = static_cast<int32_t>(Hkv);
  p.D = static_cast<int32_t>(D);
  p.pos = pos;
  p.pos64 = pos_bits == 64;
  p.inv_freq = inv_freq;
  p.R = static_cast<int32_t>(R);
  p.interleaved = interleaved ? 1 : 0;
  p.mscale = mscale;
  p.sign = inverse ? -1.0f : 1.0f;
  p.vec = D % 8 == 0 && vec_rows(q, p.q_tok, p.q_head) && vec_rows(q_out, p.qo_tok, p.qo_head) &&
          (Hkv == 0 || (vec_rows(k, p.k_tok, p.k_head) && vec_rows(k_out, p.ko_tok, p.ko_head)));
  const cudaError_t e = launch_rows(p, 0, dtype == SAGE_BF16, sms,
                                    reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? succeeded() : cuda_refused(e, "rotary launch");
}

sage_status sage_kv_append(const sage_paged_cache* cache, const sage_paged_batch* batch,
                           const void* k, const void* v, const void* q, void* q_out, int dtype,
                           int64_t Hq, const int64_t* k_strides, const int64_t* v_strides,
                           const int64_t* q_strides, const int64_t* qo_strides,
                           const double* inv_freq, int64_t R, int interleaved, float mscale,
                           void* ws, size_t ws_bytes, sage_stream_t stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  RowsParams p{};
  if ((s = paged_geo(cache, batch, ws, ws_bytes, &p.c)) != SAGE_OK) return s;
  if (cache->kind != SAGE_Q8 && cache->kind != dtype)
    return refuse(SAGE_ERR_INVALID_ARG, "dtype %d differs from the cache's kind %d", dtype,
                  cache->kind);
  const int64_t T = batch->total_q, Hkv = cache->Hkv, D = cache->D;
  if (q != nullptr && inv_freq == nullptr)
    return refuse(SAGE_ERR_INVALID_ARG, "q is given without inv_freq: there is nothing to do");
  if (q != nullptr && (Hq < 1 || Hq > 65535))
    return refuse(SAGE_ERR_INVALID_ARG, "Hq=%lld out of range", (long long)Hq);
  if (inv_freq != nullptr && (s = check_rotation(inv_freq, R, D)) != SAGE_OK) return s;
  if (T == 0 || batch->nseq == 0) return succeeded();
  if (k == nullptr || v == nullptr || !on(k, 2) || !on(v, 2) ||
      (q != nullptr && (!on(q, 2) || q_out == nullptr || !on(q_out, 2))))
    return refuse(SAGE_ERR_INVALID_ARG, "k, v (and q with q_out) must be 2-byte aligned device "
                  "pointers");
  if ((s = row_strides("k", k_strides, T, Hkv, D, &p.k_tok, &p.k_head)) != SAGE_OK) return s;
  if ((s = row_strides("v", v_strides, T, Hkv, D, &p.v_tok, &p.v_head)) != SAGE_OK) return s;
  if (q != nullptr) {
    if ((s = row_strides("q", q_strides, T, Hq, D, &p.q_tok, &p.q_head)) != SAGE_OK) return s;
    if ((s = row_strides("q_out", qo_strides, T, Hq, D, &p.qo_tok, &p.qo_head)) != SAGE_OK)
      return s;
    if (q == q_out && (p.q_tok != p.qo_tok || p.q_head != p.qo_head))
      return refuse(SAGE_ERR_INVALID_ARG, "an output in place needs its input's strides");
  }
  int sms = 0;
  if ((s = require_device(&sms)) != SAGE_OK) return s;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.T = T;
  p.Hq = q != nullptr ? static_cast<int32_t>(Hq) : 0;
  p.Hkv = static_cast<int32_t>(Hkv);
  p.D = static_cast<int32_t>(D);
  p.inv_freq = inv_freq;
  p.R = inv_freq != nullptr ? static_cast<int32_t>(R) : 0;
  p.interleaved = interleaved ? 1 : 0;
  p.mscale = mscale;
  p.sign = 1.0f;
  p.vec = vec_rows(k, p.k_tok, p.k_head) && vec_rows(v, p.v_tok, p.v_head) &&
          (q == nullptr ||
           (vec_rows(q, p.q_tok, p.q_head) && vec_rows(q_out, p.qo_tok, p.qo_head)));
  const cudaError_t e = launch_rows(p, cache->kind == SAGE_Q8 ? 2 : 1, dtype == SAGE_BF16, sms,
                                    reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? succeeded() : cuda_refused(e, "cache append launch");
}

sage_status sage_attn_paged(const sage_paged_cache* cache, const sage_paged_batch* batch,
                            const void* q, void* out, float* lse, int dtype, int64_t Hq,
                            const int64_t* q_strides, int64_t window, int64_t sinks,
                            float sm_scale, void* ws, size_t ws_bytes, sage_stream_t stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  PagedAttnParams p{};
  if ((s = paged_geo(cache, batch, ws, ws_bytes, &p.c)) != SAGE_OK) return s;
  if (cache->kind != SAGE_Q8 && cache->kind != dtype)
    return refuse(SAGE_ERR_INVALID_ARG, "dtype %d differs from the cache's kind %d", dtype,
                  cache->kind);
  if (Hq < 1 || Hq > 65535 || Hq % cache->Hkv != 0)
    return refuse(SAGE_ERR_INVALID_ARG, "Hq=%lld must be a positive multiple of Hkv=%lld",
                  (long long)Hq, (long long)cache->Hkv);
  if (window < 0 || sinks < 0)
    return refuse(SAGE_ERR_INVALID_ARG, "window=%lld and sinks=%lld must not be negative",
                  (long long)window, (long long)sinks);
  if (std::isnan(sm_scale) || std::isinf(sm_scale))
    return refuse(SAGE_ERR_INVALID_ARG, "sm_scale must be finite");
  const int64_t T = batch->total_q, D = cache->D;
  if (T == 0 || batch->nseq == 0 || batch->max_q == 0) return succeeded();
  if (static_cast<int64_t>(batch->max_q) * (Hq / cache->Hkv) > INT_MAX / 2)
    return refuse(SAGE_ERR_UNSUPPORTED, "max_q=%d times %lld query heads per kv head exceeds 2^30",
                  batch->max_q, (long long)(Hq / cache->Hkv));
  if (q == nullptr || !on(q, 2) || out == nullptr || !on(out, 16))
    return refuse(SAGE_ERR_INVALID_ARG,
                  "q must be a 2-byte and out a 16-byte aligned device pointer");
  if (lse != nullptr && !on(lse, 4))
    return refuse(SAGE_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if ((s = row_strides("q", q_strides, T, Hq, D, &p.q_tok, &p.q_head)) != SAGE_OK) return s;
  int sms = 0;
  if ((s = require_device(&sms)) != SAGE_OK) return s;
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.Hq = static_cast<int32_t>(Hq);
  p.group = static_cast<int32_t>(Hq / cache->Hkv);
  p.magic = static_cast<uint32_t>((uint64_t(1) << 32) / static_cast<uint64_t>(p.group) + 1);
  // a window as long as the longest sequence hides nothing
  p.window = window >= batch->max_kv ? 0 : static_cast<int32_t>(window);
  p.sinks = p.window == 0 ? 0 : static_cast<int32_t>(sinks < batch->max_kv ? sinks : batch->max_kv);
  p.scale_log2 = (sm_scale > 0.0f ? sm_scale : 1.0f / sqrtf(static_cast<float>(D))) *
                 1.44269504088896340736f;
  p.q_vec = vec_rows(q, p.q_tok, p.q_head);
  p.timeout_ns = device_wait_ns();
  uint8_t* parts = static_cast<uint8_t*>(ws) + kClearBytes;
  p.arrivals = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == SAGE_BF16;
  // Sequences whose rows (new tokens times the group) fit one tile of the kernel
  // for few rows go there, longer ones to the tensor-core kernel, each launch
  // skipping the other's; batches of long sequences run as the latter alone.
  const int few = paged_few_rows(p.c.Dp);
  const int64_t most = static_cast<int64_t>(batch->max_q) * p.group;
  const bool many = most > few && paged_many_serves(p.c, p.group);
  const bool all = many && T * p.group >= kAllMany * batch->nseq;
  cudaError_t e = cudaSuccess;
  if (!all) {
    p.min_rows = 0;
    p.max_rows = many ? few : INT_MAX;
    p.parts = parts;
    e = launch_paged_few(p, bf16, sms, st);
  }
  if (e == cudaSuccess && many) {
    p.min_rows = all ? 0 : few + 1;
    p.max_rows = INT_MAX;
    p.parts = parts + few_bytes();
    e = launch_paged_many(p, bf16, sms, st);
  }
  return e == cudaSuccess ? succeeded() : cuda_refused(e, "paged attention launch");
}

}  // extern "C"
