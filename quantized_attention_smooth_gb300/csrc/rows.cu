// Rotary positions and the paged cache's writer: one kernel over (token, head)
// rows.
//
//   rotation   y1 = g (x1 cos a - x2 sin a),  y2 = g (x2 cos a + x1 sin a),
//              a = pos * inv_freq[i] for channel pair i, in fp32
//   16-bit     the row rounded once to the cache's type
//   Q8         x = k - mean;  s = max|x| / 127;  code = rint(x * (127 / max|x|))
//              V code = e4m3(v * (1 / v_scale)), saturating
//              (each one IEEE fp32 operation, as in the quantisation prologue)
//
// The angle of a far position needs more bits than fp32 has: pos * inv_freq is
// formed in turns as a 64-bit fixed-point fraction, F = frac(inv_freq / 2 pi)
// * 2^64, whose product with the position modulo 2^64 is exact.  F itself is off by
// the roundings of 1 / (2 pi) and of one double multiplication (2^-53 of the turns
// each) and by its own last bit, which the position multiplies: the phase is off by
// |pos| (inv_freq 2^-52 + 2^-62) rad, less than the 2^-24 of the cut to fp32 while
// |pos inv_freq| < 2^28 and |pos| < 2^38.
//
// The work is bound by memory: each row is read once and written once.  In the
// first kernel a row belongs to 8 or 16 lanes of 8 channels (one 16-byte vector
// each); the half layout's partner channels come from another lane by a shuffle.
// A group of lanes keeps its head for all tokens of the CTA, so the per-channel
// means and scales are loaded once.  The second kernel gives a lane two vectors.
// cos and sin of a CTA's tokens are computed once into shared memory and serve
// every head.  Measured (GB300, back to back in a graph): interleaved rope of
// 16000 tokens x 80 heads x 128 fp16, 110 us, 5.9 TB/s, 88 % of the measured copy
// bandwidth; rope of one token for each of 64 sequences 3.8 us, of which the
// launch is most.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sage_device.cuh"
#include "sage_kernels.h"
#include "sage_paged.h"

namespace sage {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxToks = 8;          // tokens of one CTA
constexpr int kMaxPairToks = 64;
constexpr unsigned kAll = 0xFFFFFFFFu;

template <bool kBF16>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool kBF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Channels c0..c0+7 of a row (zeros from D on), element by element.
__device__ __forceinline__ uint4 load8_slow(const uint16_t* row, int c0, int D) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e < D) w[e / 2] |= static_cast<uint32_t>(row[c0 + e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The half layout's partners of channels c0..c0+7, element by element.
__device__ __forceinline__ uint4 load8_partner(const uint16_t* row, int c0, int R) {
  const int half = R / 2;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = c0 + e;
    if (c < R)
      w[e / 2] |= static_cast<uint32_t>(row[c < half ? c + half : c - half]) << (16 * (e & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(uint16_t* row, int c0, int D, bool vec, const uint4& v) {
  if (vec) {
    *reinterpret_cast<uint4*>(row + c0) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e < D) row[c0 + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
}

// The sequence that holds row `tok`: the last s with cu_q[s] <= tok, by a
// warp's 32-way search (each round trip to memory cuts the range by 32).
__device__ __forceinline__ int find_seq(const PagedGeo& c, int64_t tok, int lane) {
  int lo = 0, hi = c.nseq;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned b = __ballot_sync(kAll, i < hi && c.cu_q[i] <= tok);
    const int n = __popc(b);
    if (n == 0) break;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A token's position and slot, given its sequence.
__device__ __forceinline__ void place(const PagedGeo& c, int64_t tok, int s, int64_t* pos_out,
                                      int* page_out, int64_t* slot_out, int64_t* scale_out) {
  int start = 0, n = 0, len = 0, page = -1;
  int64_t pos = -1;
  if (paged_seq(c, s, &start, &n, &len) && tok >= start && tok < start + n) {
    pos = static_cast<int64_t>(len) - n + (tok - start);
    if (pos >= 0) {
      const int pn = static_cast<int>(pos) / c.page_size;
      page = paged_page(c, s, pn);
      const int slot = static_cast<int>(pos) - pn * c.page_size;
      *slot_out = page * c.page_stride + slot * c.token_stride;
      *scale_out = static_cast<int64_t>(page) * c.Hkv * c.page_size + slot;
    }
  }
  *pos_out = pos;
  *page_out = pos < 0 ? -2 : page;
}

// Each token's position and slot (append): a warp per token where a CTA has one
// for each (fewest round trips), else a thread per token (all at once).
__device__ __forceinline__ void place_tokens(const RowsParams& p, int64_t t0, int nt, int64_t* pos_s,
                                             int* page_s, int64_t* slot_s, int64_t* scale_s) {
  const PagedGeo& c = p.c;
  if (nt <= kRowThreads / 32) {
    const int i = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (i < nt) {
      const int s = find_seq(c, t0 + i, lane);
      if (lane == 0) place(c, t0 + i, s, &pos_s[i], &page_s[i], &slot_s[i], &scale_s[i]);
    }
    return;
  }
  const int i = threadIdx.x;
  if (i < nt) {
    int lo = 0, hi = c.nseq;                            // the last s with cu_q[s] <= token
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (c.cu_q[mid] <= t0 + i) lo = mid;
      else hi = mid;
    }
    place(c, t0 + i, lo, &pos_s[i], &page_s[i], &slot_s[i], &scale_s[i]);
  }
}

// cos and sin of the CTA's tokens, times the gain, 64 apart per token.
__device__ __forceinline__ void turn_table(const RowsParams& p, int nt, const int64_t* pos_s,
                                           float2* cs) {
  const int half = p.R / 2;
  for (int i = threadIdx.x; i < nt * half; i += kRowThreads) {
    const int t = i / half, f = i - t * half;
    const double turns = p.inv_freq[f] * 0.15915494309189533577;     // 1 / (2 pi)
    const uint64_t frac = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
    const uint64_t a = frac * static_cast<uint64_t>(pos_s[t]) + (1ull << 31);
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578125e-10f,
              &sn, &cn);                                             // 2^-31
    cs[t * 64 + f] = make_float2(cn * p.mscale, sn * p.mscale * p.sign);
  }
}

// kMode: 0 rope, 1 append 16-bit, 2 append Q8.  kLanes: lanes of a row.
// kShfl: the half layout's partner vector is another lane's whole vector.
template <int kMode, bool kBF16, int kLanes, bool kShfl>
__global__ void __launch_bounds__(kRowThreads, kMode == 0 ? 5 : 3)
rows_kernel(const RowsParams p) {
  __shared__ float2 cs[kMaxToks * 64];
  __shared__ int64_t pos_s[kMaxToks];
  __shared__ int page_s[kMaxToks];          // -1: no such page; -2: no such token
  __shared__ int64_t slot_s[kMaxToks], scale_s[kMaxToks];   // the slot of head 0, and its scale
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.toks;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.toks), p.T - t0));
  const int half = p.R / 2;
  const PagedGeo& c = p.c;

  if constexpr (kMode == 0) {
    if (threadIdx.x < nt) {
      pos_s[threadIdx.x] = p.pos64 ? static_cast<const int64_t*>(p.pos)[t0 + threadIdx.x]
                                   : static_cast<const int32_t*>(p.pos)[t0 + threadIdx.x];
      page_s[threadIdx.x] = 0;
    }
  } else {
    place_tokens(p, t0, nt, pos_s, page_s, slot_s, scale_s);
  }
  __syncthreads();
  if (p.inv_freq != nullptr) turn_table(p, nt, pos_s, cs);
  __syncthreads();

  const int nq = p.Hq;
  const int rows = nq + p.Hkv * (kMode == 0 ? 1 : 2);
  const int sub = threadIdx.x % kLanes;
  const int c0 = 8 * sub;
  const bool live = c0 < p.D;
  const int groups = kRowThreads / kLanes;
  // partner lane of the half layout
  int mate = sub;
  if (kShfl && c0 < p.R) mate = c0 < half ? sub + half / 8 : sub - half / 8;
  const int rstep = groups * gridDim.y;
  const int rend = (rows + rstep - 1) / rstep * rstep;   // whole warps stay in the loop
  for (int r = blockIdx.y * groups + threadIdx.x / kLanes; r < rend; r += rstep) {
    const bool has = r < rows && live;
    const int what = r < nq ? 0 : (r < nq + p.Hkv ? 1 : 2);          // q, k, v
    const int h = what == 0 ? r : (what == 1 ? r - nq : r - nq - p.Hkv);
    const uint16_t* src = what == 0 ? p.q + h * p.q_head
                          : what == 1 ? p.k + h * p.k_head : p.v + h * p.v_head;
    const int64_t tok_stride = what == 0 ? p.q_tok : what == 1 ? p.k_tok : p.v_tok;
    const bool turn = p.inv_freq != nullptr && what != 2;
    float chan[8];                          // Q8: k mean, or 1 / v scale
    if constexpr (kMode == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) chan[e] = 0.0f;
      if (has && what != 0) {
        const float* src4 = (what == 1 ? c.k_mean : c.v_scale) + h * c.Dp + c0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          chan[e] = src4[e];
          if (what == 2) chan[e] = chan[e] > 0.0f ? __fdiv_rn(1.0f, chan[e]) : 0.0f;
        }
      }
    }
    constexpr int kUnroll = kShfl ? 4 : 1;
    for (int tb = 0; tb < nt; tb += kUnroll) {
      uint4 raw[kUnroll], rawp[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (has && tb + u < nt) {
          const uint16_t* row = src + (t0 + tb + u) * tok_stride;
          raw[u] = p.vec ? *reinterpret_cast<const uint4*>(row + c0) : load8_slow(row, c0, p.D);
          if constexpr (!kShfl)
            rawp[u] = turn && !p.interleaved ? load8_partner(row, c0, p.R) : raw[u];
        }
      }
      __syncwarp();                         // in place: every lane has read its row
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int t = tb + u;
        if (t >= nt) break;                 // the same for every lane
        if constexpr (kShfl) {
          rawp[u].x = __shfl_sync(kAll, raw[u].x, mate, kLanes);
          rawp[u].y = __shfl_sync(kAll, raw[u].y, mate, kLanes);
          rawp[u].z = __shfl_sync(kAll, raw[u].z, mate, kLanes);
          rawp[u].w = __shfl_sync(kAll, raw[u].w, mate, kLanes);
        }
        float x[8];
        unpack8<kBF16>(raw[u], x);
        if (turn && c0 < p.R) {
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c0 + 2 * i < p.R) {
                const float2 a = cs[t * 64 + c0 / 2 + i];
                const float x1 = x[2 * i], x2 = x[2 * i + 1];
                x[2 * i] = x1 * a.x - x2 * a.y;
                x[2 * i + 1] = x2 * a.x + x1 * a.y;
              }
          } else {
            float y[8];
            unpack8<kBF16>(rawp[u], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int ch = c0 + e;
              if (ch < p.R) {
                const bool low = ch < half;
                const float2 a = cs[t * 64 + (low ? ch : ch - half)];
                x[e] = low ? x[e] * a.x - y[e] * a.y : x[e] * a.x + y[e] * a.y;
              }
            }
          }
        }
        if constexpr (kMode == 0) {
          if (has) {
            uint16_t* dst = what == 0 ? p.q_out + (t0 + t) * p.qo_tok + h * p.qo_head
                                      : p.k_out + (t0 + t) * p.ko_tok + h * p.ko_head;
            store8(dst, c0, p.D, p.vec, pack8<kBF16>(x));
          }
        } else {
          if (what == 0) {
            if (has && page_s[t] != -2)
              store8(p.q_out + (t0 + t) * p.qo_tok + h * p.qo_head, c0, p.D, p.vec,
                     pack8<kBF16>(x));
          }
          const int page = page_s[t];
          const int64_t at = slot_s[t] + h * c.head_stride + c0;
          const bool put = has && what != 0 && page >= 0;
          if constexpr (kMode == 1) {
            if (put) {
              uint16_t* base = reinterpret_cast<uint16_t*>(what == 1 ? c.k : c.v);
              *reinterpret_cast<uint4*>(base + at) = turn ? pack8<kBF16>(x) : raw[u];
            }
          } else {
            float top = 0.0f;
            if (what == 1) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e] = __fsub_rn(x[e], chan[e]);
                top = fmaxf(top, fabsf(x[e]));
              }
            }
            // lanes of one row share `what`; the shuffles run in every lane
#pragma unroll
            for (int d = kLanes / 2; d > 0; d /= 2)
              top = fmaxf(top, __shfl_xor_sync(kAll, top, d, kLanes));
            if (put && what == 1) {
              const float inv = top > 0.0f ? __fdiv_rn(127.0f, top) : 0.0f;
              uint32_t w[2] = {0, 0};
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e / 4] |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(x[e], inv))) & 0xFFu)
                            << (8 * (e & 3));
              *reinterpret_cast<uint2*>(c.k + at) = make_uint2(w[0], w[1]);
              if (sub == 0)
                c.k_scale[scale_s[t] + static_cast<int64_t>(h) * c.page_size] =
                    __fdiv_rn(top, 127.0f);
            } else if (put) {
              uint32_t w[2];
#pragma unroll
              for (int i = 0; i < 2; ++i)
                w[i] = pack_e4m3x2(__fmul_rn(x[4 * i], chan[4 * i]),
                                   __fmul_rn(x[4 * i + 1], chan[4 * i + 1])) |
                       pack_e4m3x2(__fmul_rn(x[4 * i + 2], chan[4 * i + 2]),
                                   __fmul_rn(x[4 * i + 3], chan[4 * i + 3])) << 16;
              *reinterpret_cast<uint2*>(c.v + at) = make_uint2(w[0], w[1]);
            }
          }
        }
      }
      __syncwarp();
    }
  }
}

// ---- The usual case: rows in whole 16-byte vectors, rotations whose pairs are
// whole vectors.  A lane holds two vectors of a row, in the half layout the two
// that turn into each other (no partner from another lane, one cos and sin for
// both), else neighbours; a row takes ceil(D / 16) lanes, so that 80 channels
// fill 30 of 32 lanes with six rows.  q, k and v rows go in passes of their own
// (no warp does two kinds).  Arithmetic bounds the Q8 cache's rows: there a lane
// keeps its head through the CTA's tokens, with the head's means or multipliers
// in registers.

__device__ __forceinline__ int wrap(int x, int n) { return x >= n ? x - n : x; }

struct Tokens {
  int64_t pos[kMaxPairToks], slot[kMaxPairToks], scale[kMaxPairToks];
  int page[kMaxPairToks];
};

// kMode as above; kWhat: 0 q, 1 k, 2 v.
template <int kMode, int kWhat, bool kBF16>
__device__ __forceinline__ void pair_pass(const RowsParams& p, const Tokens& tk, const float2* cs,
                                          int64_t t0, int nt) {
  const PagedGeo& c = p.c;
  constexpr bool kCodes = kMode == 2 && kWhat != 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.D + 15) / 16, fit = 32 / per;      // lanes of a row; rows of a warp
  const int slot = lane / per, sub = lane - slot * per;
  const int base = slot * per;
  const bool turn = kWhat != 2 && p.inv_freq != nullptr;
  // this lane's vectors, as first channels
  const bool halves = turn && !p.interleaved && sub < p.R / 16;
  const int ca = halves ? 8 * sub : 16 * sub, cb = halves ? ca + p.R / 2 : ca + 8;
  const bool two = cb < p.D;                            // D % 16 == 8: the last lane has one
  const int heads = kWhat == 0 ? p.Hq : p.Hkv;
  const int groups = kRowThreads / 32 * fit, group = warp * fit + slot;
  // Codes: a group keeps its head; else rows are dealt one after another.
  const int at_once = kCodes ? min(heads, groups) : heads;
  const int step = kCodes ? groups / at_once : 0;       // tokens side by side
  const uint16_t* const rows = kWhat == 0 ? p.q : kWhat == 1 ? p.k : p.v;
  const int64_t tok_stride = kWhat == 0 ? p.q_tok : kWhat == 1 ? p.k_tok : p.v_tok;
  const int64_t head_stride = kWhat == 0 ? p.q_head : kWhat == 1 ? p.k_head : p.v_head;

  for (int hb = 0; hb < heads; hb += at_once) {
    int t = group / at_once, h = hb + group - t * at_once;
    const bool mine = slot < fit && h < heads && (!kCodes || t < step);
    float chan[16];                                     // codes: means, or 1 / scale
    if constexpr (kCodes) {
      const float* src = (kWhat == 1 ? c.k_mean : c.v_scale) + h * c.Dp;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int ch = (e < 8 ? ca : cb) + e % 8;
        chan[e] = mine && ch < p.D ? src[ch] : 0.0f;
        if (kWhat == 2) chan[e] = chan[e] > 0.0f ? __fdiv_rn(1.0f, chan[e]) : 0.0f;
      }
    }
    // the next row: the same head `step` tokens on, or `groups` rows on
    auto advance = [&](int& tt, int& hh) {
      if constexpr (kCodes) {
        tt += step;
      } else {
        hh += groups;
        while (hh >= heads) {
          hh -= heads;
          ++tt;
        }
      }
    };
    constexpr int kAhead = kCodes ? 1 : 3;              // rows whose loads run ahead
    uint4 ring[kAhead][2];
    int lt = t, lh = h;                                 // the next row to load
    const uint16_t* at = rows + (t0 + lt) * tok_stride + lh * head_stride;   // codes: moves on
    auto load = [&](uint4 (&r)[2]) {
      r[0] = r[1] = make_uint4(0, 0, 0, 0);
      if (mine && lt < nt) {
        const uint16_t* src =
            kCodes ? at : rows + (t0 + lt) * tok_stride + lh * head_stride;
        r[0] = *reinterpret_cast<const uint4*>(src + ca);
        if (two) r[1] = *reinterpret_cast<const uint4*>(src + cb);
      }
      advance(lt, lh);
      if (kCodes) at += step * tok_stride;
    };
    auto handle = [&](const uint4 (&raw)[2]) {
      const bool has = mine && t < nt;
      float x[2][8];
      unpack8<kBF16>(raw[0], x[0]);
      unpack8<kBF16>(raw[1], x[1]);
      if (turn) {
        const float2* const a = cs + (has ? t : 0) * 64;
        if (halves) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 w = a[ca + e];
            const float y = x[0][e] * w.x - x[1][e] * w.y;
            x[1][e] = x[1][e] * w.x + x[0][e] * w.y;
            x[0][e] = y;
          }
        } else if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (ca + 2 * i < p.R) {
              const float2 w = a[ca / 2 + i];
              float &x1 = x[i / 4][2 * (i % 4)], &x2 = x[i / 4][2 * (i % 4) + 1];
              const float y = x1 * w.x - x2 * w.y;
              x2 = x2 * w.x + x1 * w.y;
              x1 = y;
            }
        }
      }
      const int page = kMode == 0 ? 0 : has ? tk.page[t] : -1;
      if constexpr (!kCodes) {
        const bool put = has && (kWhat == 0 ? page != -2 : page >= 0);
        if (put) {
          uint16_t* dst;
          if constexpr (kWhat == 0) dst = p.q_out + (t0 + t) * p.qo_tok + h * p.qo_head;
          else if constexpr (kMode == 0) dst = p.k_out + (t0 + t) * p.ko_tok + h * p.ko_head;
          else
            dst = reinterpret_cast<uint16_t*>(kWhat == 1 ? c.k : c.v) + tk.slot[t] +
                  h * c.head_stride;
          *reinterpret_cast<uint4*>(dst + ca) = turn ? pack8<kBF16>(x[0]) : raw[0];
          if (two) *reinterpret_cast<uint4*>(dst + cb) = turn ? pack8<kBF16>(x[1]) : raw[1];
        }
      } else {
        uint32_t w[4];
        if constexpr (kWhat == 1) {
          float top = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e / 8][e % 8] = __fsub_rn(x[e / 8][e % 8], chan[e]);
            top = fmaxf(top, fabsf(x[e / 8][e % 8]));
          }
          // the row's largest, in every lane of the row
          if ((per & (per - 1)) == 0) {
            for (int d = 1; d < per; d *= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
          } else {
            const float part = top;
            int from = sub;
            for (int k = 1; k < per; ++k) {
              from = wrap(from + 1, per);
              top = fmaxf(top, __shfl_sync(kAll, part, base + from));
            }
          }
          const float inv = top > 0.0f ? __fdiv_rn(127.0f, top) : 0.0f;
          // rint by adding 1.5 * 2^23: the low byte is the code
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              b[e] = __float_as_uint(
                  __fadd_rn(__fmul_rn(x[i / 2][4 * (i % 2) + e], inv), 12582912.0f));
            w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040),
                               0x5410);
          }
          if (sub == 0 && page >= 0)
            c.k_scale[tk.scale[t] + static_cast<int64_t>(h) * c.page_size] =
                __fdiv_rn(top, 127.0f);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* y = &x[i / 2][4 * (i % 2)];
            w[i] = pack_e4m3x2(__fmul_rn(y[0], chan[4 * i]), __fmul_rn(y[1], chan[4 * i + 1])) |
                   pack_e4m3x2(__fmul_rn(y[2], chan[4 * i + 2]), __fmul_rn(y[3], chan[4 * i + 3]))
                       << 16;
          }
        }
        if (page >= 0) {
          uint8_t* dst = (kWhat == 1 ? c.k : c.v) + tk.slot[t] + h * c.head_stride;
          if (c.wide && !halves) {
            *reinterpret_cast<uint4*>(dst + ca) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {                                      // apart, or slots on 8 bytes
            *reinterpret_cast<uint2*>(dst + ca) = make_uint2(w[0], w[1]);
            if (two) *reinterpret_cast<uint2*>(dst + cb) = make_uint2(w[2], w[3]);
          }
        }
      }
      advance(t, h);
    };
    if constexpr (kCodes) {
      load(ring[0]);
      for (int tb = 0; tb < nt; tb += step) {
        const uint4 raw[2] = {ring[0][0], ring[0][1]};
        load(ring[0]);
        handle(raw);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(ring[i]);
    // whole warps stay in the loop as long as one of their rows has a token left
    while (__any_sync(kAll, mine && t < nt)) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint4 raw[2] = {ring[i][0], ring[i][1]};
        load(ring[i]);
        __syncwarp();                                   // in place: rows are read first
        handle(raw);
      }
    }
  }
}

template <int kMode, bool kBF16>
__global__ void __launch_bounds__(kRowThreads, kMode == 2 ? 4 : 3)
pair_rows_kernel(const RowsParams p) {
  __shared__ float2 cs[kMaxPairToks * 64];
  __shared__ Tokens tk;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.toks;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.toks), p.T - t0));
  if constexpr (kMode == 0) {
    if (threadIdx.x < nt)
      tk.pos[threadIdx.x] = p.pos64 ? static_cast<const int64_t*>(p.pos)[t0 + threadIdx.x]
                                    : static_cast<const int32_t*>(p.pos)[t0 + threadIdx.x];
  } else {
    place_tokens(p, t0, nt, tk.pos, tk.page, tk.slot, tk.scale);
  }
  __syncthreads();
  if (p.inv_freq != nullptr) {
    turn_table(p, nt, tk.pos, cs);
    __syncthreads();
  }
  if (p.Hq > 0) pair_pass<kMode, 0, kBF16>(p, tk, cs, t0, nt);
  if (p.Hkv > 0) pair_pass<kMode, 1, kBF16>(p, tk, cs, t0, nt);
  if (kMode != 0) pair_pass<kMode, 2, kBF16>(p, tk, cs, t0, nt);
}

template <int kMode, bool kBF16>
cudaError_t launch_pairs(const RowsParams& p0, int sms, cudaStream_t st) {
  RowsParams p = p0;
  p.toks = 1;
  while (p.toks < kMaxPairToks && p.T / (2 * p.toks) >= 4 * sms) p.toks *= 2;
  const int64_t ctas = (p.T + p.toks - 1) / p.toks;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  pair_rows_kernel<kMode, kBF16><<<static_cast<unsigned>(ctas), kRowThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <int kMode, bool kBF16, int kLanes>
cudaError_t launch_lanes(const RowsParams& p, bool shfl, dim3 grid, cudaStream_t st) {
  if (shfl) rows_kernel<kMode, kBF16, kLanes, true><<<grid, kRowThreads, 0, st>>>(p);
  else rows_kernel<kMode, kBF16, kLanes, false><<<grid, kRowThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <int kMode>
cudaError_t launch_mode(const RowsParams& p0, bool bf16, int sms, cudaStream_t st) {
  RowsParams p = p0;
  const int lanes = p.D <= 64 ? 8 : 16;
  const int rows = p.Hq + p.Hkv * (kMode == 0 ? 1 : 2);
  const int groups = kRowThreads / lanes;
  // Few tokens: one per CTA, and its heads over several CTAs, so that every SM
  // has work; many: kMaxToks, which serve the means, scales and angles.
  p.toks = 1;
  while (p.toks < kMaxToks && p.T / (2 * p.toks) >= 4 * sms) p.toks *= 2;
  const int64_t ctas = (p.T + p.toks - 1) / p.toks;
  int64_t y = (rows + groups - 1) / groups;
  if (ctas * y > 2 * sms) y = 2 * sms / ctas > 1 ? 2 * sms / ctas : 1;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(y));
  const bool shfl = p.vec && (p.inv_freq == nullptr || p.interleaved || p.R % 16 == 0);
  if (lanes == 8)
    return bf16 ? launch_lanes<kMode, true, 8>(p, shfl, grid, st)
                : launch_lanes<kMode, false, 8>(p, shfl, grid, st);
  return bf16 ? launch_lanes<kMode, true, 16>(p, shfl, grid, st)
              : launch_lanes<kMode, false, 16>(p, shfl, grid, st);
}

}  // namespace

cudaError_t launch_rows(const RowsParams& p, int mode, bool bf16, int sms, cudaStream_t st) {
  // Two vectors a lane from 4 tokens per SM on, for whole vectors.  Measured, two
  // vectors against one (us; one call in a graph, L2 flushed):
  //   rope, half layout, 16000 tokens x (40 + 40) heads of 128      132   192
  //   16-bit append, half layout, q beside it: 24000 tokens, 32 q
  //     heads on 8 kv heads of 128                                 130   192
  //     65000 tokens, 16 on 16 heads of 80                         231   370
  //   16-bit append as it is, 65000 x 16 of 80 | 16000 x 40 of 128  128   161 | 122   120
  //   Q8 append as it is, the same two                             128   237 | 149   156
  //   Q8 append, half layout, the rows of the 16-bit one           210   220 | 280   471
  //   Q8 append, interleaved, 24000 tokens, 32 on 8 of 128          261   161
  // The last one is on the slower side.  One vector a lane has the shorter way
  // through few tokens (64: 3.8 us against 4.3; Q8 4.7 against 6.8), and rope and
  // 16-bit appends whose pairs are neighbours stay with it (110 against 118).
  const bool apart = p.inv_freq != nullptr && !p.interleaved;
  const bool neighbours = p.inv_freq != nullptr && p.interleaved;
  const bool pairs = p.vec && p.T >= 4 * static_cast<int64_t>(sms) &&
                     !(apart && p.R % 16 != 0) && !(neighbours && mode != 2);
  if (pairs) {
    if (mode == 0)
      return bf16 ? launch_pairs<0, true>(p, sms, st) : launch_pairs<0, false>(p, sms, st);
    if (mode == 1)
      return bf16 ? launch_pairs<1, true>(p, sms, st) : launch_pairs<1, false>(p, sms, st);
    return bf16 ? launch_pairs<2, true>(p, sms, st) : launch_pairs<2, false>(p, sms, st);
  }
  if (mode == 0) return launch_mode<0>(p, bf16, sms, st);
  if (mode == 1) return launch_mode<1>(p, bf16, sms, st);
  return launch_mode<2>(p, bf16, sms, st);
}

}  // namespace sage
