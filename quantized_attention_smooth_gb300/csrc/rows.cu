// Rotary positions and the paged cache's writer: one kernel over (token, head)
// rows.
//
//   rotation   y1 = g (x1 cos a - x2 sin a),  y2 = g (x2 cos a + x1 sin a),
//              a = pos * inv_freq[i] for channel pair i, in fp32
//   16-bit     the row rounded once to the cache's type
//   Q8         x = k - mean;  s = max|x| / 127;  code = rint(x * (127 / max|x|))
//              V code = e4m3(v * (1 / v_scale)), saturating
//              (each one IEEE fp32 operation, as in the quantisation prologue)
//   Q4         x = k - mean, or v * (1 / (64 v_scale)), in groups of 32 channels:
//              s = fp16(min(max|x| * fl(1/7), most)),  code = rint(x * (1 / s)), within
//              -7..7; most = 9352 (K: 7 of it fit 16 bits) or 1 (V: 7 * 64 v_scale)
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
// bandwidth (half layout 108); rope of one token for each of 64 sequences 3.8 us, of which the
// launch is most; three axes, 32768 tokens x 80 x 128 bf16, 215 us, 6.24 TB/s, 93 %.
// Packed prompts into the 4-bit cache, 76000 tokens x 16 heads x 80 fp16: 140 us, 3.7
// TB/s, issue slots 74 % full; read back 145 us, 3.6 TB/s, waiting for loads.  24000
// tokens, 32 heads of q and 8 of k and v, 128 bf16, half layout: into 16 bits 100 us,
// 5.9 TB/s; 8 bits 109; 4 bits 114.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sage_device.cuh"
#include "sage_kernels.h"
#include "sage_paged.h"
#include "sage_paged_device.cuh"

namespace sage {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxToks = 8;          // tokens of one CTA
constexpr int kMaxPairToks = 64;
constexpr unsigned kAll = 0xFFFFFFFFu;
// CTAs of an SM, as the kernels' registers allow.
constexpr int row_ctas(int mode) { return mode == 0 ? 5 : 3; }
constexpr int pair_ctas(int mode) { return mode == 2 ? 4 : 3; }
constexpr int group_ctas(bool turn) { return turn ? 3 : 4; }
constexpr int kGatherCtas = 4;
constexpr float kSeventh = 1.0f / 7.0f;
constexpr float kMostK = 9352.0f, kMostV = 1.0f;   // largest scales of a Q4 group

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

// The number that an e4m3 code stands for.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(two)));
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

// cos and sin of the CTA's tokens, times the gain, 64 apart per token.  Rotations of
// several axes take a pair's position from the axis that it follows.  kAxes false: there
// are none; few tokens have no use for the loads that ask (rope of 64: 3.8 us, with them
// 4.2; appends of 64 to 300 3 to 4 % longer with them).
template <bool kAxes>
__device__ __forceinline__ void turn_table(const RowsParams& p, int64_t t0, int nt,
                                           const int64_t* pos_s, float2* cs) {
  // A thread keeps its pair, whose fraction of a turn takes doubles: a pair and a token
  // each time, the FP64 pipe would be what a long CTA waits for.
  const int half = p.R / 2, first = threadIdx.x / half, f = threadIdx.x - first * half;
  if (first >= nt) return;
  const int rows = nt > 1 ? kRowThreads / half : 1;
  if (first >= rows) return;
  const double turns = p.inv_freq[f] * 0.15915494309189533577;       // 1 / (2 pi)
  const uint64_t frac = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
  const bool axes = kAxes && p.naxes > 0;
  const int axis =
      axes && p.axis_of != nullptr ? min(static_cast<int>(p.axis_of[f]), p.naxes - 1) : 0;
  for (int t = first; t < nt; t += rows) {
    int64_t pos;
    if (axes) {
      const int64_t at = axis * p.axis_stride + t0 + t;
      pos = p.pos64 ? static_cast<const int64_t*>(p.pos)[at] : static_cast<const int32_t*>(p.pos)[at];
    } else {
      pos = pos_s[t];
    }
    const uint64_t a = frac * static_cast<uint64_t>(pos) + (1ull << 31);
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578125e-10f,
              &sn, &cn);                                             // 2^-31
    cs[t * 64 + f] = make_float2(cn * p.mscale, sn * p.mscale * p.sign);
  }
}

// The larger of two numbers; NaN if one of them is (fmaxf would give the other).
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Q4: the group's scale from its largest, and the codes of eight channels plus 8, in
// nibbles.  A group that holds a NaN has a scale of NaN and codes of zero, so that it
// reads back as NaN; infinities take the largest scale and code.
__device__ __forceinline__ __half group_scale(float top, float most) {
  float s;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(s) : "f"(__fmul_rn(top, kSeventh)), "f"(most));
  return __float2half_rn(s);
}
__device__ __forceinline__ uint32_t pack_nibbles(const float (&x)[8], float top, float inv) {
  float n[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) n[e] = __fmul_rn(x[e], inv);
  if (!(__fmul_rn(top, inv) < 7.25f)) {         // a scale at its bounds, or NaN
    if (isnan(top)) return 0x88888888u;         // (its bits would borrow from other codes)
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = fminf(fmaxf(n[e], -7.0f), 7.0f);
  }
  // 1.5 * 2^23 + 8 rounds to whole numbers and leaves n + 8 in the lowest bits; above
  // them stands 0x4B400000, which comes off the sum of all eight
  uint32_t w = 0;
#pragma unroll
  for (int e = 7; e >= 0; --e) w = w * 16u + __float_as_uint(__fadd_rn(n[e], 12582920.0f));
  return w - 0x4B400000u * 0x11111111u;
}

// kMode: 0 rope, 1 append 16-bit, 2 append Q8, 3 append Q4.  kLanes: lanes of a row.
// kShfl: the half layout's partner vector is another lane's whole vector.
template <int kMode, bool kBF16, int kLanes, bool kShfl, bool kAxes>
__global__ void __launch_bounds__(kRowThreads, row_ctas(kMode))
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
    if (threadIdx.x < nt && !(kAxes && p.naxes > 0)) {
      pos_s[threadIdx.x] = p.pos64 ? static_cast<const int64_t*>(p.pos)[t0 + threadIdx.x]
                                   : static_cast<const int32_t*>(p.pos)[t0 + threadIdx.x];
    }
  } else {
    place_tokens(p, t0, nt, pos_s, page_s, slot_s, scale_s);
  }
  __syncthreads();
  if (p.inv_freq != nullptr) turn_table<kAxes>(p, t0, nt, pos_s, cs);
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
    float chan[8];                          // codes: k mean, or the values' factor
    if constexpr (kMode >= 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) chan[e] = 0.0f;
      if (has && what != 0) {
        const float* src4 = (what == 1 ? c.k_mean : c.v_scale) + h * c.Dp + c0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          chan[e] = src4[e];
          if (what == 2)
            chan[e] = chan[e] > 0.0f ? __fdiv_rn(1.0f, kMode == 3 ? 64.0f * chan[e] : chan[e])
                                     : 0.0f;
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
          if constexpr (kMode == 3) {
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] = what == 1 ? __fsub_rn(x[e], chan[e]) : __fmul_rn(x[e], chan[e]);
              top = max_or_nan(top, fabsf(x[e]));
            }
            // four lanes are a group
            top = max_or_nan(top, __shfl_xor_sync(kAll, top, 1));
            top = max_or_nan(top, __shfl_xor_sync(kAll, top, 2));
            if (r < rows && what != 0 && page >= 0) {
              const __half scale = group_scale(top, what == 1 ? kMostK : kMostV);
              const float s = __half2float(scale);
              const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
              if (c0 < 32 * ((p.D + 31) / 32))
                *reinterpret_cast<uint32_t*>((what == 1 ? c.k : c.v) + slot_s[t] +
                                             h * c.head_stride + c0 / 2) = pack_nibbles(x, top, inv);
              if (sub % 4 == 0)
                reinterpret_cast<__half*>(what == 1 ? c.k_groups : c.v_groups)
                    [(scale_s[t] + static_cast<int64_t>(h) * c.page_size) * (c.Dp / 32) + sub / 4] =
                        scale;
            }
          } else if constexpr (kMode == 1) {
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

// ---- Q4, many tokens: two lanes are a group of 32 channels of one head's keys or
// values and keep it for the CTA's tokens, with the means or factors in registers.  In
// the half layout a lane reads its partner channels as well (they come out of the L1) and
// turns its own.  Arithmetic bounds this: what a group costs besides its channels (the
// largest across lanes, the scale, places and stores) is shared by 16 channels a lane;
// with 8, four lanes a group, the rows of 76000 tokens x 16 heads x 80 took 211 us.
template <bool kBF16, bool kTurn, bool kVal>
__device__ __forceinline__ void group_pass(const RowsParams& p, const Tokens& tk, const float2* cs,
                                           int64_t t0, int nt) {
  const PagedGeo& c = p.c;
  constexpr int kPairs = kRowThreads / 2;
  constexpr bool kRot = kTurn && !kVal;
  const int pair = threadIdx.x >> 1, side = threadIdx.x & 1;
  const int groups = (p.D + 31) / 32, padded = c.Dp / 32, units = p.Hkv * groups;
  const int at_once = min(units, kPairs), step = kPairs / at_once;
  const int first = pair / at_once, rounds = (nt + step - 1) / step;
  const int half = p.R / 2;
  const int64_t stride = kVal ? p.v_tok : p.k_tok, ahead = step * stride;
  for (int ub = 0; ub < units; ub += at_once) {
    const int u = ub + pair - first * at_once;
    const bool mine = u < units && first < step;
    const int h = u / groups, grp = u - h * groups, c0 = 32 * grp + 16 * side;
    const int left = mine ? p.D - c0 : 0;               // channels from c0 on
    float chan[16];                                     // means, or 1 / (64 scale)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      chan[e] = e < left ? (kVal ? c.v_scale : c.k_mean)[h * c.Dp + c0 + e] : 0.0f;
      if (kVal) chan[e] = chan[e] > 0.0f ? __fdiv_rn(1.0f, 64.0f * chan[e]) : 0.0f;
    }
    const uint16_t* src = (kVal ? p.v + h * p.v_head : p.k + h * p.k_head) +
                          (t0 + first) * stride + c0;
    uint8_t* const codes = (kVal ? c.v : c.k) + h * c.head_stride + c0 / 2;
    __half* const scales = reinterpret_cast<__half*>(kVal ? c.v_groups : c.k_groups) + grp +
                           static_cast<int64_t>(h) * c.page_size * padded;
    uint4 next[2];
    auto load = [&](int t) {
      next[0] = next[1] = make_uint4(0, 0, 0, 0);
      if (t < nt) {
        if (left > 0) next[0] = *reinterpret_cast<const uint4*>(src);
        if (left > 8) next[1] = *reinterpret_cast<const uint4*>(src + 8);
      }
    };
    load(first);
    for (int r = 0; r < rounds; ++r) {
      const int t = first + r * step, at = t < nt ? t : 0;
      float x[2][8];
      unpack8<kBF16>(next[0], x[0]);
      unpack8<kBF16>(next[1], x[1]);
      if constexpr (kRot) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int ch = c0 + 8 * v;
          if (ch >= p.R || 8 * v >= left || t >= nt) continue;
          if (!p.interleaved) {
            const bool low = ch < half;
            float y[8];
            unpack8<kBF16>(*reinterpret_cast<const uint4*>(src + 8 * v + (low ? half : -half)), y);
            const float2* const a = cs + at * 64 + (low ? ch : ch - half);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 w = a[e];
              x[v][e] = low ? x[v][e] * w.x - y[e] * w.y : x[v][e] * w.x + y[e] * w.y;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (ch + 2 * i < p.R) {
                const float2 w = cs[at * 64 + ch / 2 + i];
                const float x1 = x[v][2 * i], x2 = x[v][2 * i + 1];
                x[v][2 * i] = x1 * w.x - x2 * w.y;
                x[v][2 * i + 1] = x2 * w.x + x1 * w.y;
              }
          }
        }
      }
      src += ahead;
      load(t + step);                                   // the next row's loads run ahead
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float& y = x[e / 8][e % 8];
        y = kVal ? __fmul_rn(y, chan[e]) : __fsub_rn(y, chan[e]);
        top = max_or_nan(top, fabsf(y));
      }
      top = max_or_nan(top, __shfl_xor_sync(kAll, top, 1));
      const __half scale = group_scale(top, kVal ? kMostV : kMostK);
      const float s = __half2float(scale);
      const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
      if (mine && t < nt && tk.page[at] >= 0) {
        *reinterpret_cast<uint2*>(codes + tk.slot[at]) =
            make_uint2(pack_nibbles(x[0], top, inv), pack_nibbles(x[1], top, inv));
        if (side == 0) {
          __half* const to = scales + tk.scale[at] * padded;
          *to = scale;
          if (grp == groups - 1)                        // groups behind D
            for (int e = groups; e < padded; ++e) to[e - grp] = __ushort_as_half(0);
        }
      }
    }
  }
}

template <bool kBF16, bool kTurn>
__global__ void __launch_bounds__(kRowThreads, group_ctas(kTurn))
group_rows_kernel(const RowsParams p) {
  __shared__ float2 cs[kTurn ? kMaxPairToks * 64 : 1];
  __shared__ Tokens tk;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.toks;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.toks), p.T - t0));
  place_tokens(p, t0, nt, tk.pos, tk.page, tk.slot, tk.scale);
  __syncthreads();
  if constexpr (kTurn) {
    turn_table<true>(p, t0, nt, tk.pos, cs);
    __syncthreads();
    if (p.Hq > 0) pair_pass<3, 0, kBF16>(p, tk, cs, t0, nt);
  }
  group_pass<kBF16, kTurn, false>(p, tk, cs, t0, nt);
  group_pass<kBF16, kTurn, true>(p, tk, cs, t0, nt);
}

template <int kMode, bool kBF16>
__global__ void __launch_bounds__(kRowThreads, pair_ctas(kMode))
pair_rows_kernel(const RowsParams p) {
  __shared__ float2 cs[kMaxPairToks * 64];
  __shared__ Tokens tk;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.toks;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.toks), p.T - t0));
  if constexpr (kMode == 0) {
    if (threadIdx.x < nt && p.naxes == 0)
      tk.pos[threadIdx.x] = p.pos64 ? static_cast<const int64_t*>(p.pos)[t0 + threadIdx.x]
                                    : static_cast<const int32_t*>(p.pos)[t0 + threadIdx.x];
  } else {
    place_tokens(p, t0, nt, tk.pos, tk.page, tk.slot, tk.scale);
  }
  __syncthreads();
  if (p.inv_freq != nullptr) {
    turn_table<true>(p, t0, nt, tk.pos, cs);
    __syncthreads();
  }
  if (p.Hq > 0) pair_pass<kMode, 0, kBF16>(p, tk, cs, t0, nt);
  if (p.Hkv > 0) pair_pass<kMode, 1, kBF16>(p, tk, cs, t0, nt);
  if (kMode != 0) pair_pass<kMode, 2, kBF16>(p, tk, cs, t0, nt);
}

// Tokens of a CTA, `most` at most, so that the CTAs fill whole waves of `slots`.  Each
// begins with a chain of dependent loads (sequence, page, positions) and the angles, so
// a wave and a bit take as long as two: 16-bit append of 9868 rotated tokens (617 CTAs of
// 16 on 456 slots) 38.5 us, in one wave 28.6; Q8, 9872 tokens 71 and 56; rope 48 and 38;
// read back 43.3 and 39.2.  Two smaller waves instead of one were slower (40, 66, 40).
inline int tokens_of_cta(int64_t T, int most, int64_t slots) {
  const int64_t waves = (T + most * slots - 1) / (most * slots);
  return T > 0 ? static_cast<int>((T + waves * slots - 1) / (waves * slots)) : 1;
}

template <int kMode, bool kBF16>
cudaError_t launch_pairs(const RowsParams& p0, int sms, cudaStream_t st) {
  RowsParams p = p0;
  const int per_sm = kMode == 3 ? group_ctas(p.inv_freq != nullptr) : pair_ctas(kMode);
  p.toks = tokens_of_cta(p.T, kMaxPairToks, static_cast<int64_t>(per_sm) * sms);
  const int64_t ctas = (p.T + p.toks - 1) / p.toks;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (kMode == 3 && p.inv_freq == nullptr)      // q comes with a rotation only
    group_rows_kernel<kBF16, false><<<static_cast<unsigned>(ctas), kRowThreads, 0, st>>>(p);
  else if constexpr (kMode == 3)
    group_rows_kernel<kBF16, true><<<static_cast<unsigned>(ctas), kRowThreads, 0, st>>>(p);
  else
    pair_rows_kernel<kMode, kBF16><<<static_cast<unsigned>(ctas), kRowThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <int kMode, bool kBF16, int kLanes>
cudaError_t launch_lanes(const RowsParams& p, bool shfl, dim3 grid, cudaStream_t st) {
  if (p.naxes > 0) {
    if (shfl) rows_kernel<kMode, kBF16, kLanes, true, true><<<grid, kRowThreads, 0, st>>>(p);
    else rows_kernel<kMode, kBF16, kLanes, false, true><<<grid, kRowThreads, 0, st>>>(p);
  } else {
    if (shfl) rows_kernel<kMode, kBF16, kLanes, true, false><<<grid, kRowThreads, 0, st>>>(p);
    else rows_kernel<kMode, kBF16, kLanes, false, false><<<grid, kRowThreads, 0, st>>>(p);
  }
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
  // has work; many: up to kMaxToks, which share the means, scales and angles.
  p.toks = tokens_of_cta(p.T, kMaxToks, static_cast<int64_t>(row_ctas(kMode)) * sms);
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

// ---- Reading back: thread = 8 channels of a head's keys or values, for several of
// the CTA's tokens, so that a quantised cache's means and scales stay in registers.
constexpr int kGatherToks = 32;

template <int kKind, bool kBF16>
__global__ void __launch_bounds__(kRowThreads, kGatherCtas)
gather_kernel(const RowsParams p) {
  __shared__ int64_t pos_s[kGatherToks], slot_s[kGatherToks], scale_s[kGatherToks];
  __shared__ int page_s[kGatherToks];
  const PagedGeo& c = p.c;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.toks;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.toks), p.T - t0));
  const int64_t tokens = c.cu_q[c.nseq];                // rows behind stay as they are
  place_tokens(p, t0, nt, pos_s, page_s, slot_s, scale_s);
  __syncthreads();
  const int vecs = p.D / 8, units = 2 * p.Hkv * vecs;
  const int at_once = min(units, kRowThreads), step = kRowThreads / at_once;
  const int t_first = threadIdx.x / at_once;
  if (t_first >= step) return;
  for (int u = blockIdx.y * at_once + threadIdx.x % at_once; u < units;
       u += at_once * gridDim.y) {
    const int h2 = u / vecs, c0 = 8 * (u - h2 * vecs);
    const bool val = h2 >= p.Hkv;
    const int h = val ? h2 - p.Hkv : h2;
    float chan[8];                              // K's means, V's factors
    if constexpr (kKind == kKindQ8 || kKind == kKindQ4) {
      const float* src = (val ? c.v_scale : c.k_mean) + h * c.Dp + c0;
#pragma unroll
      for (int e = 0; e < 8; ++e) chan[e] = kKind == kKindQ4 && val ? 64.0f * src[e] : src[e];
    }
    const uint8_t* const codes = val ? c.v : c.k;
    uint16_t* const out = (val ? p.q_out : p.k_out) + h * (val ? p.qo_head : p.ko_head);
    const int64_t out_tok = val ? p.qo_tok : p.ko_tok;
    constexpr int kUnroll = 4;
    for (int tb = t_first; tb < nt; tb += kUnroll * step) {
      uint4 raw[kUnroll];
      float scale[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int t = tb + k * step;
        raw[k] = make_uint4(0, 0, 0, 0);
        scale[k] = 0.0f;
        if (t >= nt || page_s[t] < 0) continue;
        const int64_t at = slot_s[t] + h * c.head_stride;
        const int64_t sc = scale_s[t] + static_cast<int64_t>(h) * c.page_size;
        if constexpr (kKind == kKindQ4) {
          raw[k].x = *reinterpret_cast<const uint32_t*>(codes + at + c0 / 2);
          scale[k] = __half2float(reinterpret_cast<const __half*>(
              val ? c.v_groups : c.k_groups)[sc * (c.Dp / 32) + c0 / 32]);
        } else if constexpr (kKind == kKindQ8) {
          const uint2 w = *reinterpret_cast<const uint2*>(codes + at + c0);
          raw[k].x = w.x;
          raw[k].y = w.y;
          scale[k] = val ? 1.0f : c.k_scale[sc];
        } else {
          raw[k] = *reinterpret_cast<const uint4*>(codes + 2 * (at + c0));
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int t = tb + k * step;
        if (t >= nt || t0 + t >= tokens) continue;
        uint4 put = raw[k];
        if constexpr (kKind == kKindQ8 || kKind == kKindQ4) {
          float x[8];
          if constexpr (kKind == kKindQ4) {
            uint32_t n[4];                      // channels 0 and 4, 1 and 5, ...
            nibbles_to_half(raw[k].x, n);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&n[e]));
              x[e] = f.x;
              x[e + 4] = f.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t b = ((e < 4 ? raw[k].x : raw[k].y) >> (8 * (e & 3))) & 0xFFu;
              x[e] = val ? e4m3_value(b) : static_cast<float>(static_cast<int8_t>(b));
            }
          }
          // one rounding each (with 4 bits the first product is exact)
          if (val) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], scale[k]), chan[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(__fmul_rn(x[e], scale[k]), chan[e]);
          }
          put = page_s[t] < 0 ? make_uint4(0, 0, 0, 0) : pack8<kBF16>(x);
        }
        store8(out + (t0 + t) * out_tok, c0, p.D, p.vec, put);
      }
    }
  }
}

template <int kKind, bool kBF16>
cudaError_t launch_gather_kind(const RowsParams& p0, int sms, cudaStream_t st) {
  RowsParams p = p0;
  const int units = 2 * p.Hkv * (p.D / 8);
  p.toks = tokens_of_cta(p.T, kGatherToks, static_cast<int64_t>(kGatherCtas) * sms);
  const int64_t ctas = (p.T + p.toks - 1) / p.toks;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  int64_t y = (units + kRowThreads - 1) / kRowThreads;
  if (ctas * y > 4 * sms) y = 4 * sms / ctas > 1 ? 4 * sms / ctas : 1;
  gather_kernel<kKind, kBF16><<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(y)),
                                kRowThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gather(const RowsParams& p, bool bf16, int sms, cudaStream_t st) {
  if (p.c.kind == kKindQ4)
    return bf16 ? launch_gather_kind<kKindQ4, true>(p, sms, st)
                : launch_gather_kind<kKindQ4, false>(p, sms, st);
  if (p.c.kind == kKindQ8)
    return bf16 ? launch_gather_kind<kKindQ8, true>(p, sms, st)
                : launch_gather_kind<kKindQ8, false>(p, sms, st);
  return launch_gather_kind<kKindF16, false>(p, sms, st);   // bits as they are, either type
}

cudaError_t launch_rows(const RowsParams& p, int mode, bool bf16, int sms, cudaStream_t st) {
  // Two vectors a lane (over four bits, two lanes a group), for whole vectors: fewer
  // instructions a row, but q, k and v go in passes of their own, one after another, and a
  // pass of few heads leaves lanes idle, so one vector a lane has the shorter way through
  // few tokens, and through more of them where heads are few.  Measured, one vector against
  // the other (us; bf16, 152 SMs; q heads on kv heads x channels, tokens):
  //                      32 on 8 x 128                      8 on 1 x 64                       16 on 16 x 80
  //                   600         3000       9000        3000       9000       27000       1000       4500
  //   rope, half     8.4  7.4   22.3 17.0   60.9 35.2    7.8 17.1   17.1 18.6   41.6 26.9    8.9  9.0   22.2 14.9
  //   16 bits as is  4.2  5.8    6.3  7.8   14.6 15.6    5.8 22.3   12.5 23.2   31.9 26.7    5.9  6.7   13.1 10.5
  //   16 bits, half  9.5  9.9   25.3 20.2   75.2 41.8    9.9 27.2   24.2 29.1   64.8 39.1   11.4 11.9   31.1 19.1
  //   16 bits, near  7.9 10.4   16.6 21.1   53.5 46.3    7.9 27.4   18.5 29.8   47.4 40.1    8.9 11.5   24.2 19.1
  //   Q8 as is       5.3 13.0    8.9 15.4   21.7 19.5    8.8  9.3   21.7  9.8   57.5 10.0    8.4 14.4   20.6 18.7
  //   Q8, half      11.4 17.0   29.8 25.2   87.3 51.2   12.9 14.5   33.0 16.6   90.3 22.7   14.5 18.1   38.3 26.0
  //   Q8, near       9.4 19.1   21.3 29.5   64.8 60.1   10.9 16.0   27.4 18.6   73.5 26.3   12.4 20.2   30.9 28.2
  //   Q4 as is       5.8 13.1    9.9 15.6   24.3 19.4    8.9  8.9   22.2  9.4   58.0  9.9    9.9 12.4   24.2 18.1
  //   Q4, half      11.4 12.9   30.4 26.4   87.3 53.0   12.9 12.5   33.5 14.4   91.3 22.7   15.3 16.1   41.7 27.3
  //   Q4, near       9.4 12.5   21.3 25.9   64.4 52.2   10.8 12.9   27.8 14.4   73.0 22.1   13.1 15.6   34.5 25.2
  // Hence a least number of tokens per SM, fixed + by_pass * (the sum over the passes of 1 /
  // (lanes of a row x heads)).  Over nine shapes from 1 to 64 heads at 300 to 60000 tokens the
  // choice takes 0.7 % longer than the faster kernel on average and 27 % at most.
  // Interleaved rope is as fast either way where rows fill the lanes of one vector each
  // (16000 tokens x 80 heads x 128: 111 118; 76000 x 40: 265 276) and stays there.
  struct Least {
    double fixed, by_pass;
  };
  constexpr Least kAsIs[4] = {{0, 0}, {14, 500}, {28, 0}, {28, 0}};   // (rope has no row as it is)
  constexpr Least kApart[4] = {{1, 500}, {1, 300}, {10, 50}, {14, 0}};
  constexpr Least kNear[4] = {{8, 1200}, {14, 500}, {24, 0}, {28, 0}};
  const bool apart = p.inv_freq != nullptr && !p.interleaved;
  const bool neighbours = p.inv_freq != nullptr && p.interleaved;
  const Least least = apart ? kApart[mode] : neighbours ? kNear[mode] : kAsIs[mode];
  const double passes = ((p.Hq > 0 ? 1.0 / p.Hq : 0.0) +
                         (p.Hkv > 0 ? (mode == 0 ? 1.0 : 2.0) / p.Hkv : 0.0)) /
                        (p.D <= 64 ? 8 : 16);
  const bool pairs = p.vec && p.T >= (least.fixed + least.by_pass * passes) * sms &&
                     !(apart && p.R % 16 != 0) && !(neighbours && mode == 0 && p.D % 64 == 0);
  if (pairs) {
    if (mode == 3)
      return bf16 ? launch_pairs<3, true>(p, sms, st) : launch_pairs<3, false>(p, sms, st);
    if (mode == 0)
      return bf16 ? launch_pairs<0, true>(p, sms, st) : launch_pairs<0, false>(p, sms, st);
    if (mode == 1)
      return bf16 ? launch_pairs<1, true>(p, sms, st) : launch_pairs<1, false>(p, sms, st);
    return bf16 ? launch_pairs<2, true>(p, sms, st) : launch_pairs<2, false>(p, sms, st);
  }
  if (mode == 0) return launch_mode<0>(p, bf16, sms, st);
  if (mode == 1) return launch_mode<1>(p, bf16, sms, st);
  if (mode == 2) return launch_mode<2>(p, bf16, sms, st);
  return launch_mode<3>(p, bf16, sms, st);
}

}  // namespace sage
