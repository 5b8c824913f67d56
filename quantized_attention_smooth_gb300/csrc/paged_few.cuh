// Attention of few new tokens per sequence over the paged cache (decoding,
// checking drafted tokens): bound by reading the cache once.
//
//   x_jr = c q_r . K_j  (base 2, fp32),  m_r a reference near max_j x_jr,
//   O_r  = sum_j 2^(x_jr - m_r) V_j,  l_r = sum_j 2^(x_jr - m_r),  out = O / l
//
// The rows of one (sequence, kv head) are its new tokens times the query heads
// of the group, so a key is loaded once for all of them.  The products run
// transposed, S^T = K Q^T and O^T = V^T P^T, on m16n8k16 tensor instructions:
// 16 keys (or channels) by 8 rows, which wastes nothing at a group of 8 or a
// few tokens of 2 or 4.  A contraction's order is free, so each lane takes the
// operands as whole 16-byte vectors of the cache: 4 lanes cover 64 bytes of a
// key for S^T, 8 lanes 128 bytes of a value row for O^T, and the fragments are
// put together by byte permutes.  Every warp streams blocks of 16 keys through a
// ring of its own in shared memory, by asynchronous copies two or three blocks
// ahead, with no barrier in the loop.  S^T's accumulators become P^T's operands
// by an 8x8 register transpose.
//
// Work is cut into units of 4 warps x 16 keys and dealt evenly to a fixed grid:
// every CTA derives its own contiguous range from the lengths (a scan over the
// sequences), so ragged batches balance and no length comes to the host.  A (sequence, head) that spans CTAs leaves fp32
// parts (max, sum, O) in the workspace, two per CTA at most; whoever finishes
// last (or a second kernel) joins them in the order of their ranges, so results
// do not depend on timing.
//
// Measured on GB300 (events around graphs of four calls): 64 sequences of
// 1024-16384 keys, 32 query heads on 8 kv heads of 128 channels, 350 us bf16
// (6.56 TB/s of K and V, 96 % of the measured copy bandwidth) and 196 us 8-bit
// (5.65 TB/s, 83 %; its conversions issue in 58 % of the cycles).  With K and V
// straight into registers, a block ahead, they took 357 and 212 us: too few bytes
// in flight for the loads' latency.  One sequence of 777 keys, 11.4 us: the plan,
// the loads' latency and the join in turn, next to no bytes.  A head of its own
// keys for each query head (D = 80, 16 heads) reaches 3.7 TB/s: seven rows of
// eight in a tile are empty and the arithmetic is the same.
//
// P is rounded to the 16-bit type of the tensor instruction (by up to 2^-8 of it in
// bf16, 2^-11 in fp16, as the output's own rounding); the sum l takes it unrounded.
// The 8-bit cache's codes are exact in fp16: K codes |n| <= 127, e4m3 values <= 448;
// bf16 queries are scaled per row by a power of two first.
//
// The 4-bit cache: x_j = sum over groups of s_jg (sum of q n over the group's channels),
// O_c = sum_j (P_j s_jg) n_jc, both on fp16 products of exact codes.  Eight rows of
// one group's 16 bytes are what ldmatrix moves: as they stand the A operands of S^T,
// transposed those of O^T, whose tiles then have one group each, so that a group's
// scale multiplies S^T's partial sums and P, in fp32.  Blocks are 32 keys (16 where
// registers are short: 171 us with them below); a fifth warp fills the others' rings by
// tensor copies and goes on to the next item while they join the last.  64 x 8520
// keys of 32 heads on 8 x 128: 161 us, 3.90 TB/s, 58 % of the measured copy bandwidth.
// No pipe is full (issue slots 50 %, ALU 42 %): the 12 warps an SM that 128 registers a
// thread leave wait for their own results through 660 instructions a step, and the
// copies alone take 128 us.  The first form, with 16 keys a step and copies by the
// warps themselves, took 205.

#pragma once

#include <atomic>
#include <type_traits>

#include "sage_kernels.h"
#include "sage_paged_device.cuh"

namespace sage {
namespace {

constexpr int kWarps = 4;                 // that take the keys
constexpr int kMaxCtas = 152 * 8;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kJoinInside = 40;   // most parts of an item, on average, that one CTA joins
static_assert(kMaxCtas * 4 <= kArrivalBytes, "a counter for every CTA");

// One part of a split item (in the workspace).
struct PartHead {
  int32_t parts, seq, head, tile;   // parts of the item from this one on; 0: none here
};
constexpr int kMaxRows = 32;
constexpr size_t kPartBytes = sizeof(PartHead) + kMaxRows * 8 + kMaxRows * 128 * 4;

// The CTA whose range holds unit x, where CTA i's begins at total i / busy.
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int busy) {
  return static_cast<int>(((x + 1) * busy - 1) / total);
}

__device__ __forceinline__ uint8_t* part_at(uint8_t* parts, int cta, int which) {
  return parts + (static_cast<size_t>(cta) * 2 + which) * kPartBytes;
}

// A part's maxima, sums and O.
__device__ __forceinline__ const float* part_floats(uint8_t* parts, int cta, int which) {
  return reinterpret_cast<const float*>(part_at(parts, cta, which) + sizeof(PartHead));
}

struct Units {
  int per, tiles;            // units of one item; row tiles of one kv head
  int64_t total;
};
template <int kRows, int kUnitBlocks, int kKeys>
__device__ __forceinline__ Units units_of(const PagedAttnParams& p, int s, int* start, int* n,
                                          int* len, int team) {
  Units u{0, 0, 0};
  if (!paged_seq(p.c, s, start, n, len)) return u;
  const int64_t rows = static_cast<int64_t>(*n) * p.group;
  if (rows < p.min_rows || rows > p.max_rows || rows == 0) return u;
  const Span sp = span_of<kKeys>(*len - *n, *len - 1, p.window, p.sinks);
  u.per = max(1, (sp.count + kUnitBlocks - 1) / kUnitBlocks);
  u.tiles = static_cast<int>((rows + kRows - 1) / kRows);
  u.total = static_cast<int64_t>(u.per) * u.tiles * (p.c.Hkv / team);
  return u;
}

template <bool kBF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kBF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// A barrier of the warps that take the keys (4 bits: a fifth one is elsewhere).
template <bool kSome>
__device__ __forceinline__ void workers_barrier() {
  if constexpr (kSome) asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
  else __syncthreads();
}

// Four 8x8 matrices of 16 bits from shared memory, a row of 16 bytes from each lane's
// address: lane 4 g + t gets word t of row g, or transposed halfword g of rows 2t, 2t + 1.
template <bool kTrans>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

// fp16 products on top of sums that stay as they are.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
               "{%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
                 "f"(c3));
}

// 16 rows of codes by the group: of rows 0-7 and 8-15 (kG 4 or 2 groups).
template <bool kTrans, int kG>
__device__ __forceinline__ void load_codes(uint32_t (&lo)[kG], uint32_t (&hi)[kG], uint32_t at) {
  if constexpr (kG == 4) {
    ldmatrix4<kTrans>(lo, at);
    ldmatrix4<kTrans>(hi, at + 8 * 64);
  } else {
    uint32_t w[4];
    ldmatrix4<kTrans>(w, at);
    lo[0] = w[0]; lo[1] = w[1]; hi[0] = w[2]; hi[1] = w[3];
  }
}

// A row's scales (kG halves).
template <int kG>
__device__ __forceinline__ void row_scales(uint32_t at, float (&s)[kG]) {
  uint32_t w[2] = {0, 0};
  if constexpr (kG == 4)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < kG / 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    s[2 * i] = f.x;
    s[2 * i + 1] = f.y;
  }
}
// A nibble u in the lowest bits of an fp16 is the number u 2^-24, four bits higher
// u 2^-20, exactly: a mask makes two operands of eight codes, and -8 of each comes off
// the sums (K).  Values become numbers n = u - 8 first, since their sums may be far
// smaller than the weights that 8 of each would add.
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
constexpr uint32_t kMinus8 = 0x80088008u, kMinus8x16 = 0x80808080u;    // -8 in both forms

// The part of a (sequence, kv head, row tile) that a CTA is at, and where it
// stands in its range of units: in shared memory, since registers that kept it
// through the loop over the keys would cost the loop spills.
struct FewItem {
  int64_t cur, off, last, total;   // unit; unit within the sequence; past the range; all
  int busy;                        // CTAs that share them
  int s, start, rows, base, head, tile, first, count, per;
  int first_cta, parts, joins;     // of a split item; whether this CTA joins it
  Span span;
};

// kForm: 0 D = Dp, every vector of a row is loaded; 1 vectors from D on are not; 2
// so too, and rows of the 8-bit cache go in 8 bytes at a time (D or a stride is an
// odd multiple of 8, so that they end or start on 8 bytes only).
// A warp's ring of blocks in shared memory, and the merge buffer that takes its
// place at an item's end.
template <int kKind, int kDp, int kNr>
struct Few {
  static constexpr int kRowB =                                        // bytes of a row
      kKind == kKindQ4 ? kDp / 2 : kDp * (kKind == kKindQ8 ? 1 : 2);
  static constexpr int kScaleB = kDp / 16;                            // a 4-bit row's scales
  // keys of a block: 32 of 4 bits as far as registers go
  static constexpr int kKeys = kKind == kKindQ4 && kNr * kDp <= 128 ? 32 : 16;
  static constexpr int kBlockB =                                      // K, V, scales
      2 * kKeys * kRowB + (kKind == kKindQ8 ? 64 : kKind == kKindQ4 ? 512 : 0);
  static constexpr int kStages = kKind == kKindQ4 ? (kDp * kKeys == 4096 ? 3 : 4)
                                                     : kRowB == 64 ? 4 : 3;
  // where a 4-bit block's scales lie, of keys and 256 bytes on of values: 16 rows on 128
  // bytes, as a tensor copy wants them
  static constexpr int kScales = 2 * kKeys * kRowB;
  static constexpr int kPitch = kDp + 4;
  static constexpr int kRing = kWarps * kStages * kBlockB;
  static constexpr int kMerge = kWarps * 8 * kNr * kPitch * 4;
  // (4 bits: beside the rings, which already take the next item's blocks)
  static constexpr int kMergeAt = kKind == kKindQ4 ? kRing : 0;
  static constexpr int kSmem = kMergeAt + (kRing - kMergeAt > kMerge ? kRing - kMergeAt : kMerge);
  static constexpr int kCtas = kRowB == 256 || kNr > 2 ? 2
                               : kNr == 2 ? (kDp == 128 ? 2 : 3)
                               : kKind == kKindQ4 ? 3 : 4;
  // 4 bits: a fifth warp makes the copies of the other four
  static constexpr int kThreads = kKind == kKindQ4 ? 160 : 128;
};

// Tensor maps of a 4-bit cache's codes, K and V.
struct Maps4 {
  CUtensorMap t[2];
};
struct NoMaps {};
template <int kKind>
using Maps = std::conditional_t<kKind == kKindQ4, Maps4, NoMaps>;

template <int kKind, bool kQBF16, int kDp, int kNr, int kForm>
__global__ void __launch_bounds__(Few<kKind, kDp, kNr>::kThreads, Few<kKind, kDp, kNr>::kCtas)
paged_few_kernel(const PagedAttnParams p, const __grid_constant__ Maps<kKind> maps) {
  constexpr bool kQ8 = kKind == kKindQ8, kQ4 = kKind == kKindQ4;
  constexpr bool kMmaBF16 = kKind == kKindBF16;
  constexpr float kDown = kBelow<kMmaBF16>, kOver = kLazy + kDown;
  constexpr int kRows = 8 * kNr;
  constexpr int kUnitBlocks = kWarps;                     // a unit: a block of each warp
  constexpr int kEl = kQ8 || kQ4 ? 1 : 2;                 // bytes of an element
  constexpr int kKw = kQ8 ? kDp / 16 : kDp / 8;           // words of a key per lane
  constexpr int kVw = kQ8 ? kDp / 32 : kDp / 16;          // words of a value per lane
  constexpr int kMt = kDp / 16;                           // 16-channel tiles of O^T
  using L = Few<kKind, kDp, kNr>;
  constexpr int kPitch = L::kPitch, kRowB = L::kRowB, kStages = L::kStages, kKeys = L::kKeys;
  constexpr int kSubs = kKeys / 16;                       // 16 keys to a product
  constexpr int kThreads = L::kThreads;
  constexpr int kChunks = kRowB / 16;                     // 16-byte vectors of a row
  extern __shared__ __align__(1024) uint8_t ring_s[];
  float (*const acc_s)[kRows * kPitch] = reinterpret_cast<float (*)[kRows * kPitch]>(ring_s + L::kMergeAt);
  __shared__ int64_t scan_s[kThreads / 32];
  __shared__ FewItem it_s[kQ4 ? 2 : 1];         // the item at hand (4 bits: and the next one)
  // 4 bits: each warp's stages, filled and read; the first key of a stage's block
  constexpr int kRings = kQ4 ? kWarps * kStages : 1;
  __shared__ uint64_t full_s[kRings], empty_s[kRings];
  __shared__ int key_s[kRings];
  __shared__ volatile int abort_s, stop_s[2];
  __shared__ float m_s[kWarps][kRows], l_s[kWarps][kRows];

  const PagedGeo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x;
  // Teams of CTAs work on as many heads side by side (4 bits only, see launch_few).
  const int team = kQ4 ? p.team : 1, member = kQ4 ? cta % team : 0;
  const int seat = kQ4 ? cta / team : cta, seats = kQ4 ? gridDim.x / team : gridDim.x;
  uint8_t* const ring = ring_s + warp * kStages * L::kBlockB;
  // where a vector of a key lies in a block (4 bits: eight rows of one vector, as ldmatrix
  // takes them)
  auto k_at = [](int row, int vec) {
    if constexpr (kQ4) return row * kRowB + ((vec ^ ((row >> (kChunks == 4 ? 1 : 2)) & (kChunks - 1))) << 4);
    return row * kRowB + ((kChunks >= 8 ? vec ^ ((row & 1) << 2) : vec) << 4);
  };
  if (!p.join_inside) asm volatile("griddepcontrol.launch_dependents;");

  if constexpr (kQ4) {
    if ((smem_u32(ring_s) & 511u) != 0) {       // the copies' swizzle goes by the address
      if (tid == 0) atomicOr(c.status, kStatusBadItem);
      if (tid < 2) reinterpret_cast<PartHead*>(part_at(p.parts, cta, tid))->parts = 0;
      return;
    }
    if (tid == 0) {
      abort_s = 0;
      for (int i = 0; i < kRings; ++i) {
        mbar_init(&full_s[i], 1 + 8);           // codes; the lanes that copy scales
        mbar_init(&empty_s[i], 1);
      }
      mbar_fence_init();
    }
  }
  // 4 bits: 32-bit shared addresses, and this lane's part of those that the loop reads:
  // rows 8 and 16 further and the values lie at fixed distances
  const uint32_t ring_u = smem_u32(ring);
  const uint32_t mat_off = kDp == 128 ? k_at(lane & 7, lane >> 3)
                                      : k_at((lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1);
  const uint32_t key_scales = 2 * kKeys * kRowB + g * L::kScaleB;
  const uint32_t val_scales = 2 * kKeys * kRowB + 256 + g * L::kScaleB;
  int stage4 = 0;                               // the stage at hand and its round's parity
  uint32_t parity4 = 0;
  bool ok = true;
  auto next_stage = [&] {
    if (++stage4 == kStages) {
      stage4 = 0;
      parity4 ^= 1u;
    }
  };
  // ---- this CTA's range of units
  const int per_thread = (c.nseq + kThreads - 1) / kThreads;
  const int s_begin = min(c.nseq, tid * per_thread), s_end = min(c.nseq, s_begin + per_thread);
  int64_t mine = 0;
  for (int s = s_begin; s < s_end; ++s) {
    int a, n, len;
    mine += units_of<kRows, kUnitBlocks, L::kKeys>(p, s, &a, &n, &len, team).total;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(kAll, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) scan_s[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan_s[w];
    total += scan_s[w];
  }
  const int64_t end = before + incl, begin = end - mine;
  // no CTA between two parts of an item is left without a unit: the join walks
  // from CTA to CTA
  const int64_t busy = min(total, static_cast<int64_t>(seats));
  const int64_t u0 = seat < busy ? total * seat / busy : 0;
  const int64_t u1 = seat < busy ? total * (seat + 1) / busy : 0;
  bool used[2] = {false, false};
  if (u0 < u1) {
    if (begin <= u0 && u0 < end) {                        // one thread
      int64_t off = u0 - begin;
      int s = s_begin;
      for (; s < s_end; ++s) {
        int a, n, len;
        const int64_t w = units_of<kRows, kUnitBlocks, L::kKeys>(p, s, &a, &n, &len, team).total;
        if (off < w) break;
        off -= w;
      }
      FewItem& it = it_s[0];
      it.s = s;
      it.off = off;
      it.cur = u0;
      it.last = u1;
      it.total = total;
      it.busy = static_cast<int>(busy);
    }
    __syncthreads();
    // an item from where its CTA stands in its range (count 0: none left), by one thread
    auto seek = [&](FewItem& it) {
        it.count = 0;
        while (it.cur < it.last && it.s < c.nseq) {
          int start, n, len;
          const Units un =
              units_of<kRows, kUnitBlocks, L::kKeys>(p, it.s, &start, &n, &len, team);
          if (it.off >= un.total) {                       // an empty sequence
            it.off = 0;
            ++it.s;
            continue;
          }
          const int64_t item = it.off / un.per;
          it.first = static_cast<int>(it.off - item * un.per);
          it.count = static_cast<int>(
              min(static_cast<int64_t>(un.per - it.first), it.last - it.cur));
          it.per = un.per;
          const int heads = static_cast<int>(item / un.tiles);
          it.head = heads * team + member;
          it.tile = static_cast<int>(item - static_cast<int64_t>(heads) * un.tiles);
          it.start = start;
          it.rows = n * p.group;
          it.base = len - n;
          it.span = span_of<L::kKeys>(len - n, len - 1, p.window, p.sinks);
          break;
        }
    };
    // 4 bits: the fifth warp's copies of units from..to-1 of an item: lanes 8 w .. 8 w + 7
    // serve warp w, by 16 keys, which share a page: codes of K and V by a tensor copy each,
    // their scales by 16 bytes a lane.  (By tensor copies as well they took longer than
    // the codes: 128 us for the copies of 64 x 8520 keys alone, 103 without.)  Pages that
    // are not there, and 16 keys that no row sees, lie outside and read zeros.
    auto send = [&](const FewItem& it, int from, int to) {
      if constexpr (kQ4) {
        const int w = lane >> 3, j8 = lane & 7, kv = j8 & 1, half = j8 >> 1;
        const Span sp = it.span;
        const int row0 = it.tile * kRows, kvh = it.head;
        const int p_hi = it.base + (min(row0 + kRows, it.rows) - 1) / p.group;
        const int sinks = p.window > 0 ? p.sinks : 0;
        const int lo = p.window > 0 ? max(0, it.base + row0 / p.group - p.window + 1) : 0;
        const int32_t* const table = c.table + it.s * c.table_stride;
        uint8_t* const dst = ring_s + w * kStages * L::kBlockB;
        const uint32_t dst_u = smem_u32(dst) + L::kScales + 16 * j8;
        const CUtensorMap* const map = &maps.t[kv];
        const int64_t page_b = static_cast<int64_t>(c.Hkv) * c.page_size * L::kScaleB;
        const int64_t head_b = static_cast<int64_t>(kvh) * c.page_size * L::kScaleB + 16 * j8;
        int k0 = -1, page[kSubs], slot[kSubs];
        bool need[kSubs];
        // a block's first key and its pages; the table's entries are used a step later, and
        // nothing here waits for them (64 x 8520 keys: 162 us, with a bound on them 180)
        auto locate = [&](int u) {
          const int vb = u * kWarps + w;
          k0 = kKeys * (vb < sp.sink ? vb : vb - sp.sink + sp.from);
          if (!(vb < sp.count && k0 <= p_hi && (k0 + kKeys - 1 >= lo || k0 < sinks))) k0 = -1;
#pragma unroll
          for (int h = 0; h < kSubs; ++h) {
            const int kh = k0 + 16 * h;
            need[h] = k0 >= 0 && kh <= p_hi && (kh + 15 >= lo || kh < sinks);
            page[h] = -1;
            slot[h] = 0;
            if (need[h]) {
              const int pn = page_of(c, kh);
              page[h] = table[pn];
              slot[h] = kh - pn * c.page_size;
            }
          }
        };
        if (from < to) locate(from);
        for (int u = from; ok && u < to; ++u) {
          const int ring_at = w * kStages + stage4;
          ok = __all_sync(kAll, mbar_wait(&empty_s[ring_at], parity4 ^ 1u, &abort_s, c.status,
                                          p.timeout_ns));
          if (!ok) break;
          if (j8 == 0) {
            key_s[ring_at] = k0;
            if (k0 >= 0) mbar_expect_tx(&full_s[ring_at], 2 * kKeys * kRowB);
            else mbar_arrive(&full_s[ring_at]);
          }
          __syncwarp();
          if (k0 >= 0) {
#pragma unroll
            for (int h = 0; h < kSubs; ++h) {
              const bool there =
                  static_cast<uint32_t>(page[h]) < static_cast<uint32_t>(c.num_pages);
              if (!there && need[h]) atomicOr(c.status, kStatusBadPage);
              if (half == h)
                tma_load_4d(dst + stage4 * L::kBlockB + (kv * kKeys + 16 * h) * kRowB, map, 0,
                            slot[h], kvh, there ? page[h] : static_cast<int>(c.num_pages),
                            &full_s[ring_at]);
              if (L::kScaleB == 8 || j8 < 4) {
                const int64_t at = there ? page[h] * page_b + head_b + slot[h] * L::kScaleB : 0;
                const uint32_t to_u = dst_u + stage4 * L::kBlockB + 128 * h;
                copy16(to_u, reinterpret_cast<const uint8_t*>(c.k_groups) + at, there ? 16 : 0);
                copy16(to_u + 256, reinterpret_cast<const uint8_t*>(c.v_groups) + at,
                       there ? 16 : 0);
              }
            }
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];"
                       :: "r"(smem_u32(&full_s[ring_at])) : "memory");
          __syncwarp();
          next_stage();
          if (u + 1 < to) locate(u + 1);
        }
      }
    };
    if (kQ4 && tid == 32 * kWarps) seek(it_s[0]);
    int nth = 0, sent = 0;                      // items begun; blocks of the item sent ahead
    while (true) {
      FewItem& it = it_s[kQ4 ? nth & 1 : 0];
      if (!kQ4 && tid == 0) seek(it);
      if (kQ4 && tid == 0) stop_s[nth & 1] = abort_s;
      __syncthreads();                          // 4 bits: the warps are through with the last item
      const int count = it.count, first_unit = it.first;
      if (count == 0 || (kQ4 && stop_s[nth & 1])) break;
      ++nth;
      if (kQ4 && warp == kWarps) {
        // the rest of this item's blocks, then the first ones of the next item, which
        // are on their way while the other warps join their parts of this one
        send(it, first_unit + sent, first_unit + count);
        FewItem& next = it_s[nth & 1];
        if (lane == 0) {                        // (the rest of `it` is the other warps')
          next.cur = it.cur + count;
          next.off = it.off + count;
          next.last = it.last;
          next.total = it.total;
          next.busy = it.busy;
          next.s = it.s;
          seek(next);
        }
        __syncwarp();
        sent = min(next.count, kStages);
        send(next, next.first, next.first + sent);
        continue;
      }
      const int row0 = it.tile * kRows;
      const int kvh = it.head, s = it.s;
      const Span sp = it.span;
      const int p_lo = it.base + row0 / p.group;
      const int p_hi = it.base + (min(row0 + kRows, it.rows) - 1) / p.group;
      const int sinks = p.window > 0 ? p.sinks : 0;
      const int lo = p.window > 0 ? max(0, p_lo - p.window + 1) : 0;        // first key of row0
      const int lo_hi = p.window > 0 ? max(0, p_hi - p.window + 1) : 0;     // of the last row

      const int end_unit = first_unit + count;
      // ---- the rows' queries, as the B operand of S^T
      uint32_t qw[kNr][kDp / 8];
      float qoff[kNr][kQ4 ? kDp / 32 : 1][2];             // 4 bits: -8 sum q of a group
      float rs[kNr][2];                                   // logit scale of rows 2t, 2t + 1
      int rpos[kNr][2];
#pragma unroll
      for (int nr = 0; nr < kNr; ++nr) {
        const int r = row0 + 8 * nr + g;
        const bool has = r < it.rows;
        const uint16_t* qrow = p.q + (static_cast<int64_t>(it.start) + r / p.group) * p.q_tok +
                               (static_cast<int64_t>(kvh) * p.group + r % p.group) * p.q_head;
#pragma unroll
        for (int i = 0; i < kDp / 32; ++i) {
          const int ch = kQ8 ? 64 * (i / 2) + 16 * t + 8 * (i % 2) : 32 * i + 8 * t;   // 8 channels
          uint32_t* w = &qw[nr][4 * i];
          w[0] = w[1] = w[2] = w[3] = 0;
          if (has && ch < c.D) {
            if (p.q_vec) {
              const uint4 v = *reinterpret_cast<const uint4*>(qrow + ch);
              w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e / 2] |= static_cast<uint32_t>(qrow[ch + e]) << (16 * (e & 1));
            }
          }
        }
        float row_scale = p.scale_log2;
        if constexpr (kQ4) {
          // Into fp16's range, times 2^(12 - e), e the exponent of the largest; channels
          // 0 and 4 of eight side by side, 1 and 5, ..., as the codes are taken apart;
          // odd ones times 2^-4, for their codes come as 16 n.
          auto lo = [](uint32_t w) {
            return kQBF16 ? __uint_as_float(w << 16)
                          : __low2float(*reinterpret_cast<const __half2*>(&w));
          };
          auto hi = [](uint32_t w) {
            return kQBF16 ? __uint_as_float(w & 0xFFFF0000u)
                          : __high2float(*reinterpret_cast<const __half2*>(&w));
          };
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < kDp / 8; ++i)
            top = fmaxf(top, fmaxf(fabsf(lo(qw[nr][i])), fabsf(hi(qw[nr][i]))));
          top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
          top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
          const int e = exponent_of(top);
          const float down = power_of_2(-e), even = 4096.0f, odd = 256.0f;
#pragma unroll
          for (int i = 0; i < kDp / 32; ++i) {
            uint32_t* w = &qw[nr][4 * i];
            const uint32_t u[4] = {w[0], w[1], w[2], w[3]};
            w[0] = pack2<false>(lo(u[0]) * down * even, lo(u[2]) * down * even);
            w[1] = pack2<false>(hi(u[0]) * down * odd, hi(u[2]) * down * odd);
            w[2] = pack2<false>(lo(u[1]) * down * even, lo(u[3]) * down * even);
            w[3] = pack2<false>(hi(u[1]) * down * odd, hi(u[3]) * down * odd);
            // codes hold n + 8: the products start from minus 8 of everything
            float off[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma<false>(off, kMinus8, kMinus8, kMinus8x16, kMinus8x16, w[0], w[1]);
            mma<false>(off, kMinus8, kMinus8, kMinus8x16, kMinus8x16, w[2], w[3]);
            qoff[nr][i][0] = off[0];
            qoff[nr][i][1] = off[1];
          }
          row_scale = row_scale * power_of_2(e) * 4096.0f;  // 2^-12 of the queries, 2^24 of the codes
        }
        if constexpr (kQ8 && kQBF16) {
          // bf16 queries into fp16's range: times 2^-e, e the exponent of the largest
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < kDp / 8; ++i) {
            top = fmaxf(top, fabsf(__uint_as_float(qw[nr][i] << 16)));
            top = fmaxf(top, fabsf(__uint_as_float(qw[nr][i] & 0xFFFF0000u)));
          }
          top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
          top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
          const int e = exponent_of(top);
          const float down = power_of_2(-e);
#pragma unroll
          for (int i = 0; i < kDp / 8; ++i)
            qw[nr][i] = pack2<false>(__uint_as_float(qw[nr][i] << 16) * down,
                                     __uint_as_float(qw[nr][i] & 0xFFFF0000u) * down);
          row_scale *= power_of_2(e);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          rs[nr][i] = __shfl_sync(kAll, row_scale, (2 * t + i) * 4);
          const int rr = row0 + 8 * nr + 2 * t + i;
          rpos[nr][i] = rr < it.rows ? it.base + rr / p.group : -1;
        }
      }

      float o[kMt][kNr][4], m[kNr][2], l[kNr][2];
#pragma unroll
      for (int nr = 0; nr < kNr; ++nr) {
        m[nr][0] = m[nr][1] = -INFINITY;
        l[nr][0] = l[nr][1] = 0.0f;
#pragma unroll
        for (int j = 0; j < kMt; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][nr][e] = 0.0f;
      }

      auto seen = [&](int j) { return j <= p_hi && (j >= lo || j < sinks); };
      if constexpr (kQ4) {
        constexpr int kG = kDp / 32, kX = kSubs * kNr;
        // waits for the block in a stage; its first key (-1: nothing that a row sees)
        auto take = [&](int at) {
          ok = __all_sync(kAll, mbar_wait(&full_s[at], parity4, &abort_s, c.status, p.timeout_ns));
          return ok ? key_s[at] : -1;
        };
        // ---- S^T of a block, times its rows' factors
        auto logits = [&](uint32_t base, float (&x)[kX][4]) {
          // lane: word t of a group of keys g and g + 8
#pragma unroll
          for (int sub = 0; sub < kSubs; ++sub) {
            uint32_t wa[kG], wb[kG];
            load_codes<false, kG>(wa, wb, base + mat_off + 16 * sub * kRowB);
            float sa[kG], sb[kG];
            row_scales<kG>(base + key_scales + 128 * sub, sa);
            row_scales<kG>(base + key_scales + 128 * sub + 8 * L::kScaleB, sb);
            if constexpr (kForm != 0)           // groups behind D: anything
#pragma unroll
              for (int i = 0; i < kG; ++i)
                if (32 * i >= c.D) sa[i] = sb[i] = 0.0f;
#pragma unroll
            for (int i = 0; i < kG; ++i) {
              const uint32_t ua = wa[i] >> 8, ub = wb[i] >> 8;
#pragma unroll
              for (int nr = 0; nr < kNr; ++nr) {
                float y[4], z[4];
                float (&w)[4] = x[sub * kNr + nr];
                mma_from(y, wa[i] & kLow, wb[i] & kLow, wa[i] & kHigh, wb[i] & kHigh,
                         qw[nr][4 * i], qw[nr][4 * i + 1], qoff[nr][i][0], qoff[nr][i][1],
                         qoff[nr][i][0], qoff[nr][i][1]);
                mma_from(z, ua & kLow, ub & kLow, ua & kHigh, ub & kHigh, qw[nr][4 * i + 2],
                         qw[nr][4 * i + 3], y[0], y[1], y[2], y[3]);
                w[0] = i == 0 ? sa[i] * z[0] : w[0] + sa[i] * z[0];
                w[1] = i == 0 ? sa[i] * z[1] : w[1] + sa[i] * z[1];
                w[2] = i == 0 ? sb[i] * z[2] : w[2] + sb[i] * z[2];
                w[3] = i == 0 ? sb[i] * z[3] : w[3] + sb[i] * z[3];
              }
            }
          }
#pragma unroll
          for (int sn = 0; sn < kX; ++sn)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[sn][e] *= rs[sn % kNr][e & 1];
        };
        // ---- masks, running maximum and sum, O^T
        auto weigh = [&](uint32_t base, float (&x)[kX][4], int cur0) {
          // (branches once for the block: a test per logit costs as much as the logits)
          const bool full_block =
              cur0 + kKeys - 1 <= p_lo && (cur0 >= lo_hi || cur0 + kKeys - 1 < sinks);
          if (!full_block) {
#pragma unroll
            for (int sn = 0; sn < kX; ++sn)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = cur0 + 16 * (sn / kNr) + g + 8 * (e >> 1);
                const int pos = rpos[sn % kNr][e & 1];
                if (!(j <= pos && (p.window <= 0 || j > pos - p.window || j < sinks)))
                  x[sn][e] = -INFINITY;
              }
          }
          bool over = false;                    // a logit has outgrown its row's reference
          float top[kNr][2];
#pragma unroll
          for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              top[nr][i] = fmaxf(x[nr][i], x[nr][i + 2]);
              if constexpr (kSubs == 2)
                top[nr][i] = fmaxf(top[nr][i], fmaxf(x[kNr + nr][i], x[kNr + nr][i + 2]));
              over |= top[nr][i] > m[nr][i] + kOver;    // with m = -inf: any logit but -inf
            }
          if (__any_sync(kAll, over)) {
            // Rare after the first block: references move with the maximum, O and l
            // follow.
            float alpha[kNr][2];
#pragma unroll
            for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float v = top[nr][i];
                v = fmaxf(v, __shfl_xor_sync(kAll, v, 4));
                v = fmaxf(v, __shfl_xor_sync(kAll, v, 8));
                v = fmaxf(v, __shfl_xor_sync(kAll, v, 16));
                const float next = v > m[nr][i] + kOver ? v - kDown : m[nr][i];
                alpha[nr][i] = next == m[nr][i] ? 1.0f : fast_exp2(m[nr][i] - next);
                m[nr][i] = next;
                l[nr][i] *= alpha[nr][i];
              }
#pragma unroll
            for (int j = 0; j < kMt; ++j)
#pragma unroll
              for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][nr][e] *= alpha[nr][e & 1];
          }
          // lane: channels 4 g .. 4 g + 3 of each group, of keys 2t and 2t + 1 (lo), and
          // of those 8 further (hi); a value's scale goes into P, by the group
          float safe[kNr][2];
#pragma unroll
          for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i) safe[nr][i] = m[nr][i] == -INFINITY ? 0.0f : m[nr][i];
#pragma unroll
          for (int sub = 0; sub < kSubs; ++sub) {
            float e4[kNr][4];
#pragma unroll
            for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                e4[nr][e] = fast_exp2(x[sub * kNr + nr][e] - safe[nr][e & 1]);
                l[nr][e & 1] += e4[nr][e];
              }
            uint32_t vl[kG], vh[kG];
            load_codes<true, kG>(vl, vh, base + mat_off + (kKeys + 16 * sub) * kRowB);
            // P times the scales of keys g and g + 8, rounded once, before P is turned round
            float sa[kG], sb[kG];
            row_scales<kG>(base + val_scales + 128 * sub, sa);
            row_scales<kG>(base + val_scales + 128 * sub + 8 * L::kScaleB, sb);
            if (!full_block) {                // scales that no row sees may be NaN
              const int j = cur0 + 16 * sub + g;
#pragma unroll
              for (int i = 0; i < kG; ++i) {
                if (!seen(j)) sa[i] = 0.0f;
                if (!seen(j + 8)) sb[i] = 0.0f;
              }
            }
#pragma unroll
            for (int i = 0; i < kG; ++i) {
              uint32_t n[2][4];               // the four channels, as numbers -8..7
              nibbles_to_half(vl[i], n[0]);
              nibbles_to_half(vh[i], n[1]);
#pragma unroll
              for (int nr = 0; nr < kNr; ++nr) {
                const uint32_t b0 =
                    transpose8x8(pack2<false>(e4[nr][0] * sa[i], e4[nr][1] * sa[i]));
                const uint32_t b1 =
                    transpose8x8(pack2<false>(e4[nr][2] * sb[i], e4[nr][3] * sb[i]));
                mma<false>(o[2 * i][nr], n[0][0], n[0][1], n[1][0], n[1][1], b0, b1);
                mma<false>(o[2 * i + 1][nr], n[0][2], n[0][3], n[1][2], n[1][3], b0, b1);
              }
            }
          }
        };
        for (int u = first_unit; ok && u < end_unit; ++u) {
          const uint32_t base = ring_u + stage4 * L::kBlockB;
          const int at = warp * kStages + stage4;
          const int cur0 = take(at);
          if (cur0 >= 0) {
            float x[kX][4];
            logits(base, x);
            weigh(base, x, cur0);
          }
          __syncwarp();                         // the block has been read
          if (lane == 0) mbar_arrive(&empty_s[at]);
          next_stage();
        }
      } else {
        const int32_t* const table = c.table + s * c.table_stride;
        const int64_t ts = c.token_stride * kEl;
        // Copies: lane -> vector lc of every kRows32-th row.  A vector's place in its row
        // is turned by the row, so that the reads below hit every bank once.
        constexpr int kRows32 = 32 / kChunks;
        const int lc = lane % kChunks, lr = lane / kChunks;
        const int lc_left = c.D - lc * (16 / kEl);          // channels from the vector's first on
        auto v_at = [](int row, int vec) {
          return (16 + row) * kRowB +
                 ((kChunks >= 8 ? vec ^ (row & 6) : vec ^ ((row >> 1) & 3)) << 4);
        };
        // this lane's vector in a block's keys and values (bytes)
        const int64_t lane_off = (kvh * c.head_stride + lr * c.token_stride) * kEl + 16 * lc;
        // Vectors of channels from D on are never loaded: zero once.
        if (kForm != 0) {
          for (int i = lane; i < kStages * L::kBlockB / 16; i += 32)
            reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
        // A step is a block of kKeys keys.  Its first key (-1: none that a row sees):
        auto key_of = [&](int unit) {
          const int vb = unit * kWarps + warp;
          const int k0 = kKeys * (vb < sp.sink ? vb : vb - sp.sink + sp.from);
          return vb < sp.count && k0 <= p_hi && (k0 + kKeys - 1 >= lo || k0 < sinks) ? k0 : -1;
        };
        int next_key0 = -1, next_page = -1;
        auto locate = [&](int unit) {             // the table's entry, used a step later
          next_key0 = key_of(unit);
          if (next_key0 >= 0) next_page = table[page_of(c, next_key0)];
        };
        // Starts the copies of the located block into a stage; rows that no row of
        // the tile sees become zero (0 times what lies there could be NaN).
        auto issue = [&](int stage) {
          const int k0 = next_key0;
          if (k0 >= 0) {
            int64_t at = 0;
            const bool there =
                static_cast<uint32_t>(next_page) < static_cast<uint32_t>(c.num_pages);
            const uint32_t dst = smem_u32(ring + stage * L::kBlockB);
            const float* scales = c.k_scale;
            if (there) {
              const int slot = k0 - page_of(c, k0) * c.page_size;
              at = (next_page * c.page_stride + static_cast<int64_t>(slot) * c.token_stride) * kEl;
              if (kQ8)
                scales += (static_cast<int64_t>(next_page) * c.Hkv + kvh) * c.page_size + slot +
                          4 * (lane & 3);
            } else if (lane == 0) {
              atomicOr(c.status, kStatusBadPage);
            }
            if (kQ8 && lane < 4)
              copy16(dst + 32 * kRowB + 16 * lane, reinterpret_cast<const uint8_t*>(scales),
                     there ? 16 : 0);
            const bool whole = there && k0 + 15 <= p_hi && (k0 >= lo || k0 + 15 < sinks);
            const uint8_t* src_k = c.k + at + lane_off;
            const uint8_t* src_v = c.v + at + lane_off;
            const int64_t down = kRows32 * ts;
#pragma unroll
            for (int i = 0; i < 16 / kRows32; ++i) {
              const int row = lr + i * kRows32;
              const bool see = whole || (there && seen(k0 + row));
              copy_part<kForm>(dst + k_at(row, lc), see ? src_k : c.k, see, lc_left);
              copy_part<kForm>(dst + v_at(row, lc), see ? src_v : c.v, see, lc_left);
              src_k += down;
              src_v += down;
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        locate(first_unit);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
          issue(i);
          next_key0 = -1;
          if (first_unit + i + 1 < end_unit) locate(first_unit + i + 1);
        }
        int stage = 0;
        for (int u = first_unit; u < end_unit; ++u) {
          asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 2) : "memory");
          __syncwarp();                           // every lane's copies; and the last stage is read
          issue(stage == 0 ? kStages - 1 : stage - 1);
          next_key0 = -1;
          if (u + kStages < end_unit) locate(u + kStages);
          const uint8_t* const block = ring + stage * L::kBlockB;
          stage = stage + 1 == kStages ? 0 : stage + 1;
          // ---- S^T, in two chains of products
          const int cur0 = key_of(u);
          if (cur0 < 0) continue;
          float x[kNr][4], x2[kNr][4];
#pragma unroll
          for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nr][e] = x2[nr][e] = 0.0f;
#pragma unroll
          for (int v = 0; v < kKw / 4; ++v) {
            const uint4 ka = *reinterpret_cast<const uint4*>(block + k_at(g, 4 * v + t));
            const uint4 kb = *reinterpret_cast<const uint4*>(block + k_at(g + 8, 4 * v + t));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
            constexpr int kPer = kQ8 ? 4 : 2;     // k-steps of a vector
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              uint32_t a0, a1, a2, a3;
              if constexpr (kQ8) {
                int8_to_half(wa[i], a0, a2);
                int8_to_half(wb[i], a1, a3);
              } else {
                a0 = wa[2 * i]; a2 = wa[2 * i + 1];
                a1 = wb[2 * i]; a3 = wb[2 * i + 1];
              }
              const int step = kPer * v + i;
#pragma unroll
              for (int nr = 0; nr < kNr; ++nr)
                mma<kMmaBF16>((step & 1) ? x2[nr] : x[nr], a0, a1, a2, a3, qw[nr][2 * step],
                              qw[nr][2 * step + 1]);
            }
          }
          float ks[2] = {1.0f, 1.0f};
          if constexpr (kQ8) {
            ks[0] = reinterpret_cast<const float*>(block + 32 * kRowB)[g];
            ks[1] = reinterpret_cast<const float*>(block + 32 * kRowB)[g + 8];
          }
          {
            // ---- logits, masks, running maximum and sum
            const bool full =
                cur0 + 15 <= p_lo && (cur0 >= lo_hi || cur0 + 15 < sinks);
            bool over = false;                    // a logit has outgrown its row's reference
#pragma unroll
            for (int nr = 0; nr < kNr; ++nr) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float v = (x[nr][e] + x2[nr][e]) * rs[nr][e & 1];
                if constexpr (kQ8) v *= ks[e >> 1];
                if (!full) {
                  const int j = cur0 + g + 8 * (e >> 1);
                  const int pos = rpos[nr][e & 1];
                  const bool see =
                      j <= pos && (p.window <= 0 || j > pos - p.window || j < sinks);
                  v = see ? v : -INFINITY;
                }
                x[nr][e] = v;
                over |= v > m[nr][e & 1] + kOver;  // with m = -inf: any logit but -inf
              }
            }
            if (__any_sync(kAll, over)) {
              // Rare after the first block: references move with the maximum, O and l
              // follow.
              float alpha[kNr][2];
#pragma unroll
              for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float v = fmaxf(x[nr][i], x[nr][i + 2]);
                  v = fmaxf(v, __shfl_xor_sync(kAll, v, 4));
                  v = fmaxf(v, __shfl_xor_sync(kAll, v, 8));
                  v = fmaxf(v, __shfl_xor_sync(kAll, v, 16));
                  const float next = v > m[nr][i] + kOver ? v - kDown : m[nr][i];
                  alpha[nr][i] = next == m[nr][i] ? 1.0f : fast_exp2(m[nr][i] - next);
                  m[nr][i] = next;
                  l[nr][i] *= alpha[nr][i];
                }
#pragma unroll
              for (int j = 0; j < kMt; ++j)
#pragma unroll
                for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[j][nr][e] *= alpha[nr][e & 1];
            }
            // ---- P^T and O^T
            uint32_t pb[kNr][2];
#pragma unroll
            for (int nr = 0; nr < kNr; ++nr) {
              float e4[4];
              const float safe[2] = {m[nr][0] == -INFINITY ? 0.0f : m[nr][0],
                                     m[nr][1] == -INFINITY ? 0.0f : m[nr][1]};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                e4[e] = fast_exp2(x[nr][e] - safe[e & 1]);
                l[nr][e & 1] += e4[e];
              }
              pb[nr][0] = transpose8x8(pack2<kMmaBF16>(e4[0], e4[1]));
              pb[nr][1] = transpose8x8(pack2<kMmaBF16>(e4[2], e4[3]));
            }
            uint32_t vw[4][kVw];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int row = 2 * t + (y & 1) + 8 * (y >> 1);
              if constexpr (kVw == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(block + v_at(row, g / 2) +
                                                                8 * (g & 1));
                vw[y][0] = v.x;
                vw[y][1] = v.y;
              } else {
#pragma unroll
                for (int i = 0; i < kVw / 4; ++i) {
                  const uint4 v = *reinterpret_cast<const uint4*>(block + v_at(row, g + 8 * i));
                  vw[y][4 * i] = v.x;
                  vw[y][4 * i + 1] = v.y;
                  vw[y][4 * i + 2] = v.z;
                  vw[y][4 * i + 3] = v.w;
                }
              }
            }
            // operands of O^T's j-th tile: a0, a1 of keys 2t, 2t + 1 and the tile's two
            // halves of channels, a2, a3 of the keys 8 further
            auto product = [&](int j, const uint32_t (&a)[4]) {
#pragma unroll
              for (int nr = 0; nr < kNr; ++nr)
                mma<kMmaBF16>(o[j][nr], a[0], a[1], a[2], a[3], pb[nr][0], pb[nr][1]);
            };
            if constexpr (kQ8) {
#pragma unroll
              for (int j = 0; j < kMt; j += 2) {          // two bytes of a word at a time
                uint32_t a[2][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const int y = 2 * (q >> 1), word = (kDp == 128 ? 2 : 1) * (q & 1) + j / 4;
                  const uint32_t two = __byte_perm(vw[y][word], vw[y + 1][word],
                                                   (j & 2) ? 0x7362 : 0x5140);
                  a[0][q] = e4m3x2_to_half2(two);
                  a[1][q] = e4m3x2_to_half2(two >> 16);
                }
                product(j, a[0]);
                product(j + 1, a[1]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < kMt; ++j) {
                uint32_t a[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const int y = 2 * (q >> 1), word = (kDp == 128 ? 4 : 2) * (q & 1) + j / 2;
                  a[q] = __byte_perm(vw[y][word], vw[y + 1][word], (j & 1) ? 0x7632 : 0x5410);
                }
                product(j, a);
              }
            }
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      workers_barrier<kQ4>();                   // the rings become the merge buffer

      // ---- join the warps
#pragma unroll
      for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = l[nr][i];
          v += __shfl_xor_sync(kAll, v, 4);
          v += __shfl_xor_sync(kAll, v, 8);
          v += __shfl_xor_sync(kAll, v, 16);
          if (g == 0) {
            m_s[warp][8 * nr + 2 * t + i] = m[nr][i];
            l_s[warp][8 * nr + 2 * t + i] = v;
          }
        }
#pragma unroll
      for (int j = 0; j < kMt; ++j)
#pragma unroll
        for (int nr = 0; nr < kNr; ++nr)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int hi = e >> 1;
            // lanes g side by side: the 32 lanes of a store hit 32 banks
            float* const row = &acc_s[warp][(8 * nr + 2 * t + (e & 1)) * kPitch];
            // 4 bits: tile j holds channels 4 g + 2 (j % 2) + hi of group j / 2
            row[(kQ4 ? 2 * j + hi : kMt * hi + j) * 8 + g] = o[j][nr][e];
          }
      workers_barrier<kQ4>();
      const bool alone = it.first == 0 && it.count == it.per;
      const int which = it.first == 0 ? 1 : 0;
      uint8_t* part = part_at(p.parts, cta, which);
      float* part_m = reinterpret_cast<float*>(part + sizeof(PartHead));
      float* part_l = part_m + kMaxRows;
      float* part_o = part_l + kMaxRows;
      if (!alone) {
        used[which] = true;
        if (tid == 0) {
          const int64_t from = it.cur - it.first;
          const int end_seat = cta_of(from + it.per - 1, it.total, it.busy);
          const int first_seat = cta_of(from, it.total, it.busy);
          it.first_cta = first_seat * team + member;
          it.parts = end_seat - first_seat + 1;
          *reinterpret_cast<PartHead*>(part) =
              PartHead{end_seat - seat + 1, it.s, it.head, it.tile};
        }
      }
      // out = O / l of four channels of a row
      auto deliver = [&](int r, int ch, float top, float sum, float4 a) {
        const int rr = it.tile * kRows + r;
        if (rr >= it.rows || ch >= c.D) return;
        const int64_t tok = static_cast<int64_t>(it.start) + rr / p.group;
        const int h = it.head * p.group + rr % p.group;
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        a.x *= inv; a.y *= inv; a.z *= inv; a.w *= inv;
        if constexpr (kQ8 || kQ4) {
          const float4 sv = *reinterpret_cast<const float4*>(c.v_scale + it.head * kDp + ch);
          constexpr float kUnit = kQ4 ? 64.0f : 1.0f;
          a.x *= kUnit * sv.x; a.y *= kUnit * sv.y; a.z *= kUnit * sv.z; a.w *= kUnit * sv.w;
        }
        *reinterpret_cast<uint2*>(p.out + (tok * p.Hq + h) * c.D + ch) =
            make_uint2(pack2<kQBF16>(a.x, a.y), pack2<kQBF16>(a.z, a.w));
        if (p.lse != nullptr && ch == 0)
          p.lse[tok * p.Hq + h] = sum == 0.0f ? -INFINITY
                                              : (top + log2f(sum)) * 0.69314718055994530942f;
      };
      for (int i = tid; i < kRows * (kDp / 4); i += 32 * kWarps) {
        const int r = i / (kDp / 4), ch = 4 * (i % (kDp / 4));
        // where channel ch stands: tile j, half hi and lane g of the products
        const int cj = kQ8 && kDp == 128 ? ch % 8 : kDp == 128 ? ch % 8 : ch % 4;
        const int chi = kQ8 && kDp == 128 ? (ch / 8) & 1 : kDp == 128 ? ch / 64 : (ch / 4) & 1;
        const int cg = kQ8 && kDp == 128 ? ch / 16 : kDp == 128 ? (ch % 64) / 8 : ch / 8;
        const int at4 = kQ4 ? ch / 32 * 32 + ch % 32 / 4 : (kMt * chi + cj) * 8 + cg;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][r]);
        const float safe = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = fast_exp2(m_s[w][r] - safe);
          sum += f * l_s[w][r];
          const float* v = &acc_s[w][r * kPitch + at4];
          a.x += f * v[0]; a.y += f * v[8]; a.z += f * v[16]; a.w += f * v[24];
        }
        if (!alone) {
          *reinterpret_cast<float4*>(part_o + r * kDp + ch) = a;
          if (ch == 0) {
            part_m[r] = top;
            part_l[r] = sum;
          }
          continue;
        }
        deliver(r, ch, top, sum, a);
      }
      if (!alone && p.join_inside) {
        // The CTA that finishes an item's last part joins them all, in their order.
        __threadfence();
        workers_barrier<kQ4>();
        if (tid == 0) {
          const uint32_t arrived = atomicAdd(&p.arrivals[it.first_cta], 1u) + 1u;
          it.joins = arrived == static_cast<uint32_t>(it.parts);
          if (it.joins) p.arrivals[it.first_cta] = 0;     // for the next call
          __threadfence();
        }
        workers_barrier<kQ4>();
        if (it.joins) {
          // the parts' maxima and sums through shared memory (as many as fit)
          constexpr int kFit = kWarps * kRows * kPitch / (2 * kRows);
          float* const ml = &acc_s[0][0];
          const int parts = it.parts, fit = min(parts, kFit);
          for (int i = tid; i < fit * kRows; i += 32 * kWarps) {
            const float* f = part_floats(p.parts, it.first_cta + i / kRows * team, i < kRows) + i % kRows;
            ml[i] = __ldcg(f);
            ml[kFit * kRows + i] = __ldcg(f + kMaxRows);
          }
          workers_barrier<kQ4>();
          for (int i = tid; i < kRows * (kDp / 4); i += 32 * kWarps) {
            const int r = i / (kDp / 4), ch = 4 * (i % (kDp / 4));
            if (it.tile * kRows + r >= it.rows) break;    // later ones are later rows
            auto max_of = [&](int j) {
              return j < kFit ? ml[j * kRows + r]
                              : __ldcg(part_floats(p.parts, it.first_cta + j * team, 0) + r);
            };
            auto sum_of = [&](int j) {
              return j < kFit ? ml[(kFit + j) * kRows + r]
                              : __ldcg(part_floats(p.parts, it.first_cta + j * team, 0) + kMaxRows + r);
            };
            float top = -INFINITY;
            for (int j = 0; j < parts; ++j) top = fmaxf(top, max_of(j));
            const float safe = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int j0 = 0; j0 < parts; j0 += 8) {
              float4 v[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                v[j] = __ldcg(reinterpret_cast<const float4*>(
                    part_floats(p.parts, it.first_cta + min(j0 + j, parts - 1) * team,
                                j0 + j == 0 || parts == 1) + 2 * kMaxRows + r * kDp + ch));
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (j0 + j < parts) {
                  const float w = fast_exp2(max_of(j0 + j) - safe);
                  sum += w * sum_of(j0 + j);
                  a.x += w * v[j].x; a.y += w * v[j].y; a.z += w * v[j].z; a.w += w * v[j].w;
                }
            }
            deliver(r, ch, top, sum, a);
          }
        }
      }
      if constexpr (!kQ4) {
        __syncthreads();
        if (tid == 0) {
          it.cur += it.count;
          it.off += it.count;
        }
      }
    }
    if (kQ4 && warp == kWarps && abort_s) {     // no copy may be in flight when the CTA exits
      for (int i = 1; i <= kStages; ++i) {
        const int st = stage4 - i;              // below 0: in the round before
        mbar_wait(&full_s[(lane >> 3) * kStages + (st < 0 ? st + kStages : st)],
                  st < 0 ? parity4 ^ 1u : parity4, nullptr, c.status, p.timeout_ns);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  }
  if (tid < 2 && !used[tid])
    reinterpret_cast<PartHead*>(part_at(p.parts, cta, tid))->parts = 0;
}

// Joins the parts of one row of the item that begins in CTA blockIdx.x and
// ends in a later one: weights 2^(m_i - max), summed in the parts' order.  An item's
// parts lie a team of CTAs apart with 4 bits (kTeams) and side by side otherwise: a
// distance that the compiler knows lets their loads run ahead (8 bits, one sequence of
// 30000 keys, 32 heads on 8 x 128: 27.4 us, with p.team 33.3).
template <bool kQBF16, int kDp, int kRows, bool kTeams>
__global__ void __launch_bounds__(128)
paged_join_kernel(const PagedAttnParams p, int ctas) {
  __shared__ float w_s[kMaxCtas];
  __shared__ float red_s[4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const PartHead h = *reinterpret_cast<const PartHead*>(part_at(p.parts, c0, 1));
  const int team = kTeams ? p.team : 1;
  const int parts = min(h.parts, (ctas - c0 + team - 1) / team);
  if (parts <= 0) return;
  int start, n, len;
  if (!paged_seq(p.c, h.seq, &start, &n, &len)) return;
  const int rr = h.tile * kRows + r;
  if (rr >= n * p.group) return;
  float top = -INFINITY;
  for (int i = tid; i < parts; i += 128) {
    const float v = reinterpret_cast<const float*>(part_at(p.parts, c0 + i * team, i == 0) +
                                                   sizeof(PartHead))[r];
    w_s[i] = v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
  if ((tid & 31) == 0) red_s[tid >> 5] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
  const float safe = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, acc = 0.0f;
  const int ch = tid;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float* f = reinterpret_cast<const float*>(part_at(p.parts, c0 + i * team, i == 0) +
                                                    sizeof(PartHead));
    const float w = fast_exp2(w_s[i] - safe);
    sum += w * f[kMaxRows + r];
    if (ch < kDp) acc += w * f[2 * kMaxRows + r * kDp + ch];
  }
  const int64_t tok = static_cast<int64_t>(start) + rr / p.group;
  const int hq = h.head * p.group + rr % p.group;
  if (ch < p.c.D) {
    float v = sum == 0.0f ? 0.0f : acc / sum;           // (a NaN shows)
    if (p.c.kind == kKindQ8) v *= p.c.v_scale[h.head * kDp + ch];
    if (p.c.kind == kKindQ4) v *= 64.0f * p.c.v_scale[h.head * kDp + ch];
    uint16_t bits;
    if constexpr (kQBF16) {
      const __nv_bfloat16 b = __float2bfloat16_rn(v);
      bits = *reinterpret_cast<const uint16_t*>(&b);
    } else {
      const __half b = __float2half_rn(v);
      bits = *reinterpret_cast<const uint16_t*>(&b);
    }
    p.out[(tok * p.Hq + hq) * p.c.D + ch] = bits;
  }
  if (p.lse != nullptr && ch == 0)
    p.lse[tok * p.Hq + hq] = sum == 0.0f ? -INFINITY
                                         : (top + log2f(sum)) * 0.69314718055994530942f;
}

template <int kKind, bool kQBF16, int kDp, int kNr, int kForm = 0>
cudaError_t launch_few(const PagedAttnParams& p, int sms, cudaStream_t st) {
  if constexpr (kForm == 0) {
    if (!p.c.wide)                              // 8-bit only: the others' rows always are
      return launch_few<kKind, kQBF16, kDp, kNr, kKind == kKindQ8 ? 2 : 1>(p, sms, st);
    if (kKind == kKindQ4 ? p.c.D <= kDp - 32 : p.c.D != kDp)
      return launch_few<kKind, kQBF16, kDp, kNr, 1>(p, sms, st);
  }
  using L = Few<kKind, kDp, kNr>;
  auto* kern = paged_few_kernel<kKind, kQBF16, kDp, kNr, kForm>;
  static std::atomic<int> resident[64] = {};   // CTAs of one SM, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int per = resident[dev].load(std::memory_order_relaxed);
  if (per == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, L::kThreads, L::kSmem);
    if (e != cudaSuccess) return e;
    per = per < 1 ? 1 : per > 8 ? 8 : per;
    resident[dev].store(per, std::memory_order_relaxed);
  }
  // at most one CTA per unit of the longest lengths the call declares
  constexpr int kUnitKeys = L::kKeys * kWarps;
  const int64_t max_units = (static_cast<int64_t>(p.c.max_kv) + kUnitKeys - 1) / kUnitKeys + 1;
  const int64_t tiles = (static_cast<int64_t>(p.c.max_q) * p.group + 8 * kNr - 1) / (8 * kNr);
  const int64_t items = tiles * p.c.Hkv * p.c.nseq;    // below 2^63; times max_units perhaps not
  int ctas = sms * per < kMaxCtas ? sms * per : kMaxCtas;
  if (items < ctas && items * max_units < ctas) ctas = static_cast<int>(items * max_units);
  PagedAttnParams prm = p;
  prm.team = 1;
  Maps<kKind> maps{};
  if constexpr (kKind == kKindQ4) {
    if (!paged_maps4(p.c, 16, maps.t, nullptr)) return cudaErrorInvalidValue;
    // Neighbouring heads are read at the same time, by a team of CTAs in step: a row of
    // 64 bytes alone is half a line of the L2, and its other half came from memory again
    // (NHD, 64 x 8520 keys: 1090 MB read instead of 631, 196 us instead of 182); where
    // heads lie apart their scales are neighbours all the same.
    while (prm.team < 8 && p.c.Hkv % (2 * prm.team) == 0) prm.team *= 2;
    ctas = ctas / prm.team * prm.team;
    if (ctas == 0) ctas = prm.team;
  }
  // Parts are joined by the CTA that finishes an item last, which saves the host a
  // launch, unless few items spread over many CTAs: one CTA would then read a
  // hundred parts or more, and a second kernel does it by the row.  (Sequence and
  // head pairs over 32768 keys, inside against second kernel: 1: 91 and 63 us, 2: 54
  // and 45, 4: 44 and 40, 8: 50 and 48, 128: 351 and 353; over 2000 keys the second
  // kernel is 1 to 2 us ahead up to 64 of them, at the price of its launch.)
  // Over four bits the second kernel is worth its launch sooner with more rows to join (tiles
  // of 16 and 24 rows; inside against second: 9.5 parts an item 43 and 36, 25 and 21; 19
  // parts 31 and 20; 2.4 and 1.6 parts 81 and 78, 29.8 and 30.8).
  constexpr int kInside = kKind == kKindQ4 && kNr > 1 ? 6 : kJoinInside;
  prm.join_inside = items >= (ctas + kInside - 1) / kInside;
  kern<<<ctas, L::kThreads, L::kSmem, st>>>(prm, maps);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess || prm.join_inside) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 8 * kNr);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_join_kernel<kQBF16, kDp, 8 * kNr, kKind == kKindQ4>, prm,
                         ctas);
  note_launch();
  return e;
}

// Row tiles of 8, 16, 24 or 32 rows: the fewest that hold a sequence's rows, as a
// wider tile costs registers and with them loads in flight.  Where the other
// kernel takes the longer sequences, the ones left here are mostly single tokens.
template <int kKind, bool kQBF16>
cudaError_t launch_kind(const PagedAttnParams& p, int sms, cudaStream_t st) {
  int64_t rows = static_cast<int64_t>(p.c.max_q) * p.group;
  if (p.max_rows < rows) rows = p.group;
  if (p.c.Dp == 128)
    return rows <= 8 ? launch_few<kKind, kQBF16, 128, 1>(p, sms, st)
                     : launch_few<kKind, kQBF16, 128, 2>(p, sms, st);
  if (rows <= 8) return launch_few<kKind, kQBF16, 64, 1>(p, sms, st);
  if (rows <= 16) return launch_few<kKind, kQBF16, 64, 2>(p, sms, st);
  if (rows <= 24) return launch_few<kKind, kQBF16, 64, 3>(p, sms, st);
  return launch_few<kKind, kQBF16, 64, 4>(p, sms, st);
}

}  // namespace
}  // namespace sage
