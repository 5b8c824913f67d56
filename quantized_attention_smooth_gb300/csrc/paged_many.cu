// Attention of many new tokens per sequence (a prompt's chunks) over the paged
// cache on the tensor cores (tcgen05): bound by the products.
//
//   S = Q K^T (128 rows x 128 keys, fp32);  x = S c;  P = 2^(x - m_ref);
//   O += P V;  l += sum P;  out = O / l
//
// The rows of one (sequence, kv head) are its new tokens times the query heads
// of the group, token by token, so that heads which share keys share a tile.
// A CTA works on a pair of 128-row tiles that share every K and V tile:
//   warps 0-3, 4-7  softmax of tile 0 and 1: thread = row = TMEM lane
//   warp 8          issues the MMAs (one thread)
//   warp 10         cuts the CTA's range of work into items for the others
//   warp 9          copies K and V tiles from the pages (16-bit cache): one
//                   tensor copy per page and 64 channels, each by its own lane
//   warps 12-15     8-bit cache only: read K and V codes, widen them to fp16
//                   (exactly) and store them where the copies would put them
// TMEM (512 columns): S0 | S1 | O0 | O1, and P_t in the first half of S_t, as
// the A operand of O_t += P_t V: shared memory then carries Q, K and V alone.
// (With P in shared memory as well, the operands' reads and writes of a key
// step come to 3000 cycles of its bandwidth against 2048 of the tensor pipe.)
// K is the B operand with channels contiguous, V the B operand with its rows
// contiguous (MN-major), so both tiles are used as they lie in the pages.
//
// Order of the MMAs:  QK_0(0) QK_1(0) | PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1) ...
// While one tile's softmax runs, the other tile's products do.  QK_t(j+1)
// overwrites P_t(j) behind PV_t(j) that reads it: one thread issues both, and
// the pipe executes them in that order.  A commit covers everything issued
// before it, so S_t(j+1) ready also means that PV_t(j) is done, and a softmax
// warp may rescale O_t itself, with nobody else at it.  It does so only when
// the row's maximum has grown by more than 2^8 since m_ref was taken (any m_ref
// gives the same result; P then stays below 2^8, or 2^15 in fp16, and keeps its
// relative precision), which after the first tiles is hardly ever.
//
// Work is cut into units of (pair of tiles, kv head, 128 keys), dealt evenly to
// one CTA per SM as one contiguous range each, derived from the lengths on the
// device; pairs that span CTAs leave fp32 parts (m, l, O) in the workspace for a
// second kernel, which joins them in order.  Key tiles that no row sees (before
// the window, behind the sinks) are never visited.  Values of keys that no row
// of the pair sees are zeroed in shared memory (0 times NaN would be NaN).
//
// Measured on GB300 (32 query heads on 8 kv heads of 128 channels; four calls in a
// graph): 2048 new tokens over 30720 cached ones, bf16, 752 us, 1417 TFLOP/s, 74 %
// of the measured bf16 peak; two causal prompts of 8192 tokens 836 us, 1316 TFLOP/s;
// chunks over the 8-bit cache 462 us, 948 TFLOP/s.  Call after call, at the power
// cap, they take 819 us (1302 TFLOP/s, 77 % of the sustained peak), 869 and 454.  A key step of both tiles takes about 2950
// cycles against 2048 of the tensor pipe: the softmax of a tile (1490 cycles, two
// and a half per instruction with one warp of it per scheduler) and its products
// (1024 and the signals' latency) follow one another, and the two tiles overlap
// only that far.  Tried and slower: the logits in four pieces with a load ahead
// (1830 cycles), two threads a row (registers spill), P in shared memory.  The
// 8-bit cache adds the key scales (64 products and 32 loads a row) and shares the
// issue slots with the widening warps: 2500 cycles a tile.

#include <atomic>
#include <cfloat>
#include <type_traits>

#include "sage_kernels.h"
#include "sage_paged_device.cuh"

namespace sage {
namespace {

constexpr int kPairRows = 256, kTileRows = 128, kKeys = 128;
constexpr int kMaxManyCtas = 152;
constexpr uint32_t kTmemCols = 512;
constexpr unsigned kAll = 0xFFFFFFFFu;
// Units that an item costs besides its key tiles: filling and draining the
// pipeline takes about as long as this many tiles.  (Two prompts of 8192 tokens:
// 945 us with 2, 847 with 3, 843 with 4, 865 with 6: the first rows' items are
// short.  32 of 512: 190, 186, 183, 192; five ragged chunks: 362, 321, 314, 327; eight of
// 2048 over the 8-bit cache: 621, 558, 524, 552.  Long chunks do not care.)
constexpr int kItemUnits = 4;

struct ManyHead {
  int32_t parts, seq, head, pair;   // parts of the item from this one on; 0: none here
  int32_t pad[60];
};
constexpr size_t kManyPartBytes = sizeof(ManyHead) + 2 * kPairRows * 4 + kPairRows * 128 * 4;
static_assert(sizeof(ManyHead) == 256, "parts stay 256-byte aligned");

__device__ __forceinline__ uint8_t* many_part(uint8_t* parts, int cta, int which) {
  return parts + (static_cast<size_t>(cta) * 2 + which) * kManyPartBytes;
}

template <int kKind, int kDp>
struct Many {
  static constexpr bool kQ8 = kKind == kKindQ8;
  static constexpr int kThreads = kQ8 ? 512 : 384;
  static constexpr int kPanel = kTileRows * 128;               // 128 rows x 64 channels
  static constexpr int kTileBytes = kDp / 64 * kPanel;         // Q, K or V tile of 16 bits
  static constexpr int kStages = kQ8 ? (kDp == 128 ? 3 : 6) : (kDp == 128 ? 5 : 10);
  // 8-bit cache: codes as they lie in the pages, a tile and its key scales a stage
  static constexpr int kRawStages = kDp == 128 ? 3 : 6;
  // (the scales of each copied page on 128 bytes, as a tensor copy needs them)
  static constexpr int kRawBytes = kKeys * kDp + 1024;
  static constexpr int kScaleRing = 4;                         // key scales of 4 tiles
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
  static constexpr int kScaleOff = kRawOff + (kQ8 ? kRawStages * kRawBytes : 0);
  static constexpr int kBarOff = kScaleOff + (kQ8 ? kScaleRing * kKeys * 4 : 0);
  // full[stages], empty[stages], q_ready[2], s_full[2], p_ready[2], o_full[2], drain,
  // item_full[items], item_empty[items], raw_full[raw], raw_empty[raw]
  static constexpr int kItems = 4;
  static constexpr int kC = kQ8 ? 2 : 4;         // a softmax run's keys, in 32s (registers)
  static constexpr int kNumBars = 2 * kStages + 9 + 2 * kItems + 2 * kRawStages;
  static constexpr int kMiscOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kItemOff = kMiscOff + 256;
  static constexpr int kAlloc = kItemOff + kItems * 128;
  // warps that take items: softmax, MMA, copies, and the 8-bit cache's widening
  static constexpr int kTakers = 8 + 1 + 1 + (kQ8 ? 4 : 0);
  static_assert(kAlloc <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// D (+)= A[tmem] B[smem]: A is 128 rows of 16-bit pairs, one pair a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .b64 bd;\n\t.reg .pred p;\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n}"
      :: "r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
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

// One lane of a converged warp, the same one each time.  A branch on it, and
// operands that come out of a shuffle, tell the compiler that the values are
// the warp's: the MMAs then take them from uniform registers.  (From a branch on
// the lane number each MMA cost about 90 cycles to issue, for 64 to run.)
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n}"
               : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kAll, x, 0); }

// A position in a ring of kN barriers and the parity of its present round.
template <int kN>
struct Ring {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == kN) {
      at = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
         "r"(smem_u32(bar))
      : "memory");
}

// The part of a (sequence, kv head, pair) that a CTA works on, as the scheduling
// warp leaves it in shared memory for the other roles (registers that they
// would keep for it across an item cost spills in their loops).
struct Item {
  int s, head, pair, start, rows;
  int base;                  // position of the sequence's row 0
  int p_hi;                  // position of the pair's last row
  int lo;                    // first key of the window of the first row
  int first, count, per;     // key tiles: from, how many (0: no more items), of how many
  int sink, from;            // Span
  int before;                // key tiles of the CTA's earlier items
  int parts;                 // CTAs from this one on that work on the pair
  struct {
    int lo, hi;              // positions of the tile's first and last row
    int tok, off;            // its first row's token, and query head within the group
  } tile[2];
  __device__ __forceinline__ int key0(int i) const {     // first key of the i-th tile
    const int v = first + i;
    return kKeys * (v < sink ? v : v - sink + from);
  }
  __device__ __forceinline__ bool two() const { return pair * kPairRows + kTileRows < rows; }
};
static_assert(sizeof(Item) <= 128, "items lie 128 bytes apart");

__device__ __forceinline__ bool served(const PagedAttnParams& p, int s, int* start, int* n,
                                       int* len, int* rows) {
  if (!paged_seq(p.c, s, start, n, len)) return false;
  *rows = *n * p.group;
  return *rows > 0 && *rows >= p.min_rows && *rows <= p.max_rows;
}

__device__ __forceinline__ Span pair_span(const PagedAttnParams& p, int base, int rows, int pair,
                                          int* p_lo, int* p_hi) {
  *p_lo = base + pair * kPairRows / p.group;
  *p_hi = base + (min((pair + 1) * kPairRows, rows) - 1) / p.group;
  Span r = span_of<kKeys>(*p_lo, *p_hi, p.window, p.sinks);
  r.count = max(1, r.count);             // a pair that sees nothing still writes its zeros
  return r;
}

// A CTA's place in the units.  An item takes kItemUnits + tiles units, the first
// ones without a tile; a CTA whose range ends among those leaves the item to the
// next one.
struct Walk {
  int s, pair, head, unit;
  int64_t left, at, all;     // units left; where it stands in all units
  int busy;                  // CTAs that share them
};

// x / group for a row's x < group + 256, by a multiplication: exact while
// x * group < 2^32 (groups up to 16384).
__device__ __forceinline__ int by_group(const PagedAttnParams& p, int x) {
  return p.group == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.magic));
}

// Inclusive sum over the block's threads; ends with a barrier.
template <int kThreads>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(kAll, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t all = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return v + before;
}

__device__ __forceinline__ uint32_t below(int x) {       // the x lowest bits
  return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u;
}

template <int kKind, bool kQBF16, int kDp>
__global__ void __launch_bounds__(kKind == kKindQ8 ? 512 : 384, 1)
paged_many_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_s, const PagedAttnParams p) {
  using L = Many<kKind, kDp>;
  constexpr bool kQ8 = L::kQ8;
  constexpr bool kMmaBF16 = kKind == kKindBF16;
  constexpr float kDown = kBelow<kMmaBF16>, kOver = kLazy + kDown;
  constexpr int kStages = L::kStages;
  constexpr int kC = L::kC;
  // The driver places dynamic shared memory behind its 1 KB reservation of a
  // block; a base off the swizzle's grid is reported and the CTA does nothing.
  extern __shared__ __align__(1024) uint8_t smem[];
  const PagedGeo& c = p.c;
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(c.status, kStatusBadItem);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  asm volatile("griddepcontrol.launch_dependents;");

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + kStages;
  uint64_t* q_ready = empty + kStages;
  uint64_t* s_full = q_ready + 2;
  uint64_t* p_ready = s_full + 2;
  uint64_t* o_full = p_ready + 2;
  uint64_t* drain = o_full + 2;
  uint64_t* item_full = drain + 1;
  uint64_t* item_empty = item_full + L::kItems;
  uint64_t* raw_full = item_empty + L::kItems;
  uint64_t* raw_empty = raw_full + L::kRawStages;
  int* scan_s = reinterpret_cast<int*>(smem);     // the plan's; the queries come there later
  int64_t* sums_s = reinterpret_cast<int64_t*>(smem + L::kMiscOff);        // 16
  Walk* walk_s = reinterpret_cast<Walk*>(smem + L::kMiscOff + 128);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 196);

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], kQ8 ? 128 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_ready[t], kTileRows);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], kTileRows);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < L::kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], L::kTakers);
    }
    for (int i = 0; i < L::kRawStages; ++i) {
      mbar_init(&raw_full[i], p.tensor_copies ? 1 : 32);
      mbar_init(&raw_empty[i], 128);
    }
    mbar_fence_init();
  }
  if (warp == 8) tmem_alloc(tmem_slot, kTmemCols);

  // ---- this CTA's range of units: pairs per sequence, then tiles per pair
  Walk walk{0, 0, 0, 0, 0, 0, 0, 0};
  {
    constexpr int T = L::kThreads;
    const int spt = (c.nseq + T - 1) / T;
    const int sb = min(c.nseq, tid * spt), se = min(c.nseq, sb + spt);
    int64_t pairs = 0, all_pairs = 0, all = 0;
    for (int s = sb; s < se; ++s) {
      int a, n, len, rows;
      if (served(p, s, &a, &n, &len, &rows)) pairs += (rows + kPairRows - 1) / kPairRows;
    }
    const int64_t pair_end = block_scan<T>(pairs, sums_s, &all_pairs);
    scan_s[tid] = static_cast<int>(pair_end);
    __syncthreads();
    const int64_t ppt = (all_pairs + T - 1) / T;
    const int64_t pb = min(all_pairs, tid * ppt), pe = min(all_pairs, pb + ppt);
    // the pair pb: its thread's chunk of sequences by bisection, then a walk
    int s0 = 0, p0 = 0;
    if (pb < pe) {
      int lo = 0, hi = T - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (scan_s[mid] > pb) hi = mid;
        else lo = mid + 1;
      }
      int64_t rest = pb - (lo > 0 ? scan_s[lo - 1] : 0);
      for (s0 = lo * spt; s0 < c.nseq; ++s0) {
        int a, n, len, rows;
        if (!served(p, s0, &a, &n, &len, &rows)) continue;
        const int np = (rows + kPairRows - 1) / kPairRows;
        if (rest < np) break;
        rest -= np;
      }
      p0 = static_cast<int>(rest);
    }
    // visits this thread's pairs; f(s, pair, tiles) returns true to stop
    auto visit = [&](auto f) {
      int s = s0, pair = p0;
      for (int64_t i = pb; i < pe; ++s, pair = 0) {
        int a, n, len, rows;
        if (s >= c.nseq) return;
        if (!served(p, s, &a, &n, &len, &rows)) continue;
        for (; i < pe && pair * kPairRows < rows; ++i, ++pair) {
          int plo, phi;
          if (f(s, pair, pair_span(p, len - n, rows, pair, &plo, &phi).count)) return;
        }
      }
    };
    int64_t mine = 0;
    visit([&](int, int, int tiles) { mine += tiles + kItemUnits; return false; });
    mine *= c.Hkv;
    const int64_t end = block_scan<T>(mine, sums_s, &all), begin = end - mine;
    const int64_t busy = min(all, static_cast<int64_t>(ctas));
    const int64_t u0 = cta < busy ? all * cta / busy : 0;
    const int64_t u1 = cta < busy ? all * (cta + 1) / busy : 0;
    if (u0 < u1 && begin <= u0 && u0 < end) {             // one thread
      int64_t off = u0 - begin;
      visit([&](int s, int pair, int tiles) {
        const int64_t per = tiles + kItemUnits, w = per * c.Hkv;
        if (off >= w) {
          off -= w;
          return false;
        }
        *walk_s = Walk{s, pair, static_cast<int>(off / per), static_cast<int>(off % per),
                       u1 - u0, u0, all, static_cast<int>(busy)};
        return true;
      });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (u0 < u1) walk = *walk_s;
  }
  const uint32_t tbase = *tmem_slot;
  const int wg = warp >> 2;
  auto item_at = [&](int i) -> const Item& {
    return *reinterpret_cast<const Item*>(smem + L::kItemOff + 128 * i);
  };
  // waits for the next item; false at the end, or if a wait ran out
  auto take = [&](const Ring<L::kItems>& at) {
    return __all_sync(kAll, mbar_wait(&item_full[at.at], at.parity, abort_flag, c.status,
                                      p.timeout_ns)) &&
           item_at(at.at).count > 0;
  };
  auto give_back = [&](const Ring<L::kItems>& at) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[at.at]);
  };

  if (wg == 2) {
    if constexpr (kQ8) regs_decrease<72>();
    else regs_decrease<80>();
    if (warp == 10) {
      // ================================================== items
      Ring<L::kItems> at;
      bool ok = true, more = true;
      int start = 0, n = 0, len = 0, rows = 0, p_lo = 0, p_hi = 0, tiles = 0;
      Span span{0, 0, 0};
      bool fresh = true;
      while (ok && more) {
        int first = 0, count = 0, parts = 0;
        while (count <= 0 && walk.left > 0 && walk.s < c.nseq) {
          if (fresh || walk.head == 0) {        // a new pair
            if (((fresh || walk.pair == 0) && !served(p, walk.s, &start, &n, &len, &rows)) ||
                walk.pair * kPairRows >= rows) {
              ++walk.s;
              walk.pair = walk.head = walk.unit = 0;
              continue;
            }
            span = pair_span(p, len - n, rows, walk.pair, &p_lo, &p_hi);
            fresh = false;
          }
          first = max(0, walk.unit - kItemUnits);
          const int64_t upto = walk.unit + walk.left - kItemUnits;   // tiles before the end
          count = static_cast<int>(min(static_cast<int64_t>(span.count), upto)) - first;
          const int rest = span.count + kItemUnits - walk.unit;
          // the CTA with the item's last unit: CTA i's range begins at all * i / busy
          parts = static_cast<int>(((walk.at + rest) * walk.busy - 1) / walk.all) - cta + 1;
          walk.at += rest;
          walk.left -= rest;
          walk.unit = 0;
          if (count <= 0 && ++walk.head == c.Hkv) {
            walk.head = 0;
            ++walk.pair;
          }
        }
        more = count > 0;
        ok = __all_sync(kAll, mbar_wait(&item_empty[at.at], at.parity ^ 1u, abort_flag, c.status,
                                        p.timeout_ns));
        if (!ok) break;
        if (lane == 0) {
          Item& x = *reinterpret_cast<Item*>(smem + L::kItemOff + 128 * at.at);
          x.count = max(count, 0);
          if (more) {
            x.s = walk.s;
            x.head = walk.head;
            x.pair = walk.pair;
            x.start = start;
            x.rows = rows;
            x.base = len - n;
            x.p_hi = p_hi;
            x.lo = p.window > 0 ? max(0, p_lo - p.window + 1) : 0;
            x.first = first;
            x.per = span.count;
            x.sink = span.sink;
            x.from = span.from;
            x.before = tiles;
            x.parts = parts;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int row0 = walk.pair * kPairRows + t * kTileRows;
              const int tok = row0 / p.group;
              x.tile[t].tok = tok;
              x.tile[t].off = row0 - tok * p.group;
              x.tile[t].lo = x.base + tok;
              x.tile[t].hi = x.base + (min(row0 + kTileRows, rows) - 1) / p.group;
            }
          }
          mbar_arrive(&item_full[at.at]);
        }
        __syncwarp();
        tiles += count;
        if (++walk.head == c.Hkv) {
          walk.head = 0;
          ++walk.pair;
        }
        at.next();
      }
    } else if (warp == 9 && kQ8 && p.tensor_copies) {
      // ================================================== copies of codes, by the page
      const int rows_box = min(c.page_size, kKeys), boxes = kKeys / rows_box;
      Ring<L::kRawStages> ring;                 // K and V tiles alternate
      int issued = 0;
      bool ok = true;
      for (Ring<L::kItems> at; ok && take(at); give_back(at), at.next()) {
        const Item& it = item_at(at.at);
        const int sinks = p.window > 0 ? p.sinks : 0;
        const int count = it.count, head = it.head;
        for (int i = 0; ok && i < count; ++i) {
          const int key0 = it.key0(i);
          int page = static_cast<int>(c.num_pages), slot = 0;
          if (lane < boxes) {
            const int k = key0 + lane * rows_box;
            if (k <= it.p_hi && (k + rows_box - 1 >= it.lo || k < sinks)) {
              const int pn = page_of(c, k);
              const int pg = paged_page(c, it.s, pn);
              if (pg >= 0) page = pg;           // else the copy lies outside and reads zeros
              slot = k - pn * c.page_size;
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(kAll, mbar_wait(&raw_empty[ring.at], ring.parity ^ 1u, abort_flag,
                                            c.status, p.timeout_ns));
            if (!ok) break;
            if (lane == 0)
              mbar_expect_tx(&raw_full[ring.at], kKeys * kDp + (kv == 0 ? kKeys * 4 : 0));
            __syncwarp();
            if (lane < boxes) {
              uint8_t* dst = smem + L::kRawOff + ring.at * L::kRawBytes;
              tma_load_4d(dst + lane * rows_box * kDp, kv == 0 ? &tm_k : &tm_v, 0, slot, head,
                          page, &raw_full[ring.at]);
              if (kv == 0)
                tma_load_3d(dst + kKeys * kDp + lane * max(rows_box * 4, 128), &tm_s, slot, head, page,
                            &raw_full[ring.at]);
            }
            ring.next();
            issued = min(issued + 1, L::kRawStages);
          }
        }
      }
      // no copy may still be in flight when the CTA exits
      for (int i = 1; i <= issued; ++i) {
        const int st = ring.at - i;             // below 0: in the round before
        mbar_wait(&raw_full[st < 0 ? st + L::kRawStages : st],
                  st < 0 ? ring.parity ^ 1u : ring.parity, nullptr, c.status, p.timeout_ns);
      }
    } else if (warp == 9 && kQ8) {
      // ================================================== copies of codes, for rows
      // and pages that tensor copies cannot take (D or a stride an odd multiple of
      // 8, page sizes that neither divide nor are multiples of 128); five times
      // slower (three chunks of 1000 tokens over 9000: 2738 us against 484)
      Ring<L::kRawStages> ring;                 // K and V tiles alternate
      bool ok = true;
      const bool wide = c.wide;                 // rows in vectors of 16 bytes, else of 8
      const int shift = (kDp == 128 ? 3 : 2) + (wide ? 0 : 1);   // log2 of a row's lanes
      const int width = wide ? 16 : 8, col = (lane & ((1 << shift) - 1)) * width;
      const int step = 32 >> shift;
      for (Ring<L::kItems> at; ok && take(at); give_back(at), at.next()) {
        const Item& it = item_at(at.at);
        const int sinks = p.window > 0 ? p.sinks : 0;
        const int count = it.count, head = it.head, lo = it.lo, p_hi = it.p_hi;
        for (int i = 0; ok && i < count; ++i) {
          const int key0 = it.key0(i);
          // lane b < 8 finds the page of keys 16 b .. 16 b + 15
          int page = -1, slot = 0;
          const int kb = key0 + 16 * (lane & 7);
          if (lane < 8 && kb <= p_hi && (kb + 15 >= lo || kb < sinks)) {
            const int pn = page_of(c, kb);
            page = paged_page(c, it.s, pn);
            slot = kb - pn * c.page_size;
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(kAll, mbar_wait(&raw_empty[ring.at], ring.parity ^ 1u, abort_flag,
                                            c.status, p.timeout_ns));
            if (!ok) break;
            const uint32_t dst = smem_u32(smem + L::kRawOff + ring.at * L::kRawBytes);
            const uint8_t* const codes = kv == 0 ? c.k : c.v;
#pragma unroll 4
            for (int r = lane >> shift; r < kKeys; r += step) {
              const int pg = __shfl_sync(kAll, page, r / 16), sl = __shfl_sync(kAll, slot, r / 16);
              const int key = key0 + r;
              const bool see = pg >= 0 && col < c.D && key <= p_hi && (key >= lo || key < sinks);
              const uint8_t* src = codes;       // not read unless seen
              if (see)
                src += pg * c.page_stride + (sl + (r & 15)) * c.token_stride +
                       head * c.head_stride + col;
              if (wide)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                             :: "r"(dst + r * kDp + col), "l"(src), "r"(see ? 16 : 0) : "memory");
              else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                             :: "r"(dst + r * kDp + col), "l"(src), "r"(see ? 8 : 0) : "memory");
            }
            if (kv == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = lane + 32 * j;
                const int pg = __shfl_sync(kAll, page, r / 16),
                          sl = __shfl_sync(kAll, slot, r / 16);
                const int key = key0 + r;
                const bool see = pg >= 0 && key <= p_hi && (key >= lo || key < sinks);
                const float* src = c.k_scale;
                if (see)
                  src += (static_cast<int64_t>(pg) * c.Hkv + head) * c.page_size + sl + (r & 15);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                             :: "r"(dst + kKeys * kDp + 4 * r), "l"(src), "r"(see ? 4 : 0)
                             : "memory");
              }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];"
                         :: "r"(smem_u32(&raw_full[ring.at])) : "memory");
            ring.next();
          }
        }
      }
      // no copy may still be in flight when the CTA exits
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 9 && !kQ8) {
      // ================================================== copies of K and V
      const int rows_box = min(c.page_size, kKeys), boxes = kKeys / rows_box;
      Ring<kStages> ring;                       // K and V tiles alternate
      int issued = 0;
      bool ok = true;
      for (Ring<L::kItems> at; ok && take(at); give_back(at), at.next()) {
        const Item& it = item_at(at.at);
        const int sinks = p.window > 0 ? p.sinks : 0;
        const int count = it.count, head = it.head;
        for (int i = 0; ok && i < count; ++i) {
          const int key0 = it.key0(i);
          // lane b finds the page of box b
          int page = static_cast<int>(c.num_pages), slot = 0;
          if (lane < boxes) {
            const int k = key0 + lane * rows_box;
            if (k <= it.p_hi && (k + rows_box - 1 >= it.lo || k < sinks)) {
              const int pg = paged_page(c, it.s, page_of(c, k));
              if (pg >= 0) page = pg;           // else the copy lies outside and reads zeros
              slot = k - page_of(c, k) * c.page_size;
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(kAll, mbar_wait(&empty[ring.at], ring.parity ^ 1u, abort_flag,
                                            c.status, p.timeout_ns));
            if (!ok) break;
            if (lane == 0) mbar_expect_tx(&full[ring.at], L::kTileBytes);
            __syncwarp();
            if (lane < boxes) {
              uint8_t* dst = smem + L::kRingOff + ring.at * L::kTileBytes + lane * rows_box * 128;
#pragma unroll
              for (int a = 0; a < kDp / 64; ++a)
                tma_load_4d(dst + a * L::kPanel, kv == 0 ? &tm_k : &tm_v, 64 * a, slot, head, page,
                            &full[ring.at]);
            }
            ring.next();
            issued = min(issued + 1, kStages);
          }
        }
      }
      // no copy may still be in flight when the CTA exits
      for (int i = 1; i <= issued; ++i) {
        const int st = ring.at - i;             // below 0: in the round before
        mbar_wait(&full[st < 0 ? st + kStages : st], st < 0 ? ring.parity ^ 1u : ring.parity,
                  nullptr, c.status, p.timeout_ns);
      }
    } else if (warp == 8) {
      // ================================================== MMAs
      constexpr uint32_t kFmt = kMmaBF16 ? 1u : 0u;
      constexpr uint32_t kIdQk = make_idesc(kFmt, kFmt, kTileRows, kKeys);
      // only the caller's channels, in 16s: k-steps of S, columns of O
      const int d16 = (c.D + 15) / 16;
      const uint32_t id_pv = uniform(make_idesc(kFmt, kFmt, kTileRows, 16) & ~(0x3Fu << 17) |
                                     (static_cast<uint32_t>(2 * d16) << 17) | (1u << 16));
      const uint32_t q_lo = sdesc_sw128_lo(smem_u32(smem));
      const uint32_t ring_lo = sdesc_sw128_lo(smem_u32(smem + L::kRingOff));
      // V: rows of 64 channels contiguous (MN-major), the next 64 channels a panel
      // further (leading offset), the next 8 keys 1024 bytes further (stride offset)
      const uint32_t v_lo = ((smem_u32(smem + L::kRingOff) & 0x3FFFFu) >> 4) |
                            (static_cast<uint32_t>(L::kPanel >> 4) << 16);
      const uint32_t tb = uniform(tbase);
      // S_t = Q_t K^T and O_t (+)= P_t V, for one elected lane
      auto qk = [&](auto tc, uint32_t k_lo) {
        constexpr int t = decltype(tc)::value;
        if (d16 == kDp / 16) {
#pragma unroll
          for (int k = 0; k < kDp / 16; ++k) {
            const uint32_t off = ((k / 4) * L::kPanel + (k % 4) * 32) >> 4;
            mma_f16_ss_lo(tb + t * 128, q_lo + ((t * L::kTileBytes) >> 4) + off, k_lo + off, kIdQk,
                          k > 0 ? 1u : 0u);
          }
          return;
        }
#pragma unroll
        for (int k = 0; k < kDp / 16; ++k) {
          const uint32_t off = ((k / 4) * L::kPanel + (k % 4) * 32) >> 4;
          if (k < d16)
            mma_f16_ss_lo(tb + t * 128, q_lo + ((t * L::kTileBytes) >> 4) + off, k_lo + off, kIdQk,
                          k > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](auto tc, uint32_t val_lo, uint32_t add) {
        constexpr int t = decltype(tc)::value;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(tb + 256 + t * kDp, tb + t * 128 + 8 * k, val_lo + ((k * 2048) >> 4),
                 kSdescSw128Hi, id_pv, k > 0 ? 1u : add);
      };
      constexpr std::integral_constant<int, 0> T0{};
      constexpr std::integral_constant<int, 1> T1{};
      Ring<kStages> ring;
      uint32_t items[2] = {0, 0}, steps[2] = {0, 0};
      bool ok = true, issued = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kAll, mbar_wait(bar, parity & 1, abort_flag, c.status, p.timeout_ns));
      };
      auto ring_lo_at = [&](uint32_t lo0) {
        return uniform(lo0 + ring.at * (L::kTileBytes >> 4));
      };
      for (Ring<L::kItems> item; ok && take(item); give_back(item), item.next()) {
        const Item& it = item_at(item.at);
        const bool two = it.two();
        const int count = it.count, sinks = p.window > 0 ? p.sinks : 0;
        ok = wait(&q_ready[0], items[0]++);
        if (ok && two) ok = wait(&q_ready[1], items[1]++);
        ok = ok && wait(&full[ring.at], ring.parity);
        if (!ok) break;
        tc_fence_after();
        issued = true;
        uint32_t k_lo = ring_lo_at(ring_lo);
        if (elect_one()) {
          qk(T0, k_lo);
          tc_commit(&s_full[0]);
          if (two) {
            qk(T1, k_lo);
            tc_commit(&s_full[1]);
          }
          tc_commit(&empty[ring.at]);
        }
        __syncwarp();
        ring.next();
        for (int i = 0; ok && i < count; ++i) {
          const bool more = i + 1 < count;
          ok = wait(&full[ring.at], ring.parity);
          if (!ok) break;
          if constexpr (!kQ8) {
            const int key0 = it.key0(i);
            if (!(key0 + kKeys - 1 <= it.p_hi && (key0 >= it.lo || key0 + kKeys - 1 < sinks))) {
              // values of keys that no row of the pair sees
              for (int r = lane; r < kKeys; r += 32) {
                const int key = key0 + r;
                if (key <= it.p_hi && (key >= it.lo || key < sinks)) continue;
                uint4* row = reinterpret_cast<uint4*>(smem + L::kRingOff +
                                                      ring.at * L::kTileBytes + r * 128);
#pragma unroll
                for (int a = 0; a < kDp / 64; ++a)
#pragma unroll
                  for (int q = 0; q < 8; ++q) row[a * (L::kPanel / 16) + q] = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          const uint32_t val_lo = ring_lo_at(v_lo);
          uint64_t* const v_empty = &empty[ring.at];
          ring.next();
          // ---- tile 0: PV, then the next QK^T
          ok = wait(&p_ready[0], steps[0]++);
          if (ok && more) ok = wait(&full[ring.at], ring.parity);
          if (!ok) break;
          tc_fence_after();
          if (more) k_lo = ring_lo_at(ring_lo);
          if (elect_one()) {
            pv(T0, val_lo, i > 0 ? 1u : 0u);
            if (!two) tc_commit(v_empty);
            if (more) {
              qk(T0, k_lo);
              tc_commit(&s_full[0]);
              if (!two) tc_commit(&empty[ring.at]);
            } else {
              tc_commit(&o_full[0]);
            }
          }
          __syncwarp();
          if (two) {
            // ---- tile 1
            ok = wait(&p_ready[1], steps[1]++);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              pv(T1, val_lo, i > 0 ? 1u : 0u);
              tc_commit(v_empty);
              if (more) {
                qk(T1, k_lo);
                tc_commit(&s_full[1]);
                tc_commit(&empty[ring.at]);
              } else {
                tc_commit(&o_full[1]);
              }
            }
            __syncwarp();
          }
          if (more) ring.next();
        }
      }
      if (issued) {                             // every MMA ends before TMEM is released
        if (elect_one()) tc_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0, nullptr, c.status, p.timeout_ns);
      }
    }
  } else if (wg == 3) {
    // ==================================================== 8-bit cache: widen
    if constexpr (kQ8) {
      regs_decrease<88>();
      constexpr int kRowLanes = kDp / 16;       // 16-byte vectors of a row
      constexpr int kIter = kKeys * kRowLanes / 128;
      const int id = tid - 384, r0 = id / kRowLanes, ch = id % kRowLanes * 16;
      float* const scales = reinterpret_cast<float*>(smem + L::kScaleOff);
      const int box = p.tensor_copies ? min(c.page_size, kKeys) : kKeys;
      const int scale_at = kKeys * kDp + id / box * max(4 * box, 128) + id % box * 4;
      Ring<kStages> ring;
      Ring<L::kRawStages> raw;
      bool ok = true;
      for (Ring<L::kItems> at; ok && take(at); give_back(at), at.next()) {
        const Item& it = item_at(at.at);
        const int count = it.count, before = it.before, lo = it.lo, p_hi = it.p_hi;
        const int sinks = p.window > 0 ? p.sinks : 0;
        for (int i = 0; ok && i < count; ++i) {
          const int key0 = it.key0(i);
          const bool part =
              !(key0 + kKeys - 1 <= p_hi && (key0 >= lo || key0 + kKeys - 1 < sinks));
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(kAll, mbar_wait(&raw_full[raw.at], raw.parity, abort_flag, c.status,
                                            p.timeout_ns) &&
                                      mbar_wait(&empty[ring.at], ring.parity ^ 1u, abort_flag,
                                                c.status, p.timeout_ns));
            if (!ok) break;
            const uint8_t* const codes = smem + L::kRawOff + raw.at * L::kRawBytes;
            uint8_t* const tile = smem + L::kRingOff + ring.at * L::kTileBytes +
                                  (ch / 64) * L::kPanel;
            uint4 w[kIter];
#pragma unroll
            for (int j = 0; j < kIter; ++j)
              w[j] = *reinterpret_cast<const uint4*>(codes + (r0 + j * (128 / kRowLanes)) * kDp +
                                                     ch);
            if (kv == 1 && part) {              // values of keys that no row of the pair sees
#pragma unroll
              for (int j = 0; j < kIter; ++j) {
                const int key = key0 + r0 + j * (128 / kRowLanes);
                if (!(key <= p_hi && (key >= lo || key < sinks))) w[j] = make_uint4(0, 0, 0, 0);
              }
            }
            if (kv == 0)
              scales[(before + i) % L::kScaleRing * kKeys + id] =
                  *reinterpret_cast<const float*>(codes + scale_at);
#pragma unroll
            for (int j = 0; j < kIter; ++j) {
              const int r = r0 + j * (128 / kRowLanes);
              const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
              uint32_t h[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (kv == 0) {
                  int8_to_half(u[q], h[2 * q], h[2 * q + 1]);
                } else {
                  h[2 * q] = e4m3x2_to_half2(u[q]);
                  h[2 * q + 1] = e4m3x2_to_half2(u[q] >> 16);
                }
              }
              const int q0 = (ch % 64) / 8;
              uint4* row = reinterpret_cast<uint4*>(tile + r * 128);
              row[q0 ^ (r & 7)] = make_uint4(h[0], h[1], h[2], h[3]);
              row[(q0 + 1) ^ (r & 7)] = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&full[ring.at]);
            mbar_arrive(&raw_empty[raw.at]);
            ring.next();
            raw.next();
          }
        }
      }
    }
  } else {
    // ==================================================== softmax of tile wg
    if constexpr (kQ8) regs_increase<176>();
    else regs_increase<208>();
    const int t = wg, r = tid - t * kTileRows;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lane_off + t * 128, to = tbase + lane_off + 256 + t * kDp;
    uint32_t items = 0, steps = 0;
    bool ok = true;
    bool used[2] = {false, false};
    // the next item that has rows in this tile
    auto advance = [&](Ring<L::kItems>& at) {
      for (; take(at); give_back(at), at.next())
        if (t == 0 || item_at(at.at).two()) return true;
      return false;
    };
    // The queries of this warp's 32 rows into shared memory, swizzled as a copy
    // would; returns this lane's row's factor from S to base-2 logits.  The lanes
    // of a row load neighbouring vectors (a row per lane would touch 32 lines a
    // load: 5000 cycles an item against 900).
    auto load_q = [&](const Item& x) {
      constexpr int kVecs = kDp / 8, kRowsAtOnce = 32 / kVecs;
      const int i = lane % kVecs, sub = lane / kVecs;
      uint8_t* const dst = smem + t * L::kTileBytes + (i / 8) * L::kPanel;
      float sc = p.scale_log2;
      const int row_end = x.rows - x.pair * kPairRows - t * kTileRows;
      const int off = x.tile[t].off;
      const uint16_t* const q0 = p.q + (static_cast<int64_t>(x.start) + x.tile[t].tok) * p.q_tok +
                                 static_cast<int64_t>(x.head) * p.group * p.q_head + 8 * i;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint4 v[kVecs / 2];
#pragma unroll
        for (int j = 0; j < kVecs / 2; ++j) {
          const int row = (warp & 3) * 32 + (half * (kVecs / 2) + j) * kRowsAtOnce + sub;
          v[j] = make_uint4(0, 0, 0, 0);
          if (row < row_end && 8 * i < c.D) {
            const int dt = by_group(p, off + row);
            const uint16_t* q = q0 + dt * p.q_tok + (off + row - dt * p.group) * p.q_head;
            if (p.q_vec) {
              v[j] = *reinterpret_cast<const uint4*>(q);
            } else {
              uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
              for (int e = 0; e < 8; ++e)
                u[e / 2] |= static_cast<uint32_t>(q[e]) << (16 * (e & 1));
              v[j] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kVecs / 2; ++j) {
          const int in_warp = (half * (kVecs / 2) + j) * kRowsAtOnce + sub;
          if constexpr (kQ8 && kQBF16) {
            // bf16 queries into fp16's range: times 2^-e, e the exponent of the row's largest
            const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              top = fmaxf(top, fabsf(__uint_as_float(u[e] << 16)));
              top = fmaxf(top, fabsf(__uint_as_float(u[e] & 0xFFFF0000u)));
            }
#pragma unroll
            for (int d = kVecs / 2; d > 0; d /= 2)
              top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
            const int ex = exponent_of(top);
            const float down = power_of_2(-ex);
            auto half2 = [&](uint32_t w2) {
              return pack2<false>(__uint_as_float(w2 << 16) * down,
                                  __uint_as_float(w2 & 0xFFFF0000u) * down);
            };
            v[j] = make_uint4(half2(u[0]), half2(u[1]), half2(u[2]), half2(u[3]));
#pragma unroll
            for (int g = 0; g < kRowsAtOnce; ++g) {
              const int e = __shfl_sync(kAll, ex, g * kVecs);
              // not 0, however small the row and the scale: hidden logits are -inf
              if (lane == in_warp - sub + g) sc = fmaxf(p.scale_log2 * power_of_2(e), FLT_MIN);
            }
          }
          const int row = (warp & 3) * 32 + in_warp;
          *reinterpret_cast<uint4*>(dst + row * 128 + (((i % 8) ^ (row & 7)) << 4)) = v[j];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      mbar_arrive(&q_ready[t]);
      return sc;
    };
    Ring<L::kItems> at;
    bool have = advance(at);
    float sc = have ? load_q(item_at(at.at)) : 0.0f;
    while (ok && have) {
      const Item& it = item_at(at.at);
      const int row_end = it.rows - it.pair * kPairRows - t * kTileRows;   // rows of this tile
      const bool has = r < row_end;
      const int dt = by_group(p, it.tile[t].off + r);         // this row's token, from the tile's
      const int pos = has ? it.tile[t].lo + dt : -1;
      const int t_lo = it.tile[t].lo, t_hi = it.tile[t].hi;
      const int count = it.count, before = it.before;
      const int sinks = p.window > 0 ? p.sinks : 0;
      float ref = -INFINITY, l = 0.0f;
      for (int i = 0; i < count; ++i) {
        ok = __all_sync(kAll, mbar_wait(&s_full[t], steps++ & 1, abort_flag, c.status,
                                        p.timeout_ns));
        if (!ok) break;
        tc_fence_after();
        const int key0 = it.key0(i);
        const bool masked =
            !(key0 + kKeys - 1 <= t_lo &&
              (p.window <= 0 || key0 >= t_hi - p.window + 1 || key0 + kKeys - 1 < sinks));
        // Exponentials against the reference at hand, and the maximum beside them,
        // in one straight run of independent instructions.  Only if a row's
        // maximum turns out to have outgrown its reference (always on an item's
        // first tile), the reference moves and the run is taken again; S is still
        // there, as P is stored last.
        uint32_t w[64];
        float2 a01, a23;
        // logits of 32 kC keys from the key0-th on, without the factor sc
        auto logits = [&](auto& x, int c0, auto masked_c) {
#pragma unroll
          for (int q = 0; q < kC; ++q) tmem_ld32(ts + 32 * (c0 + q), x[q]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < kC; ++q) reg_fence(x[q]);
          if constexpr (kQ8) {
            const float4* ks = reinterpret_cast<const float4*>(
                smem + L::kScaleOff + (((before + i) % L::kScaleRing) * kKeys + 32 * c0) * 4);
#pragma unroll
            for (int e = 0; e < 8 * kC; ++e) {
              const float4 k4 = ks[e];
              uint32_t* y = &x[e / 8][(e % 8) * 4];
              const float2 u = __fmul2_rn(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                                          make_float2(k4.x, k4.y));
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])),
                                          make_float2(k4.z, k4.w));
              y[0] = __float_as_uint(u.x);
              y[1] = __float_as_uint(u.y);
              y[2] = __float_as_uint(v.x);
              y[3] = __float_as_uint(v.y);
            }
          }
          if constexpr (decltype(masked_c)::value) {
#pragma unroll
            for (int q = 0; q < kC; ++q) {
              const int k = key0 + 32 * (c0 + q);
              const int hi = pos + 1 - k;                            // keys below: not later
              const int lo = p.window > 0 ? pos - p.window + 1 - k : 0;   // below: too early
              const uint32_t early = below(lo) & ~below(sinks - k);
              const uint32_t see = below(hi) & ~early;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see >> e) & 1u)) x[q][e] = 0xFF800000u;       // -inf
            }
          }
        };
        auto weigh = [&](auto masked_c) {
          const float safe = ref == -INFINITY ? 0.0f : ref;
          const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-safe, -safe);
          a01 = make_float2(0.0f, 0.0f);
          a23 = make_float2(0.0f, 0.0f);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c0 = 0; c0 < 4; c0 += kC) {
            uint32_t x[kC][32];
            logits(x, c0, masked_c);
#pragma unroll
            for (int e = 0; e < 8 * kC; ++e) {
              const uint32_t* y = &x[e / 8][(e % 8) * 4];
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(y[k]));
              const float2 d01 = __ffma2_rn(
                  make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, nm2);
              const float2 d23 = __ffma2_rn(
                  make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), sc2, nm2);
              const float2 p01 = make_float2(fast_exp2(d01.x), fast_exp2(d01.y));
              const float2 p23 = make_float2(fast_exp2(d23.x), fast_exp2(d23.y));
              w[16 * c0 + 2 * e] = pack2<kMmaBF16>(p01.x, p01.y);
              w[16 * c0 + 2 * e + 1] = pack2<kMmaBF16>(p23.x, p23.y);
              a01 = __fadd2_rn(a01, p01);
              a23 = __fadd2_rn(a23, p23);
            }
          }
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        };
        while (true) {
          const float top = masked ? weigh(std::true_type{}) : weigh(std::false_type{});
          const bool grew = top > ref + kOver || (ref == -INFINITY && top > -INFINITY);
          if (!__any_sync(kAll, grew)) break;
          const float next = grew ? top - kDown : ref;
          const float alpha = grew ? fast_exp2(ref - next) : 1.0f;  // 0 from -inf
          if (i > 0) {
#pragma unroll
            for (int q = 0; q < kDp / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(to + 16 * q, o);
              tmem_ld_wait();
              reg_fence(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(to + 16 * q, o);
            }
          }
          l *= alpha;
          ref = next;
        }
        tmem_st32(ts, reinterpret_cast<const uint32_t (&)[32]>(w[0]));
        tmem_st32(ts + 32, reinterpret_cast<const uint32_t (&)[32]>(w[32]));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_ready[t]);
        l += (a01.x + a01.y) + (a23.x + a23.y);
      }
      if (!ok) break;
      // The next item's queries go out before this one's results: every QK^T of
      // this tile has been read, so its first one can run meanwhile.  (It
      // overwrites S_t behind the last PV that reads P_t; O_t is only
      // overwritten once this thread has delivered the next P.)
      // Only the very next item is waited for here: one further on may need the
      // slot of this one, which is given back below.
      Ring<L::kItems> nx = at;
      nx.next();
      have = take(nx);
      const bool ready = have && (t == 0 || item_at(nx.at).two());
      float next_sc = 0.0f;
      if (ready) next_sc = load_q(item_at(nx.at));
      // ---- out = O / l, or a part
      ok = __all_sync(kAll, mbar_wait(&o_full[t], items++ & 1, abort_flag, c.status,
                                      p.timeout_ns));
      if (!ok) break;
      tc_fence_after();
      const bool whole = it.first == 0 && it.count == it.per;
      if (whole) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const int64_t orow = (static_cast<int64_t>(it.start) + it.tile[t].tok + dt) * p.Hq +
                             it.head * p.group + it.tile[t].off + r - dt * p.group;
        const float* sv = c.v_scale + it.head * kDp;
        // Four lanes trade their rows' 16-byte vectors, so that each store writes
        // 64 bytes of a row (a row per lane would write 32 half sectors).
        const int j = lane & 3;
        int64_t rows4[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) rows4[m] = __shfl_sync(kAll, orow, (lane & ~3) + m);
#pragma unroll 1
        for (int q = 0; q < kDp / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(to + 32 * q, o);
          tmem_ld_wait();
          reg_fence(o);
          uint32_t u[4][4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a = __uint_as_float(o[8 * v + 2 * e]) * inv;
              float b = __uint_as_float(o[8 * v + 2 * e + 1]) * inv;
              if constexpr (kQ8) {
                a *= sv[32 * q + 8 * v + 2 * e];
                b *= sv[32 * q + 8 * v + 2 * e + 1];
              }
              u[v][e] = pack2<kQBF16>(a, b);
            }
          // a 4 x 4 transpose of vectors: by pairs of lanes, then by pairs of pairs
#pragma unroll
          for (int d = 1; d <= 2; d *= 2)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (!(v & d)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t give = (j & d) ? u[v][e] : u[v + d][e];
                  const uint32_t got = __shfl_xor_sync(kAll, give, d);
                  if (j & d) u[v][e] = got;
                  else u[v + d][e] = got;
                }
              }
          const int ch = 32 * q + 8 * j;
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if ((r & ~3) + m < row_end && ch < c.D)
              *reinterpret_cast<uint4*>(p.out + rows4[m] * c.D + ch) =
                  make_uint4(u[m][0], u[m][1], u[m][2], u[m][3]);
        }
        if (has && p.lse != nullptr)
          p.lse[orow] = l > 0.0f ? (ref + log2f(l)) * 0.69314718055994530942f : -INFINITY;
      } else {
        const int which = it.first == 0 ? 1 : 0;
        uint8_t* part = many_part(p.parts, cta, which);
        used[which] = true;
        if (t == 0 && r == 0) {
          ManyHead* h = reinterpret_cast<ManyHead*>(part);
          h->parts = it.parts;
          h->seq = it.s;
          h->head = it.head;
          h->pair = it.pair;
        }
        const int row = t * kTileRows + r;
        float* ml = reinterpret_cast<float*>(part + sizeof(ManyHead));
        ml[row] = ref;
        ml[kPairRows + row] = l;
        float4* po = reinterpret_cast<float4*>(ml + 2 * kPairRows);
#pragma unroll
        for (int q = 0; q < kDp / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(to + 32 * q, o);
          tmem_ld_wait();
          reg_fence(o);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            po[(8 * q + v) * kPairRows + row] =
                make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                            __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
        }
      }
      tc_fence_before();                        // O_t has been read
      give_back(at);
      if (have && !ready) {                     // an item without rows in this tile
        give_back(nx);
        nx.next();
        have = advance(nx);
        if (have) next_sc = load_q(item_at(nx.at));
      }
      at = nx;
      sc = next_sc;
    }
    if (tid == 0) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (!used[w]) reinterpret_cast<ManyHead*>(many_part(p.parts, cta, w))->parts = 0;
    }
  }

  // ---- teardown: all roles have drained; release tensor memory
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// Joins 32 rows of the pair that begins in CTA blockIdx.x and ends in a later
// one: weights 2^(m_i - max), summed in the parts' order.
template <bool kQBF16, int kDp>
__global__ void __launch_bounds__(256)
paged_many_join_kernel(const PagedAttnParams p, int ctas) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x;
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), grp = threadIdx.x >> 5;
  const ManyHead* h = reinterpret_cast<const ManyHead*>(many_part(p.parts, c0, 1));
  const int parts = min(h->parts, ctas - c0);
  if (parts <= 0) return;
  int start, n, len;
  if (!paged_seq(p.c, h->seq, &start, &n, &len)) return;
  const int rows = n * p.group, rr = h->pair * kPairRows + row;
  if (rr >= rows) return;
  auto ml = [&](int i) {
    return reinterpret_cast<const float*>(many_part(p.parts, c0 + i, i == 0) + sizeof(ManyHead));
  };
  float top = -INFINITY;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, ml(i)[row]);
  const float safe = top == -INFINITY ? 0.0f : top;
  constexpr int kVec = kDp / 32;                 // float4s of a thread
  float sum = 0.0f;
  float4 acc[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = 0; i < parts; ++i) {
    const float* f = ml(i);
    const float w = fast_exp2(f[row] - safe);
    sum += w * f[kPairRows + row];
    const float4* po = reinterpret_cast<const float4*>(f + 2 * kPairRows);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const float4 o = po[(grp + 8 * v) * kPairRows + row];
      acc[v].x += w * o.x; acc[v].y += w * o.y; acc[v].z += w * o.z; acc[v].w += w * o.w;
    }
  }
  const int64_t tok = static_cast<int64_t>(start) + rr / p.group;
  const int hq = h->head * p.group + rr % p.group;
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int ch = 4 * (grp + 8 * v);
    if (ch >= p.c.D) continue;
    float4 a = acc[v];
    a.x *= inv; a.y *= inv; a.z *= inv; a.w *= inv;
    if (p.c.kind == kKindQ8) {
      const float4 s = *reinterpret_cast<const float4*>(p.c.v_scale + h->head * kDp + ch);
      a.x *= s.x; a.y *= s.y; a.z *= s.z; a.w *= s.w;
    }
    *reinterpret_cast<uint2*>(p.out + (tok * p.Hq + hq) * p.c.D + ch) =
        make_uint2(pack2<kQBF16>(a.x, a.y), pack2<kQBF16>(a.z, a.w));
  }
  if (p.lse != nullptr && grp == 0)
    p.lse[tok * p.Hq + hq] = sum > 0.0f ? (top + log2f(sum)) * 0.69314718055994530942f
                                        : -INFINITY;
}

// Whether pages are whole boxes of a 128-key tile, or hold whole tiles, with
// strides that a tensor map takes (below 2^40 bytes).
bool page_boxes(const PagedGeo& c) {
  if (c.page_size < kKeys ? kKeys % c.page_size != 0 : c.page_size % kKeys != 0) return false;
  return c.page_stride < (int64_t(1) << 39) && c.token_stride < (int64_t(1) << 39) &&
         c.head_stride < (int64_t(1) << 39);
}

template <int kKind, bool kQBF16, int kDp>
cudaError_t launch_many(const PagedAttnParams& p, int sms, cudaStream_t st) {
  using L = Many<kKind, kDp>;
  auto* kern = paged_many_kernel<kKind, kQBF16, kDp>;
  static std::atomic<bool> configured[64] = {};   // a kernel attribute, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  CUtensorMap mk{}, mv{}, ms{};
  PagedAttnParams prm = p;
  const PagedGeo& c = p.c;
  const uint64_t el = kKind == kKindQ8 ? 1 : 2;                // bytes of an element
  prm.tensor_copies = kKind != kKindQ8 || (page_boxes(c) && c.wide);
  if (prm.tensor_copies) {
    const uint64_t dims[4] = {static_cast<uint64_t>(c.D), static_cast<uint64_t>(c.page_size),
                              static_cast<uint64_t>(c.Hkv), static_cast<uint64_t>(c.num_pages)};
    const uint64_t strides[3] = {static_cast<uint64_t>(c.token_stride) * el,
                                 static_cast<uint64_t>(c.head_stride) * el,
                                 static_cast<uint64_t>(c.page_stride) * el};
    const uint32_t rows = static_cast<uint32_t>(c.page_size < kKeys ? c.page_size : kKeys);
    const uint32_t box[4] = {kKind == kKindQ8 ? static_cast<uint32_t>(kDp) : 64u, rows, 1, 1};
    const CUtensorMapDataType type =
        kKind == kKindQ8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle swizzle =
        kKind == kKindQ8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    bool made = encode_tiled(&mk, type, 4, c.k, dims, strides, box, swizzle) &&
                encode_tiled(&mv, type, 4, c.v, dims, strides, box, swizzle);
    if (made && kKind == kKindQ8) {
      const uint64_t sdims[3] = {dims[1], dims[2], dims[3]};
      const uint64_t sstrides[2] = {dims[1] * 4, dims[1] * dims[2] * 4};
      const uint32_t sbox[3] = {rows, 1, 1};
      made = encode_tiled(&ms, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, c.k_scale, sdims, sstrides,
                          sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    if (!made) return cudaErrorInvalidValue;
  }
  // one CTA per SM, and no more than the units of the lengths the call declares
  const int64_t pairs = (static_cast<int64_t>(p.c.max_q) * p.group + kPairRows - 1) / kPairRows;
  const int64_t items = pairs * p.c.nseq * p.c.Hkv;   // below 2^58; times the tiles perhaps not
  const int64_t tiles = (static_cast<int64_t>(p.c.max_kv) + kKeys - 1) / kKeys + 1;
  int ctas = sms < kMaxManyCtas ? sms : kMaxManyCtas;
  if (items < ctas && items * tiles < ctas) ctas = static_cast<int>(items * tiles);
  kern<<<ctas, L::kThreads, L::kAlloc, st>>>(mk, mv, ms, prm);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), kPairRows / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_many_join_kernel<kQBF16, kDp>, p, ctas);
  note_launch();
  return e;
}

template <int kKind, bool kQBF16>
cudaError_t launch_many_dim(const PagedAttnParams& p, int sms, cudaStream_t st) {
  return p.c.Dp == 64 ? launch_many<kKind, kQBF16, 64>(p, sms, st)
                      : launch_many<kKind, kQBF16, 128>(p, sms, st);
}

}  // namespace

size_t paged_many_bytes() { return 2 * static_cast<size_t>(kMaxManyCtas) * kManyPartBytes; }

// 16-bit pages are copied as boxes of whole pages or 128 slots, by tensor maps;
// codes of 8 bits need not be.
bool paged_many_serves(const PagedGeo& c, int group) {
  if (group > 16384) return false;
  return c.kind == kKindQ8 || page_boxes(c);
}

cudaError_t launch_paged_many(const PagedAttnParams& p, bool bf16, int sms, cudaStream_t st) {
  if (p.c.kind == kKindQ8)
    return bf16 ? launch_many_dim<kKindQ8, true>(p, sms, st)
                : launch_many_dim<kKindQ8, false>(p, sms, st);
  return bf16 ? launch_many_dim<kKindBF16, true>(p, sms, st)
              : launch_many_dim<kKindF16, false>(p, sms, st);
}

}  // namespace sage
