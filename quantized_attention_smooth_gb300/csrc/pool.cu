// Block tables, slot maps and the page pool's stack, from request lengths.
//
//   have_i = ceil(len_i / page),  need_i = ceil((len_i + new_i) / page) - have_i,
//   first_i = sum of need before i;  granted: need_i = 0, or first_i + need_i <= left
//   k-th new page of i: stack[left - 1 - first_i - k];  left -= granted needs
//   row t of i: position len_i + t, slot table_i[position / page] * page + position % page
//
// and a cut the other way round: the k-th page of all that go back lies at
// stack[left' - 1 - k], so that it undoes a step.
//
// A step moves little (64 requests over 1028 columns: 0.5 MB) and is a chain of a
// few dependent loads, so it runs as one launch of one cluster: its first CTA scans
// the requests, a thread each, and leaves 16 bytes a sequence; the cluster's barrier
// hands them to the others, which write tables, positions and slots.  A request that
// is given twice is found by a mark per request, which the first CTA clears again.
// Measured (GB300, in a graph): a step and a cut of 64 requests over 1028 columns 14 us,
// of 256 prompts (52000 rows, 264 columns) 21 us; their bytes would take 0.2.

#include <climits>

#include "sage_kernels.h"
#include "sage_paged.h"

namespace sage {
namespace {

constexpr int kThreads = 1024, kCluster = 8;
constexpr int kStaged = 1024;        // sequences whose entries fit in shared memory
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ int pages_of(const PoolParams& p, int64_t tokens) {
  return static_cast<int>((tokens + p.page_size - 1) / p.page_size);
}

// Inclusive sums over the block of two numbers a thread, and their totals.
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t* all_a, int64_t* all_b) {
  __shared__ int64_t sums[2][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t x = __shfl_up_sync(kAll, a, d), y = __shfl_up_sync(kAll, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sums[0][warp] = a;
    sums[1][warp] = b;
  }
  __syncthreads();
  // every warp sums the warps' totals for itself
  int64_t x = sums[0][lane], y = sums[1][lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t u = __shfl_up_sync(kAll, x, d), v = __shfl_up_sync(kAll, y, d);
    if (lane >= d) {
      x += u;
      y += v;
    }
  }
  *all_a = __shfl_sync(kAll, x, 31);
  *all_b = __shfl_sync(kAll, y, 31);
  const int64_t before_a = __shfl_sync(kAll, x, (warp + 31) & 31);
  const int64_t before_b = __shfl_sync(kAll, y, (warp + 31) & 31);
  if (warp > 0) {
    a += before_a;
    b += before_b;
  }
  __syncthreads();
}

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// Marks every request with its first place in the call (counted from the end, so
// that the largest mark is the first place).
__device__ __forceinline__ void mark_requests(const PoolParams& p) {
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int r = p.requests[i];
    if (r >= 0 && r < p.max_requests) atomicMax(&p.marks[r], static_cast<uint32_t>(p.n - i));
  }
  __syncthreads();
}
// Whether place i holds a request of the pool that no earlier place holds.
__device__ __forceinline__ bool first_place(const PoolParams& p, int i, int r) {
  return r >= 0 && r < p.max_requests &&
         __ldcg(&p.marks[r]) == static_cast<uint32_t>(p.n - i);
}
__device__ __forceinline__ void clear_marks(const PoolParams& p) {
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int r = p.requests[i];
    if (r >= 0 && r < p.max_requests) p.marks[r] = 0;
  }
}

// The stack's height; a number that cannot be one is reported and taken as the
// nearest that can.
__device__ __forceinline__ int height(const PoolParams& p) {
  const int left = p.left[0];
  if (left >= 0 && left <= p.num_pages) return left;
  if (threadIdx.x == 0) atomicOr(p.status, kStatusBadPool);
  return left < 0 ? 0 : p.num_pages;
}

// A sequence's entry in the workspace: its length before the step (-1: denied), the
// stack's place of its first new page, pages that it has and pages that it gets.
__device__ __forceinline__ void plan_step(const PoolParams& p) {
  const int left = height(p);
  mark_requests(p);
  int64_t rows = 0, taken = 0;
  int given = left, denied = 0;
  for (int i0 = 0; i0 < p.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int r = -1, old = 0, fresh = 0, have = 0, need = 0;
    bool fine = false;
    if (i < p.n) {
      r = p.requests[i];
      fresh = p.new_lens[i];
      if (first_place(p, i, r)) {
        old = p.lens[r];
        const int64_t all = static_cast<int64_t>(old) + fresh;
        fine = old >= 0 && fresh >= 0 && fresh <= p.max_q && all <= p.max_kv;
        if (fine) {
          const int end = pages_of(p, all);
          fine = end <= p.width && end <= p.plan_width;
        }
        if (old >= 0 && pages_of(p, old) <= p.width) have = pages_of(p, old);
      }
      if (fresh < 0) fresh = 0;
    }
    int64_t row = fresh, all_rows, upto, all_need;
    // the rows' places first: a sequence beyond them needs no pages
    int64_t none = 0, all_none;
    scan2(row, none, &all_rows, &all_none);
    if (rows + row > p.rows) fine = false;
    if (i < p.n && !fine) atomicOr(p.status, kStatusBadPool);
    if (fine) need = pages_of(p, static_cast<int64_t>(old) + fresh) - have;
    upto = need;
    int64_t refused = 0, all_refused;
    scan2(upto, refused, &all_need, &all_refused);
    const bool granted = fine && (need == 0 || taken + upto <= left);
    const int64_t first = taken + upto - need;
    if (i < p.n) {
      const int64_t at = rows + row - fresh;
      p.cu_q[i] = static_cast<int>(min(at, static_cast<int64_t>(INT_MAX)));
      p.kv_lens[i] = granted ? old + fresh : 0;
      p.seqs[i] = make_int4(granted ? old : -1, static_cast<int>(max(left - 1 - first, int64_t(-1))),
                            have, granted ? need : 0);
      if (granted) {
        p.lens[r] = old + fresh;
        if (need > 0) given = min(given, static_cast<int>(left - first - need));
      } else {
        ++denied;
      }
    }
    rows += all_rows;
    taken += all_need;
  }
  // the lowest place that was taken, and how many were denied
  __shared__ int low, count;
  if (threadIdx.x == 0) {
    low = left;
    count = 0;
  }
  __syncthreads();
  if (given < left) atomicMin(&low, given);
  if (denied > 0) atomicAdd(&count, denied);
  clear_marks(p);
  __syncthreads();
  if (threadIdx.x == 0) {
    p.cu_q[p.n] = static_cast<int>(min(rows, static_cast<int64_t>(INT_MAX)));
    p.left[0] = low;
    p.denied[0] = count;
  }
}

// A page of a sequence: its own, or the stack's.
__device__ __forceinline__ int page_at(const PoolParams& p, const int32_t* row, const int4& q,
                                       int j) {
  return j < q.z ? row[j] : p.free_pages[q.y - (j - q.z)];
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
step_kernel(const PoolParams p) {
  // Up to kStaged sequences each CTA keeps the entries, rows and requests by itself: the
  // search for a row's sequence is a chain of log2 n loads (256 prompts, from the L2 and
  // a row at a time: 28 us, so 21).  More sequences are read where they lie.
  __shared__ int4 seqs_s[kStaged];
  __shared__ int cu_s[kStaged + 1], requests_s[kStaged];
  if (blockIdx.x == 0) plan_step(p);
  cluster_barrier();
  const bool staged = p.n <= kStaged;
  if (staged) {
    for (int i = threadIdx.x; i <= p.n; i += kThreads) {
      cu_s[i] = __ldcg(&p.cu_q[i]);
      if (i < p.n) {
        seqs_s[i] = __ldcg(&p.seqs[i]);
        requests_s[i] = p.requests[i];
      }
    }
    __syncthreads();
  }
  const int* const cu = staged ? cu_s : p.cu_q;
  const int4* const seqs = staged ? seqs_s : p.seqs;
  const int* const requests = staged ? requests_s : p.requests;
  const int id = blockIdx.x * kThreads + threadIdx.x, threads = kCluster * kThreads;
  // ---- the tables: a warp per 128 columns of a row
  const int lane = threadIdx.x & 31, warps = threads / 32;
  const int chunks = (p.plan_width + 127) / 128;
  for (int64_t u = id / 32; u < static_cast<int64_t>(p.n) * chunks; u += warps) {
    const int i = static_cast<int>(u / chunks);
    const int j0 = static_cast<int>(u - static_cast<int64_t>(i) * chunks) * 128;
    const int4 q = seqs[i];
    int32_t* const own = p.table + (q.z + q.w > 0 ? requests[i] * p.table_stride : 0);
    int32_t* const out = p.block_table + i * p.plan_stride;
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k + lane;
      page[k] = j < p.plan_width && j < q.z + q.w ? page_at(p, own, q, j) : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k + lane;
      if (j >= p.plan_width) continue;
      if (j >= q.z && j < q.z + q.w) own[j] = page[k];
      out[j] = page[k];
    }
  }
  // ---- the rows, four at a time; those from cu[n] on stay as they are
  if (p.positions == nullptr && p.slots == nullptr) return;
  const int64_t total = min(static_cast<int64_t>(cu[p.n]), p.rows);
  constexpr int kUnroll = 4;
  for (int64_t tb = id; tb < total; tb += kUnroll * threads) {
    int64_t pos[kUnroll];
    int page[kUnroll], in[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t t = tb + k * threads;
      pos[k] = page[k] = -1;
      in[k] = 0;
      if (t >= total) continue;
      int lo = 0, hi = p.n;                     // the last i with cu[i] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int4 q = seqs[lo];
      if (q.x >= 0) {
        const int at = q.x + static_cast<int>(t - cu[lo]);
        const int j = p.page_shift >= 0 ? at >> p.page_shift : at / p.page_size;
        pos[k] = at;
        in[k] = at - j * p.page_size;
        page[k] = page_at(p, p.table + requests[lo] * p.table_stride, q, j);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t t = tb + k * threads;
      if (t >= total) continue;
      if (p.positions != nullptr) p.positions[t] = pos[k];
      if (p.slots != nullptr)
        p.slots[t] = pos[k] < 0 ? -1 : static_cast<int64_t>(page[k]) * p.page_size + in[k];
    }
  }
}

// A sequence's entry: its first page to go, how many go, and how many pages before
// them go (from the call's first sequence on).
__device__ __forceinline__ void plan_trim(const PoolParams& p) {
  const int left = height(p);
  mark_requests(p);
  int64_t gone = 0;
  for (int i0 = 0; i0 < p.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int r = -1, kept = 0, back = 0;
    if (i < p.n) {
      r = p.requests[i];
      const int keep = p.new_lens != nullptr ? p.new_lens[i] : 0;
      const bool fine = first_place(p, i, r) && keep >= 0;
      if (!fine) {
        atomicOr(p.status, kStatusBadPool);
      } else {
        const int len = p.lens[r];
        if (keep < len && pages_of(p, len) <= p.width) {
          kept = pages_of(p, keep);
          back = pages_of(p, len) - kept;
          p.lens[r] = keep;
        } else if (keep < len || len < 0) {
          atomicOr(p.status, kStatusBadPool);
        }
      }
    }
    int64_t upto = back, all, none = 0, all_none;
    scan2(upto, none, &all, &all_none);
    if (i < p.n)
      p.seqs[i] = make_int4(kept, back, static_cast<int>(min(gone + upto - back, int64_t(INT_MAX))), 0);
    gone += all;
  }
  clear_marks(p);
  __syncthreads();
  if (threadIdx.x == 0) {
    // more pages than the stack has room for: some went back twice
    if (left + gone > p.num_pages) atomicOr(p.status, kStatusBadPool);
    p.left[0] = static_cast<int>(min(left + gone, static_cast<int64_t>(p.num_pages)));
  }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
trim_kernel(const PoolParams p) {
  if (blockIdx.x == 0) plan_trim(p);
  cluster_barrier();
  const int id = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
  const int height = __ldcg(&p.left[0]);
  for (int i = id / 32; i < p.n; i += kCluster * kThreads / 32) {
    const int4 q = __ldcg(&p.seqs[i]);
    if (q.y == 0) continue;
    const int32_t* const own = p.table + p.requests[i] * p.table_stride + q.x;
    for (int k = lane; k < q.y; k += 32) {
      const int64_t at = static_cast<int64_t>(height) - 1 - q.z - k;
      if (at >= 0) p.free_pages[at] = own[k];
    }
  }
}

}  // namespace

cudaError_t launch_paged_step(const PoolParams& p, cudaStream_t st) {
  step_kernel<<<kCluster, kThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_paged_trim(const PoolParams& p, cudaStream_t st) {
  trim_kernel<<<kCluster, kThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace sage
