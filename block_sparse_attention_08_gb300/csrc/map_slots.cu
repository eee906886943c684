// map_slots.cu -- page-table rows and the slot of every new token of a serving
// step, from the requests' lengths and a stack of free pages.
//
// With old = len - new, request r holds ceil(old / 128) pages and needs
// ceil(len / 128); over the requests, two running sums place everything: of
// the new tokens (row cu[r] of the token buffers) and of the opened pages (the
// off[r]-th page from the top of the stack).  Token i of request r sits at
// position p = old + i, slot table[r, p / 128] * 128 + p % 128.
//
// The call moves a few bytes per request and 12 per token, so it is bound by
// launch and load latency.  One launch does all of it: every CTA takes its own
// share of the token rows and of the opened pages and runs the sums over all
// requests itself, kMsChunk requests at a time, in shared memory; no CTA waits
// for another.  A token in an opened page takes the id from the stack, not
// from the table entry that another CTA may be writing.  3.2 us in
// a graph for 64 single tokens, 4.2 us for 509 requests with 14 k tokens (6.5 us
// with 2048 rows to a CTA: the loads of a thread's four rows followed each other;
// an empty launch is 1.3 us).
#include "launch.h"

namespace msa {

constexpr int kMsThreads = 512;
constexpr int kMsChunk = kMsThreads;   // one request per thread and pass
constexpr int kMsCtas = 4 * kNumSMs;   // resident at once; up to here each thread has one token row

struct MsSum {
  long long tokens, pages;
};

// Exclusive sums over the CTA's threads; `total` gets the sums of all.
__device__ __forceinline__ MsSum ms_scan(MsSum x, MsSum* warp_sums, MsSum* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  MsSum s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, s.tokens, d), p = __shfl_up_sync(0xffffffffu, s.pages, d);
    if (lane >= d) {
      s.tokens += t;
      s.pages += p;
    }
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  MsSum before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < kMsThreads / 32; ++w) {
    const MsSum v = warp_sums[w];
    if (w < warp) {
      before.tokens += v.tokens;
      before.pages += v.pages;
    }
    all.tokens += v.tokens;
    all.pages += v.pages;
  }
  *total = all;
  return MsSum{before.tokens + s.tokens - x.tokens, before.pages + s.pages - x.pages};
}

// Pages of n positions (n + kBlock - 1 may pass 2^31).
__device__ __forceinline__ int ms_pages(int n) { return static_cast<int>((static_cast<unsigned>(n) + kBlock - 1) / kBlock); }

// The last i < n with a[i] <= x (a[0] <= x).
__device__ __forceinline__ int ms_last_le(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kMsThreads) map_slots_kernel(SlotsLaunch a, int rows) {
  // per request of the pass: first row, first opened page, old length
  __shared__ int cu[kMsChunk + 1], off[kMsChunk + 1], old[kMsChunk];
  __shared__ MsSum warp_sums[kMsThreads / 32];
  __shared__ int cut_at;
  const int tid = threadIdx.x;
  const long long row0 = static_cast<long long>(blockIdx.x) * rows;
  const long long row1 = min(a.capacity, row0 + rows);
  // the kernel before has completed; the next may be launched behind this one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  long long free_top = *a.num_free;
  if (free_top < 0 || free_top > a.free_capacity) free_top = 0;
  // the id of the j-th opened page, -1 if the stack holds a bad one
  auto opened = [&](long long j) {
    const int id = a.free_pages[free_top - 1 - j];
    return id >= 0 && id < a.num_pages ? id : -1;
  };
  long long tokens = 0, pages = 0;  // mapped by the passes so far
  bool cut = false;                 // a request did not fit: none from it on is mapped

  for (int r0 = 0; r0 < a.batch; r0 += kMsChunk) {
    const int r = r0 + tid, n = min(kMsChunk, a.batch - r0);
    MsSum mine{0, 0};
    int len = 0, fresh = 0;
    if (r < a.batch) {
      len = a.seq_lens[r];
      fresh = a.new_lens[r];
      if (fresh < 0 || fresh > len || (static_cast<long long>(len) + kBlock - 1) / kBlock > a.max_blocks) {
        if (blockIdx.x == 0) record_error(a.err, MSA_DEVERR_LENGTH, r);
        fresh = 0;
        len = 0;
      }
      mine.tokens = fresh;
      mine.pages = (static_cast<long long>(len) + kBlock - 1) / kBlock -
                   (static_cast<long long>(len) - fresh + kBlock - 1) / kBlock;
    }
    if (tid == 0) cut_at = cut ? 0 : n;
    MsSum total;
    const MsSum before = ms_scan(mine, warp_sums, &total);  // (holds a barrier after the store of cut_at)
    const bool fits = tokens + before.tokens + mine.tokens <= a.capacity && pages + before.pages + mine.pages <= free_top;
    if (!cut && tid < n && !fits) atomicMin(&cut_at, tid);
    __syncthreads();
    const int m = cut_at;  // the requests of this pass that are mapped: the sums up to it fit in int32
    if (tid < m) {
      cu[tid] = static_cast<int>(tokens + before.tokens);
      off[tid] = static_cast<int>(pages + before.pages);
      old[tid] = len - fresh;
      if (tid == m - 1) {
        cu[m] = cu[tid] + fresh;
        off[m] = off[tid] + static_cast<int>(mine.pages);
      }
    }
    if (m == 0 && tid == 0) {
      cu[0] = static_cast<int>(tokens);
      off[0] = static_cast<int>(pages);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
      if (tid < n) a.cu[r] = cu[min(tid, m)];
      if (tid == m && m < n && !cut) record_error(a.err, MSA_DEVERR_FULL, r);
    }
    // this CTA's token rows among the pass's
    for (long long t = max(row0, static_cast<long long>(cu[0])) + tid; t < min(row1, static_cast<long long>(cu[m]));
         t += kMsThreads) {
      const int i = ms_last_le(cu, m, static_cast<int>(t));
      const int p = old[i] + static_cast<int>(t) - cu[i];
      const int page = p / kBlock, have = ms_pages(old[i]);
      int id;
      if (page >= have) {
        id = opened(off[i] + page - have);
      } else {
        id = a.page_table[static_cast<long long>(r0 + i) * a.max_blocks + page];
        if (id < 0 || id >= a.num_pages) id = -1;
      }
      if (id < 0) record_error(a.err, MSA_DEVERR_PAGE, t);
      a.slots[t] = id < 0 ? -1 : static_cast<int64_t>(id) * kBlock + p % kBlock;
      a.positions[t] = p;
    }
    // this CTA's opened pages among the pass's
    for (int j = off[0] + blockIdx.x * kMsThreads + tid; j < off[m]; j += gridDim.x * kMsThreads) {
      const int i = ms_last_le(off, m, j);
      const int page = ms_pages(old[i]) + j - off[i];
      a.page_table[static_cast<long long>(r0 + i) * a.max_blocks + page] = opened(j);
    }
    cut = cut || m < n;
    tokens = cu[m];
    pages = off[m];
    __syncthreads();  // the arrays are rewritten by the next pass
  }
  for (long long t = max(row0, tokens) + tid; t < row1; t += kMsThreads) {
    a.slots[t] = -1;
    a.positions[t] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.batch] = static_cast<int>(tokens);
    *a.num_free_out = static_cast<int>(free_top - pages);
  }
}

cudaError_t launch_map_slots(const SlotsLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e0 = launch_prologue(); e0 != cudaSuccess) return e0;
  constexpr long long kOnce = static_cast<long long>(kMsCtas) * kMsThreads;
  const long long rows = (L.capacity + kOnce - 1) / kOnce * kMsThreads, grid = (L.capacity + rows - 1) / rows;
  return launch_dependent(map_slots_kernel, dim3(static_cast<unsigned>(grid)), kMsThreads, 0, stream, L,
                          static_cast<int>(rows));
}

}  // namespace msa
