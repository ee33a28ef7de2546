// The pages of a paged KV cache: which request holds which page, and the
// copying of a page when a sequence forks.
//
// Book-keeping lives on the device, in three int32 arrays that a step's calls
// read and write in stream order, so a decode loop never waits for the host:
// block_table [B, max_pages] (page ids, -1 past a row's pages), n_pages [B] and
// refcount [pool]. A page is free iff its count is 0, and requests get the
// lowest free ids in row order: every result follows from the arrays alone,
// whatever order the atomics ran in (they only add and subtract integers).
#pragma once

#include "common.cuh"

namespace md {
namespace pages {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 16;                   // counts per thread and scan tile: four loads in flight
constexpr int kTile = kThreads * kPerThread;
constexpr int kMaxRows = 16384;                  // rows of a resize: their running needs sit in shared memory
constexpr int kMaxForks = kThreads;              // forks of a call: one thread each

__device__ __forceinline__ int warp_incl_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Inclusive sum over the block's threads; `total` receives the block's sum.
// `part` is kWarps ints of shared memory; all threads call it.
__device__ __forceinline__ int block_incl_scan(int v, int* part, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_incl_scan(v);
  __syncthreads();                               // the previous scan's sums have been read
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) part[lane] = warp_incl_scan(part[lane]);
  __syncthreads();
  total = part[kWarps - 1];
  return v + (warp > 0 ? part[warp - 1] : 0);
}

// Drops one reference each to the pages of entries[0 .. n), `lanes` lanes of a warp
// sharing the work, four atomics of a lane in flight (their results are checked). A
// page that is not in the pool, or that nobody holds, is flagged and its count
// stays. The entries become -1 if `clear`.
__device__ __forceinline__ void drop_pages(int32_t* refcount, int pool, int32_t* entries, int n, int lane, int lanes,
                                           bool clear) {
  for (int i0 = lane; i0 < n; i0 += 4 * lanes) {
    int page[4], held[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = i0 + k * lanes < n ? entries[i0 + k * lanes] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) held[k] = page[k] >= 0 && page[k] < pool ? atomicSub(&refcount[page[k]], 1) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i0 + k * lanes >= n) continue;
      if (held[k] <= 0) {
        if (page[k] >= 0 && page[k] < pool) atomicAdd(&refcount[page[k]], 1);
        set_status(MD_DEV_BAD_PAGE);
      }
      if (clear) entries[i0 + k * lanes] = -1;
    }
  }
}

// Bit i of the result: page base + kPerThread * threadIdx.x + i is free. Counts
// are read past L1: the block's own atomics may just have changed them.
__device__ __forceinline__ uint32_t free_bits(const int32_t* refcount, int pool, int base) {
  const int p0 = base + int(threadIdx.x) * kPerThread;
  uint32_t m = 0;
  if (p0 + kPerThread <= pool) {
    int4 c[kPerThread / 4];
#pragma unroll
    for (int i = 0; i < kPerThread / 4; ++i) c[i] = __ldcg(reinterpret_cast<const int4*>(refcount + p0) + i);
#pragma unroll
    for (int i = 0; i < kPerThread / 4; ++i)
      m |= ((c[i].x == 0 ? 1u : 0u) | (c[i].y == 0 ? 2u : 0u) | (c[i].z == 0 ? 4u : 0u) | (c[i].w == 0 ? 8u : 0u)) << (4 * i);
  } else {
    for (int i = 0; i < kPerThread; ++i)
      if (p0 + i < pool && __ldcg(refcount + p0 + i) == 0) m |= 1u << i;
  }
  return m;
}

// Calls take(rank, page) for the `want` lowest free pages (rank 0 .. want - 1), or
// for all of them if there are fewer; returns how many it found. The pool is
// read once, up to the last page taken.
template <typename Take>
__device__ __forceinline__ int take_lowest_free(const int32_t* refcount, int pool, int want, int* part, Take take) {
  int seen = 0;
  for (int base = 0; base < pool && seen < want; base += kTile) {   // uniform over the block
    uint32_t m = free_bits(refcount, pool, base);
    const int n = __popc(m);
    int total;
    int rank = seen + block_incl_scan(n, part, total) - n;
    for (; m != 0 && rank < want; m &= m - 1, ++rank) take(rank, base + int(threadIdx.x) * kPerThread + __ffs(m) - 1);
    seen += total;
  }
  return min(seen, want);
}

// ------------------------------------------------------------------ resize

struct ResizeArgs {
  int32_t* table;           // [B, max_pages]
  int32_t* n_pages;         // [B]
  int32_t* refcount;        // [pool]
  const int32_t* length;    // [B]
  int B, max_pages, pool, page, extra;
};

// Pages row b should hold, or -1 if the row is to be left alone (its count or
// its length cannot be right).
__device__ __forceinline__ int wanted_pages(const ResizeArgs& a, int b, int held) {
  if (held < 0 || held > a.max_pages) return -1;
  const int len = a.length[b];
  if (len < 0) return 0;
  const long long want = ((long long)len + a.extra + a.page - 1) / a.page;
  return want > a.max_pages ? -1 : int(want);
}

// One CTA. Rows that hold too much give their last pages back, then the lowest
// free pages go to the rows that need more, in row order. A few KB of traffic
// plus 4 B per page of the pool (read when some row needs a page): latency-bound.
__global__ void __launch_bounds__(kThreads) pages_resize_kernel(ResizeArgs a) {
  pdl_wait_primary();          // lengths come from the previous kernels
  pdl_launch_dependents();
  extern __shared__ int32_t upto[];              // [B]: pages needed by rows 0 .. b
  __shared__ int part[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // give back: a lane looks at a row, then the warp works through those that hold too
  // much, long ones together, short ones four at a time
  for (int k0 = 0; k0 * kWarps < a.B; k0 += 32) {
    const int b = (k0 + lane) * kWarps + warp;
    int held = 0, want = 0;
    if (b < a.B) {
      held = a.n_pages[b];
      want = wanted_pages(a, b, held);
      if (want < 0) {
        set_status(held < 0 || held > a.max_pages ? MD_DEV_BAD_PAGE : MD_DEV_BAD_PREFIX);
        held = want;                             // left alone
      }
    }
    uint32_t shrinks = __ballot_sync(0xffffffffu, held > want);
    const uint32_t longs = __ballot_sync(0xffffffffu, held - want > 32);
    for (uint32_t m = longs; m != 0; m &= m - 1) {
      const int i = __ffs(m) - 1;
      const int rw = __shfl_sync(0xffffffffu, want, i), rh = __shfl_sync(0xffffffffu, held, i);
      const int rb = __shfl_sync(0xffffffffu, b, i);
      drop_pages(a.refcount, a.pool, a.table + size_t(rb) * a.max_pages + rw, rh - rw, lane, 32, true);
    }
    for (uint32_t m = shrinks & ~longs; m != 0;) {
      uint32_t mine = 0;                         // this quarter of the warp's row, as a bit
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t low = m & (0u - m);
        if (k == lane >> 3) mine = low;
        m ^= low;
      }
      const int i = mine ? __ffs(mine) - 1 : 0;
      const int rw = __shfl_sync(0xffffffffu, want, i), rh = __shfl_sync(0xffffffffu, held, i);
      const int rb = __shfl_sync(0xffffffffu, b, i);
      if (mine) drop_pages(a.refcount, a.pool, a.table + size_t(rb) * a.max_pages + rw, rh - rw, lane & 7, 8, true);
    }
    if (held > want) a.n_pages[b] = want;
  }
  __syncthreads();

  int all = 0;                                   // running needs of the rows
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0;
    if (b < a.B) {
      const int held = a.n_pages[b], want = wanted_pages(a, b, held);
      need = want < 0 ? 0 : max(0, want - held);   // a row left alone: its count may be anything
    }
    int total;
    const int incl = block_incl_scan(need, part, total);
    if (b < a.B) upto[b] = all + incl;
    all += total;
  }
  if (all == 0) return;
  auto row_of = [&](int rank) -> int {           // the first row whose running need exceeds the rank
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] > rank) hi = mid; else lo = mid + 1;
    }
    return lo;
  };
  auto before = [&](int b) { return b > 0 ? upto[b - 1] : 0; };
  const int found = take_lowest_free(a.refcount, a.pool, all, part, [&](int rank, int page) {
    const int b = row_of(rank);
    a.table[size_t(b) * a.max_pages + a.n_pages[b] + (rank - before(b))] = page;
    a.refcount[page] = 1;
  });
  __syncthreads();
  // rows are served as long as their needs and those of the rows before them fit:
  // the first that does not gives back what it got
  int served = found;
  if (found < all) {
    const int b = row_of(found);
    served = before(b);
    int32_t* row = a.table + size_t(b) * a.max_pages + a.n_pages[b];
    for (int i = threadIdx.x; i < found - served; i += kThreads) {
      a.refcount[row[i]] = 0;
      row[i] = -1;
    }
    if (threadIdx.x == 0) set_status(MD_DEV_NO_PAGES);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const int need = upto[b] - before(b);
    if (need > 0 && upto[b] <= served) a.n_pages[b] += need;
  }
}

// -------------------------------------------------------------------- fork

struct ForkJob {
  int32_t from, to, rows, pad;   // rows == 0: nothing to copy
};

struct ForkArgs {
  int32_t* table;           // [B, max_pages]
  int32_t* n_pages;         // [B]
  int32_t* refcount;        // [pool]
  int32_t* length;          // [B]
  const int32_t* src;       // [n]
  const int32_t* dst;       // [n]
  ForkJob* jobs;            // [n]
  int B, n, max_pages, pool, page;
};

// One CTA, one thread per fork for the decisions, one warp per fork for the
// rows of the table. Sources are never destinations of the same call, so no
// row is read and written.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(ForkArgs a) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ int s_src[kMaxForks], s_dst[kMaxForks], s_fresh[kMaxForks], s_owner[kMaxForks];
  __shared__ int part[kWarps];
  const int i = threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int src = -1, dst = -1, len = -1, last_page = -1;
  if (i < a.n) {
    src = a.src[i];
    dst = a.dst[i];
  }
  s_src[i] = src;
  s_dst[i] = dst;
  __syncthreads();
  bool valid = i < a.n && src != -1;             // src -1: an unused entry
  if (valid) {
    int bad = 0;
    if (src < 0 || src >= a.B || dst < 0 || dst >= a.B) {
      bad = MD_DEV_BAD_ROW;
    } else {
      for (int j = 0; j < a.n; ++j)
        if (s_src[j] == dst || (j < i && s_src[j] != -1 && s_dst[j] == dst)) bad = MD_DEV_BAD_ROW;
      if (!bad) {
        len = a.length[src];
        const int hs = a.n_pages[src], hd = a.n_pages[dst];
        if (hs < 0 || hs > a.max_pages || hd < 0 || hd > a.max_pages) bad = MD_DEV_BAD_PAGE;
        else if (len > (long long)hs * a.page) bad = MD_DEV_BAD_PREFIX;
        if (!bad && len > 0 && len % a.page > 0) {   // the page to be copied
          last_page = a.table[size_t(src) * a.max_pages + len / a.page];
          if (last_page < 0 || last_page >= a.pool) bad = MD_DEV_BAD_PAGE;
        }
      }
    }
    if (bad) {
      set_status(bad);
      valid = false;
    }
  }
  const int full = valid && len > 0 ? len / a.page : 0;
  const int rows = valid && len > 0 ? len % a.page : 0;
  __syncthreads();
  s_src[i] = valid ? src : -1;
  s_fresh[i] = -1;
  __syncthreads();
  // the destinations' former pages go back first
  for (int f = warp; f < a.n; f += kWarps) {
    if (s_src[f] < 0) continue;
    const int d = s_dst[f], held = a.n_pages[d];
    drop_pages(a.refcount, a.pool, a.table + size_t(d) * a.max_pages, held, lane, 32, false);
  }
  __syncthreads();
  // a new page for every fork that ends inside one, lowest ids in list order
  const int need = rows > 0 ? 1 : 0;
  int total;
  const int incl = block_incl_scan(need, part, total);
  if (total > 0) {
    if (need) s_owner[incl - 1] = i;
    __syncthreads();
    const int found = take_lowest_free(a.refcount, a.pool, total, part, [&](int rank, int page) {
      s_fresh[s_owner[rank]] = page;
      a.refcount[page] = 1;
    });
    if (found < total && threadIdx.x == 0) set_status(MD_DEV_NO_PAGES);
  }
  __syncthreads();
  const bool empty = !valid || len < 0 || (need && s_fresh[i] < 0);   // an idle source, or no page left
  __shared__ int s_full[kMaxForks];
  s_full[i] = empty ? -1 : full;
  if (i < a.n) {
    a.jobs[i] = !empty && rows > 0 ? ForkJob{last_page, s_fresh[i], rows, 0} : ForkJob{0, 0, 0, 0};
  }
  __syncthreads();
  for (int f = warp; f < a.n; f += kWarps) {
    if (s_src[f] < 0) continue;
    const int32_t* from = a.table + size_t(s_src[f]) * a.max_pages;
    int32_t* to = a.table + size_t(s_dst[f]) * a.max_pages;
    const int nf = s_full[f], held = a.n_pages[s_dst[f]];
    const int last = max(max(nf, 0) + 1, held);  // entries past the former pages are -1 already
    for (int p = lane; p < min(last, a.max_pages); p += 32) {
      int page = -1;
      if (p < nf) {
        page = from[p];
        if (page < 0 || page >= a.pool) set_status(MD_DEV_BAD_PAGE);
        else atomicAdd(&a.refcount[page], 1);
      } else if (p == nf) {
        page = s_fresh[f];
      }
      to[p] = page;
    }
  }
  __syncthreads();
  if (valid) {
    a.n_pages[dst] = empty ? 0 : full + need;
    a.length[dst] = empty ? -1 : len;
  }
}

// Copies the first `rows` slots of a fork's last page, every layer and head of
// K and V. A head's slots of a page are contiguous: `rows` * dh elements, four
// 16-byte loads of a thread in flight (a page of 64 slots of 128 in one round).
// One CTA per (kCopyHeads layers' heads, K or V, fork); bytes-bound, 4 * rows * dh B
// a head read and written.
constexpr int kCopyThreads = 256, kCopyLoads = 4, kCopyHeads = 4;

__global__ void __launch_bounds__(kCopyThreads) pages_fork_copy_kernel(uint4* k_pages, uint4* v_pages, const ForkJob* jobs,
                                                                       int layers, int pool, int Hkv, int page, int row16) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const ForkJob job = jobs[blockIdx.z];
  if (job.rows == 0) return;
  uint4* base = blockIdx.y ? v_pages : k_pages;
  const int n = job.rows * row16, heads = layers * Hkv;
  for (int lh = blockIdx.x * kCopyHeads; lh < min(heads, int(blockIdx.x + 1) * kCopyHeads); ++lh) {
    const int layer = lh / Hkv, hk = lh - layer * Hkv;
    const uint4* from = base + ((size_t(layer) * pool + job.from) * Hkv + hk) * page * row16;
    uint4* to = base + ((size_t(layer) * pool + job.to) * Hkv + hk) * page * row16;
    for (int i0 = threadIdx.x; i0 < n; i0 += kCopyLoads * kCopyThreads) {
      uint4 x[kCopyLoads];
#pragma unroll
      for (int k = 0; k < kCopyLoads; ++k)
        if (i0 + k * kCopyThreads < n) x[k] = from[i0 + k * kCopyThreads];
#pragma unroll
      for (int k = 0; k < kCopyLoads; ++k)
        if (i0 + k * kCopyThreads < n) to[i0 + k * kCopyThreads] = x[k];
    }
  }
}

}  // namespace pages
}  // namespace md
