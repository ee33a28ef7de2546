// Advancing along the accepted branch in a paged cache, every layer at once.
//
// As commit.cuh: slot P + i receives slot P + path[i], i = 1 .. L (the root's
// K/V are in place). A thread owns one 16-byte column of one (layer, head, K or
// V) and carries all its rows in registers, read before any is written (a
// destination slot can be another row's source), so nothing is staged and no
// thread waits for another. Traffic 4 * dh B per moved row, head and layer
// (K and V, read and written); a few MB at most: latency-bound.
#pragma once

#include "common.cuh"

namespace md {
namespace commit_paged {

constexpr int kThreads = 128;

struct Args {
  uint4 *kp, *vp;              // [layers, pool, Hkv, page, dh]
  const int32_t* table;        // [B, max_pages]
  const int32_t* prefix_len;   // [B]
  const int32_t* accept_len;   // [B]
  const int32_t* path;         // [B, K + 1]
  const int32_t* bonus;        // [B]
  int32_t* new_prefix_len;     // [B]
  int32_t* next_root;          // [B]
  int32_t* next_head_row;      // [B]
  int layers, pool, page, max_pages, Hkv, row16, K;
};

__global__ void __launch_bounds__(kThreads) tree_commit_paged_kernel(const __grid_constant__ TreeParams tp, Args a) {
  pdl_wait_primary();          // path and lengths come from the acceptance kernels
  pdl_launch_dependents();
  const int b = blockIdx.y;
  __shared__ long long from[MD_MAX_K + 1], to[MD_MAX_K + 1];   // rows of the pool of layer 0, head 0
  __shared__ int moves_s, bad_s, node[MD_MAX_K + 1];
  const int P = a.prefix_len[b], L = a.accept_len[b];
  const bool lead = blockIdx.x == 0 && threadIdx.x == 0;
  if (P == -1) {               // an idle slot of the batch
    if (lead) {
      a.new_prefix_len[b] = -1;
      a.next_root[b] = -1;
      a.next_head_row[b] = -1;
    }
    return;
  }
  if (threadIdx.x < 32) {
    // lane i checks and resolves node i of the path
    const int i = threadIdx.x;
    int bad = 0;
    if (P < 0 || (long long)P + tp.T > (long long)a.max_pages * a.page || L < 0 || L > tp.max_depth || L > a.K) {
      bad = MD_DEV_BAD_PATH;
    } else if (i <= L) {
      const int n = a.path[size_t(b) * (a.K + 1) + i];
      const int up = i > 0 ? a.path[size_t(b) * (a.K + 1) + i - 1] : -1;
      if (n < 0 || n >= tp.T || tp.depth[n] != i || (i > 0 && tp.parent[n] != up)) {
        bad = MD_DEV_BAD_PATH;
      } else {
        const int32_t* row = a.table + size_t(b) * a.max_pages;
        const int sp = row[(P + n) / a.page], dp = row[(P + i) / a.page];
        // also for a row in place: without a page its K/V were never written
        if (sp < 0 || sp >= a.pool || dp < 0 || dp >= a.pool) bad = MD_DEV_BAD_PAGE;
        from[i] = (long long)sp * a.Hkv * a.page + (P + n) % a.page;
        to[i] = (long long)dp * a.Hkv * a.page + (P + i) % a.page;
        node[i] = n;
      }
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    // the rows that move, compacted to the front
    const bool moves = !bad && i <= L && node[i] != i;
    const uint32_t m = __ballot_sync(0xffffffffu, moves);
    const long long f = i <= MD_MAX_K ? from[i] : 0, d = i <= MD_MAX_K ? to[i] : 0;
    __syncwarp();
    if (moves) {
      const int at = __popc(m & ((1u << i) - 1u));
      from[at] = f;
      to[at] = d;
    }
    if (i == 0) {
      moves_s = __popc(m);
      bad_s = bad;
    }
  }
  __syncthreads();
  if (lead) {
    if (bad_s) set_status(bad_s);
    a.new_prefix_len[b] = bad_s ? P : P + L + 1;
    a.next_root[b] = a.bonus[b];
    a.next_head_row[b] = bad_s ? -1 : b * tp.T + node[L];
  }
  const int moves = moves_s;
  if (moves == 0) return;
  const size_t cols = size_t(2) * a.layers * a.Hkv * a.row16;
  for (size_t col = size_t(blockIdx.x) * kThreads + threadIdx.x; col < cols; col += size_t(gridDim.x) * kThreads) {
    const int c = int(col % a.row16);
    size_t r = col / a.row16;
    const int hk = int(r % a.Hkv);
    r /= a.Hkv;
    const size_t layer = r >> 1;
    uint4* base = ((r & 1) ? a.vp : a.kp) + ((layer * a.pool * a.Hkv + hk) * a.page) * a.row16 + c;
    uint4 x[MD_MAX_K];
#pragma unroll
    for (int i = 0; i < MD_MAX_K; ++i)
      if (i < moves) x[i] = base[from[i] * a.row16];
#pragma unroll
    for (int i = 0; i < MD_MAX_K; ++i)
      if (i < moves) base[to[i] * a.row16] = x[i];
  }
}

}  // namespace commit_paged
}  // namespace md
