// Tree-masked attention over a paged KV cache.
//
//   out[b,t,h,:] = sum_j softmax_j(scale q[b,t,h,:] . K_j) V_j
//
// over the prefix slots j < P_b and the tree slots P_b + a of the ancestors a of
// node t (itself included), slot s of request b being row s % page of page
// block_table[b, s / page].
#pragma once

#include "common.cuh"

namespace md {
namespace attn_paged {

struct Args {
  const uint16_t* q;           // [B, T, Hq, dh]
  const uint16_t *kp, *vp;     // [pool, Hkv, page, dh]
  const int32_t* table;        // [B, max_pages]
  const int32_t* prefix_len;   // [B]
  void* out;                   // [B, T, Hq, dh] fp32 or bf16
  int B, Hq, Hkv, pool, page, max_pages;
  float scale_log2;
  int out_bf16;
};

constexpr int kThreads = 128;

// One warp per (request, node, query head): one pass over its keys with a
// running maximum and sum. Every row reads its keys again (5 ms for a 70B-shaped
// tree of 65 nodes over 4096 slots): a first form to check against.
template <int DH>
__global__ void __launch_bounds__(kThreads) attn_paged_rows_kernel(const __grid_constant__ TreeParams tp, Args a) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int E = DH / 32;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int b = blockIdx.y;
  if (row >= tp.T * a.Hq) return;
  const int t = row / a.Hq, h = row - t * a.Hq, hk = h / (a.Hq / a.Hkv);
  const int P = a.prefix_len[b];
  const bool bad = P < 0 || (long long)P + tp.T > (long long)a.max_pages * a.page;
  if (bad && P != -1 && row == 0 && lane == 0) set_status(MD_DEV_BAD_PREFIX);
  const size_t orow = (size_t(b) * tp.T * a.Hq + row) * DH;
  float qv[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = bf16_to_f32(a.q[orow + e * 32 + lane]);
    acc[e] = 0.f;
  }
  const int n = bad ? 0 : P + tp.T;
  for (int s = 0; s < n; ++s) {
    const int node = s - P;
    if (node >= 0 && !((tp.anc[t][node >> 5] >> (node & 31)) & 1u)) continue;
    const int pg = a.table[size_t(b) * a.max_pages + s / a.page];
    float kv[E], vv[E], x = 0.f;
    if (pg >= 0 && pg < a.pool) {
      const size_t at = ((size_t(pg) * a.Hkv + hk) * a.page + s % a.page) * DH;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        kv[e] = bf16_to_f32(a.kp[at + e * 32 + lane]);
        vv[e] = bf16_to_f32(a.vp[at + e * 32 + lane]);
      }
    } else {
      if (lane == 0) set_status(MD_DEV_BAD_PAGE);
#pragma unroll
      for (int e = 0; e < E; ++e) kv[e] = vv[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(qv[e], kv[e], x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale_log2;
    const float m2 = fmaxf(m, x);
    const float f = m == -INFINITY ? 0.f : exp2f(m - m2), p = exp2f(x - m2);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + p * vv[e];
    m = m2;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float o = n > 0 ? acc[e] / l : 0.f;
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[orow + e * 32 + lane] = uint16_t(pack_bf16x2(o, 0.f));
    else static_cast<float*>(a.out)[orow + e * 32 + lane] = o;
  }
}

}  // namespace attn_paged
}  // namespace md
