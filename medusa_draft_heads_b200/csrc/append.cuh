// Norms, rotation and cache write of a step's new tokens, in one pass.
//
// Per token and head: y = x * rsqrt(mean(x^2) + eps) * w (queries and keys, if
// they have norm weights), then each pair of elements is turned by the token's
// angle pos * inv_freq. Queries go to a dense tensor, keys and values into the
// token's slot of the paged cache. Everything is read and written once:
// 4 * (Hq + 2 Hkv) * dh B per token, DRAM-bound for prompts and a launch's
// latency for a step's tree.
#pragma once

#include "common.cuh"

namespace md {
namespace append {

constexpr int kThreads = 256;

struct Args {
  const uint16_t *q, *k, *v;                          // element strides below; a head's dh elements are contiguous
  long long qb, qt, qh, kb, kt, kh, vb, vt, vh;       // strides of request, token, head
  const int32_t* pos;          // [B, T]
  const float* inv_freq;       // [rot / 2]
  const uint16_t *q_norm, *k_norm;                    // [dh] or NULL
  uint16_t* q_out;             // [B, T, Hq, dh]
  uint16_t *k_pages, *v_pages; // [pool, Hkv, page, dh]
  const int32_t* table;        // [B, max_pages]
  const int32_t* prefix_len;   // [B]
  const int32_t* n_new;        // [B] or NULL
  int T, Hq, Hkv, rot, interleaved, max_pages, pool, page;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// One CTA per (token, share of its heads): DH / 8 lanes per head, 8 elements a
// lane, so a norm's sum and a pair's partner are shuffles within the head's
// lanes. The token's rot / 2 angles are formed once per CTA: the turn
// pos * inv_freq / 2 pi and its remainder in fp64 (in fp32 the angle of a
// position near 10^5 would be off by 2^-8 and more), cosine and sine of the
// remainder in fp32.
template <int DH>
__global__ void __launch_bounds__(kThreads) qk_rope_append_kernel(Args a) {
  constexpr int LPH = DH / 8;
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float s_cos[DH / 2], s_sin[DH / 2];
  const int b = blockIdx.x / a.T, t = blockIdx.x - b * a.T;
  const int P = a.prefix_len[b];
  if (P == -1) return;                                // an idle slot of the batch
  if (a.n_new && t >= a.n_new[b]) return;             // padding behind a request's tokens
  const int half = a.rot / 2;
  if (int(threadIdx.x) < half) {
    const double turn = double(a.pos[blockIdx.x]) * double(a.inv_freq[threadIdx.x]) * 0.15915494309189535;
    const float r = float(turn - rint(turn));
    sincospif(2.f * r, &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
  }
  // the token's slot in the cache (-1: nowhere to write)
  long long slot_row = -1;
  if (P >= 0 && (long long)P + t < (long long)a.max_pages * a.page) {
    const int pg = a.table[size_t(b) * a.max_pages + (P + t) / a.page];
    if (pg >= 0 && pg < a.pool) slot_row = (long long)pg * a.Hkv * a.page + (P + t) % a.page;
    else if (threadIdx.x == 0) set_status(MD_DEV_BAD_PAGE);
  } else if (threadIdx.x == 0) {
    set_status(MD_DEV_BAD_PREFIX);
  }
  __syncthreads();
  const int c = threadIdx.x % LPH;                    // this lane's eighth .. of the head: elements 8c .. 8c + 7
  const int heads = a.Hq + 2 * a.Hkv;
  const int hpc = kThreads / LPH;                     // heads a pass of the CTA covers
  for (int h0 = blockIdx.y * hpc; h0 < heads; h0 += gridDim.y * hpc) {
    const int h = h0 + threadIdx.x / LPH;
    const bool on = h < heads;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (on) {
      const uint16_t* src = is_q   ? a.q + b * a.qb + t * a.qt + h * a.qh
                            : is_k ? a.k + b * a.kb + t * a.kt + (h - a.Hq) * a.kh
                                   : a.v + b * a.vb + t * a.vt + (h - a.Hq - a.Hkv) * a.vh;
      u = reinterpret_cast<const uint4*>(src)[c];
    }
    float x[8];
    unpack8(u, x);
    const uint16_t* w = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (w) {
      float wf[8];
      unpack8(reinterpret_cast<const uint4*>(w)[c], wf);
      const float inv = rsqrtf(ss * (1.f / DH) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wf[i];
    }
    if (a.interleaved) {                              // pairs (2i, 2i + 1)
      if (8 * c < a.rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float cs = s_cos[4 * c + i], sn = s_sin[4 * c + i];
          const float x0 = x[2 * i], x1 = x[2 * i + 1];
          x[2 * i] = x0 * cs - x1 * sn;
          x[2 * i + 1] = x1 * cs + x0 * sn;
        }
      }
    } else {                                          // pairs (i, i + rot / 2)
      const int hl = half / 8;                        // lanes of half the rotated elements
      const bool first = c < hl, turns = 8 * c < a.rot;
      const int lane = threadIdx.x & 31;
      const int partner = !turns ? lane : first ? lane + hl : lane - hl;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, x[i], partner);
        if (turns) {
          const int f = 8 * (first ? c : c - hl) + i;
          x[i] = first ? x[i] * s_cos[f] - o * s_sin[f] : x[i] * s_cos[f] + o * s_sin[f];
        }
      }
    }
    if (!on) continue;
    if (is_q) {
      reinterpret_cast<uint4*>(a.q_out + (size_t(blockIdx.x) * a.Hq + h) * DH)[c] = pack8(x);
    } else if (slot_row >= 0) {
      uint16_t* pool = is_k ? a.k_pages : a.v_pages;
      const int hk = is_k ? h - a.Hq : h - a.Hq - a.Hkv;
      // values go through bit for bit
      reinterpret_cast<uint4*>(pool + (size_t(slot_row) + size_t(hk) * a.page) * DH)[c] = is_k ? pack8(x) : u;
    }
  }
}

}  // namespace append
}  // namespace md
