// Norms, rotation and cache write of a step's new tokens, in one pass.
//
// Per token and head: y = x * rsqrt(mean(x^2) + eps) * w (queries and keys, if
// they have norm weights), then each pair of elements is turned by the token's
// angle pos * inv_freq. Queries go to a dense tensor, keys and values into the
// token's slot of the paged cache. Everything is read and written once:
// 4 * (Hq + 2 Hkv) * dh B per token. A prompt runs at 76 to 79 % of a copy's rate with
// 81 % of the issue slots taken; a step's tree is a launch's latency.
#pragma once

#include "common.cuh"

namespace md {
namespace append {

constexpr int kThreads = 256;
constexpr int kRun = 16;              // tokens of a CTA, at most

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
  int run, block;              // tokens of a CTA; heads it takes at a time
  int T, Hq, Hkv, rot, interleaved, max_pages, pool, page;
  float eps;
};

__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
  x[0] = bf16lo(u.x);
  x[1] = bf16hi(u.x);
  x[2] = bf16lo(u.y);
  x[3] = bf16hi(u.y);
}
__device__ __forceinline__ uint2 pack4(const float* x) { return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); }

// One CTA per (run of up to kRun tokens of a request, share of the heads). DH / 8
// lanes per head take two pieces of 4 elements each, placed so that a rotated
// pair's two elements are one lane's: 4c and rot / 2 + 4c (halves), or 8c and 8c + 4
// (adjacent pairs, and elements that are not turned). A lane's head is the same for
// every token of the run, so its pointers are set once, and the next token's pieces
// load while one is worked on. The angles of the run's tokens are
// formed at the start: the turn pos * inv_freq / 2 pi and its remainder in fp64 (in
// fp32 the angle of a position near 10^5 would be off by 2^-8 and more), cosine
// and sine of the remainder in fp32.
// MANY: all heads of a token fit half of the CTA's lanes or fewer, which then take
// several tokens at once (8 heads of 64: 13.7 against 22.7 us for 16k tokens; the
// general form is slower where it is not needed, 151 against 111 us for a prompt).
template <int DH, bool MANY>
__global__ void __launch_bounds__(kThreads) qk_rope_append_kernel(Args a) {
  constexpr int LPH = DH / 8;
  constexpr int kHeads = kThreads / LPH;              // heads of a block
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ __align__(16) float s_cos[kRun][DH / 2], s_sin[kRun][DH / 2];
  __shared__ long long s_row[kRun];                   // the token's row of the pools (head 0), or -1
  const int runs = (a.T + a.run - 1) / a.run;
  const int b = blockIdx.x / runs, t0 = (blockIdx.x - b * runs) * a.run;
  const int P = a.prefix_len[b];
  const int n_new = a.n_new ? min(a.n_new[b], a.T) : a.T;
  // an idle slot of the batch, or padding behind a request's tokens
  const int ntok = P == -1 ? 0 : min(a.run, n_new - t0);
  if (ntok <= 0) return;
  const int half = a.rot / 2;
  const int c = threadIdx.x % LPH, sub = threadIdx.x / LPH;
  const int heads = a.Hq + 2 * a.Hkv;
  const bool turns = 8 * c < a.rot;
  const bool halves = turns && !a.interleaved;
  const int e0 = halves ? 4 * c : 8 * c, e1 = halves ? half + 4 * c : 8 * c + 4;   // the lane's pieces
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int tk = i / half, f = i - tk * half;
    const double turn = double(a.pos[size_t(b) * a.T + t0 + tk]) * double(a.inv_freq[f]) * 0.15915494309189535;
    const float r = float(turn - rint(turn));
    sincospif(2.f * r, &s_sin[tk][f], &s_cos[tk][f]);
  }
  if (int(threadIdx.x) < ntok) {
    long long row = -1;
    const long long slot = (long long)P + t0 + threadIdx.x;
    if (P >= 0 && slot < (long long)a.max_pages * a.page) {
      const int pi = int(slot / a.page), pg = a.table[size_t(b) * a.max_pages + pi];
      if (pg >= 0 && pg < a.pool) row = (long long)pg * a.Hkv * a.page + (slot - (long long)pi * a.page);
      else set_status(MD_DEV_BAD_PAGE);
    } else {
      set_status(MD_DEV_BAD_PREFIX);
    }
    s_row[threadIdx.x] = row;
  }
  const int at_once = MANY ? kHeads / a.block : 1, tk0 = MANY ? sub / a.block : 0;
  bool ready = false;                                 // the angles and rows are in shared memory
  for (int h0 = int(blockIdx.y) * a.block; h0 < heads; h0 += int(gridDim.y) * a.block) {
    const int h = h0 + sub - tk0 * a.block;
    // 0 query, 1 key, 2 value, 3 none
    const int kind = sub >= at_once * a.block ? 3 : h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : h < heads ? 2 : 3;
    const long long t = t0 + tk0;
    const uint16_t* src = kind == 0   ? a.q + b * a.qb + t * a.qt + h * a.qh
                          : kind == 1 ? a.k + b * a.kb + t * a.kt + (h - a.Hq) * a.kh
                                      : a.v + b * a.vb + t * a.vt + (h - a.Hq - a.Hkv) * a.vh;
    const long long step = at_once * (kind == 0 ? a.qt : kind == 1 ? a.kt : a.vt);
    uint16_t* dst = kind == 0   ? a.q_out + ((size_t(b) * a.T + t0) * a.Hq + h) * DH
                    : kind == 1 ? a.k_pages + size_t(h - a.Hq) * a.page * DH
                                : a.v_pages + size_t(h - a.Hq - a.Hkv) * a.page * DH;
    uint2 u[2] = {make_uint2(0, 0), make_uint2(0, 0)}, next[2];
    if (kind < 3 && tk0 < ntok) {
      u[0] = *reinterpret_cast<const uint2*>(src + e0);
      u[1] = *reinterpret_cast<const uint2*>(src + e1);
    }
    if (!ready) __syncthreads();
    ready = true;
    for (int n = 0; n < ntok; n += at_once) {         // the same count for every lane: the sums are shuffles
      const int tk = n + tk0;
      src += step;
      if (tk + at_once < ntok && kind < 3) {
        next[0] = *reinterpret_cast<const uint2*>(src + e0);
        next[1] = *reinterpret_cast<const uint2*>(src + e1);
      }
      const int at = MANY ? min(tk, kRun - 1) : tk;
      const float4 cs = *reinterpret_cast<const float4*>(&s_cos[at][turns ? 4 * c : 0]);
      const float4 sn = *reinterpret_cast<const float4*>(&s_sin[at][turns ? 4 * c : 0]);
      const long long row = s_row[at];
      const uint16_t* w = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
      float x[8];
      unpack4(u[0], x);
      unpack4(u[1], x + 4);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      if (w) {
        float g[8];
        unpack4(*reinterpret_cast<const uint2*>(w + e0), g);
        unpack4(*reinterpret_cast<const uint2*>(w + e1), g + 4);
        const float inv = rsqrtf(ss * (1.f / DH) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * g[e];
      }
      if (turns) {
        const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
        float y[8];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          if (a.interleaved) {
            y[2 * f] = x[2 * f] * cv[f] - x[2 * f + 1] * sv[f];
            y[2 * f + 1] = x[2 * f + 1] * cv[f] + x[2 * f] * sv[f];
          } else {
            y[f] = x[f] * cv[f] - x[4 + f] * sv[f];
            y[4 + f] = x[4 + f] * cv[f] + x[f] * sv[f];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e];
      }
      uint16_t* to = kind == 0 ? dst + size_t(tk) * a.Hq * DH : dst + row * DH;
      if ((!MANY || tk < ntok) && (kind == 0 || (kind < 3 && row >= 0))) {
        // values go through bit for bit
        *reinterpret_cast<uint2*>(to + e0) = kind == 2 ? u[0] : pack4(x);
        *reinterpret_cast<uint2*>(to + e1) = kind == 2 ? u[1] : pack4(x + 4);
      }
      u[0] = next[0];
      u[1] = next[1];
    }
  }
}

}  // namespace append
}  // namespace md
