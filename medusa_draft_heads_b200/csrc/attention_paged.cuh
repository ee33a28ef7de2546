// Tree-masked attention over a paged KV cache, on the tensor cores (tcgen05).
//
//   out[b,t,h,:] = sum_j softmax_j(scale q[b,t,h,:] . K_j) V_j
//
// over the prefix slots j < P_b and the tree slots P_b + a of the ancestors a of
// node t (itself included), slot s of request b being row s % page of page
// block_table[b, s / page]. The T * G query rows (node, head of the group) of a
// KV head share its keys, so scores and weighted sums are dense products.
//
// CTA = (KV split, unit of up to two 128-row tiles, KV head, request). It walks
// its chunks of 128 keys with two softmax warpgroups, each with a stream of its
// own: S (128 columns of TMEM, overwritten in place by the weights P) and O
// (DH columns).
//   - two tiles: stream w is row tile w, and both walk every chunk, so a chunk
//     fetched once serves 256 rows;
//   - one tile (a request with few rows: decoding, chains, the odd last tile):
//     the streams take the chunks in turn and are joined at the end.
// While one stream's warps run its softmax the tensor cores work for the other.
//
//   warp 0      K: one TMA copy per page piece and 64-column block, each lane a
//               piece (its page id from the block table), three slots
//   warp 1      one thread issues, per (stream, chunk): O += P V, then the
//               stream's next S = Q K^T. A stream's S landing implies that its
//               previous P V landed too (they complete in issue order), so the
//               softmax may rescale O in place.
//   warp 2      V, as K; two slots, a third where the second Q tile would be
//   warp 3      the Q tiles
//   warps 4-11  softmax: thread = row. Running maximum m (moved only when a
//               chunk exceeds it by 2^8, O and the sum then rescaled), weights
//               P = exp2(S - m), their sum in fp32.
//
// P is rounded to bf16 for the product with V (the relative error of a weight,
// 2^-9, averages out over the keys, and the bf16 output is rounded to the same
// precision). For fp32 outputs P is split into hi + lo bf16 parts (to 2^-14) and
// P V runs twice.
//
// The KV splits of a unit are the CTAs of a cluster: O and (m, sum) of every
// stream are staged in shared memory, and each CTA combines its share of the
// rows from all of them (distributed shared memory). Splits are made of the
// request's own length on the device, so a table wider than the sequences
// costs nothing.
//
// Slots behind the tree's last hold anything, NaN included: their scores are
// replaced, and their V rows zeroed in shared memory (0 * NaN would reach O). A
// tree node's V that is not finite must reach only the rows that see the node:
// such elements are zeroed in shared memory too and added to those rows'
// results at the end.
#pragma once

#include "common.cuh"

namespace md {
namespace attn_paged {

constexpr int kBM = 128;              // rows of a tile
constexpr int kBN = 128;              // keys of a chunk
constexpr int kThreads = 384;
constexpr int kSoftThreads = 256;
constexpr int kKStages = 3;
constexpr int kVStages = 3;           // the third only with one row tile
constexpr int kMaxSplits = 16;        // CTAs of a cluster (above 8 by opt-in)
constexpr float kRescaleLog2 = 8.0f;
constexpr uint32_t kTmemCols = 512;   // S0, S1, O0, O1: 128 columns each

template <int DH>
struct Cfg {
  static constexpr int KB = DH / 64;                       // 64-column blocks
  static constexpr uint32_t kTile = KB * 128 * 128;        // 128 rows x DH bf16, 128-byte swizzle
  static constexpr int kLd = DH + 4;                       // padded fp32 row of the staged O
  // Q0, Q1 (or a V slot), 3 K slots, 2 V slots
  static constexpr uint32_t kRing = 7 * kTile;
  static constexpr int kSmem = int(kRing) + 512 + 1024;    // + barriers, alignment
  static_assert(2 * kBM * (kLd * 4 + 8) <= int(kRing), "staged O, (m, sum)");
};

struct Args {
  const uint16_t* v_pages;     // [pool, Hkv, page, dh] (the slow path of a V that is not finite)
  const int32_t* table;        // [B, max_pages]
  const int32_t* prefix_len;   // [B]
  void* out;                   // [B, T, Hq, dh]
  int B, Hq, Hkv, G, pool, page, max_pages;
  int piece;                   // rows of a TMA copy: the largest power of two dividing page, at most 128
  int tpt;                     // tree nodes of a row tile
  int units, splits, sort;
  float scale_log2;
};

__device__ __forceinline__ float exp2_sfu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 columns of this thread's TMEM lane, requested only: tmem_ld_wait() and then
// settle() come before their first use.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps uses of v[0..31] behind the wait above it.
__device__ __forceinline__ void settle(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}

// Visibility of the 64 keys n0 .. n0 + 63 (n = slot - P) as bit j: prefix keys
// (n < 0) always, tree node n iff it is in the row's ancestor set.
__device__ __forceinline__ uint64_t visible_bits(uint64_t lo, uint64_t hi, int n0) {
  if (n0 <= -64) return ~0ull;
  if (n0 >= 128) return 0ull;
  if (n0 < 0) return (lo << (-n0)) | ((1ull << (-n0)) - 1ull);
  if (n0 == 0) return lo;
  if (n0 < 64) return (lo >> n0) | (hi << (64 - n0));
  if (n0 == 64) return hi;
  return hi >> (n0 - 64);
}

__device__ __forceinline__ bool bf16_finite(uint32_t v) { return (v & 0x7F80u) != 0x7F80u; }

// The copies of one chunk of K or V into a ring slot, each lane a page piece.
// Pieces behind the last slot are not copied. All lanes of a warp call it.
template <int DH>
__device__ __forceinline__ void load_chunk(uint32_t dst, const CUtensorMap* map, uint32_t bar, const int32_t* row, int key0,
                                           int nkeys, int hk, const Args& a) {
  using C = Cfg<DH>;
  const int lane = threadIdx.x & 31;
  const int left = min(kBN, nkeys - key0);
  const int pieces = (left + a.piece - 1) / a.piece;
  if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(pieces * a.piece) * DH * 2);
  __syncwarp();
  if (lane < pieces) {
    const int key = key0 + lane * a.piece;
    const int pi = key / a.page;
    int pg = row[pi];
    if (pg < 0 || pg >= a.pool) {
      set_status(MD_DEV_BAD_PAGE);
      pg = a.pool;                       // past the pool: the copy fills zeros
    }
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
      tma_load_3d(dst + kb * (kBN * 128) + lane * a.piece * 128, map, kb * 64, key - pi * a.page, pg * a.Hkv + hk, bar);
  }
}

template <int DH, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeParams tp, Args a) {
  using C = Cfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem;                                    // 2 tiles (the second may be V slot 2)
  uint8_t* sK = smem + 2 * C::kTile;                     // 3 slots
  uint8_t* sV = sK + kKStages * C::kTile;                // 2 slots
  float2* sML = reinterpret_cast<float2*>(smem + 2 * kBM * C::kLd * 4);   // [2][128], behind the staged O
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* q_full = bars;                // 1
  uint64_t* k_full = q_full + 1;          // 3
  uint64_t* k_empty = k_full + kKStages;  // 3
  uint64_t* v_full = k_empty + kKStages;  // 3
  uint64_t* v_empty = v_full + kVStages;  // 3
  uint64_t* s_full = v_empty + kVStages;  // 2
  uint64_t* p_full = s_full + 2;          // 2
  uint64_t* mma_done = p_full + 2;        // 1
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  int* req = reinterpret_cast<int*>(tmem_slot + 1);
  int* bad_v = req + 1;

  const int split = blockIdx.x, unit = blockIdx.y % a.units, hk = blockIdx.y / a.units;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = tp.T;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(q_full), 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_u32(&k_full[i]), 1);
      mbar_init(smem_u32(&k_empty[i]), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(smem_u32(&v_full[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 4);
    }
    mbar_init(smem_u32(mma_done), 1);
    fence_barrier_init();
    *req = blockIdx.z;
    *bad_v = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  pdl_wait_primary();          // inputs may come from earlier kernels
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // More CTAs than one wave: requests from the longest prefix down, so that
  // short ones fill the tail.
  if (a.sort) {
    for (int c = threadIdx.x; c < a.B; c += kThreads) {
      const int pc = a.prefix_len[c];
      int rank = 0;
      for (int j = 0; j < a.B; ++j) {
        const int pj = a.prefix_len[j];
        rank += (pj > pc || (pj == pc && j < c)) ? 1 : 0;
      }
      if (rank == int(blockIdx.z)) *req = c;
    }
    __syncthreads();
  }
  const int b = *req;
  const uint32_t tmem = *tmem_slot;
  const int P = a.prefix_len[b];
  const bool bad = P < 0 || (long long)P + T > (long long)a.max_pages * a.page;
  if (bad && P != -1 && split == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(MD_DEV_BAD_PREFIX);
  const int nkeys = bad ? 0 : P + T;
  const int nch_all = (nkeys + kBN - 1) / kBN;
  const int c_begin = int((long long)nch_all * split / a.splits);
  const int nch = int((long long)nch_all * (split + 1) / a.splits) - c_begin;
  const int tok0 = unit * 2 * a.tpt;                   // nodes of this unit
  const bool two = T - tok0 > a.tpt;                   // two row tiles
  const int vst = two ? 2 : 3;                         // V slots in use
  const int32_t* trow = a.table + size_t(b) * a.max_pages;
  auto v_slot = [&](int s) -> uint8_t* { return s < 2 ? sV + s * C::kTile : sQ + C::kTile; };

  if (warp == 0) {
    // ------------------------------------ K ------------------------------------
    bool ok = true;
    const int withhold = *const_cast<volatile int*>(&g_withhold_chunk);   // test hook, normally -1
    int n = 0;
    for (int c = 0; c < nch; ++c) {
      if (c == withhold) continue;
      const int st = c % kKStages;
      if (c >= kKStages && !mbar_wait(smem_u32(&k_empty[st]), ((c / kKStages) - 1) & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      load_chunk<DH>(smem_u32(sK + st * C::kTile), &kmap, smem_u32(&k_full[st]), trow, (c_begin + c) * kBN, nkeys, hk, a);
      n = c + 1;
    }
    // every copy issued into this CTA's shared memory lands before it may exit
    for (int c = (n > kKStages ? n - kKStages : 0); c < n; ++c)
      if (c != withhold) ok = mbar_wait(smem_u32(&k_full[c % kKStages]), (c / kKStages) & 1) && ok;
    if (!ok && lane == 0) set_status(MD_DEV_TIMEOUT);
  } else if (warp == 2) {
    // ------------------------------------ V ------------------------------------
    bool ok = true;
    const int withhold = *const_cast<volatile int*>(&g_withhold_chunk);
    int n = 0;
    for (int c = 0; c < nch; ++c) {
      if (c == withhold) continue;
      const int st = c % vst;
      if (c >= vst && !mbar_wait(smem_u32(&v_empty[st]), ((c / vst) - 1) & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      load_chunk<DH>(smem_u32(v_slot(st)), &vmap, smem_u32(&v_full[st]), trow, (c_begin + c) * kBN, nkeys, hk, a);
      n = c + 1;
    }
    for (int c = (n > vst ? n - vst : 0); c < n; ++c)
      if (c != withhold) ok = mbar_wait(smem_u32(&v_full[c % vst]), (c / vst) & 1) && ok;
    if (!ok && lane == 0) set_status(MD_DEV_TIMEOUT);
  } else if (warp == 3) {
    // ------------------------------------ Q ------------------------------------
    if (lane == 0 && nch > 0) {
      const uint32_t qb = smem_u32(q_full);
      const int tiles = two ? 2 : 1;
      mbar_arrive_expect_tx(qb, uint32_t(tiles * a.tpt * a.G) * DH * 2);
      for (int w = 0; w < tiles; ++w)
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_3d(smem_u32(sQ + w * C::kTile + kb * (kBM * 128)), &qmap, kb * 64, hk * a.G,
                      b * T + tok0 + w * a.tpt, qb);
      if (!mbar_wait(qb, 0)) set_status(MD_DEV_TIMEOUT);
    }
  } else if (warp == 1) {
    // ----------------------------------- MMA -----------------------------------
    if (lane == 0 && nch > 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(kBM, kBN, 0, 0);
      constexpr uint32_t idesc_o = umma_idesc_bf16(kBM, DH, 0, 1);
      bool ok = mbar_wait(smem_u32(q_full), 0);
      // S_w = Q K_c^T; the last stream to use the chunk frees its slot
      auto issue_s = [&](int c, int w) -> bool {
        const int st = c % kKStages;
        if (!mbar_wait(smem_u32(&k_full[st]), (c / kKStages) & 1)) return false;
        tc_fence_after();
        const uint32_t sq = smem_u32(sQ + (two ? w : 0) * C::kTile), sk = smem_u32(sK + st * C::kTile);
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb) {
          const uint64_t ad = umma_desc_sw128(sq + kb * (kBM * 128), 16, 1024);
          const uint64_t bd = umma_desc_sw128(sk + kb * (kBN * 128), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16(tmem + w * 128, ad + uint64_t((kk * 32) >> 4), bd + uint64_t((kk * 32) >> 4), idesc_s, (kb | kk) != 0);
        }
        umma_commit(smem_u32(&s_full[w]));
        if (!two || w == 1) umma_commit(smem_u32(&k_empty[st]));
        return true;
      };
      const int step = two ? 1 : 2;                      // a stream's next chunk
      if (ok) ok = issue_s(0, 0);
      if (ok && two) ok = issue_s(0, 1);
      if (ok && !two && nch > 1) ok = issue_s(1, 1);
      const int jobs = two ? 2 * nch : nch;
      for (int j = 0; j < jobs && ok; ++j) {
        const int w = j & 1, c = two ? j >> 1 : j, nth = j >> 1;     // nth chunk of this stream
        const int st = c % vst;
        if (!mbar_wait(smem_u32(&p_full[w]), nth & 1) || !mbar_wait(smem_u32(&v_full[st]), (c / vst) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bd = umma_desc_sw128(smem_u32(v_slot(st)), kBN * 128, 1024);
#pragma unroll
        for (int part = 0; part < (F32 ? 2 : 1); ++part)
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            umma_f16_tmem_a(tmem + 256 + w * 128, tmem + w * 128 + uint32_t((kk >> 1) * 32 + part * 16 + (kk & 1) * 8),
                            bd + uint64_t((kk * 2048) >> 4), idesc_o, (nth | part | kk) != 0);
        if (!two || w == 1) umma_commit(smem_u32(&v_empty[st]));
        if (c + step < nch) ok = issue_s(c + step, w);
      }
      // every MMA issued so far completes before TMEM is read out or released
      umma_commit(smem_u32(mma_done));
      if (!mbar_wait(smem_u32(mma_done), 0)) ok = false;
      if (!ok) set_status(MD_DEV_TIMEOUT);
    }
  } else {
    // --------------------------------- softmax ---------------------------------
    const int w = (warp - 4) >> 2;                       // stream
    const int q = warp & 3;                              // TMEM lane quarter
    const int r = q * 32 + lane;                         // row of the tile
    const int tile_tok = tok0 + (two ? w * a.tpt : 0);
    const int t = tile_tok + r / a.G;
    const bool live = r < a.tpt * a.G && t < T;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint32_t lane_off = uint32_t(q * 32) << 16;
    const uint32_t tS = tmem + lane_off + uint32_t(w * 128), tO = tmem + lane_off + uint32_t(256 + w * 128);
    const int tt = live ? t : 0;
    const uint64_t anc_lo = (uint64_t(tp.anc[tt][1]) << 32) | tp.anc[tt][0];
    const uint64_t anc_hi = (uint64_t(tp.anc[tt][3]) << 32) | tp.anc[tt][2];
    const float sc = a.scale_log2;
    const int my_jobs = two ? nch : (nch - w + 1) / 2;
    float run_m = -INFINITY, run_l = 0.f;
    bool ok = true;
    for (int j = 0; j < my_jobs; ++j) {
      const int c = two ? j : 2 * j + w;
      if (ok && !mbar_wait(smem_u32(&s_full[w]), j & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const int key0 = (c_begin + c) * kBN;
      if (warp_live) {
        // two readings of S, 64 and 32 columns at a time: the whole row in registers spills
        const bool masked = key0 + kBN > P;              // tree slots, or slots behind them
        float s[64];
        float m8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          tmem_ld32_async(tS + 64 * g, s);
          tmem_ld32_async(tS + 64 * g + 32, s + 32);
          tmem_ld_wait();
          settle(s);
          settle(s + 32);
          if (masked) {
            const uint64_t vis = visible_bits(anc_lo, anc_hi, key0 + 64 * g - P);
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = ((vis >> i) & 1ull) ? s[i] : -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) m8[i & 7] = fmaxf(m8[i & 7], s[i]);
        }
        tmem_ld32_async(tS, s);                          // the first columns of the second reading
        float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
        mx = (mx == -INFINITY) ? -INFINITY : mx * sc;
        const bool up = mx > run_m + kRescaleLog2 || (run_m == -INFINITY && mx != -INFINITY);
        const float m_new = up ? mx : run_m;
        const float fold = (up && run_m != -INFINITY) ? exp2f(run_m - m_new) : 1.f;
        if (__any_sync(0xffffffffu, fold != 1.f)) {
#pragma unroll
          for (int e0 = 0; e0 < DH; e0 += 32) {
            float o[32];
            tmem_ld32(tO + e0, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= fold;
            tmem_st32(tO + e0, o);
          }
        }
        run_l *= fold;
        run_m = m_new;
        const float mb = (run_m == -INFINITY) ? 0.f : run_m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < kBN / 32; ++g) {
          float* x = s + 32 * (g & 1);
          tmem_ld_wait();
          settle(x);
          if (g < 3) tmem_ld32_async(tS + 32 * (g + 1), s + 32 * ((g + 1) & 1));
          if (masked) {
            const uint32_t vis = uint32_t(visible_bits(anc_lo, anc_hi, key0 + 32 * g - P));
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = ((vis >> i) & 1u) ? x[i] : -INFINITY;
          }
          uint32_t ph[16], pl[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float p0 = exp2_sfu(fmaf(x[i], sc, -mb));
            const float p1 = exp2_sfu(fmaf(x[i + 1], sc, -mb));
            sum[(i >> 1) & 3] += p0 + p1;
            if constexpr (F32) {
              const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
              ph[i >> 1] = __byte_perm(u0, u1, 0x7632);              // truncated to bf16
              const float r0 = p0 - __uint_as_float(u0 & 0xFFFF0000u);
              const float r1 = p1 - __uint_as_float(u1 & 0xFFFF0000u);
              pl[i >> 1] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
            } else {
              ph[i >> 1] = pack_bf16x2(p0, p1);
            }
          }
          tmem_st16u(tS + 32 * g, ph);                   // over the 32 scores just read
          if constexpr (F32) tmem_st16u(tS + 32 * g + 16, pl);
        }
        tmem_st_wait();
        run_l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // V rows that P's zeros must not meet
      if (key0 + kBN > P && (!two || w == 0)) {
        const int st = c % vst;
        if (!mbar_wait(smem_u32(&v_full[st]), (c / vst) & 1)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* v = v_slot(st);
        const int valid = min(kBN, nkeys - key0);
        const int tree0 = max(0, P - key0);              // first row of a tree node
        for (int i = r; i < kBN * C::KB * 8; i += kBM) { // 16-byte pieces, kb-major
          const int row = (i >> 3) & (kBN - 1);
          uint4* piece = reinterpret_cast<uint4*>(v) + i;
          if (row >= valid) {
            *piece = make_uint4(0, 0, 0, 0);
          } else if (row >= tree0 && T > 1) {
            uint4 x = *piece;
            uint32_t u[4] = {x.x, x.y, x.z, x.w};
            bool fix = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!bf16_finite(u[e])) { u[e] &= 0xFFFF0000u; fix = true; }
              if (!bf16_finite(u[e] >> 16)) { u[e] &= 0x0000FFFFu; fix = true; }
            }
            if (fix) {
              *piece = make_uint4(u[0], u[1], u[2], u[3]);
              *bad_v = 1;
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[w]));
    }
    if (!ok) set_status(MD_DEV_TIMEOUT);
    // the stream's O and (m, sum), staged over the idle tiles and ring: every MMA
    // of the CTA is done, so nothing reads or fills them any more
    bool staged = ok && my_jobs > 0;
    if (nch > 0) staged = __all_sync(0xffffffffu, mbar_wait(smem_u32(mma_done), 0)) && staged;
    named_bar_sync(1, kSoftThreads);                     // both streams are past their last look at the ring
    float* sO = reinterpret_cast<float*>(smem) + size_t(w) * kBM * C::kLd;
    if (staged && warp_live) {
      tc_fence_after();
#pragma unroll
      for (int e0 = 0; e0 < DH; e0 += 32) {
        float o[32];
        tmem_ld32(tO + e0, o);
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(sO + r * C::kLd + e0 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
      if (*bad_v && live) {
        // elements of visible nodes' V that are not finite, left out of P V
        for (int n = 0; n < T; ++n) {
          if (!((tp.anc[t][n >> 5] >> (n & 31)) & 1u)) continue;
          const int slot = P + n, c = slot / kBN - c_begin;
          if (c < 0 || c >= nch || (!two && (c & 1) != w)) continue;
          const int pg = trow[slot / a.page];
          if (pg < 0 || pg >= a.pool) continue;
          const uint16_t* v = a.v_pages + ((size_t(pg) * a.Hkv + hk) * a.page + slot % a.page) * DH;
          for (int e = 0; e < DH; ++e)
            if (!bf16_finite(v[e])) sO[r * C::kLd + e] += bf16_to_f32(v[e]);
        }
      }
    }
    sML[w * kBM + r] = make_float2(staged ? run_m : -INFINITY, staged ? run_l : 0.f);
  }

  // ------------------- join the streams and splits of each row -------------------
  __syncwarp();
  cluster_sync();                        // every split's streams are staged
  if (warp >= 4) {
    // a row's partial results: (split, stream) with one tile, (split) with two
    const int np = two ? a.splits : 2 * a.splits;
    const int ntok = min(two ? 2 * a.tpt : a.tpt, T - tok0);
    const int rows = ntok * a.G;                         // dense over the unit's (node, head) pairs
    const int tile_rows = a.tpt * a.G;
    const int crank = int(cluster_ctarank());
    const int r0 = rows * crank / a.splits, r1 = rows * (crank + 1) / a.splits;
    constexpr int kLanes = DH / 4;                       // float4 columns: 32 or 16 lanes a row
    constexpr int kRowsPerWarp = 32 / kLanes;
    const int sub = lane / kLanes, col = lane % kLanes;
    for (int i0 = r0 + (warp - 4) * kRowsPerWarp; i0 < r1; i0 += 8 * kRowsPerWarp) {
      const int i = min(i0 + sub, r1 - 1);               // the last pair may repeat a row
      const int w0 = i / tile_rows, row = i - w0 * tile_rows;          // stream (two tiles) and row in it
      // lane p holds partial p of this warp's row (two rows a warp: 16 lanes each)
      float m_p = -INFINITY, l_p = 0.f, m2 = -INFINITY, l2 = 0.f;
      auto ml_of = [&](int p) -> float2 {
        const int sp = two ? p : p >> 1, st = two ? w0 : p & 1;
        return ld_cluster_f2(mapa_shared(smem_u32(&sML[st * kBM + row]), uint32_t(sp)));
      };
      if (col < np) { const float2 x = ml_of(col); m_p = x.x; l_p = x.y; }
      if (kLanes == 16 && col + 16 < np) { const float2 x = ml_of(col + 16); m2 = x.x; l2 = x.y; }
      float mx = fmaxf(m_p, m2);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float w_p = (m_p == -INFINITY) ? 0.f : exp2f(m_p - mx), w_2 = (m2 == -INFINITY) ? 0.f : exp2f(m2 - mx);
      float L = l_p * w_p + l2 * w_2;
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int p = 0; p < np; ++p) {
        const int from = sub * kLanes + (p & (kLanes - 1));
        const float wgt = __shfl_sync(0xffffffffu, (kLanes == 16 && p >= 16) ? w_2 : w_p, from);
        const float mm = __shfl_sync(0xffffffffu, (kLanes == 16 && p >= 16) ? m2 : m_p, from);
        if (mm != -INFINITY) {                           // a stream without chunks staged nothing
          const int sp = two ? p : p >> 1, st = two ? w0 : p & 1;
          const float* src = reinterpret_cast<float*>(smem) + (size_t(st) * kBM + row) * C::kLd + col * 4;
          const float4 o = ld_cluster_f4(mapa_shared(smem_u32(src), uint32_t(sp)));
          acc.x = fmaf(o.x, wgt, acc.x);
          acc.y = fmaf(o.y, wgt, acc.y);
          acc.z = fmaf(o.z, wgt, acc.z);
          acc.w = fmaf(o.w, wgt, acc.w);
        }
      }
      const float inv = 1.f / L;
      float4 y = bad ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (i0 + sub < r1) {
        const int tn = tok0 + i / a.G, h = hk * a.G + i % a.G;
        const size_t at = ((size_t(b) * T + tn) * a.Hq + h) * DH + col * 4;
        if constexpr (F32)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      }
    }
  }
  __syncwarp();
  cluster_sync();                        // peers are done reading this CTA's shared memory
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace attn_paged
}  // namespace md
