// Tree-masked attention over a paged KV cache, on the tensor cores (tcgen05).
//
//   out[b,t,h,:] = sum_j softmax_j(scale q[b,t,h,:] . K_j) V_j
//
// over the prefix slots j < P_b and the tree slots P_b + a of the ancestors a of
// node t (itself included), slot s of request b being row s % page of page
// block_table[b, s / page]. The T * G query rows (node, head of the group) of a
// KV head share its keys, so scores and weighted sums are dense products.
//
// CTA = (KV split, unit of one or two 128-row tiles, KV head, request). Two streams
// (one, with half of everything, where there are many short requests: Cfg),
// each with scores S, weights P (written over S) and an accumulator O in TMEM, walk
// the split's keys in jobs of 64:
//   - two tiles: stream w is row tile w and takes every job, so that a chunk of
//     keys fetched once serves 256 rows;
//   - one tile (decoding, chains, the odd last tile, or where more CTAs pay): the
//     streams take the jobs in turn and are joined at the end.
// While one stream's warps run a job's softmax the tensor cores work for the other,
// and (bf16 results) for this stream's next job, whose S goes to a second buffer.
//
//   warp 0      K: chunks of 128 keys, one TMA copy per page piece and 64-column
//               block, each lane a piece (its page id from the block table)
//   warp 2      V, as K; then the look at the chunks that reach the tree (below)
//   warps 1, 3  MMAs of stream 0 and 1 (warp 3 also fetches the Q tiles): O += P V
//               of a job, then S = Q K^T of the next one in its buffer. Both take
//               their operands in issue order, so S may overwrite P behind its P V.
//   warps 4-19  softmax: a row of a stream is two threads, 32 keys of a job each;
//               they exchange maxima through shared memory. The reference maximum m
//               moves only when a job exceeds it by 2^8: O and the sum are then
//               rescaled in place, once the stream's last P V has landed. P =
//               exp2(S - m); sums in fp32.
//
// P is rounded to bf16 for the product with V where the result is bf16: a weight's
// error, at most 2^-8 of it either way, averages out over the keys as V does, and the
// result is rounded to the same precision (0.0023 of the result against 64 bits,
// 0.0017 being the last rounding's own: two roundings of one size). A second part of P
// leaves 0.0017 and was not worth its product: 70B batch of 8 125 us against 103, 70B
// tree 27 against 22.6. For fp32 results P is three bf16 parts, 24 bits, and P V
// three products; S then has one buffer, the parts needing the other's columns. The
// tensor cores' accumulator drops what it cannot hold at every step (8e-6 of the result
// over 20000 keys), so after every 128 keys O is added to a sum in local memory:
// with N(0, 1) inputs 8e-7 of the result from 128 to 660000 slots (256 keys a stretch
// 1.2e-6, 192 1.0e-6), with values of one sign 2.3e-6, as the dropped parts add up.
//
// The KV splits of a unit are the CTAs of a cluster: O and (m, sum) of every
// stream are staged in shared memory, and each CTA combines its share of the
// rows from all of them (distributed shared memory). Splits are made of the
// request's own length on the device, so that none is empty in a wide table; how many
// there are, and the CTAs' shape, go by the table's width (paged_attn_plan).
//
// Slots behind the tree's last hold anything, NaN included: their scores are
// replaced, and their V rows zeroed in shared memory (0 * NaN would reach O). A
// tree node's V that is not finite must reach only the rows that see the node:
// such elements are zeroed in shared memory too and added to those rows'
// results at the end.
//
// What bounds it. Long prefixes with few rows: bytes (16 requests of 20k to 33k
// slots, one node: 264 us, 6.4 TB/s, 97 % of a copy's rate, replayed from a cool start;
// call after call the power cap takes the clocks to 1.6 GHz, 310 us, 83 %). Many rows: the two-tile
// walk takes 1.76 us a chunk of 128 keys where its tensor work takes 1.34 (measured
// without the softmax: S with N = 64 is held back by shared memory, 43 clocks an MMA
// against 32) and the special-function unit 1.08; 70B batch of 8: 103 us, 0.66
// PFLOP/s. One request: set-up, first loads, the splits' joining and the launch,
// about 8 us, are as much as the walk (70B tree over 4096 slots: 22.5 us). Many
// requests of few keys: the same fixed part once a CTA, halved by two CTAs an SM.
#pragma once

#include <climits>

#include "attention_tc.cuh"
#include "common.cuh"

namespace md {
namespace attn_paged {

using attn_tc::exp2_sfu;
using attn_tc::visible_bits;

constexpr int kBM = 128;              // rows of a tile
constexpr int kSub = 64;              // keys of a job: half a chunk
constexpr int kMaxStages = 3;
constexpr int kMaxSplits = 16;        // CTAs of a cluster (above 8 by opt-in)
constexpr float kRescaleLog2 = 8.0f;

// STREAMS = 2: one CTA per SM, as above. STREAMS = 1: half a CTA of everything (one
// stream, one row tile, chunks of 64 keys), two to an SM, so that one's set-up and
// read-out run beside the other's walk: for grids of many short requests (256 of 200
// slots, 8 KV heads, one node: 189 us with two streams, 105 with one).
template <int DH, bool F32, int STREAMS>
struct Cfg {
  static constexpr int kBN = 64 * STREAMS;                 // keys of a chunk (a slot of the rings)
  static constexpr int kSoftThreads = 256 * STREAMS;
  static constexpr int kThreads = 128 + kSoftThreads;
  static constexpr int kKStages = STREAMS == 2 ? 3 : 2;
  static constexpr uint32_t kTmemCols = 256 * STREAMS;     // S and O of each stream: 128 columns each
  // bf16 results: two S buffers a stream, so that the next scores are ready when a
  // job ends; fp32 ones: the three parts of P take the columns of the second
  static constexpr int kBufs = F32 ? 1 : 2;
  static constexpr int kParts = F32 ? 3 : 1;               // bf16 parts of P
  // jobs (of 64 keys) in one accumulator; fp32 results: then it is added to a sum
  // outside the tensor cores, whose accumulator drops what it cannot hold at every step
  static constexpr int kStretch = F32 ? 2 : INT_MAX;
  static constexpr int KB = DH / 64;                       // 64-column blocks
  static constexpr uint32_t kQTile = KB * kBM * 128;       // 128 rows x DH bf16, 128-byte swizzle
  static constexpr uint32_t kTile = KB * kBN * 128;        // a chunk of K or V
  static constexpr int kLd = DH + 4;                       // padded fp32 row of the staged O
  // a Q tile per stream (the second may be a V slot), the K slots, 2 V slots
  static constexpr uint32_t kRing = STREAMS * kQTile + (kKStages + 2) * kTile;
  static constexpr int kSmem = int(kRing) + 512 + 1024 * STREAMS;   // + barriers, row maxima
  static_assert(STREAMS * kBM * (kLd * 4 + 8) + (STREAMS * kBM + 2 * kMaxSplits) * 12 <= int(kRing),
                "staged O, (m, sum), weights");
};

struct Args {
  const uint16_t* v_pages;     // [pool, Hkv, page, dh] (the slow path of a V that is not finite)
  const int32_t* table;        // [B, max_pages]
  const int32_t* prefix_len;   // [B]
  void* out;                   // [B, T, Hq, dh]
  int B, Hq, Hkv, G, pool, page, max_pages;
  int piece;                   // rows of a TMA copy: the largest power of two dividing page, within a chunk
  int tpt;                     // tree nodes of a row tile
  int tpu;                     // row tiles of a unit: 1 or 2
  int units, splits, sort;
  float scale_log2;
};

// Two fp32 in one 64-bit register: the packed FMA and add of sm_100.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f32x2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// NaN if one of them is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// 4-D tiled TMA load (no multicast).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// 16 columns, loaded and stored (few registers beside a row of scores).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]) : "memory");
}

// The MMAs and commits of attention_paged, issued by one elected lane of a
// converged warp. The election sits inside the instruction's own predicate: code
// around it stays convergent, so operands are computed and kept in uniform
// registers, which is where an MMA takes them from (under a lane's branch each
// operand of each MMA is moved there on its own: 80 clocks an MMA).
__device__ __forceinline__ void umma_f16_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f16_tmem_a_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                      uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// mbar_wait, for waits that are short and many: the bounded form's clock and limit
// (a timer and a global load) are only read once the phase is really late.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity);
}

__device__ __forceinline__ f32x2 exp2_sfu2(f32x2 x) {
  float a, b;
  unpair(x, a, b);
  return pair(exp2_sfu(a), exp2_sfu(b));
}

// An fp32's leading 16 bits as a value, and those of two packed as bf16x2.
__device__ __forceinline__ float high_part(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

template <int ID, int THREADS>
__device__ __forceinline__ void fixed_bar_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

template <int N>
struct IntTag {
  static constexpr int value = N;
};

__device__ __forceinline__ bool bf16_finite(uint32_t v) { return (v & 0x7F80u) != 0x7F80u; }

// Where the page piece of this lane lies for the chunk at key0: its page's row of the
// tensor map and its first slot in the page. Loaded a chunk ahead of its use.
struct Piece {
  int page, at;
};
template <int BN>
__device__ __forceinline__ Piece piece_of(const int32_t* row, int key0, int nkeys, const Args& a) {
  const int key = key0 + int(threadIdx.x & 31) * a.piece;
  Piece p = {0, 0};
  if (key < min(nkeys, key0 + BN)) {
    const int pi = key / a.page;
    p.page = row[pi];
    p.at = key - pi * a.page;
  }
  return p;
}

// The copies of one chunk of K or V into a ring slot, each lane a page piece.
// Pieces behind the last slot are not copied. All lanes of a warp call it.
template <int DH, bool F32, int STREAMS>
__device__ __forceinline__ void load_chunk(uint32_t dst, const CUtensorMap* map, uint32_t bar, Piece p, int key0, int nkeys,
                                           int hk, const Args& a) {
  using C = Cfg<DH, F32, STREAMS>;
  constexpr int kBN = C::kBN;
  const int lane = threadIdx.x & 31;
  const int pieces = (min(kBN, nkeys - key0) + a.piece - 1) / a.piece;
  if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(pieces * a.piece) * DH * 2);
  __syncwarp();
  if (lane < pieces) {
    if (p.page < 0 || p.page >= a.pool) {
      set_status(MD_DEV_BAD_PAGE);
      p.page = a.pool;                   // past the pool: the copy fills zeros
    }
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
      tma_load_3d(dst + kb * (kBN * 128) + lane * a.piece * 128, map, kb * 64, p.at, p.page * a.Hkv + hk, bar);
  }
}

template <int DH, bool F32, int STREAMS>
__global__ void __launch_bounds__(Cfg<DH, F32, STREAMS>::kThreads, 3 - STREAMS)
    attn_paged_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeParams tp, Args a) {
  using C = Cfg<DH, F32, STREAMS>;
  constexpr int kBN = C::kBN, kKStages = C::kKStages;
  constexpr bool kPair = STREAMS == 2;
  constexpr int kAllBar = 1 + 4 * STREAMS;               // named barrier of the softmax warps, behind those of pairs
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                                    // a tile per stream (the second may be V slot 2)
  uint8_t* sK = smem + STREAMS * C::kQTile;              // the K slots
  uint8_t* sV = sK + kKStages * C::kTile;                // 2 slots
  float2* sML = reinterpret_cast<float2*>(smem + STREAMS * kBM * C::kLd * 4);   // [streams][128], behind the staged O
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* q_full = bars;                // 1
  uint64_t* k_full = q_full + 1;          // up to 3
  uint64_t* k_empty = k_full + kMaxStages;
  uint64_t* v_full = k_empty + kMaxStages;
  uint64_t* v_empty = v_full + kMaxStages;
  uint64_t* s_full = v_empty + kMaxStages;  // [streams][2 buffers]
  uint64_t* p_full = s_full + 4;          // [2][2]
  uint64_t* o_full = p_full + 4;          // [2]
  uint64_t* v_fixed = o_full + 2;         // [2]: the chunks that reach the tree, behind the V warp's look
  uint64_t* mma_done = v_fixed + 2;       // 1
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  int* req = reinterpret_cast<int*>(tmem_slot + 1);
  int* bad_v = req + 1;
  float* s_part = reinterpret_cast<float*>(smem + C::kRing + 512);        // [2 streams][2 halves][128]: row maxima, sums

  const int split = blockIdx.x, unit = blockIdx.y % a.units, hk = blockIdx.y / a.units;
  const int warp = __reduce_max_sync(0xffffffffu, int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int T = tp.T;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(q_full), 1);
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_u32(&k_full[i]), 1);
      mbar_init(smem_u32(&k_empty[i]), STREAMS);         // every stream has used it
      mbar_init(smem_u32(&v_full[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), STREAMS);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&o_full[i]), 1);
      mbar_init(smem_u32(&v_fixed[i]), 1);
    }
    mbar_init(smem_u32(mma_done), STREAMS);
    fence_barrier_init();
    *req = blockIdx.z;
    *bad_v = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (lane == 0) {
    if (warp == 0) prefetch_tensormap(&kmap);
    if (warp == 2) prefetch_tensormap(&vmap);
    if (warp == 3) prefetch_tensormap(&qmap);
  }
  pdl_wait_primary();          // inputs may come from earlier kernels
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // More CTAs than one wave: requests from the longest prefix down, so that
  // short ones fill the tail.
  if (a.sort) {
    for (int c = threadIdx.x; c < a.B; c += C::kThreads) {
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
  // at most 2^25 chunks and 16 splits
  const int c_begin = int(uint32_t(nch_all) * uint32_t(split) / uint32_t(a.splits));
  const int nch = int(uint32_t(nch_all) * uint32_t(split + 1) / uint32_t(a.splits)) - c_begin;
  // jobs' keys: halves of chunks, without a last half that is all behind the keys
  const int nsub = nch == 0 ? 0 : (min(nkeys, (c_begin + nch) * kBN) - c_begin * kBN + kSub - 1) / kSub;
  const int tok0 = unit * a.tpu * a.tpt;               // nodes of this unit
  const bool two = kPair && a.tpu == 2 && T - tok0 > a.tpt;   // two row tiles
  const int vst = !kPair || two ? 2 : 3;               // V slots in use
  const int c_tree = max(0, (P - c_begin * kBN) / kBN);   // first chunk with tree slots (at most two have any), if below nch
  const int32_t* trow = a.table + size_t(b) * a.max_pages;
  auto v_slot = [&](int s) -> uint8_t* { return s < 2 ? sV + s * C::kTile : sQ + C::kQTile; };

  if (warp == 0) {
    // ------------------------------------ K ------------------------------------
    bool ok = true;
    const int withhold = *const_cast<volatile int*>(&g_withhold_chunk);   // test hook, normally -1
    int n = 0;
    Piece next = piece_of<kBN>(trow, c_begin * kBN, nch > 0 ? nkeys : 0, a);
    for (int c = 0; c < nch; ++c) {
      const int key0 = (c_begin + c) * kBN;
      const Piece p = next;
      if (c + 1 < nch) next = piece_of<kBN>(trow, key0 + kBN, nkeys, a);
      if (c == withhold) continue;
      const int st = c % kKStages;
      if (c >= kKStages && !wait_phase(smem_u32(&k_empty[st]), ((c / kKStages) - 1) & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      load_chunk<DH, F32, STREAMS>(smem_u32(sK + st * C::kTile), &kmap, smem_u32(&k_full[st]), p, key0, nkeys, hk, a);
      n = c + 1;
    }
    // every copy issued into this CTA's shared memory lands before it may exit
    for (int c = (n > kKStages ? n - kKStages : 0); c < n; ++c)
      if (c != withhold) ok = wait_phase(smem_u32(&k_full[c % kKStages]), (c / kKStages) & 1) && ok;
    if (!ok && lane == 0) set_status(MD_DEV_TIMEOUT);
  } else if (warp == 2) {
    // ------------------------------------ V ------------------------------------
    bool ok = true;
    const int withhold = *const_cast<volatile int*>(&g_withhold_chunk);
    int n = 0;
    Piece next = piece_of<kBN>(trow, c_begin * kBN, nch > 0 ? nkeys : 0, a);
    for (int c = 0; c < nch; ++c) {
      const int key0 = (c_begin + c) * kBN;
      const Piece p = next;
      if (c + 1 < nch) next = piece_of<kBN>(trow, key0 + kBN, nkeys, a);
      if (c == withhold) continue;
      const int st = c % vst;
      if (c >= vst && !wait_phase(smem_u32(&v_empty[st]), ((c / vst) - 1) & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      load_chunk<DH, F32, STREAMS>(smem_u32(v_slot(st)), &vmap, smem_u32(&v_full[st]), p, key0, nkeys, hk, a);
      n = c + 1;
    }
    // V rows that P's zeros must not meet: slots behind the last key, and what is
    // not finite in the tree's (a node may not reach the rows that do not see it)
    for (int c = c_tree; c < nch && ok; ++c) {
      ok = __all_sync(0xffffffffu, c != withhold && wait_phase(smem_u32(&v_full[c % vst]), (c / vst) & 1));
      if (!ok) break;
      const int key0 = (c_begin + c) * kBN, valid = min(kBN, nkeys - key0);
      const int first = T > 1 ? max(0, P - key0) : valid;
      bool fixed = false;
      for (int kb = 0; kb < C::KB; ++kb) {
        uint4* v = reinterpret_cast<uint4*>(v_slot(c % vst) + kb * (kBN * 128));   // 8 pieces of 16 bytes a row
#pragma unroll 4
        for (int i = first * 8 + lane; i < valid * 8; i += 32) {
          uint4 x = v[i];
          uint32_t h[4] = {x.x, x.y, x.z, x.w};
          bool fix = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!bf16_finite(h[e])) { h[e] &= 0xFFFF0000u; fix = true; }
            if (!bf16_finite(h[e] >> 16)) { h[e] &= 0x0000FFFFu; fix = true; }
          }
          if (fix) v[i] = make_uint4(h[0], h[1], h[2], h[3]);
          fixed |= fix;
        }
        for (int i = valid * 8 + lane; i < kBN * 8; i += 32) v[i] = make_uint4(0, 0, 0, 0);
      }
      if (fixed) *bad_v = 1;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&v_fixed[c - c_tree]));
    }
    for (int c = (n > vst ? n - vst : 0); c < n; ++c)
      if (c != withhold) ok = wait_phase(smem_u32(&v_full[c % vst]), (c / vst) & 1) && ok;
    if (!ok && lane == 0) set_status(MD_DEV_TIMEOUT);
  } else if (warp < 4) {
    // --------------------------- MMAs: warp 1 + 2 w, stream w ---------------------------
    // The whole warp walks the stream's jobs, convergent; one elected lane issues.
    // A warp per stream: one stream's waits do not keep the other's MMAs back.
    if (nch > 0 && (warp >> 1) < STREAMS) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(kBM, kSub, 0, 0);
      constexpr uint32_t idesc_o = umma_idesc_bf16(kBM, DH, 0, 1);
      const int w = kPair ? warp >> 1 : 0;
      const uint32_t tS = __reduce_max_sync(0xffffffffu, tmem) + w * 128, tO = tS + STREAMS * 128;
      const int n = __reduce_max_sync(0xffffffffu, nsub), ct = __reduce_max_sync(0xffffffffu, c_tree);
      const uint32_t q_desc = smem_u32(sQ), k_desc = smem_u32(sK), v_desc = smem_u32(sV);
      if (w == STREAMS - 1 && lane == 0) {               // the Q tiles
        const uint32_t qb = smem_u32(q_full);
        const int tiles = two ? 2 : 1;
        mbar_arrive_expect_tx(qb, uint32_t(tiles * a.tpt * a.G) * DH * 2);
        for (int i = 0; i < tiles; ++i)
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_4d(smem_u32(sQ + i * C::kQTile + kb * (kBM * 128)), &qmap, kb * 64, hk * a.G, tok0 + i * a.tpt, b, qb);
      }
      __syncwarp();
      bool ok = __all_sync(0xffffffffu, wait_phase(smem_u32(q_full), 0));
      // TILES row tiles: a job is half a chunk, the next job the next half (2), or the
      // same half of the next chunk, the other stream having taken the other (1)
      auto walk = [&](auto tiles_tag) {
        constexpr int TILES = decltype(tiles_tag)::value;
        constexpr int VST = TILES == 2 || !kPair ? 2 : 3;
        const int jobs = TILES == 2 || !kPair ? n : (n - w + 1) / 2;
        int ks = 0, kph = 0, vs = 0, vph = 0;            // slot and phase of the next job's K and V
        auto half_of = [&](int j) { return TILES == 2 ? j & 1 : w; };      // of the job's chunk
        auto issue_s = [&](int j, int buf) {
          const int half = half_of(j);
          if (TILES == 1 || half == 0) {                 // a chunk this stream has not used yet
            ok = __all_sync(0xffffffffu, wait_phase(smem_u32(&k_full[ks]), kph));
            tc_fence_after();
          }
          if (!ok) return;
          const uint64_t ad = umma_desc_sw128(q_desc + (TILES == 2 ? w : 0) * C::kQTile, 16, 1024);
          const uint64_t bd = umma_desc_sw128(k_desc + ks * C::kTile + half * (kSub * 128), 16, 1024);
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_elect(tS + buf * kSub, ad + uint64_t((kb * (kBM * 128) + kk * 32) >> 4),
                             bd + uint64_t((kb * (kBN * 128) + kk * 32) >> 4), idesc_s, (kb | kk) != 0);
          umma_commit_elect(smem_u32(&s_full[2 * w + buf]));
          if (TILES == 1 || half == 1 || j == jobs - 1) {
            umma_commit_elect(smem_u32(&k_empty[ks]));
            if (++ks == kKStages) { ks = 0; kph ^= 1; }
          }
        };
        // O += P V of job j, then the S that follows in its buffer
        auto job = [&](int j, int buf, int ph) {
          const int half = half_of(j);
          if (TILES == 1 || half == 0) {                 // a chunk this stream has not used yet
            const int c = TILES == 1 ? j : j >> 1;
            ok = c < ct ? wait_phase(smem_u32(&v_full[vs]), vph) : wait_phase(smem_u32(&v_fixed[c - ct]), 0);
          }
          ok = __all_sync(0xffffffffu, ok && wait_phase(smem_u32(&p_full[2 * w + buf]), ph));
          if (!ok) return;
          tc_fence_after();
          const uint32_t vb = (VST == 3 && vs == 2 ? q_desc + C::kQTile : v_desc + vs * C::kTile) + half * (kSub * 128);
          const uint64_t bd = umma_desc_sw128(vb, kBN * 128, 1024);
#pragma unroll
          for (int part = 0; part < C::kParts; ++part)
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk)
              umma_f16_tmem_a_elect(tO, tS + buf * kSub + uint32_t(part * (kSub / 2) + kk * 8), bd + uint64_t((kk * 2048) >> 4),
                                    idesc_o, (part | kk) != 0 ? 1u : uint32_t(j % C::kStretch != 0));
          umma_commit_elect(smem_u32(&o_full[w]));
          if (TILES == 1 || half == 1 || j == jobs - 1) {
            umma_commit_elect(smem_u32(&v_empty[vs]));
            if (++vs == VST) { vs = 0; vph ^= 1; }
          }
          if (j + C::kBufs < jobs) issue_s(j + C::kBufs, buf);
        };
#pragma unroll
        for (int j = 0; j < C::kBufs; ++j)
          if (j < jobs && ok) issue_s(j, j);
        int ph = 0;
        for (int j0 = 0; j0 < jobs && ok; j0 += C::kBufs, ph ^= 1)
#pragma unroll
          for (int i = 0; i < C::kBufs; ++i)
            if (j0 + i < jobs && ok) job(j0 + i, i, ph);
      };
      if (ok) {
        if constexpr (kPair) {
          if (two) walk(IntTag<2>{});
          else walk(IntTag<1>{});
        } else {
          walk(IntTag<1>{});
        }
      }
      // every MMA issued so far completes before TMEM is read out or released
      umma_commit_elect(smem_u32(mma_done));
      if (!wait_phase(smem_u32(mma_done), 0)) ok = false;
      if (!ok && lane == 0) set_status(MD_DEV_TIMEOUT);
    }
  } else {
    // --------------------------------- softmax ---------------------------------
    const int w = kPair ? (warp - 4) >> 3 : 0;           // stream
    const int half = ((warp - 4) >> 2) & 1;              // of a job's keys, and of O's columns
    const int q = warp & 3;                              // TMEM lane quarter
    // The two halves' warps. Two CTAs to an SM: ids known to the compiler, as an id in a
    // register reserves all 16 barriers of a CTA, which then has the SM to itself.
    auto pair_sync = [&] {
      if constexpr (kPair) {
        named_bar_sync(1 + w * 4 + q, 64);
      } else {
        switch (q) {
          case 0: fixed_bar_sync<1, 64>(); break;
          case 1: fixed_bar_sync<2, 64>(); break;
          case 2: fixed_bar_sync<3, 64>(); break;
          default: fixed_bar_sync<4, 64>();
        }
      }
    };
    const int r = q * 32 + lane;                         // row of the tile
    const int tile_tok = tok0 + (two ? w * a.tpt : 0);
    const int t = tile_tok + r / a.G;
    const bool live = r < a.tpt * a.G && t < T;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint32_t lane_off = uint32_t(q * 32) << 16;
    const uint32_t tS = tmem + lane_off + uint32_t(w * 128), tO = tmem + lane_off + uint32_t((STREAMS + w) * 128);
    const int tt = live ? t : 0;
    const uint64_t anc_lo = (uint64_t(tp.anc[tt][1]) << 32) | tp.anc[tt][0];
    const uint64_t anc_hi = (uint64_t(tp.anc[tt][3]) << 32) | tp.anc[tt][2];
    const float sc = a.scale_log2;
    const int my_jobs = two || !kPair ? nsub : (nsub - w + 1) / 2;
    float run_m = -INFINITY, run_l = 0.f;
    // fp32 results: the finished stretches' sum, this thread's half of the row (indexed
    // in rolled loops: local memory), against the maximum keep_m
    [[maybe_unused]] float keep[F32 ? DH / 2 : 1];
    [[maybe_unused]] float keep_m = -INFINITY;
    bool ok = true;
    for (int j = 0; j < my_jobs; ++j) {
      const int u = two || !kPair ? j : 2 * j + w;       // 64 keys of the range
      const int buf = j % C::kBufs;
      // A wait that gives up only skips work: every iteration runs the halves' barriers.
      ok = __all_sync(0xffffffffu, ok && wait_phase(smem_u32(&s_full[2 * w + buf]), (j / C::kBufs) & 1));
      tc_fence_after();
      const uint32_t tSb = tS + buf * kSub;
      const int key0 = c_begin * kBN + u * kSub;
      if (warp_live) {
        if constexpr (F32) {
          if (j > 0 && j % C::kStretch == 0 && ok) {
            // S of this job was issued behind the last P V: O is complete, and the next
            // P V, which overwrites it, waits for this job's P
            const float f = keep_m == -INFINITY || keep_m == run_m ? 1.f : exp2f(keep_m - run_m);
            keep_m = run_m;
#pragma unroll 1
            for (int e0 = 0; e0 < DH / 2; e0 += 16) {
              float o[16];
              tmem_ld16(tO + half * (DH / 2) + e0, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) keep[e0 + e] = j == C::kStretch ? o[e] : fmaf(keep[e0 + e], f, o[e]);
            }
          }
        }
        float s[32];
        if (ok) tmem_ld32_async(tSb + half * 32, s);
        tmem_ld_wait();
        settle(s);
        const bool masked = key0 + kSub > P;             // tree slots, or slots behind them
        if (masked) {
          const uint32_t vis = uint32_t(visible_bits(anc_lo, anc_hi, key0 + half * 32 - P));
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = ((vis >> i) & 1u) ? s[i] : -INFINITY;
        }
        float m4[4];                                     // four chains of three-way maxima
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m4[k] = max3(s[k], s[k + 4], s[k + 8]);
          m4[k] = max3(m4[k], s[k + 12], s[k + 16]);
          m4[k] = max3(m4[k], s[k + 20], s[k + 24]);
          m4[k] = max3(m4[k], s[k + 28], s[k + 28]);
        }
        float mx = max3(max3(m4[0], m4[1], m4[2]), m4[3], m4[3]);
        // the row's maximum over both halves; behind the second barrier both have
        // read their scores, and either may write P over them
        pair_sync();                                     // the last job's maxima have been read
        s_part[(2 * w + half) * kBM + r] = mx;
        pair_sync();
        const float mo = s_part[(2 * w + (half ^ 1)) * kBM + r];
        mx = max3(mx, mo, mo);
        // a score that is NaN or infinite makes the row NaN, as its softmax is
        if (!(mx < INFINITY)) run_l = __int_as_float(0x7FC00000);
        mx = (mx == -INFINITY) ? -INFINITY : mx * sc;
        const bool up = mx > run_m + kRescaleLog2 || (run_m == -INFINITY && mx != -INFINITY);
        if (__any_sync(0xffffffffu, up)) {
          const float fold = (up && run_m != -INFINITY) ? exp2f(run_m - mx) : 1.f;
          if (__any_sync(0xffffffffu, fold != 1.f)) {
            // O is rescaled in place, half of its columns here: this stream's last P V has
            // landed (the one before it has, as S of this job was issued behind it)
            if (ok) ok = __all_sync(0xffffffffu, wait_phase(smem_u32(&o_full[w]), (j - 1) & 1));
            tc_fence_after();
#pragma unroll 1
            for (int e0 = half * (DH / 2); e0 < (half + 1) * (DH / 2); e0 += 16) {
              float o[16];
              tmem_ld16(tO + e0, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= fold;
              tmem_st16(tO + e0, o);
            }
          }
          run_l *= fold;
          run_m = up ? mx : run_m;
        }
        const float mb = (run_m == -INFINITY) ? 0.f : run_m;
        const f32x2 sc2 = pair(sc, sc), mb2 = pair(-mb, -mb);
        f32x2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        uint32_t p0[16];
        [[maybe_unused]] uint32_t p1[16], p2[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a0, a1;
          unpair(fma2(pair(s[2 * i], s[2 * i + 1]), sc2, mb2), a0, a1);
          a0 = exp2_sfu(a0);
          a1 = exp2_sfu(a1);
          sum[i & 1] = add2(sum[i & 1], pair(a0, a1));
          if constexpr (F32) {
            // truncated parts, 8 bits each: the remainders are exact
            p0[i] = high_halves(a0, a1);
            const float b0 = a0 - high_part(a0), b1 = a1 - high_part(a1);
            p1[i] = high_halves(b0, b1);
            p2[i] = pack_bf16x2(b0 - high_part(b0), b1 - high_part(b1));
          } else {
            p0[i] = pack_bf16x2(a0, a1);
          }
        }
        tmem_st16u(tSb + half * 16, p0);
        if constexpr (F32) {
          tmem_st16u(tSb + kSub / 2 + half * 16, p1);
          tmem_st16u(tSb + kSub + half * 16, p2);
        }
        tmem_st_wait();
        float l0, l1;
        unpair(add2(sum[0], sum[1]), l0, l1);
        run_l += l0 + l1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&p_full[2 * w + buf]));
    }
    if (!ok) set_status(MD_DEV_TIMEOUT);
    // the stream's O and (m, sum), staged over the idle tiles and ring: every MMA
    // of the CTA is done, so nothing reads or fills them any more
    bool staged = ok && my_jobs > 0;
    if (nch > 0) staged = __all_sync(0xffffffffu, wait_phase(smem_u32(mma_done), 0)) && staged;
    if (c_tree < nch) staged = __all_sync(0xffffffffu, wait_phase(smem_u32(&v_fixed[nch - 1 - c_tree]), 0)) && staged;   // *bad_v
    if (warp_live) pair_sync();                          // the last maxima have been read
    if (half == 1) s_part[(2 * w + 1) * kBM + r] = run_l;
    fixed_bar_sync<kAllBar, C::kSoftThreads>();          // both streams are past their last look at the ring
    if (half == 0)
      sML[w * kBM + r] = staged ? make_float2(run_m, run_l + s_part[(2 * w + 1) * kBM + r]) : make_float2(-INFINITY, 0.f);
    // With one tile both streams' results are of the same rows: stream 0 stages its own
    // against their common maximum, stream 1 adds to it.
    float* sO = reinterpret_cast<float*>(smem) + (two ? size_t(w) * kBM * C::kLd : 0) + r * C::kLd;
    float fold = 1.f;
    float2 both = make_float2(-INFINITY, 0.f);
    bool onto = false;                                   // stream 1: stream 0 staged this row
    if (kPair && !two) {
      fixed_bar_sync<kAllBar, C::kSoftThreads>();
      const float2 x = sML[r], y = sML[kBM + r];
      const float m = fmaxf(x.x, y.x);
      const float f0 = x.x == -INFINITY ? 0.f : exp2_sfu(x.x - m), f1 = y.x == -INFINITY ? 0.f : exp2_sfu(y.x - m);
      both = make_float2(m, (x.x == -INFINITY ? 0.f : x.y * f0) + (y.x == -INFINITY ? 0.f : y.y * f1));
      fold = w == 0 ? f0 : f1;
      onto = w == 1 && x.x != -INFINITY;
      staged = staged && __any_sync(0xffffffffu, (w == 0 ? x.x : y.x) != -INFINITY);
      if (w == 1) fixed_bar_sync<kAllBar, C::kSoftThreads>(); // stream 0's rows are staged
    }
    if (staged && warp_live) {
      tc_fence_after();
#pragma unroll 1
      for (int e0 = half * (DH / 2); e0 < (half + 1) * (DH / 2); e0 += 16) {
        float o[16];
        tmem_ld16(tO + e0, o);
        if constexpr (F32) {
          if (my_jobs > C::kStretch) {
            const float f = keep_m == -INFINITY || keep_m == run_m ? 1.f : exp2f(keep_m - run_m);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(keep[e0 - half * (DH / 2) + e], f, o[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          float4* to = reinterpret_cast<float4*>(sO + e0 + e);
          float4 v = make_float4(o[e] * fold, o[e + 1] * fold, o[e + 2] * fold, o[e + 3] * fold);
          if (onto) {
            const float4 x = *to;
            if (fold == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);   // nothing of this row in stream 1
            v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
          }
          *to = v;
        }
      }
      if (*bad_v && live) {
        // elements of visible nodes' V that are not finite, left out of P V
        for (int n = 0; n < T; ++n) {
          if (!((tp.anc[t][n >> 5] >> (n & 31)) & 1u)) continue;
          const int slot = P + n, u = (slot - c_begin * kBN) / kSub;
          if (slot < c_begin * kBN || u >= nsub || (kPair && !two && (u & 1) != w)) continue;
          const int pg = trow[slot / a.page];
          if (pg < 0 || pg >= a.pool) continue;
          const uint16_t* v = a.v_pages + ((size_t(pg) * a.Hkv + hk) * a.page + slot % a.page) * DH;
          for (int e = half * (DH / 2); e < (half + 1) * (DH / 2); ++e)
            if (!bf16_finite(v[e])) sO[e] += bf16_to_f32(v[e]);
        }
      }
    }
    if (kPair && !two) {
      if (w == 0) fixed_bar_sync<kAllBar, C::kSoftThreads>();
      else if (half == 0) sML[r] = both;                 // every thread has read the streams' own
    }

    // ----------------- join the streams and splits of each row -----------------
    __syncwarp();
    cluster_sync();                      // every split's streams are staged
    const int np = a.splits;                             // a row's partial results
    const int ntok = min(two ? 2 * a.tpt : a.tpt, T - tok0);
    const int rows = ntok * a.G;                         // dense over the unit's (node, head) pairs
    const int tile_rows = a.tpt * a.G;
    const int crank = int(cluster_ctarank());
    const int r0 = rows * crank / a.splits, r1 = rows * (crank + 1) / a.splits;
    const int tid = threadIdx.x - (C::kThreads - C::kSoftThreads);
    // This code runs once a CTA, so what it costs is fetching it: loops stay rolled.
    // Weights of the partial results first: sW[row][p] = 2^(m_p - m) / L, or -1 where
    // nothing was staged; from (m, sum) of every partial, copied to sP[row][p].
    float2* sP = sML + STREAMS * kBM;
    float* sW = reinterpret_cast<float*>(sP + STREAMS * kBM + 2 * kMaxSplits);
    const int nw = (r1 - r0) * np;
    if (tid < nw) {                                      // at most 2 * 128 + 16 pairs
      const int i = tid / np, p = tid - i * np;
      const int w0 = (r0 + i) / tile_rows, row = r0 + i - w0 * tile_rows;   // stream (two tiles) and row in it
      sP[tid] = ld_cluster_f2(mapa_shared(smem_u32(&sML[w0 * kBM + row]), uint32_t(p)));
    }
    fixed_bar_sync<kAllBar, C::kSoftThreads>();
    if (tid < nw) {
      const int i = tid / np;
      float mx = -INFINITY, L = 0.f;
#pragma unroll 2
      for (int p = 0; p < np; ++p) mx = fmaxf(mx, sP[i * np + p].x);
#pragma unroll 2
      for (int p = 0; p < np; ++p) {
        const float2 ml = sP[i * np + p];
        L += ml.x == -INFINITY ? 0.f : ml.y * exp2_sfu(ml.x - mx);
      }
      const float m = sP[tid].x;
      sW[tid] = m == -INFINITY ? -1.f : exp2_sfu(m - mx) / L;
    }
    fixed_bar_sync<kAllBar, C::kSoftThreads>();
    // rows as float4 columns, up to kP of a thread's loads from the cluster in flight
    constexpr int kF4 = DH / 4, kP = 8;
    const int items = (r1 - r0) * kF4;
#pragma unroll 1
    for (int i = tid; i < items; i += C::kSoftThreads) {
      const int pr = r0 + i / kF4;                       // (node, head) pair of the unit
      const int w0 = pr / tile_rows, row = pr - w0 * tile_rows;
      const float* sw = sW + (i / kF4) * np;
      const uint32_t src = smem_u32(smem) + uint32_t(((w0 * kBM + row) * C::kLd + (i % kF4) * 4) * 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int p0 = 0; p0 < np; p0 += kP) {
        float4 o[kP];
        float wgt[kP];
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          const int p = p0 + e;
          wgt[e] = p < np ? sw[p] : -1.f;
          o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (!(wgt[e] < 0.f)) o[e] = ld_cluster_f4(mapa_shared(src, uint32_t(p)));
        }
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          const float x = wgt[e] < 0.f ? 0.f : wgt[e];
          acc.x = fmaf(o[e].x, x, acc.x);
          acc.y = fmaf(o[e].y, x, acc.y);
          acc.z = fmaf(o[e].z, x, acc.z);
          acc.w = fmaf(o[e].w, x, acc.w);
        }
      }
      if (bad) acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const size_t at = ((size_t(b) * T + tok0 + pr / a.G) * a.Hq + hk * a.G + pr % a.G) * DH + (i % kF4) * 4;
      if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = acc;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
    __syncwarp();
    cluster_sync();                      // peers are done reading this CTA's shared memory
  }
  if (warp < 4) {                        // the other warps' part of the softmax warps' two cluster barriers
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace attn_paged
}  // namespace md
