// libmedusa: C ABI entry points (validation, launch planning, launches).
//
// One translation unit holds every kernel so that the device status word is a
// single module-scope variable without relocatable device code.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <utility>

#include "common.cuh"
#include "heads.cuh"
#include "heads_gemm.cuh"
#include "heads_gemm2.cuh"
#include "heads_skinny.cuh"
#include "tree_build.cuh"
#include "attention.cuh"
#include "attention_tc.cuh"
#include "accept.cuh"
#include "commit.cuh"
#include "append.cuh"
#include "attention_paged.cuh"
#include "commit_paged.cuh"
#include "pages.cuh"
#include "hydra.cuh"
#include "reject.cuh"

struct md_tree {
  md::TreeParams tp;
  int32_t K;
  int32_t kph[MD_MAX_K];
};

namespace {

using md::TreeParams;

constexpr int kMaxDevices = 64;

// Host caches below are filled lazily and may be filled by several threads at
// once; each writer stores the same value, and atomics make that well defined.
int num_sms() {
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

md_status cuda_ok(cudaError_t e) {
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MD_ERR_CUDA;
  }
  return MD_OK;
}

md_status last_launch() { return cuda_ok(cudaGetLastError()); }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> cached{nullptr};
  EncodeTiledFn fn = cached.load(std::memory_order_acquire);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<EncodeTiledFn>(p);
      cached.store(fn, std::memory_order_release);
    }
  }
  return fn;
}

// 2-D bf16 tensor map over a row-major [rows, cols] matrix; box [box_rows, box_cols].
md_status make_map_2d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                      uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MD_ERR_CUDA;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MD_OK : MD_ERR_CUDA;
}

// Launch with programmatic stream serialization: the kernel may be scheduled
// while its predecessor on the stream finishes; it waits (griddepcontrol.wait)
// before reading anything the predecessor writes.
template <typename... KArgs, typename... Args>
md_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t st,
                     Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

// The top-k merge is launched in plain stream order: as a dependent launch
// (which lets its CTAs start and wait beside the still-running projection)
// the calls ran slower, although the merge alone is faster (a four-level
// Hydra draft at 70B shapes took 1.50 ms that way against 1.46 ms in plain
// order; more shared memory per merge CTA or a later trigger did not change
// it). The kernel's own griddepcontrol instructions are no-ops in this form,
// and the launch after it can still be a dependent one.
inline md_status launch_merge(const md::heads::MergeArgs& ma, int blocks, cudaStream_t st) {
  md::heads::heads_merge_kernel<<<blocks, md::heads::kMergeThreads, 0, st>>>(ma);
  return cuda_ok(cudaGetLastError());
}

template <typename Kernel>
md_status set_smem(Kernel k, int bytes) {
  return cuda_ok(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

// ----------------------------- heads launchers -----------------------------

// One epoch per call of the streaming heads kernels: their tickets carry it
// (epoch_arrive), so the workspace needs no clearing between calls and the
// first kernel is launched dependent on the kernel before it. Never 0, so
// zeroed memory holds no epoch.
uint32_t next_epoch() {
  static std::atomic<uint32_t> counter{0};
  uint32_t e;
  do {
    e = counter.fetch_add(1, std::memory_order_relaxed) + 1u;
  } while (e == 0);
  return e;
}

template <int M>
md_status launch_heads(const md::heads::Plan& pl, const md_bf16* h, const md_bf16* W1, const md_bf16* b1,
                       const md_bf16* Wv, const int32_t* kph, int32_t* topk_ids, float* topk_vals, float* logits_dbg,
                       const float* gumbel_u, float inv_tau, uint8_t* ws, cudaStream_t st) {
  using namespace md::heads;
  md_status s;
  // phase 1
  W1Args wa;
  wa.h = h; wa.W1 = W1; wa.b1 = b1;
  wa.zt = reinterpret_cast<uint16_t*>(ws + pl.off_zt);
  wa.part = reinterpret_cast<float*>(ws + pl.off_part);
  wa.counters = reinterpret_cast<unsigned long long*>(ws + pl.off_cnt);
  wa.d = pl.d; wa.K = pl.K; wa.splits = pl.splits; wa.rows = pl.rows; wa.ntile_o = pl.ntile_o;
  wa.shared = 0;
  wa.epoch = next_epoch();
  const int w1_smem = pl.rows * 16 + kConsumerWarps * M * kW1TileO * 4;
  if ((s = set_smem(heads_w1_kernel<M>, w1_smem)) != MD_OK) return s;
  if ((s = launch_pdl(heads_w1_kernel<M>, dim3(pl.ntile_o, pl.splits, pl.K), dim3(kW1Threads), w1_smem, st, wa)) !=
      MD_OK)
    return s;

  // phase 2 (programmatic dependent launch: its TMA of Wv may start before phase 1 ends)
  CUtensorMap map;
  if ((s = make_map_2d(&map, Wv, uint64_t(pl.V), uint64_t(pl.K) * pl.d, kTileV, kStageRows)) != MD_OK) return s;
  VocabArgs va;
  va.zt = wa.zt;
  va.cand_val = reinterpret_cast<float*>(ws + pl.off_cval);
  va.cand_id = reinterpret_cast<int*>(ws + pl.off_cid);
  va.logits_dbg = logits_dbg;
  va.gumbel_u = gumbel_u;
  va.inv_tau = inv_tau;
  va.stream_k = pl.stream_k;
  va.tickets = reinterpret_cast<unsigned long long*>(ws + pl.off_tick);
  va.epoch = wa.epoch;
  va.spart = reinterpret_cast<float*>(ws + pl.off_spart);
  va.d = pl.d; va.V = pl.V; va.K = pl.K; va.kmax = pl.kmax; va.ntiles = pl.ntiles; va.units = pl.units;
  va.nstages = pl.nstages;
  va.shared = 0; va.kh = pl.K;
  for (int k = 0; k < MD_MAX_K; ++k) va.kph[k] = k < pl.K ? kph[k] : 0;
  const int v_smem = vocab_smem_bytes(M, pl.nstages);
  if ((s = set_smem(heads_vocab_kernel<M>, v_smem)) != MD_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.grid);
  cfg.blockDim = dim3((kConsumerWarps + 1) * 32);
  cfg.dynamicSmemBytes = v_smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((s = cuda_ok(cudaLaunchKernelEx(&cfg, heads_vocab_kernel<M>, map, va))) != MD_OK) return s;

  // phase 3
  MergeArgs ma;
  ma.cand_val = va.cand_val; ma.cand_id = va.cand_id;
  ma.topk_ids = topk_ids; ma.topk_vals = topk_vals;
  ma.K = pl.K; ma.kmax = pl.kmax; ma.nslots = pl.grid;
  ma.partitioned = 1; ma.units = pl.units; ma.ntiles = pl.ntiles; ma.kh = pl.K;
  ma.stages = va.stream_k ? pl.d / kStageRows : 0;
  for (int k = 0; k < MD_MAX_K; ++k) ma.kph[k] = va.kph[k];
  md::heads::set_merge_ranges(ma);
  return launch_merge(ma, pl.M * pl.K, st);
}

// Workspace of the tensor-core path: z [K, M, d] bf16 and the candidates
// [M, K, per_mt2, kmax] (one list per row, head and CTA / CTA pair of the
// row's tile). More than one 128-row tile: CTA pairs (256-row tiles).
struct GemmPlan {
  int mtiles, ntiles1, ntiles2;
  bool pair;              // CTA-pair kernel (M > 128)
  int groups;             // row tiles (single CTAs) or row-tile pairs (pairs)
  int cluster;            // pair kernel: CTAs per cluster (2), else 0
  int per_mt1, per_mt2;   // CTAs (pairs) per group of the two GEMMs
  int grid1, grid2;
  size_t off_z, off_cval, off_cid, bytes;
};

// Clusters of `cs` CTAs of the pair kernel that can be resident at once
// (0 when such a cluster cannot be placed).
int pair_max_clusters(int cs) {
  static std::mutex mu;
  static int cache[9] = {-1, -1, -1, -1, -1, -1, -1, -1, -1};
  std::lock_guard<std::mutex> lock(mu);
  if (cache[cs] >= 0) return cache[cs];
  auto kern = md::gemm::heads_gemm_pair_kernel<md::gemm::EPI_TOPK, 16>;
  int n = 0;
  if (set_smem(kern, md::gemm::kSmemP) == MD_OK) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cs * 64);
    cfg.blockDim = dim3(md::gemm::kThreads);
    cfg.dynamicSmemBytes = md::gemm::kSmemP;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
  }
  cache[cs] = n;
  return n;
}

// CTAs (pairs) per group: as many as can be resident side by side with the
// other groups, at most one per (head, column tile) unit.
inline int gemm_per_mt(int slots, int groups, int units) { return std::max(1, std::min(slots / groups, units)); }

GemmPlan gemm_plan(int M, int d, int V, int K, int kmax) {
  using md::heads::align256;
  GemmPlan p;
  p.mtiles = (M + md::gemm::kBM - 1) / md::gemm::kBM;
  p.ntiles1 = (d + md::gemm::kBN - 1) / md::gemm::kBN;
  p.ntiles2 = (V + md::gemm::kBN - 1) / md::gemm::kBN;
  p.pair = p.mtiles > 1;
  p.groups = p.pair ? (p.mtiles + 1) / 2 : p.mtiles;
  int slots = num_sms();
  p.cluster = 0;
  if (p.pair) {
    // one cluster per pair: clusters of all the row-pair groups of a unit range
    // (one GPC) measured slower, with fewer resident CTAs and no fewer HBM reads
    p.cluster = 2;
    slots = std::max(1, pair_max_clusters(p.cluster));   // resident pairs
  }
  p.per_mt1 = gemm_per_mt(slots, p.groups, K * p.ntiles1);
  p.per_mt2 = gemm_per_mt(slots, p.groups, K * p.ntiles2);
  p.grid1 = p.groups * p.per_mt1 * (p.pair ? 2 : 1);
  p.grid2 = p.groups * p.per_mt2 * (p.pair ? 2 : 1);
  size_t o = 0;
  p.off_z = o;    o = align256(o + size_t(K) * M * d * 2);
  p.off_cval = o; o = align256(o + size_t(M) * K * p.per_mt2 * kmax * 4);
  p.off_cid = o;  o = align256(o + size_t(M) * K * p.per_mt2 * kmax * 4);
  p.bytes = o;
  return p;
}

// 3-D bf16 tensor map over [n2][n1][n0] (n0 contiguous), box [1][b1][b0], 128-byte swizzle.
md_status make_map_3d_sw128(CUtensorMap* map, const void* base, uint64_t n0, uint64_t n1, uint64_t n2, uint32_t b0,
                            uint32_t b1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MD_ERR_CUDA;
  cuuint64_t dims[3] = {n0, n1, n2};
  cuuint64_t strides[2] = {n0 * 2, n0 * n1 * 2};
  cuuint32_t box[3] = {b0, b1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MD_OK : MD_ERR_CUDA;
}

template <int EPI, int KK>
md_status launch_gemm(const CUtensorMap& amap, const CUtensorMap& bmap, const md::gemm::Args& ga, int grid,
                      int cluster, bool pdl, cudaStream_t st) {
  md_status s;
  const bool pair = cluster > 0;
  auto kern = pair ? md::gemm::heads_gemm_pair_kernel<EPI, KK> : md::gemm::heads_gemm_kernel<EPI, KK>;
  const int smem = pair ? md::gemm::kSmemP : md::gemm::kSmem;
  if ((s = set_smem(kern, smem)) != MD_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(md::gemm::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kern, amap, bmap, ga));
}

template <int KK>
md_status launch_heads_gemm(int M, int d, int V, int K, int kmax, const md_bf16* h, const md_bf16* W1,
                            const md_bf16* b1, const md_bf16* Wv, const int32_t* kph, int32_t* topk_ids,
                            float* topk_vals, float* logits_dbg, const float* gumbel_u, float inv_tau, uint8_t* ws,
                            cudaStream_t st) {
  using namespace md::gemm;
  const GemmPlan pl = gemm_plan(M, d, V, K, kmax);
  md_status s;
  Args ga = {};
  ga.M = M; ga.d = d; ga.K = K; ga.kmax = kmax;
  ga.h = h; ga.b1 = b1;
  ga.zg = reinterpret_cast<uint16_t*>(ws + pl.off_z);
  ga.cand_val = reinterpret_cast<float*>(ws + pl.off_cval);
  ga.cand_id = reinterpret_cast<int*>(ws + pl.off_cid);
  ga.logits_dbg = logits_dbg;
  for (int k = 0; k < MD_MAX_K; ++k) ga.kph[k] = k < K ? kph[k] : 0;

  // phase 1: z = bf16(h + SiLU(h W1_k + b1_k))
  CUtensorMap amap, bmap;
  if ((s = make_map_3d_sw128(&amap, h, d, M, 1, kBK, kBM)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&bmap, W1, d, d, K, 64, kBK)) != MD_OK) return s;
  ga.N = d; ga.ntiles = pl.ntiles1; ga.per_mt = pl.per_mt1; ga.groups = pl.groups; ga.a_shared = 1;
  if ((s = launch_gemm<EPI_SILU, KK>(amap, bmap, ga, pl.grid1, pl.cluster, false, st)) != MD_OK) return s;

  // phase 2: logits tile = z_k Wv_k, per-row top-k of every 256-column tile
  if ((s = make_map_3d_sw128(&amap, ga.zg, d, M, K, kBK, kBM)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&bmap, Wv, V, d, K, 64, kBK)) != MD_OK) return s;
  ga.N = V; ga.ntiles = pl.ntiles2; ga.per_mt = pl.per_mt2; ga.groups = pl.groups; ga.a_shared = 0;
  ga.gumbel_u = gumbel_u;
  ga.inv_tau = inv_tau;
  if ((s = launch_gemm<EPI_TOPK, KK>(amap, bmap, ga, pl.grid2, pl.cluster, true, st)) != MD_OK) return s;

  // phase 3: merge the tiles' candidates
  md::heads::MergeArgs ma;
  ma.cand_val = ga.cand_val; ma.cand_id = ga.cand_id;
  ma.topk_ids = topk_ids; ma.topk_vals = topk_vals;
  ma.K = K; ma.kmax = kmax; ma.nslots = pl.per_mt2;
  ma.partitioned = 1; ma.units = K * pl.ntiles2; ma.ntiles = pl.ntiles2; ma.kh = K;
  ma.stages = 0;
  for (int k = 0; k < MD_MAX_K; ++k) ma.kph[k] = ga.kph[k];
  md::heads::set_merge_ranges(ma);
  return launch_merge(ma, M * K, st);
}

// ---------------- tensor-core heads with the weights as M (2 .. 32 rows) ----------------
// Workspace: z [K, NR, d] bf16, two partial-sum slots per CTA, one ticket per
// unit of both phases, and the phase-2 candidates [M, K, G2, kmax].
struct SkinnyPlan {
  int NR;                  // rows padded to 16 or 32 (the MMA's N)
  int S, nt1, nt2;         // stages per unit, column tiles of phase 1 (d) and phase 2 (V)
  int G1, G2;              // CTAs of the two phases
  size_t off_z, off_part, off_tick, off_cval, off_cid, bytes;
};

inline bool skinny_rows(int M) { return M >= md::skinny::kMinRows && M <= md::skinny::kMaxRows; }

// The CUDA-core stream serves one row; from two rows the tensor cores (its
// FMA work grows with M: 1.50 vs 1.32 ms at two rows of 70B heads); from 33
// rows the 128-row GEMM tiles (1.44 ms at 65 rows against 1.48 ms for the
// weights-as-M kernel at 64: N = 64 leaves four stages and a heavier epilogue).
inline bool stream_rows(int M) { return M < md::skinny::kMinRows; }

SkinnyPlan skinny_plan(int M, int d, int V, int K, int kmax) {
  using md::heads::align256;
  SkinnyPlan p;
  p.NR = M <= 16 ? 16 : 32;
  p.S = d / md::skinny::kBK;
  p.nt1 = (d + md::skinny::kTile - 1) / md::skinny::kTile;
  p.nt2 = (V + md::skinny::kTile - 1) / md::skinny::kTile;
  p.G1 = int(std::min<long long>(num_sms(), (long long)K * p.nt1 * p.S));
  p.G2 = int(std::min<long long>(num_sms(), (long long)K * p.nt2 * p.S));
  size_t o = 0;
  p.off_z = o;    o = align256(o + size_t(K) * p.NR * d * 2);
  p.off_part = o; o = align256(o + size_t(std::max(p.G1, p.G2)) * 2 * M * md::skinny::kTile * 4);
  p.off_tick = o; o = align256(o + size_t(K) * (p.nt1 + p.nt2) * 8);   // epoch tickets
  p.off_cval = o; o = align256(o + size_t(M) * K * p.G2 * kmax * 4);
  p.off_cid = o;  o = align256(o + size_t(M) * K * p.G2 * kmax * 4);
  p.bytes = o;
  return p;
}

template <int EPI, int NR>
md_status launch_skinny(const CUtensorMap& wmap, const CUtensorMap& xmap, const md::skinny::Args& a, int grid,
                        bool pdl, cudaStream_t st) {
  auto kern = md::skinny::heads_skinny_kernel<EPI, NR>;
  const int smem = md::skinny::Cfg<NR>::kSmem;
  md_status s;
  if ((s = set_smem(kern, smem)) != MD_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(md::skinny::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kern, wmap, xmap, a));
}

template <int NR>
md_status launch_heads_skinny(const SkinnyPlan& pl, int M, int d, int V, int K, int kmax, const md_bf16* h,
                              const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv, const int32_t* kph,
                              int32_t* topk_ids, float* topk_vals, float* logits_dbg, const float* gumbel_u,
                              float inv_tau, uint8_t* ws, cudaStream_t st) {
  using namespace md::skinny;
  md_status s;
  Args a = {};
  a.M = M; a.d = d; a.Kh = K; a.S = pl.S; a.kmax = kmax; a.kh = 0;
  a.h = h; a.b1 = b1;
  a.z = reinterpret_cast<uint16_t*>(ws + pl.off_z);
  a.NRz = NR; a.zg_mk = 0;
  a.part = reinterpret_cast<float*>(ws + pl.off_part);
  unsigned long long* tick = reinterpret_cast<unsigned long long*>(ws + pl.off_tick);
  a.epoch = next_epoch();      // both phases' tickets (distinct words): nothing to clear
  for (int k = 0; k < MD_MAX_K; ++k) a.kph[k] = k < K ? kph[k] : 0;

  // phase 1: z = bf16(h + SiLU(h W1_k + b1_k)) -- W1_k^T as the MMA's A, h^T as its B
  CUtensorMap wmap, xmap;
  if ((s = make_map_3d_sw128(&wmap, W1, d, d, K, 64, kBK)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&xmap, h, d, M, 1, kBK, NR)) != MD_OK) return s;
  a.N = d; a.ntiles = pl.nt1; a.tickets = tick;
  if ((s = launch_skinny<EPI_SILU, NR>(wmap, xmap, a, pl.G1, true, st)) != MD_OK) return s;

  // phase 2: logits = z_k Wv_k, running top-k per (row, head, CTA)
  if ((s = make_map_3d_sw128(&wmap, Wv, V, d, K, 64, kBK)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&xmap, a.z, d, NR, K, kBK, NR)) != MD_OK) return s;
  a.N = V; a.ntiles = pl.nt2; a.tickets = tick + size_t(K) * pl.nt1;
  a.cand_val = reinterpret_cast<float*>(ws + pl.off_cval);
  a.cand_id = reinterpret_cast<int*>(ws + pl.off_cid);
  a.logits_dbg = logits_dbg; a.gumbel_u = gumbel_u; a.inv_tau = inv_tau;
  if ((s = launch_skinny<EPI_TOPK, NR>(wmap, xmap, a, pl.G2, true, st)) != MD_OK) return s;

  // phase 3: merge the CTAs' lists
  md::heads::MergeArgs ma;
  ma.cand_val = a.cand_val; ma.cand_id = a.cand_id;
  ma.topk_ids = topk_ids; ma.topk_vals = topk_vals;
  ma.K = K; ma.kmax = kmax; ma.nslots = pl.G2;
  ma.partitioned = 1; ma.units = K * pl.nt2; ma.ntiles = pl.nt2; ma.kh = K;
  ma.stages = pl.S;
  for (int k = 0; k < MD_MAX_K; ++k) ma.kph[k] = a.kph[k];
  md::heads::set_merge_ranges(ma);
  return launch_merge(ma, M * K, st);
}

// ------------------- shared vocabulary projection (one Wv) -------------------
// Phase 1 is the per-head residual block; phase 2 treats the M*K rows
// (m, k) -> m*K + k as rows of one head against the single projection.

struct SharedPlan {
  bool stream;                 // M*K == 1: CUDA-core weight stream
  bool skinny;                 // 2 <= M*K <= 32: tensor cores with the weights as M; else row-tile GEMMs
  md::heads::Plan p1, p2;      // streaming: phase-1 plan (M rows, K heads), phase-2 plan (M*K rows, 1 head)
  GemmPlan g1, g2;             // tensor cores: phase 1 (M rows, K heads), phase 2 (M*K rows, 1 head)
  size_t off2, bytes;
  size_t tick2, spart2, cval2, cid2;   // streaming: phase-2 tickets, partials, candidates (from off2)
  // weights as M: rows padded to NR1 (phase 1, M) and NR2 (phase 2, M*K)
  int NR1, NR2, S, nt1, nt2, G1, G2;
  size_t off_z, off_part, off_tick, off_cval, off_cid;
};

inline int skinny_pad(int rows) { return rows <= 16 ? 16 : 32; }

SharedPlan shared_plan(int M, int d, int V, int K, int kmax) {
  using md::heads::align256;
  SharedPlan p{};
  p.stream = M * K == 1;
  p.skinny = !p.stream && skinny_rows(M * K);
  if (p.skinny) {
    p.NR1 = skinny_pad(M);
    p.NR2 = skinny_pad(M * K);
    p.S = d / md::skinny::kBK;
    p.nt1 = (d + md::skinny::kTile - 1) / md::skinny::kTile;
    p.nt2 = (V + md::skinny::kTile - 1) / md::skinny::kTile;
    p.G1 = int(std::min<long long>(num_sms(), (long long)K * p.nt1 * p.S));
    p.G2 = int(std::min<long long>(num_sms(), (long long)p.nt2 * p.S));
    size_t o = 0;
    p.off_z = o;    o = align256(o + size_t(p.NR2) * d * 2);
    p.off_part = o; o = align256(o + size_t(std::max(p.G1, p.G2)) * 2 * (M * K) * md::skinny::kTile * 4);
    p.off_tick = o; o = align256(o + size_t(K * p.nt1 + p.nt2) * 8);   // epoch tickets
    p.off_cval = o; o = align256(o + size_t(M) * K * p.G2 * kmax * 4);
    p.off_cid = o;  o = align256(o + size_t(M) * K * p.G2 * kmax * 4);
    p.bytes = o;
  } else if (p.stream) {
    p.p1 = md::heads::make_plan(M, d, V, K, kmax, num_sms());
    p.p2 = md::heads::make_plan(M * K, d, V, 1, kmax, num_sms());
    p.off2 = align256(p.p1.off_cval);                    // phase-2 data after phase-1 data
    p.tick2 = 0;
    p.spart2 = p.p2.off_spart - p.p2.off_tick;
    p.cval2 = p.p2.off_cval - p.p2.off_tick;
    p.cid2 = p.p2.off_cid - p.p2.off_tick;
    p.bytes = p.off2 + (p.p2.bytes - p.p2.off_tick);
  } else {
    p.g1 = gemm_plan(M, d, V, K, kmax);                   // z [M*K, d] lives at g1.off_z
    p.g2 = gemm_plan(M * K, d, V, 1, kmax);
    p.off2 = align256(p.g1.off_z + size_t(K) * M * d * 2);
    p.bytes = p.off2 + (p.g2.bytes - p.g2.off_cval);
  }
  return p;
}

// One projection for all heads on the tensor cores with the weights as M:
// phase 1 is the K heads' residual blocks on the M rows (z row (m, k) written
// to row m*K + k), phase 2 one head over the M*K rows, row m*K + k keeping
// head k's top-k size.
template <int NR1, int NR2>
md_status launch_heads_shared_skinny(const SharedPlan& sp, int M, int d, int V, int K, int kmax, const md_bf16* h,
                                     const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv, const int32_t* kph,
                                     int32_t* topk_ids, float* topk_vals, float* logits_dbg, uint8_t* ws,
                                     cudaStream_t st) {
  using namespace md::skinny;
  md_status s;
  Args a = {};
  a.d = d; a.S = sp.S; a.kmax = kmax;
  a.h = h; a.b1 = b1;
  a.z = reinterpret_cast<uint16_t*>(ws + sp.off_z);
  a.NRz = NR2; a.zg_mk = 1;
  a.part = reinterpret_cast<float*>(ws + sp.off_part);
  unsigned long long* tick = reinterpret_cast<unsigned long long*>(ws + sp.off_tick);
  a.epoch = next_epoch();      // both phases' tickets (distinct words): nothing to clear
  for (int k = 0; k < MD_MAX_K; ++k) a.kph[k] = k < K ? kph[k] : 0;

  CUtensorMap wmap, xmap;
  if ((s = make_map_3d_sw128(&wmap, W1, d, d, K, 64, kBK)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&xmap, h, d, M, 1, kBK, NR1)) != MD_OK) return s;
  a.M = M; a.Kh = K; a.N = d; a.ntiles = sp.nt1; a.tickets = tick; a.kh = 0;
  if ((s = launch_skinny<EPI_SILU, NR1>(wmap, xmap, a, sp.G1, true, st)) != MD_OK) return s;

  if ((s = make_map_3d_sw128(&wmap, Wv, V, d, 1, 64, kBK)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&xmap, a.z, d, NR2, 1, kBK, NR2)) != MD_OK) return s;
  a.M = M * K; a.Kh = 1; a.N = V; a.ntiles = sp.nt2; a.tickets = tick + size_t(K) * sp.nt1; a.kh = K;
  a.zg_mk = 0;
  a.cand_val = reinterpret_cast<float*>(ws + sp.off_cval);
  a.cand_id = reinterpret_cast<int*>(ws + sp.off_cid);
  a.logits_dbg = logits_dbg; a.gumbel_u = nullptr; a.inv_tau = 1.f;
  if ((s = launch_skinny<EPI_TOPK, NR2>(wmap, xmap, a, sp.G2, true, st)) != MD_OK) return s;

  md::heads::MergeArgs ma;
  ma.cand_val = a.cand_val; ma.cand_id = a.cand_id;
  ma.topk_ids = topk_ids; ma.topk_vals = topk_vals;
  ma.K = 1; ma.kmax = kmax; ma.nslots = sp.G2;
  ma.partitioned = 1; ma.units = sp.nt2; ma.ntiles = sp.nt2; ma.kh = K;
  ma.stages = sp.S;
  for (int k = 0; k < MD_MAX_K; ++k) ma.kph[k] = a.kph[k];
  md::heads::set_merge_ranges(ma);
  return launch_merge(ma, M * K, st);
}

template <int MK>
md_status launch_heads_shared_stream(const SharedPlan& sp, int M, const md_bf16* h, const md_bf16* W1,
                                     const md_bf16* b1, const md_bf16* Wv, const int32_t* kph, int32_t* topk_ids,
                                     float* topk_vals, float* logits_dbg, uint8_t* ws, cudaStream_t st) {
  using namespace md::heads;
  const Plan& p1 = sp.p1;
  const Plan& p2 = sp.p2;
  md_status s;
  W1Args wa;
  wa.h = h; wa.W1 = W1; wa.b1 = b1;
  wa.zt = reinterpret_cast<uint16_t*>(ws + p1.off_zt);
  wa.part = reinterpret_cast<float*>(ws + p1.off_part);
  wa.counters = reinterpret_cast<unsigned long long*>(ws + p1.off_cnt);
  wa.d = p1.d; wa.K = p1.K; wa.splits = p1.splits; wa.rows = p1.rows; wa.ntile_o = p1.ntile_o;
  wa.shared = 1;
  wa.epoch = next_epoch();     // phase-1 counters and the shared projection's tickets (its own plan p2)
  auto run_w1 = [&](auto kern, int smem) -> md_status {
    md_status r;
    if ((r = set_smem(kern, smem)) != MD_OK) return r;
    return launch_pdl(kern, dim3(p1.ntile_o, p1.splits, p1.K), dim3(kW1Threads), smem, st, wa);
  };
  switch (M) {   // phase-1 rows (M * K <= 4)
    case 1: s = run_w1(heads_w1_kernel<1>, p1.rows * 16 + kConsumerWarps * 1 * kW1TileO * 4); break;
    case 2: s = run_w1(heads_w1_kernel<2>, p1.rows * 16 + kConsumerWarps * 2 * kW1TileO * 4); break;
    case 3: s = run_w1(heads_w1_kernel<3>, p1.rows * 16 + kConsumerWarps * 3 * kW1TileO * 4); break;
    case 4: s = run_w1(heads_w1_kernel<4>, p1.rows * 16 + kConsumerWarps * 4 * kW1TileO * 4); break;
    default: return MD_ERR_UNSUPPORTED;
  }
  if (s != MD_OK) return s;
  CUtensorMap map;
  if ((s = make_map_2d(&map, Wv, uint64_t(p2.V), uint64_t(p2.d), kTileV, kStageRows)) != MD_OK) return s;
  VocabArgs va;
  va.zt = wa.zt;
  va.cand_val = reinterpret_cast<float*>(ws + sp.off2 + sp.cval2);
  va.cand_id = reinterpret_cast<int*>(ws + sp.off2 + sp.cid2);
  va.logits_dbg = logits_dbg;
  va.gumbel_u = nullptr;
  va.inv_tau = 1.f;
  va.stream_k = p2.stream_k;
  va.tickets = reinterpret_cast<unsigned long long*>(ws + sp.off2 + sp.tick2);
  va.epoch = wa.epoch;
  va.spart = reinterpret_cast<float*>(ws + sp.off2 + sp.spart2);
  va.d = p2.d; va.V = p2.V; va.K = 1; va.kmax = p2.kmax; va.ntiles = p2.ntiles; va.units = p2.units;
  va.nstages = p2.nstages;
  va.shared = 1; va.kh = p1.K;
  for (int k = 0; k < MD_MAX_K; ++k) va.kph[k] = k < p1.K ? kph[k] : 0;
  const int v_smem = vocab_smem_bytes(MK, p2.nstages);
  if ((s = set_smem(heads_vocab_kernel<MK>, v_smem)) != MD_OK) return s;
  if ((s = launch_pdl(heads_vocab_kernel<MK>, dim3(p2.grid), dim3((kConsumerWarps + 1) * 32), v_smem, st, map,
                      va)) != MD_OK)
    return s;
  MergeArgs ma;
  ma.cand_val = va.cand_val; ma.cand_id = va.cand_id;
  ma.topk_ids = topk_ids; ma.topk_vals = topk_vals;
  ma.K = 1; ma.kmax = p2.kmax; ma.nslots = p2.grid;
  ma.partitioned = 1; ma.units = p2.units; ma.ntiles = p2.ntiles; ma.kh = p1.K;
  ma.stages = va.stream_k ? p2.d / kStageRows : 0;
  for (int k = 0; k < MD_MAX_K; ++k) ma.kph[k] = va.kph[k];
  md::heads::set_merge_ranges(ma);
  return launch_merge(ma, MK, st);
}

template <int KK>
md_status launch_heads_shared_gemm(const SharedPlan& sp, int M, int d, int V, int K, int kmax, const md_bf16* h,
                                   const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv, const int32_t* kph,
                                   int32_t* topk_ids, float* topk_vals, float* logits_dbg, uint8_t* ws,
                                   cudaStream_t st) {
  using namespace md::gemm;
  md_status s;
  const int MK = M * K;
  Args ga = {};
  ga.d = d; ga.kmax = kmax; ga.h = h; ga.b1 = b1;
  ga.zg = reinterpret_cast<uint16_t*>(ws + sp.g1.off_z);
  ga.cand_val = reinterpret_cast<float*>(ws + sp.off2);
  ga.cand_id = reinterpret_cast<int*>(ws + sp.off2 + (sp.g2.off_cid - sp.g2.off_cval));
  ga.logits_dbg = logits_dbg;
  for (int k = 0; k < MD_MAX_K; ++k) ga.kph[k] = k < K ? kph[k] : 0;
  // phase 1: per-head residual blocks, z rows written in (row, head) order
  CUtensorMap amap, bmap;
  if ((s = make_map_3d_sw128(&amap, h, d, M, 1, kBK, kBM)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&bmap, W1, d, d, K, 64, kBK)) != MD_OK) return s;
  ga.M = M; ga.K = K; ga.N = d; ga.ntiles = sp.g1.ntiles1; ga.per_mt = sp.g1.per_mt1; ga.groups = sp.g1.groups;
  ga.a_shared = 1; ga.zg_mk = 1; ga.kh = 0;
  if ((s = launch_gemm<EPI_SILU, KK>(amap, bmap, ga, sp.g1.grid1, sp.g1.cluster, false, st)) != MD_OK) return s;
  // phase 2: the M*K rows against the one projection
  if ((s = make_map_3d_sw128(&amap, ga.zg, d, MK, 1, kBK, kBM)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&bmap, Wv, V, d, 1, 64, kBK)) != MD_OK) return s;
  ga.M = MK; ga.K = 1; ga.N = V; ga.ntiles = sp.g2.ntiles2; ga.per_mt = sp.g2.per_mt2; ga.groups = sp.g2.groups;
  ga.a_shared = 1; ga.zg_mk = 0; ga.kh = K;
  if ((s = launch_gemm<EPI_TOPK, KK>(amap, bmap, ga, sp.g2.grid2, sp.g2.cluster, true, st)) != MD_OK) return s;
  md::heads::MergeArgs ma;
  ma.cand_val = ga.cand_val; ma.cand_id = ga.cand_id;
  ma.topk_ids = topk_ids; ma.topk_vals = topk_vals;
  ma.K = 1; ma.kmax = kmax; ma.nslots = sp.g2.per_mt2;
  ma.partitioned = 1; ma.units = sp.g2.ntiles2; ma.ntiles = sp.g2.ntiles2; ma.kh = K;
  ma.stages = 0;
  for (int k = 0; k < MD_MAX_K; ++k) ma.kph[k] = ga.kph[k];
  md::heads::set_merge_ranges(ma);
  return launch_merge(ma, MK, st);
}

md_status heads_check(int32_t M, int32_t d, int32_t V, int32_t K, int32_t kmax) {
  if (M <= 0 || d <= 0 || V <= 0 || K <= 0 || kmax <= 0) return MD_ERR_INVALID_ARG;
  if (K > MD_MAX_K || kmax > MD_MAX_KMAX) return MD_ERR_UNSUPPORTED;
  if (M > md::gemm::kMaxM) return MD_ERR_UNSUPPORTED;
  // the merge loads every candidate of one (row, head) at once: at most one
  // list of kmax entries per producer CTA, and producers run one CTA per SM
  if (num_sms() * kmax > md::heads::kMergeCap) return MD_ERR_UNSUPPORTED;
  if (d % 64 != 0 || V % 8 != 0 || V < 256) return MD_ERR_UNSUPPORTED;
  if (size_t(K) * d >= (size_t(1) << 31) || V >= (1 << 30)) return MD_ERR_UNSUPPORTED;
  return MD_OK;
}

// ---------------------------- accept planning ------------------------------

struct AcceptPlan {
  int nchunks, chunk_len;
  size_t bytes;
};

AcceptPlan accept_plan(int B, int T, int V) {
  AcceptPlan p;
  const int rows = B * T;
  const int max_chunks = (V + 1023) / 1024;
  // as many row chunks as fit one wave of resident CTAs (~4 per SM: enough
  // loads in flight), so that no second partial wave trails the scan
  static std::atomic<int> per_sm_cache{0};
  int per_sm = per_sm_cache.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    int nb = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, md::acc::accept_rows_kernel, md::acc::kRowThreads, 0) !=
            cudaSuccess ||
        nb <= 0) {
      cudaGetLastError();
      nb = 4;
    }
    per_sm = nb;
    per_sm_cache.store(nb, std::memory_order_relaxed);
  }
  int n = per_sm * num_sms() / rows;
  n = std::max(1, std::min(n, max_chunks));
  int len = (V + n - 1) / n;
  len = (len + 1023) / 1024 * 1024;
  p.chunk_len = len;
  p.nchunks = (V + len - 1) / len;
  p.bytes = size_t(rows) * p.nchunks * md::acc::kPartFloats * 4;
  return p;
}

// --------------------------- attention planning ----------------------------

struct AttnPlan {
  bool tc;                  // tensor-core path (the GQA group divides 128)
  int G, R, max_chunks;     // CUDA-core path
  int rtiles, splits, cps;  // tensor-core path
  int ch;                   // tensor-core path: keys per chunk (64: two CTAs per SM; 128: one)
  size_t off_ml, off_cnt, bytes;
};

// Clusters of `cs` CTAs of the tensor-core attention kernel (head dim DH,
// CH-key chunks) that can be resident at once (0 when none can be placed).
template <int DH, int CH>
int attn_max_clusters(int cs) {
  static std::mutex mu;
  static int cache[md::attn_tc::kMaxSplits + 1] = {-1, -1, -1, -1, -1, -1, -1, -1, -1};
  std::lock_guard<std::mutex> lock(mu);
  if (cache[cs] >= 0) return cache[cs];
  using C = md::attn_tc::Cfg<DH, CH>;
  auto kern = md::attn_tc::attn_tc_kernel<DH, CH>;
  int n = 0;
  if (set_smem(kern, C::kSmem) == MD_OK) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cs, 64);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
  }
  cache[cs] = n;
  return n;
}

AttnPlan attn_plan(int B, int T, int Hq, int Hkv, int dh, int S_max) {
  using md::heads::align256;
  AttnPlan p;
  p.G = Hq / Hkv;
  p.R = T * p.G;
  p.tc = (128 % p.G) == 0;
  if (p.tc) {
    // One wave of CTAs: (splits x row tiles x KV heads x requests) <= #SMs.
    // (Finer splits that even out unequal prefix lengths measured slower: every
    // CTA pays a prologue and epilogue of a few chunks' time and the merge.)
    p.rtiles = (p.R + 127) / 128;
    const int base = B * Hkv * p.rtiles;
    // Chunk size. 128-key chunks issue fewer MMAs per key and win while the
    // tiles fit one wave of CTAs (70B, B = 1: 25 vs 31 us). Past one wave,
    // 64-key chunks run two CTAs per SM (one CTA's prologue and split merge
    // overlap the other's chunk loop), and win when they halve the waves
    // enough: a two-CTA wave measured ~1.7 one-CTA waves (8B sweep, B = 32:
    // 256 or 768 tiles, 8-18 % faster; B = 16 and the batched 70B, 320-384
    // tiles, 2-11 % slower).
    const int sms = num_sms();
    const int waves128 = (base + sms - 1) / sms, waves64 = (base + 2 * sms - 1) / (2 * sms);
    p.ch = (base > sms && 17 * waves64 < 10 * waves128) ? 64 : 128;
    const int chunks = (S_max + p.ch - 1) / p.ch;
    int splits = std::max(1, sms * (p.ch == 64 ? 2 : 1) / base);
    splits = std::min(std::min(splits, chunks), md::attn_tc::kMaxSplits);
    // every tile's cluster resident at once (clusters must fit a GPC, so the
    // cluster occupancy, not the SM count alone, bounds them)
    if (p.ch == 64)
      while (splits > 1 && (dh == 128 ? attn_max_clusters<128, 64>(splits) : attn_max_clusters<64, 64>(splits)) < base)
        --splits;
    p.cps = (chunks + splits - 1) / splits;
    p.splits = (chunks + p.cps - 1) / p.cps;
    p.max_chunks = chunks;
    p.off_ml = p.off_cnt = 0;
    p.bytes = 256;          // the splits merge through distributed shared memory: no scratch
  } else {
    p.rtiles = p.splits = p.cps = p.ch = 0;
    p.max_chunks = (S_max + md::attn::kChunk - 1) / md::attn::kChunk;
    const size_t rows = size_t(B) * Hkv * p.max_chunks * p.R;
    p.off_ml = align256(rows * dh * 4);
    p.off_cnt = p.bytes = p.off_ml + align256(rows * 8);
  }
  return p;
}

template <int DH, int CH>
md_status launch_attn_tc(const AttnPlan& pl, const md_bf16* q, const md_bf16* kc, const md_bf16* vc,
                         const int32_t* prefix_len, int S_max, const md_tree* tree, int B, int Hq, int Hkv, float sc,
                         float* out, void* ws, cudaStream_t st) {
  using namespace md::attn_tc;
  md_status s;
  const int T = tree->tp.T;
  CUtensorMap qmap, kmap, vmap;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MD_ERR_CUDA;
  {
    // q [B*T][Hq][dh]: box {64, G, 128/G} = 128 rows of (tree token, head of the group)
    cuuint64_t dims[3] = {cuuint64_t(DH), cuuint64_t(Hq), cuuint64_t(B) * T};
    cuuint64_t strides[2] = {cuuint64_t(DH) * 2, cuuint64_t(Hq) * DH * 2};
    cuuint32_t box[3] = {64, cuuint32_t(pl.G), cuuint32_t(128 / pl.G)};
    cuuint32_t estr[3] = {1, 1, 1};
    if (fn(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<md_bf16*>(q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MD_ERR_CUDA;
  }
  if ((s = make_map_3d_sw128(&kmap, kc, DH, S_max, uint64_t(B) * Hkv, 64, CH)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&vmap, vc, DH, S_max, uint64_t(B) * Hkv, 64, CH)) != MD_OK) return s;
  (void)ws;
  Args a;
  a.prefix_len = prefix_len;
  a.out = out;
  a.B = B; a.S_max = S_max; a.Hq = Hq; a.Hkv = Hkv; a.G = pl.G; a.R = pl.R; a.rtiles = pl.rtiles;
  a.splits = pl.splits; a.chunks_per_split = pl.cps;
  a.scale_log2 = sc * 1.4426950408889634f;
  constexpr int sm = Cfg<DH, CH>::kSmem;
  if ((s = set_smem(attn_tc_kernel<DH, CH>, sm)) != MD_OK) return s;
  // the KV splits of a tile form one cluster (they merge through its shared memory)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.splits, Hkv * pl.rtiles, B);
  cfg.blockDim = dim3(Cfg<DH, CH>::kThreads);
  cfg.dynamicSmemBytes = sm;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pl.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_ok(cudaLaunchKernelEx(&cfg, attn_tc_kernel<DH, CH>, qmap, kmap, vmap, tree->tp, a));
}

// ------------------------ paged attention planning -------------------------

template <int DH, bool F32, int STREAMS>
void paged_attn_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, dim3 grid, cudaStream_t st) {
  *cfg = {};
  cfg->gridDim = grid;
  cfg->blockDim = dim3(md::attn_paged::Cfg<DH, F32, STREAMS>::kThreads);
  cfg->dynamicSmemBytes = md::attn_paged::Cfg<DH, F32, STREAMS>::kSmem;
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = grid.x;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// Function attributes last for the process: set once per device (a call of
// cudaFuncSetAttribute costs about a microsecond).
template <int DH, bool F32, int STREAMS>
md_status paged_attn_attributes() {
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  md_status s = cuda_ok(cudaGetDevice(&dev));
  if (s != MD_OK) return s;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return MD_OK;
  auto kern = md::attn_paged::attn_paged_kernel<DH, F32, STREAMS>;
  if ((s = set_smem(kern, md::attn_paged::Cfg<DH, F32, STREAMS>::kSmem)) != MD_OK) return s;
  if ((s = cuda_ok(cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))) != MD_OK) return s;
  if (dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return MD_OK;
}

// CTAs resident at once in clusters of `splits` on the current device, dev.
template <int DH, bool F32, int STREAMS>
int paged_attn_slots(int dev, int splits) {
  static std::atomic<int> cache[kMaxDevices][md::attn_paged::kMaxSplits + 1];
  int n = cache[dev][splits].load(std::memory_order_relaxed);
  if (n == 0) {                          // stored as count + 1
    int clusters = 0;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    paged_attn_config<DH, F32, STREAMS>(&cfg, attr, dim3(splits, 64), nullptr);
    cfg.numAttrs = 1;
    if (paged_attn_attributes<DH, F32, STREAMS>() != MD_OK ||
        cudaOccupancyMaxActiveClusters(&clusters, md::attn_paged::attn_paged_kernel<DH, F32, STREAMS>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      clusters = 0;
    }
    n = clusters * splits + 1;
    cache[dev][splits].store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

struct PagedAttnPlan {
  int tpt, tpu, units, splits, sort, streams;
};

// Row tiles hold whole nodes (G rows each); a unit is one or two tiles, and its
// KV range is cut into splits. The shape with the least estimated time (us) is
// taken, from measured costs: a CTA's fixed part (launch, first loads, read-out)
// 8 and 10 for one and two tiles, 0.5 and 1.5 more to join splits; a chunk of 128 keys
// 0.8 for one tile, 1.1 if other tiles' CTAs read the same keys from L2, 1.75 for two,
// 1.9 for one tile and one stream beside another such CTA, twice
// that for fp32 results (one score buffer, three P V products); CTAs
// past one wave fill the SMs as they come, with half a CTA's time left uneven; and
// no call is faster than its keys' bytes from memory, 1.1 times that in one wave (a
// batch's lengths differ, and its longest request then keeps one CTA). Chunks are
// counted by what the table can hold: the lengths are on the device. In a table much
// wider than the sequences the bytes' time hides the shapes' differences, and the first
// one stands: 32 requests of 500 slots take 13.5 us in a tight table and 26 from 2048
// slots on, the 70B batch of 8 over 4000 slots 111 us up to 32768 and 257 at 131072.
//   70B tree, B = 1 (40 tiles, 33 chunks): one tile, 3 splits 23.7 us; two tiles, 5
//     splits 26.7. B = 8: one tile 124, two tiles 113.6.
//   Decoding, 8 KV heads, 4096 slots: 1 split 32.9, 4 15.3, 8 12.5, 12 (two waves)
//     22.6. 16 requests of 26000: 1 split 261, 2 276; of 20001 to 32768: 316, 270.
//   One stream against two, 32/8 heads, one node: 256 requests of 200 slots 105 against
//     189, of 2000 365 against 446; 64 of 200 20.7 against 41.7; 32 of 500 13.2 against
//     24.9; 64 of 17 nodes over 200 33.9 against 53.3, 256 of 200 in fp32 158 against 223.
PagedAttnPlan paged_attn_plan(int B, int T, int Hq, int Hkv, int dh, int page, int max_pages, bool f32) {
  PagedAttnPlan p;
  const int G = Hq / Hkv;
  p.tpt = md::attn_paged::kBM / G;
  p.tpu = p.splits = 1;
  p.sort = 0;
  p.streams = 2;
  const int tiles = p.units = (T + p.tpt - 1) / p.tpt;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return p;
  const int chunks = int((int64_t(max_pages) * page + 127) / 128);
  const double bytes_us = 4.0 * B * Hkv * dh * 128 * chunks / 6.5e6;
  auto slots_of = [&](int streams, int s) -> int {
    if (streams == 1) return 2 * num_sms();   // the occupancy calculator counts a kernel with TMEM as one an SM
    return dh == 128 ? (f32 ? paged_attn_slots<128, true, 2>(dev, s) : paged_attn_slots<128, false, 2>(dev, s))
                     : (f32 ? paged_attn_slots<64, true, 2>(dev, s) : paged_attn_slots<64, false, 2>(dev, s));
  };
  double best = 0;
  // Shape 0: one stream a CTA, two CTAs an SM, for one row tile (with more, two tiles a
  // CTA are as fast: 16 requests of 300 slots, two tiles, 25.2 us against 24.1). T <= 64,
  // as its look at the tree's V spans two chunks of 64 keys. No splits: where two share
  // an SM, a CTA that holds TMEM must not wait for its cluster's others, which may be
  // waiting for TMEM that another kernel's CTA holds. Shapes 1 and 2: two streams, one
  // or two tiles.
  for (int shape = tiles == 1 && T <= 64 ? 0 : 1; shape <= 2 && shape <= tiles; ++shape) {
    const int tpu = std::max(shape, 1), streams = shape == 0 ? 1 : 2;
    const int units = (tiles + tpu - 1) / tpu;
    const int64_t base = int64_t(B) * Hkv * units;
    for (int s = 1; s <= (shape == 0 ? 1 : md::attn_paged::kMaxSplits) && s <= chunks; ++s) {
      const int slots = slots_of(streams, s);
      if (slots < s) continue;
      const int per_cta = (chunks + s - 1) / s;
      const double slow = f32 ? 2.0 : 1.0;
      const double one = per_cta * slow * (shape == 0 ? 1.9 : tiles > 1 ? 1.1 : 0.8) + 8.0 + (s > 1 ? 0.5 : 0.0);
      const double two = per_cta * slow * 1.75 + 10.0 + (s > 1 ? 1.5 : 0.0);
      const double longest = tpu == 2 ? two : one;
      const double all = tpu == 2 ? (tiles / 2) * two + (tiles % 2) * one : tiles * one;   // a KV head's units, one split
      const bool waves = base * s > slots;
      double us = waves ? double(B) * Hkv * s * all / slots + 0.5 * longest : longest;
      if (us < bytes_us + 8.0) us = (bytes_us + 8.0) * (waves || B == 1 ? 1.0 : 1.1);
      if (best == 0 || us < best) {
        best = us;
        p.tpu = tpu;
        p.streams = streams;
        p.units = units;
        p.splits = s;
        p.sort = B > 1 && B <= 256 && waves;   // ranking costs B^2 / 640 steps a CTA; many requests even out
      }
    }
  }
  return p;
}

template <int DH, bool F32, int STREAMS>
md_status launch_attn_paged(const md::attn_paged::Args& a, const md_bf16* q, const md_bf16* k_pages,
                            const md_tree* tree, cudaStream_t st) {
  using namespace md::attn_paged;
  md_status s;
  CUtensorMap qmap, kmap, vmap;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MD_ERR_CUDA;
  {
    // q [B][T][Hq][dh]: a box holds a tile's nodes, the G heads of one KV head each; rows
    // past the last node come as zeros, which the tensor cores multiply at less power
    // (decoding runs into the power cap on the rows it does not need)
    cuuint64_t dims[4] = {cuuint64_t(DH), cuuint64_t(a.Hq), cuuint64_t(tree->tp.T), cuuint64_t(a.B)};
    cuuint64_t strides[3] = {cuuint64_t(DH) * 2, cuuint64_t(a.Hq) * DH * 2, cuuint64_t(tree->tp.T) * a.Hq * DH * 2};
    cuuint32_t box[4] = {64, cuuint32_t(a.G), cuuint32_t(a.tpt), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    if (fn(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<md_bf16*>(q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MD_ERR_CUDA;
  }
  const uint64_t heads = uint64_t(a.pool) * a.Hkv;
  if ((s = make_map_3d_sw128(&kmap, k_pages, DH, a.page, heads, 64, a.piece)) != MD_OK) return s;
  if ((s = make_map_3d_sw128(&vmap, a.v_pages, DH, a.page, heads, 64, a.piece)) != MD_OK) return s;
  if ((s = paged_attn_attributes<DH, F32, STREAMS>()) != MD_OK) return s;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  paged_attn_config<DH, F32, STREAMS>(&cfg, attr, dim3(a.splits, a.Hkv * a.units, a.B), st);
  return cuda_ok(cudaLaunchKernelEx(&cfg, attn_paged_kernel<DH, F32, STREAMS>, qmap, kmap, vmap, tree->tp, a));
}

// ----------------------------- Hydra planning ------------------------------
// Level l drafts the children of the depth-l nodes that have children: B * n[l]
// head rows, top-k rows row0[l] + b * n[l] + slot[p] of one [rows, kmax] array.

struct HydraPlan {
  int L;                              // levels: the depth of the deepest node
  int n[MD_MAX_K];                    // nodes with children at depth l (per request)
  int row0[MD_MAX_K];                 // first top-k row of level l
  int rows;                           // top-k rows of all levels
  int8_t slot[MD_MAX_T];              // node -> index among its depth's nodes with children (-1: none)
  int8_t node[MD_MAX_K][MD_MAX_T];    // level l, index q -> node
  size_t heads_bytes[MD_MAX_K];       // heads workspace of each level (its own region: the
  size_t off_heads[MD_MAX_K];         // each level's heads workspace
  size_t off_x, off_ids, off_vals, bytes;
};

md_status hydra_plan(const md_tree* tree, int B, int d, int V, int kmax, HydraPlan* out) {
  using md::heads::align256;
  const TreeParams& tp = tree->tp;
  HydraPlan p;
  std::memset(&p, 0, sizeof(p));
  p.L = tp.max_depth;
  bool has_child[MD_MAX_T] = {};
  for (int j = 1; j < tp.T; ++j) has_child[tp.parent[j]] = true;
  for (int j = 0; j < tp.T; ++j) {
    p.slot[j] = -1;
    if (!has_child[j]) continue;
    const int l = tp.depth[j];
    p.node[l][p.n[l]] = int8_t(j);
    p.slot[j] = int8_t(p.n[l]++);
  }
  md_status s = heads_check(1, d, V, 1, kmax);
  if (s != MD_OK) return s;
  int rows = 0, maxn = 1;
  for (int l = 0; l < p.L; ++l) {
    p.row0[l] = rows;
    rows += B * p.n[l];
    maxn = std::max(maxn, p.n[l]);
    if (tree->kph[l] > kmax) return MD_ERR_INVALID_ARG;
    size_t hb = 0;
    if ((s = md_heads_workspace(B * p.n[l], d, V, 1, kmax, &hb)) != MD_OK) return s;
    p.heads_bytes[l] = hb;
  }
  p.rows = rows;
  size_t o = 0;
  p.off_x = o;     o = align256(o + size_t(B) * maxn * d * 2);
  p.off_ids = o;   o = align256(o + size_t(std::max(rows, 1)) * kmax * 4);
  p.off_vals = o;  o = align256(o + size_t(std::max(rows, 1)) * kmax * 4);
  for (int l = 0; l < p.L; ++l) {
    p.off_heads[l] = o;
    o = align256(o + p.heads_bytes[l]);
  }
  p.bytes = o;
  *out = p;
  return MD_OK;
}

// md_medusa_heads and md_medusa_heads_sampled: checks, then the streaming
// (one row), weights-as-M (2 .. 32 rows) or row-tile tensor-core path.
// gumbel_u null: top-k of the logits; else the top-k of the Gumbel keys
// logit * inv_tau - ln(-ln u).
md_status heads_call(const md_bf16* h, const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv, int32_t M,
                     int32_t d, int32_t V, int32_t K, const int32_t* k_per_head, int32_t kmax, int32_t* topk_ids,
                     float* topk_vals, float* logits_dbg, const float* gumbel_u, float inv_tau, void* ws,
                     size_t ws_bytes, void* stream) {
  if (!h || !W1 || !b1 || !Wv || !k_per_head || !topk_ids || !topk_vals) return MD_ERR_INVALID_ARG;
  md_status s = heads_check(M, d, V, K, kmax);
  if (s != MD_OK) return s;
  for (int k = 0; k < K; ++k)
    if (k_per_head[k] < 1 || k_per_head[k] > kmax || k_per_head[k] > V) return MD_ERR_INVALID_ARG;
  if (!aligned(h, 2) || !aligned(W1, 16) || !aligned(b1, 2) || !aligned(Wv, 16) || !aligned(topk_ids, 4) ||
      !aligned(topk_vals, 4) || (logits_dbg && !aligned(logits_dbg, 4)))
    return MD_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (skinny_rows(M)) {
    // tensor cores with the weights as M: h, W1, Wv feed TMA directly
    if (!aligned(h, 16) || !aligned(b1, 16)) return MD_ERR_INVALID_ARG;
    const SkinnyPlan pl = skinny_plan(M, d, V, K, kmax);
    if (!ws || ws_bytes < pl.bytes || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
    if (pl.NR == 16)
      return launch_heads_skinny<16>(pl, M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals,
                                     logits_dbg, gumbel_u, inv_tau, w, st);
    return launch_heads_skinny<32>(pl, M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals,
                                   logits_dbg, gumbel_u, inv_tau, w, st);
  }
  if (!stream_rows(M)) {
    // tensor-core path: h, W1, Wv feed TMA directly (16-byte aligned rows: d % 64, V % 8)
    if (!aligned(h, 16) || !aligned(b1, 16)) return MD_ERR_INVALID_ARG;
    if (!ws || ws_bytes < gemm_plan(M, d, V, K, kmax).bytes || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
    int mk = 0;
    for (int k = 0; k < K; ++k) mk = std::max(mk, int(k_per_head[k]));
    if (mk <= 4)
      return launch_heads_gemm<4>(M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg,
                                  gumbel_u, inv_tau, w, st);
    if (mk <= 8)
      return launch_heads_gemm<8>(M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg,
                                  gumbel_u, inv_tau, w, st);
    return launch_heads_gemm<16>(M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg,
                                 gumbel_u, inv_tau, w, st);
  }
  const md::heads::Plan pl = md::heads::make_plan(M, d, V, K, kmax, num_sms());
  if (!ws || ws_bytes < pl.bytes || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  if (M != 1) return MD_ERR_UNSUPPORTED;
  return launch_heads<1>(pl, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg, gumbel_u, inv_tau, w, st);
}

// Scratch of md_medusa_heads_static: a fixed array in the library's device
// image (every GPU that loads the library holds it until the process exits).
__device__ __align__(256) uint8_t g_heads_static_scratch[MD_HEADS_STATIC_SCRATCH_BYTES];

// Device address of g_heads_static_scratch on the current device. Host code
// cannot use the symbol itself (on the host it names a stand-in, not device
// memory), so the address is looked up once per device, with that device
// current, and cached.
md_status static_scratch_address(void** out) {
  static std::mutex mu;
  static void* addr[kMaxDevices] = {nullptr};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MD_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_heads_static_scratch) != cudaSuccess || !p) {
      (void)cudaGetLastError();
      return MD_ERR_CUDA;
    }
    addr[dev] = p;
  }
  *out = addr[dev];
  return MD_OK;
}

}  // namespace

extern "C" {

md_status md_tree_create(const int32_t* parent, const int32_t* head_rank, int32_t T, int32_t K,
                         const int32_t* k_per_head, md_tree** out) {
  if (!parent || !head_rank || !k_per_head || !out) return MD_ERR_INVALID_ARG;
  *out = nullptr;
  if (T < 1 || T > MD_MAX_T || K < 1 || K > MD_MAX_K) return MD_ERR_INVALID_ARG;
  if (parent[0] != -1) return MD_ERR_INVALID_ARG;
  for (int k = 0; k < K; ++k)
    if (k_per_head[k] < 1 || k_per_head[k] > MD_MAX_KMAX) return MD_ERR_INVALID_ARG;
  md_tree* t = new (std::nothrow) md_tree;
  if (!t) return MD_ERR_INVALID_ARG;
  std::memset(t, 0, sizeof(*t));
  TreeParams& tp = t->tp;
  tp.T = T;
  tp.W = (T + 31) / 32;
  tp.K = K;
  t->K = K;
  for (int k = 0; k < K; ++k) t->kph[k] = k_per_head[k];
  tp.parent[0] = -1;
  tp.depth[0] = 0;
  tp.rank[0] = 0;
  tp.anc[0][0] = 1u;
  int maxd = 0;
  for (int j = 1; j < T; ++j) {
    const int p = parent[j];
    if (p < 0 || p >= j) { delete t; return MD_ERR_INVALID_ARG; }
    const int d = tp.depth[p] + 1;
    if (d > K) { delete t; return MD_ERR_INVALID_ARG; }
    const int r = head_rank[j];
    if (r < 0 || r >= k_per_head[d - 1]) { delete t; return MD_ERR_INVALID_ARG; }
    for (int i = 1; i < j; ++i)
      if (parent[i] == p && head_rank[i] == r) { delete t; return MD_ERR_INVALID_ARG; }
    tp.parent[j] = int8_t(p);
    tp.depth[j] = int8_t(d);
    tp.rank[j] = int8_t(r);
    for (int w = 0; w < 4; ++w) tp.anc[j][w] = tp.anc[p][w];
    tp.anc[j][j >> 5] |= 1u << (j & 31);
    maxd = d > maxd ? d : maxd;
  }
  tp.max_depth = maxd;
  *out = t;
  return MD_OK;
}

md_status md_tree_destroy(md_tree* tree) {
  delete tree;
  return MD_OK;
}

md_status md_tree_info(const md_tree* tree, int32_t* T, int32_t* max_depth) {
  if (!tree) return MD_ERR_INVALID_ARG;
  if (T) *T = tree->tp.T;
  if (max_depth) *max_depth = tree->tp.max_depth;
  return MD_OK;
}

md_status md_heads_workspace(int32_t M, int32_t d, int32_t V, int32_t K, int32_t kmax, size_t* bytes) {
  if (!bytes) return MD_ERR_INVALID_ARG;
  md_status s = heads_check(M, d, V, K, kmax);
  if (s != MD_OK) return s;
  *bytes = stream_rows(M)   ? md::heads::make_plan(M, d, V, K, kmax, num_sms()).bytes
           : skinny_rows(M) ? skinny_plan(M, d, V, K, kmax).bytes
                            : gemm_plan(M, d, V, K, kmax).bytes;
  return MD_OK;
}

md_status md_medusa_heads(const md_bf16* h, const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv, int32_t M,
                          int32_t d, int32_t V, int32_t K, const int32_t* k_per_head, int32_t kmax,
                          int32_t* topk_ids, float* topk_vals, float* logits_dbg, void* ws, size_t ws_bytes,
                          void* stream) {
  return heads_call(h, W1, b1, Wv, M, d, V, K, k_per_head, kmax, topk_ids, topk_vals, logits_dbg, nullptr, 1.f, ws,
                    ws_bytes, stream);
}

md_status md_medusa_heads_sampled(const md_bf16* h, const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv,
                                  int32_t M, int32_t d, int32_t V, int32_t K, const int32_t* k_per_head,
                                  int32_t kmax, float temperature, const float* uniforms, int32_t* topk_ids,
                                  float* topk_keys, float* logits, void* ws, size_t ws_bytes, void* stream) {
  if (!uniforms || !logits) return MD_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return MD_ERR_INVALID_ARG;
  if (!aligned(uniforms, 16) || !aligned(logits, 16)) return MD_ERR_INVALID_ARG;
  return heads_call(h, W1, b1, Wv, M, d, V, K, k_per_head, kmax, topk_ids, topk_keys, logits, uniforms,
                    1.0f / temperature, ws, ws_bytes, stream);
}

md_status md_heads_shared_workspace(int32_t M, int32_t d, int32_t V, int32_t K, int32_t kmax, size_t* bytes) {
  if (!bytes) return MD_ERR_INVALID_ARG;
  md_status s = heads_check(M, d, V, K, kmax);
  if (s != MD_OK) return s;
  if (size_t(M) * K > size_t(md::gemm::kMaxM)) return MD_ERR_UNSUPPORTED;
  *bytes = shared_plan(M, d, V, K, kmax).bytes;
  return MD_OK;
}

md_status md_medusa_heads_shared(const md_bf16* h, const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv,
                                 int32_t M, int32_t d, int32_t V, int32_t K, const int32_t* k_per_head, int32_t kmax,
                                 int32_t* topk_ids, float* topk_vals, float* logits_dbg, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (!h || !W1 || !b1 || !Wv || !k_per_head || !topk_ids || !topk_vals) return MD_ERR_INVALID_ARG;
  size_t need = 0;
  md_status s = md_heads_shared_workspace(M, d, V, K, kmax, &need);
  if (s != MD_OK) return s;
  int mk = 0;
  for (int k = 0; k < K; ++k) {
    if (k_per_head[k] < 1 || k_per_head[k] > kmax || k_per_head[k] > V) return MD_ERR_INVALID_ARG;
    mk = std::max(mk, int(k_per_head[k]));
  }
  if (!aligned(h, 16) || !aligned(W1, 16) || !aligned(b1, 16) || !aligned(Wv, 16) || !aligned(topk_ids, 4) ||
      !aligned(topk_vals, 4) || (logits_dbg && !aligned(logits_dbg, 16)))
    return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  const SharedPlan sp = shared_plan(M, d, V, K, kmax);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (sp.skinny) {
#define MD_SHARED_SKINNY(a, b)                                                                                   \
  if (sp.NR1 == a && sp.NR2 == b)                                                                                \
    return launch_heads_shared_skinny<a, b>(sp, M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, \
                                            logits_dbg, w, st);
    MD_SHARED_SKINNY(16, 16)
    MD_SHARED_SKINNY(16, 32)
    MD_SHARED_SKINNY(32, 32)
#undef MD_SHARED_SKINNY
    return MD_ERR_UNSUPPORTED;
  }
  if (sp.stream)
    return launch_heads_shared_stream<1>(sp, M, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg, w, st);
  if (mk <= 4)
    return launch_heads_shared_gemm<4>(sp, M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg, w, st);
  if (mk <= 8)
    return launch_heads_shared_gemm<8>(sp, M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg, w, st);
  return launch_heads_shared_gemm<16>(sp, M, d, V, K, kmax, h, W1, b1, Wv, k_per_head, topk_ids, topk_vals, logits_dbg, w, st);
}

md_status md_medusa_heads_static(const md_bf16* h, const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv,
                                 int32_t M, int32_t d, int32_t V, int32_t K, const int32_t* k_per_head, int32_t kmax,
                                 int32_t* topk_ids, float* topk_vals, float* logits_dbg, void* stream) {
  // the argument checks of md_medusa_heads come before the scratch-size check
  if (!h || !W1 || !b1 || !Wv || !k_per_head || !topk_ids || !topk_vals) return MD_ERR_INVALID_ARG;
  size_t need = 0;
  md_status s = md_heads_workspace(M, d, V, K, kmax, &need);
  if (s != MD_OK) return s;
  for (int k = 0; k < K; ++k)
    if (k_per_head[k] < 1 || k_per_head[k] > kmax || k_per_head[k] > V) return MD_ERR_INVALID_ARG;
  if (need > size_t(MD_HEADS_STATIC_SCRATCH_BYTES)) return MD_ERR_WORKSPACE;
  void* scratch = nullptr;
  if ((s = static_scratch_address(&scratch)) != MD_OK) return s;
  return md_medusa_heads(h, W1, b1, Wv, M, d, V, K, k_per_head, kmax, topk_ids, topk_vals, logits_dbg, scratch,
                         size_t(MD_HEADS_STATIC_SCRATCH_BYTES), stream);
}

md_status md_tree_build(const md_tree* tree, const int32_t* topk_ids, int32_t M, int32_t kmax,
                        const int32_t* head_row, const int32_t* root_token, const int32_t* prefix_len, int32_t B,
                        int32_t* tokens, int32_t* parent, uint32_t* anc, int32_t* pos, void* stream) {
  if (!tree || !topk_ids || !root_token || !prefix_len || !tokens || !parent || !anc || !pos)
    return MD_ERR_INVALID_ARG;
  if (M < 1 || B < 1 || kmax < 1 || kmax > MD_MAX_KMAX) return MD_ERR_INVALID_ARG;
  if (!head_row && M < B) return MD_ERR_INVALID_ARG;
  for (int k = 0; k < tree->K; ++k)
    if (tree->kph[k] > kmax) return MD_ERR_INVALID_ARG;
  md::tree::BuildArgs a;
  a.topk_ids = topk_ids; a.head_row = head_row; a.root_token = root_token; a.prefix_len = prefix_len;
  a.tokens = tokens; a.parent = parent; a.anc = anc; a.pos = pos;
  a.M = M; a.K = tree->K; a.kmax = kmax;
  return launch_pdl(md::tree::tree_build_kernel, dim3(B), dim3(MD_MAX_T), 0, static_cast<cudaStream_t>(stream),
                    tree->tp, a);
}

md_status md_hydra_workspace(const md_tree* tree, int32_t B, int32_t d, int32_t V, int32_t kmax, size_t* bytes) {
  if (!tree || !bytes || B < 1 || d < 1 || V < 1 || kmax < 1) return MD_ERR_INVALID_ARG;
  HydraPlan p;
  md_status s = hydra_plan(tree, B, d, V, kmax, &p);
  if (s != MD_OK) return s;
  *bytes = p.bytes;
  return MD_OK;
}

md_status md_hydra_draft(const md_tree* tree, const md_bf16* h, int32_t M, const int32_t* head_row,
                         const md_bf16* E, const md_bf16* W1, const md_bf16* b1, const md_bf16* Wv, int32_t d,
                         int32_t V, int32_t K, int32_t kmax, const int32_t* root_token, const int32_t* prefix_len,
                         int32_t B, int32_t* tokens, int32_t* parent, uint32_t* anc, int32_t* pos,
                         float* logits_dbg, void* ws, size_t ws_bytes, void* stream) {
  if (!tree || !h || !E || !W1 || !b1 || !Wv || !root_token || !prefix_len || !tokens || !parent || !anc || !pos)
    return MD_ERR_INVALID_ARG;
  if (M < 1 || B < 1 || K != tree->K) return MD_ERR_INVALID_ARG;
  if (!head_row && M < B) return MD_ERR_INVALID_ARG;
  size_t need = 0;
  md_status s = md_hydra_workspace(tree, B, d, V, kmax, &need);
  if (s != MD_OK) return s;
  if (!aligned(h, 16) || !aligned(E, 16) || !aligned(W1, 16) || !aligned(b1, 16) || !aligned(Wv, 16) ||
      (logits_dbg && !aligned(logits_dbg, 4)))
    return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  HydraPlan p;
  if ((s = hydra_plan(tree, B, d, V, kmax, &p)) != MD_OK) return s;
  const TreeParams& tp = tree->tp;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint16_t* x = reinterpret_cast<uint16_t*>(w + p.off_x);
  int32_t* ids = reinterpret_cast<int32_t*>(w + p.off_ids);
  float* vals = reinterpret_cast<float*>(w + p.off_vals);
  // the heads kernels' tickets carry a per-call epoch: nothing is cleared, and
  // the levels' kernels follow one another as dependent launches
  for (int l = 0; l < p.L; ++l) {
    md::hydra::GatherArgs ga;
    std::memset(&ga, 0, sizeof(ga));
    ga.h = h; ga.E = E; ga.head_row = head_row; ga.root_token = root_token; ga.prefix_len = prefix_len;
    ga.prev_ids = l == 0 ? nullptr : ids + size_t(p.row0[l - 1]) * kmax;
    ga.x = x;
    ga.M = M; ga.d = d; ga.V = V; ga.kmax = kmax;
    ga.n_prev = l == 0 ? 0 : p.n[l - 1];
    for (int q = 0; q < p.n[l]; ++q) {
      const int node = p.node[l][q];
      ga.pslot[q] = l == 0 ? int8_t(0) : p.slot[tp.parent[node]];
      ga.prank[q] = tp.rank[node];
    }
    if ((s = launch_pdl(md::hydra::hydra_gather_kernel, dim3(p.n[l], B), dim3(md::hydra::kGatherThreads), 0, st,
                        ga)) != MD_OK)
      return s;
    const size_t r0 = size_t(p.row0[l]);
    if ((s = heads_call(x, W1 + size_t(l) * d * d, b1 + size_t(l) * d, Wv + size_t(l) * d * V, B * p.n[l], d, V, 1,
                        &tree->kph[l], kmax, ids + r0 * kmax, vals + r0 * kmax,
                        logits_dbg ? logits_dbg + r0 * V : nullptr, nullptr, 1.f, w + p.off_heads[l],
                        p.heads_bytes[l], stream)) != MD_OK)
      return s;
  }
  md::hydra::TokenArgs ta;
  std::memset(&ta, 0, sizeof(ta));
  ta.ids = ids; ta.root_token = root_token; ta.prefix_len = prefix_len;
  ta.tokens = tokens; ta.parent = parent; ta.anc = anc; ta.pos = pos;
  ta.kmax = kmax;
  for (int l = 0; l < MD_MAX_K; ++l) {
    ta.row0[l] = l < p.L ? p.row0[l] : 0;
    ta.n[l] = l < p.L ? p.n[l] : 0;
  }
  for (int j = 0; j < MD_MAX_T; ++j) ta.slot[j] = p.slot[j];
  return launch_pdl(md::hydra::hydra_tokens_kernel, dim3(B), dim3(MD_MAX_T), 0, st, tp, ta);
}

md_status md_attention_workspace(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t dh, int32_t S_max,
                                 size_t* bytes) {
  if (!bytes || B < 1 || T < 1 || Hq < 1 || Hkv < 1 || S_max < 1) return MD_ERR_INVALID_ARG;
  if (T > MD_MAX_T || (dh != 64 && dh != 128) || Hq % Hkv != 0 || Hq / Hkv > 16) return MD_ERR_UNSUPPORTED;
  *bytes = attn_plan(B, T, Hq, Hkv, dh, S_max).bytes;
  return MD_OK;
}

md_status md_tree_attention(const md_bf16* q, const md_bf16* k_cache, const md_bf16* v_cache,
                            const int32_t* prefix_len, int32_t S_max, const md_tree* tree, int32_t B, int32_t Hq,
                            int32_t Hkv, int32_t dh, float scale, float* out, void* ws, size_t ws_bytes,
                            void* stream) {
  if (!q || !k_cache || !v_cache || !prefix_len || !tree || !out) return MD_ERR_INVALID_ARG;
  const int T = tree->tp.T;
  size_t need = 0;
  md_status s = md_attention_workspace(B, T, Hq, Hkv, dh, S_max, &need);
  if (s != MD_OK) return s;
  if (S_max < T || !(scale >= 0.f) || !std::isfinite(scale)) return MD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  const AttnPlan pl = attn_plan(B, T, Hq, Hkv, dh, S_max);
  const float sc = scale > 0.f ? scale : 1.0f / std::sqrt(float(dh));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (pl.tc) {
    if (pl.ch == 64)
      return dh == 128 ? launch_attn_tc<128, 64>(pl, q, k_cache, v_cache, prefix_len, S_max, tree, B, Hq, Hkv, sc, out,
                                                 ws, st)
                       : launch_attn_tc<64, 64>(pl, q, k_cache, v_cache, prefix_len, S_max, tree, B, Hq, Hkv, sc, out,
                                                ws, st);
    return dh == 128 ? launch_attn_tc<128, 128>(pl, q, k_cache, v_cache, prefix_len, S_max, tree, B, Hq, Hkv, sc, out,
                                                ws, st)
                     : launch_attn_tc<64, 128>(pl, q, k_cache, v_cache, prefix_len, S_max, tree, B, Hq, Hkv, sc, out,
                                               ws, st);
  }
  md::attn::Args a;
  a.q = q; a.kc = k_cache; a.vc = v_cache; a.prefix_len = prefix_len;
  a.part_acc = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + pl.off_ml);
  a.out = out;
  a.S_max = S_max; a.Hq = Hq; a.Hkv = Hkv; a.G = pl.G; a.R = pl.R; a.max_chunks = pl.max_chunks;
  a.scale_log2 = sc * 1.4426950408889634f;
  const dim3 grid(pl.max_chunks, Hkv, B);
  if (dh == 128) {
    constexpr int sm = md::attn::smem_bytes<128>();
    if ((s = set_smem(md::attn::attn_chunk_kernel<128>, sm)) != MD_OK) return s;
    md::attn::attn_chunk_kernel<128><<<grid, md::attn::kThreads, sm, st>>>(tree->tp, a);
    if ((s = last_launch()) != MD_OK) return s;
    md::attn::attn_merge_kernel<128><<<dim3(T * Hq, B), 128, 0, st>>>(tree->tp, a);
  } else {
    constexpr int sm = md::attn::smem_bytes<64>();
    if ((s = set_smem(md::attn::attn_chunk_kernel<64>, sm)) != MD_OK) return s;
    md::attn::attn_chunk_kernel<64><<<grid, md::attn::kThreads, sm, st>>>(tree->tp, a);
    if ((s = last_launch()) != MD_OK) return s;
    md::attn::attn_merge_kernel<64><<<dim3(T * Hq, B), 64, 0, st>>>(tree->tp, a);
  }
  return last_launch();
}

md_status md_accept_workspace(int32_t B, int32_t T, int32_t V, size_t* bytes) {
  if (!bytes || B < 1 || T < 1 || V < 1) return MD_ERR_INVALID_ARG;
  if (T > MD_MAX_T || V % 8 != 0) return MD_ERR_UNSUPPORTED;
  *bytes = accept_plan(B, T, V).bytes;
  return MD_OK;
}

md_status md_tree_accept(const float* logits, int32_t V, const int32_t* tokens, const md_tree* tree, int32_t B,
                         int32_t K, int32_t mode, float temperature, float eps, float alpha, int32_t* accept_len,
                         int32_t* path, int32_t* bonus, void* ws, size_t ws_bytes, void* stream) {
  if (!logits || !tokens || !tree || !accept_len || !path || !bonus) return MD_ERR_INVALID_ARG;
  const int T = tree->tp.T;
  size_t need = 0;
  md_status s = md_accept_workspace(B, T, V, &need);
  if (s != MD_OK) return s;
  if (K < tree->tp.max_depth || K < 0) return MD_ERR_INVALID_ARG;
  if (mode != MD_ACCEPT_GREEDY && mode != MD_ACCEPT_TYPICAL) return MD_ERR_INVALID_ARG;
  if (mode == MD_ACCEPT_TYPICAL &&
      (!(temperature > 0.f) || !std::isfinite(temperature) || !(eps >= 0.f) || !(alpha >= 0.f)))
    return MD_ERR_INVALID_ARG;
  if (!aligned(logits, 16)) return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  const AcceptPlan pl = accept_plan(B, T, V);
  md::acc::Args a;
  a.logits = logits; a.tokens = tokens; a.accept_len = accept_len; a.path = path; a.bonus = bonus;
  a.part = static_cast<float*>(ws);
  a.ysamp = nullptr;
  a.T = T; a.V = V; a.K = K; a.nchunks = pl.nchunks; a.chunk_len = pl.chunk_len; a.mode = mode;
  a.inv_temp = mode == MD_ACCEPT_TYPICAL ? 1.0f / temperature : 1.0f;
  a.log_eps = std::log(eps);
  a.log_alpha = std::log(alpha);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = launch_pdl(md::acc::accept_rows_kernel, dim3(pl.nchunks, B * T), dim3(md::acc::kRowThreads), 0, st, a)) !=
      MD_OK)
    return s;
  return launch_pdl(md::acc::accept_walk_kernel, dim3(B), dim3(MD_MAX_T), 0, st, tree->tp, a);
}

md_status md_tree_accept_sampled(const float* logits, int32_t V, const int32_t* tokens, const md_tree* tree,
                                 int32_t B, int32_t K, float temperature, const float* uniforms,
                                 int32_t* accept_len, int32_t* path, int32_t* bonus, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (!logits || !tokens || !tree || !uniforms || !accept_len || !path || !bonus) return MD_ERR_INVALID_ARG;
  const int T = tree->tp.T;
  size_t need = 0;
  md_status s = md_accept_workspace(B, T, V, &need);
  if (s != MD_OK) return s;
  if (V > md::acc::kSampleTile * md::acc::kSampleMaxTiles) return MD_ERR_UNSUPPORTED;
  if (K < tree->tp.max_depth || K < 0) return MD_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return MD_ERR_INVALID_ARG;
  if (!aligned(logits, 16)) return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the per-row draws take the front of the workspace (B*T ints <= its size)
  int32_t* ysamp = static_cast<int32_t*>(ws);
  md::acc::SampleArgs sa;
  sa.logits = logits; sa.uniforms = uniforms; sa.ysamp = ysamp; sa.V = V;
  sa.inv_temp_log2e = 1.4426950408889634f / temperature;
  if ((s = launch_pdl(md::acc::accept_sample_kernel, dim3(B * T), dim3(md::acc::kSampleThreads), 0, st, sa)) !=
      MD_OK)
    return s;
  md::acc::Args a;
  a.logits = logits; a.tokens = tokens; a.accept_len = accept_len; a.path = path; a.bonus = bonus;
  a.part = nullptr;
  a.ysamp = ysamp;
  a.T = T; a.V = V; a.K = K; a.nchunks = 0; a.chunk_len = 0; a.mode = MD_ACCEPT_GREEDY;
  a.inv_temp = 1.0f; a.log_eps = 0.f; a.log_alpha = 0.f;
  return launch_pdl(md::acc::accept_walk_kernel, dim3(B), dim3(MD_MAX_T), 0, st, tree->tp, a);
}

md_status md_tree_accept_rejection(const float* logits, int32_t V, const int32_t* tokens, const md_tree* tree,
                                   int32_t B, int32_t K, float temperature, const float* head_logits, int32_t M,
                                   int32_t Kh, const int32_t* head_row, float temperature_q, const float* u_accept,
                                   const float* u_residual, int32_t* accept_len, int32_t* path, int32_t* bonus,
                                   void* stream) {
  using namespace md::rej;
  if (!logits || !tokens || !tree || !head_logits || !u_accept || !u_residual || !accept_len || !path || !bonus)
    return MD_ERR_INVALID_ARG;
  const TreeParams& tp = tree->tp;
  if (B < 1 || V < 1 || M < 1 || K < tp.max_depth || K > MD_MAX_K || Kh < tp.max_depth) return MD_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !(temperature_q > 0.f) || !std::isfinite(temperature_q))
    return MD_ERR_INVALID_ARG;
  const int slice = (V + kCtas - 1) / kCtas;
  if (slice > kMaxSlice) return MD_ERR_UNSUPPORTED;
  // the children of every node must carry the ranks 0 .. m-1 (the first m draws)
  for (int t = 0; t < tp.T; ++t) {
    int m = 0, rmax = -1;
    for (int j = 1; j < tp.T; ++j)
      if (tp.parent[j] == t) {
        ++m;
        rmax = std::max(rmax, int(tp.rank[j]));
      }
    if (m > 0 && rmax != m - 1) return MD_ERR_UNSUPPORTED;
  }
  Args a;
  a.logits = logits; a.head_logits = head_logits; a.head_row = head_row; a.tokens = tokens;
  a.u_acc = u_accept; a.u_res = u_residual; a.accept_len = accept_len; a.path = path; a.bonus = bonus;
  a.V = V; a.T = tp.T; a.K = K; a.M = M; a.Kh = Kh; a.slice = slice;
  a.inv_tau = 1.0f / temperature;
  a.inv_tau_q = 1.0f / temperature_q;
  md_status s;
  if ((s = set_smem(reject_accept_kernel, kSmem)) != MD_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas, B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_ok(cudaLaunchKernelEx(&cfg, reject_accept_kernel, tp, a));
}

md_status md_tree_commit(md_bf16* k_cache, md_bf16* v_cache, int32_t S_max, int32_t Hkv, int32_t dh,
                         const md_tree* tree, int32_t B, const int32_t* prefix_len, const int32_t* accept_len,
                         const int32_t* path, int32_t K, const int32_t* bonus, int32_t* new_prefix_len,
                         int32_t* next_root, int32_t* next_head_row, void* stream) {
  if (!k_cache || !v_cache || !tree || !prefix_len || !accept_len || !path || !bonus || !new_prefix_len ||
      !next_root || !next_head_row)
    return MD_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || S_max < tree->tp.T || K < tree->tp.max_depth || K > MD_MAX_K) return MD_ERR_INVALID_ARG;
  if (dh != 64 && dh != 128) return MD_ERR_UNSUPPORTED;
  if (new_prefix_len == prefix_len || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return MD_ERR_INVALID_ARG;
  md::commit::Args a;
  a.kc = k_cache; a.vc = v_cache; a.prefix_len = prefix_len; a.accept_len = accept_len; a.path = path;
  a.bonus = bonus; a.new_prefix_len = new_prefix_len; a.next_root = next_root; a.next_head_row = next_head_row;
  a.S_max = S_max; a.Hkv = Hkv; a.dh = dh; a.K = K;
  const int smem = 2 * (MD_MAX_K + 1) * dh * 2;
  return launch_pdl(md::commit::tree_commit_kernel, dim3(Hkv, B), dim3(md::commit::kThreads), smem,
                    static_cast<cudaStream_t>(stream), tree->tp, a);
}

// ------------------------------- paged cache -------------------------------

namespace {

// Sizes every paged call checks: a pool whose page rows a 32-bit TMA coordinate reaches.
md_status paged_check(int32_t B, int32_t pool_pages, int32_t page_size, int32_t max_pages, int32_t Hkv, int32_t dh) {
  if (B < 1 || pool_pages < 1 || page_size < 1 || max_pages < 1 || Hkv < 1) return MD_ERR_INVALID_ARG;
  if (dh != 64 && dh != 128) return MD_ERR_UNSUPPORTED;
  // slots, table entries and page rows (one page past the pool included) are int32
  if (B > 65535 || (int64_t(pool_pages) + 1) * Hkv > INT32_MAX || int64_t(max_pages) * page_size > INT32_MAX - 256 ||
      int64_t(B) * max_pages > INT32_MAX)
    return MD_ERR_UNSUPPORTED;
  return MD_OK;
}

}  // namespace

md_status md_attention_paged_workspace(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t dh, int32_t page_size,
                                       int32_t max_pages, size_t* bytes) {
  if (!bytes || T < 1 || Hq < 1) return MD_ERR_INVALID_ARG;
  md_status s = paged_check(B, 1, page_size, max_pages, Hkv, dh);
  if (s != MD_OK) return s;
  if (T > MD_MAX_T || Hq % Hkv != 0 || Hq / Hkv > 16 || Hkv > 4095 || page_size % 16 != 0) return MD_ERR_UNSUPPORTED;
  *bytes = 256;
  return MD_OK;
}

md_status md_tree_attention_paged(const md_bf16* q, const md_bf16* k_pages, const md_bf16* v_pages, int32_t pool_pages,
                                  int32_t page_size, const int32_t* block_table, int32_t max_pages,
                                  const int32_t* prefix_len, const md_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                  int32_t dh, float scale, void* out, int32_t out_type, void* ws, size_t ws_bytes,
                                  void* stream) {
  if (!q || !k_pages || !v_pages || !block_table || !prefix_len || !tree || !out) return MD_ERR_INVALID_ARG;
  size_t need = 0;
  md_status s = md_attention_paged_workspace(B, tree->tp.T, Hq, Hkv, dh, page_size, max_pages, &need);
  if (s != MD_OK) return s;
  if ((s = paged_check(B, pool_pages, page_size, max_pages, Hkv, dh)) != MD_OK) return s;
  if (!(scale >= 0.f) || !std::isfinite(scale) || (out_type != MD_OUT_F32 && out_type != MD_OUT_BF16))
    return MD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || out == q)
    return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  const PagedAttnPlan pl = paged_attn_plan(B, tree->tp.T, Hq, Hkv, dh, page_size, max_pages, out_type == MD_OUT_F32);
  md::attn_paged::Args a;
  a.v_pages = v_pages; a.table = block_table; a.prefix_len = prefix_len; a.out = out;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.pool = pool_pages; a.page = page_size; a.max_pages = max_pages;
  a.piece = std::min(page_size & -page_size, 64 * pl.streams);   // rows of a TMA copy, within a chunk
  a.tpt = pl.tpt; a.tpu = pl.tpu; a.units = pl.units; a.splits = pl.splits; a.sort = pl.sort;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(float(dh))) * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = out_type == MD_OUT_F32, one = pl.streams == 1;
  auto launch = dh == 128 ? (f32 ? (one ? launch_attn_paged<128, true, 1> : launch_attn_paged<128, true, 2>)
                                 : (one ? launch_attn_paged<128, false, 1> : launch_attn_paged<128, false, 2>))
                          : (f32 ? (one ? launch_attn_paged<64, true, 1> : launch_attn_paged<64, true, 2>)
                                 : (one ? launch_attn_paged<64, false, 1> : launch_attn_paged<64, false, 2>));
  return launch(a, q, k_pages, tree, st);
}

md_status md_qk_rope_append(const md_bf16* q, const md_bf16* k, const md_bf16* v, const int64_t* strides,
                            const int32_t* pos, const float* inv_freq, int32_t rot, int32_t interleaved,
                            const md_bf16* q_norm, const md_bf16* k_norm, float eps, md_bf16* q_out, md_bf16* k_pages,
                            md_bf16* v_pages, int32_t pool_pages, int32_t page_size, const int32_t* block_table,
                            int32_t max_pages, const int32_t* prefix_len, const int32_t* n_new, int32_t B, int32_t T,
                            int32_t Hq, int32_t Hkv, int32_t dh, void* stream) {
  if (!q || !k || !v || !strides || !pos || !inv_freq || !q_out || !k_pages || !v_pages || !block_table || !prefix_len)
    return MD_ERR_INVALID_ARG;
  if (T < 1 || Hq < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return MD_ERR_INVALID_ARG;
  md_status s = paged_check(B, pool_pages, page_size, max_pages, Hkv, dh);
  if (s != MD_OK) return s;
  if (rot < 16 || rot > dh || rot % 16 != 0 || int64_t(B) * T > INT32_MAX || int64_t(Hq) + 2 * int64_t(Hkv) > 65535)
    return MD_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, v, q_out, k_pages, v_pages, q_norm, k_norm};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return MD_ERR_INVALID_ARG;
  for (int i = 0; i < 9; ++i)
    if (strides[i] % 8 != 0) return MD_ERR_INVALID_ARG;
  md::append::Args a;
  a.q = q; a.k = k; a.v = v;
  a.qb = strides[0]; a.qt = strides[1]; a.qh = strides[2];
  a.kb = strides[3]; a.kt = strides[4]; a.kh = strides[5];
  a.vb = strides[6]; a.vt = strides[7]; a.vh = strides[8];
  a.pos = pos; a.inv_freq = inv_freq; a.q_norm = q_norm; a.k_norm = k_norm; a.q_out = q_out;
  a.k_pages = k_pages; a.v_pages = v_pages; a.table = block_table; a.prefix_len = prefix_len; a.n_new = n_new;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.rot = rot; a.interleaved = interleaved != 0;
  a.max_pages = max_pages; a.pool = pool_pages; a.page = page_size; a.eps = eps;
  // A CTA takes a run of tokens and a block of heads. Runs as long as about eight
  // CTAs a SM are left: a tree's 65 tokens of 80 heads fill the SMs with runs of one (3.1
  // us; a CTA per token 6.2); prompts use the angles and pointers of a CTA longest,
  // and all the blocks of a token in turn (24k tokens of 48 heads: runs of 4 / 8 / 16
  // 120 / 111 / 109 us; a CTA per block of heads 119).
  const int64_t heads = int64_t(Hq) + 2 * Hkv, at_once = md::append::kThreads / (dh / 8);
  const int blocks = int((heads + at_once - 1) / at_once);
  a.block = int((heads + blocks - 1) / blocks);
  const int64_t ctas = int64_t(num_sms()) * 8;
  const bool all_heads = int64_t(B) * T >= ctas * md::append::kRun;
  const int64_t fill = int64_t(B) * T * (all_heads ? 1 : blocks) / ctas;
  a.run = int(std::max<int64_t>(1, std::min<int64_t>(fill, md::append::kRun)));
  const dim3 grid(unsigned(int64_t(B) * ((T + a.run - 1) / a.run)), all_heads ? 1 : blocks);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool many = 2 * heads <= at_once;
  auto kern = dh == 128 ? (many ? md::append::qk_rope_append_kernel<128, true> : md::append::qk_rope_append_kernel<128, false>)
                        : (many ? md::append::qk_rope_append_kernel<64, true> : md::append::qk_rope_append_kernel<64, false>);
  return launch_pdl(kern, grid, dim3(md::append::kThreads), 0, st, a);
}

md_status md_tree_commit_paged(md_bf16* k_pages, md_bf16* v_pages, int32_t layers, int32_t pool_pages,
                               int32_t page_size, const int32_t* block_table, int32_t max_pages, int32_t Hkv,
                               int32_t dh, const md_tree* tree, int32_t B, const int32_t* prefix_len,
                               const int32_t* accept_len, const int32_t* path, int32_t K, const int32_t* bonus,
                               int32_t* new_prefix_len, int32_t* next_root, int32_t* next_head_row, void* stream) {
  if (!k_pages || !v_pages || !block_table || !tree || !prefix_len || !accept_len || !path || !bonus ||
      !new_prefix_len || !next_root || !next_head_row)
    return MD_ERR_INVALID_ARG;
  if (layers < 1 || K < tree->tp.max_depth || K > MD_MAX_K) return MD_ERR_INVALID_ARG;
  md_status s = paged_check(B, pool_pages, page_size, max_pages, Hkv, dh);
  if (s != MD_OK) return s;
  if (new_prefix_len == prefix_len || !aligned(k_pages, 16) || !aligned(v_pages, 16)) return MD_ERR_INVALID_ARG;
  md::commit_paged::Args a;
  a.kp = reinterpret_cast<uint4*>(k_pages); a.vp = reinterpret_cast<uint4*>(v_pages);
  a.table = block_table; a.prefix_len = prefix_len; a.accept_len = accept_len; a.path = path; a.bonus = bonus;
  a.new_prefix_len = new_prefix_len; a.next_root = next_root; a.next_head_row = next_head_row;
  a.layers = layers; a.pool = pool_pages; a.page = page_size; a.max_pages = max_pages; a.Hkv = Hkv; a.row16 = dh / 8;
  a.K = K;
  const int64_t cols = int64_t(2) * layers * Hkv * a.row16;
  const int64_t blocks = (cols + md::commit_paged::kThreads - 1) / md::commit_paged::kThreads;
  return launch_pdl(md::commit_paged::tree_commit_paged_kernel, dim3(unsigned(std::min<int64_t>(blocks, 1 << 20)), B),
                    dim3(md::commit_paged::kThreads), 0, static_cast<cudaStream_t>(stream), tree->tp, a);
}

md_status md_pages_resize(int32_t* block_table, int32_t* n_pages, int32_t* refcount, const int32_t* length, int32_t B,
                          int32_t max_pages, int32_t pool_pages, int32_t page_size, int32_t extra, void* stream) {
  if (!block_table || !n_pages || !refcount || !length || extra < 0) return MD_ERR_INVALID_ARG;
  md_status s = paged_check(B, pool_pages, page_size, max_pages, 1, 64);
  if (s != MD_OK) return s;
  if (B > md::pages::kMaxRows) return MD_ERR_UNSUPPORTED;
  if (!aligned(refcount, 16)) return MD_ERR_INVALID_ARG;
  md::pages::ResizeArgs a;
  a.table = block_table; a.n_pages = n_pages; a.refcount = refcount; a.length = length;
  a.B = B; a.max_pages = max_pages; a.pool = pool_pages; a.page = page_size; a.extra = extra;
  const int smem = B * 4;
  if (smem > 32768 && (s = set_smem(md::pages::pages_resize_kernel, md::pages::kMaxRows * 4)) != MD_OK) return s;
  return launch_pdl(md::pages::pages_resize_kernel, dim3(1), dim3(md::pages::kThreads), smem,
                    static_cast<cudaStream_t>(stream), a);
}

md_status md_pages_fork_workspace(int32_t B, int32_t n, size_t* bytes) {
  if (!bytes || B < 1 || n < 1) return MD_ERR_INVALID_ARG;
  if (n > md::pages::kMaxForks) return MD_ERR_UNSUPPORTED;
  *bytes = md::heads::align256(size_t(n) * sizeof(md::pages::ForkJob));
  return MD_OK;
}

md_status md_pages_fork(md_bf16* k_pages, md_bf16* v_pages, int32_t layers, int32_t pool_pages, int32_t Hkv,
                        int32_t page_size, int32_t dh, int32_t* block_table, int32_t* n_pages, int32_t* refcount,
                        int32_t* length, int32_t B, int32_t max_pages, const int32_t* src, const int32_t* dst,
                        int32_t n, void* ws, size_t ws_bytes, void* stream) {
  if (!k_pages || !v_pages || !block_table || !n_pages || !refcount || !length || !src || !dst) return MD_ERR_INVALID_ARG;
  size_t need = 0;
  md_status s = md_pages_fork_workspace(B, n, &need);
  if (s != MD_OK) return s;
  if (layers < 1) return MD_ERR_INVALID_ARG;
  if ((s = paged_check(B, pool_pages, page_size, max_pages, Hkv, dh)) != MD_OK) return s;
  // the copy counts layers' heads, and a head's 16-byte pieces of a page, in 32 bits
  if (int64_t(layers) * Hkv > INT32_MAX - md::pages::kCopyHeads ||
      int64_t(page_size) * (dh / 8) > INT32_MAX - md::pages::kCopyLoads * md::pages::kCopyThreads)
    return MD_ERR_UNSUPPORTED;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(refcount, 16)) return MD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  md::pages::ForkArgs a;
  a.table = block_table; a.n_pages = n_pages; a.refcount = refcount; a.length = length; a.src = src; a.dst = dst;
  a.jobs = static_cast<md::pages::ForkJob*>(ws);
  a.B = B; a.n = n; a.max_pages = max_pages; a.pool = pool_pages; a.page = page_size;
  if ((s = launch_pdl(md::pages::pages_fork_kernel, dim3(1), dim3(md::pages::kThreads), 0, st, a)) != MD_OK) return s;
  const dim3 grid((layers * Hkv + md::pages::kCopyHeads - 1) / md::pages::kCopyHeads, 2, n);
  return launch_pdl(md::pages::pages_fork_copy_kernel, grid, dim3(md::pages::kCopyThreads), 0, st,
                    reinterpret_cast<uint4*>(k_pages), reinterpret_cast<uint4*>(v_pages),
                    static_cast<const md::pages::ForkJob*>(a.jobs), layers, pool_pages, Hkv, page_size, dh / 8);
}

md_status md_get_device_status(void* stream, int32_t* out, int32_t clear) {
  if (!out) return MD_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  md_status s;
  if ((s = cuda_ok(cudaStreamSynchronize(st))) != MD_OK) return s;
  int v = 0;
  if ((s = cuda_ok(cudaMemcpyFromSymbol(&v, md::g_device_status, sizeof(int)))) != MD_OK) return s;
  *out = v;
  if (clear) {
    const int zero = 0;
    if ((s = cuda_ok(cudaMemcpyToSymbol(md::g_device_status, &zero, sizeof(int)))) != MD_OK) return s;
  }
  return MD_OK;
}

md_status md_set_wait_limit(uint64_t ns) {
  const unsigned long long v = ns == 0 ? md::kWaitLimitNs : (unsigned long long)ns;
  return cuda_ok(cudaMemcpyToSymbol(md::g_wait_limit_ns, &v, sizeof(v)));
}

md_status md_test_withhold_attention_chunk(int32_t chunk) {
  if (chunk < -1) return MD_ERR_INVALID_ARG;
  const int v = chunk;
  return cuda_ok(cudaMemcpyToSymbol(md::g_withhold_chunk, &v, sizeof(v)));
}

namespace {

// Read-only stream: 8 independent 16-byte loads per thread in flight.
__global__ void __launch_bounds__(512) stream_read_kernel(const uint4* __restrict__ p, size_t n16, uint32_t* sink) {
  constexpr int U = 8;
  uint32_t acc = 0;
  const size_t stride = size_t(gridDim.x) * blockDim.x;
  size_t i = size_t(blockIdx.x) * blockDim.x + threadIdx.x;
  for (; i + (U - 1) * stride < n16; i += U * stride) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = md::ld_stream_v4(p + i + u * stride);
#pragma unroll
    for (int u = 0; u < U; ++u) acc ^= v[u].x ^ v[u].y ^ v[u].z ^ v[u].w;
  }
  for (; i < n16; i += stride) {
    const uint4 v = md::ld_stream_v4(p + i);
    acc ^= v.x ^ v.y ^ v.z ^ v.w;
  }
  if (acc == 0x9E3779B9u) *sink = acc;   // keeps the loads; almost never written
}

}  // namespace

md_status md_stream_read(const void* buf, size_t bytes, uint32_t* sink, void* stream) {
  if (!buf || !sink || bytes % 16 != 0 || !aligned(buf, 16) || !aligned(sink, 4)) return MD_ERR_INVALID_ARG;
  if (bytes == 0) return MD_OK;
  stream_read_kernel<<<dim3(num_sms() * 4), 512, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint4*>(buf), bytes / 16, sink);
  return last_launch();
}

const char* md_status_string(md_status status) {
  switch (status) {
    case MD_OK: return "ok";
    case MD_ERR_INVALID_ARG: return "invalid argument";
    case MD_ERR_UNSUPPORTED: return "unsupported size or layout";
    case MD_ERR_CUDA: return "CUDA runtime error";
    case MD_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case MD_ERR_TIMEOUT: return "a bounded device wait gave up";
    default: return "unknown status";
  }
}

int32_t md_version(void) { return 100; }

}  // extern "C"
