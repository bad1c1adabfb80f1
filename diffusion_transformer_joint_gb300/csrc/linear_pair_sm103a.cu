// flux_linear for many rows, on sm_103a (GB300): a bf16 GEMM on tcgen05 CTA
// pairs whose epilogue applies the bias, the activation, the gate and the
// residual.
//
//   out[b, s, :] = residual[b, s, :] + gate[b, :] * act([x | x2][b, s, :] W^T + bias)
//
// Tiles: 256 token rows of one batch element x `tn` accumulator columns, 64
// channels per pipeline stage (one 128-byte swizzle row of bf16). The tile's
// columns are tn output features; for SwiGLU tn/2 gate features and the
// linear features of the same tn/2 outputs, so that the epilogue holds both
// factors of what it writes. tn is a launch parameter (the MMA's N is part of
// its instruction descriptor), chosen by pick_tile.
//
// CTA pairs (clusters of two, one CTA per SM): one M256 N=tn K16 MMA per 16
// channels, issued by the even CTA and reading both CTAs' shared memory. Each
// CTA copies its own 128 token rows and half of the tile's W rows. x2
// continues the channels of x: its stages follow those of x, from tensor maps
// of their own, so that the concatenation is never written to memory and the
// ragged last stage of either part is filled with zeros on both operands.
//
// Persistent: a pair walks tiles round robin. Tiles are numbered in groups of
// kGroup row blocks, feature tiles major and row blocks minor inside a group,
// so that the pairs running at the same time form a block of about kGroup row
// blocks x (pairs / kGroup) feature tiles and share both operands in L2.
//
// 8 warps per CTA:
//   warp 0: TMA producer (6-stage ring);
//   warp 1: MMA issuer in the even CTA (whole warp, elect.sync issues);
//   warp 2: TMEM allocation (two 256-column accumulators, pair-wide);
//   warps 4-7: epilogue, one TMEM lane (token row) per thread, 32 features at
//   a time. A warp stages its 32 rows x 32 features in a 2 KB box (64-byte
//   swizzle, a ring of four per warp). With a residual the box is first filled
//   by a TMA copy of the residual, issued two boxes ahead (the first two of a
//   tile before its accumulator is waited for), and updated in place; lane 0
//   stores the box with one TMA copy. Rows past S and features past N are
//   neither read nor written.
// The two accumulators let the epilogue of one tile overlap the next tile's
// MMAs. Every wait is bounded; a wait that runs out aborts the CTA and sets
// the status word to FLUX_ERR_DEVICE_TIMEOUT.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "linear_common.cuh"

namespace flux {
namespace {

constexpr int kRows = 128;  // token rows per CTA (256 per pair)
constexpr int kMaxTn = 256;
constexpr int kK = 64;  // channels per stage
constexpr int kStages = 6;
constexpr int kGroup = 9;
constexpr uint32_t kABytes = kRows * kK * 2;         // 16 KB: this CTA's token rows
constexpr uint32_t kBBytes = kMaxTn / 2 * kK * 2;    // up to 16 KB: its half of the W rows
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr int kThreads = 256;
constexpr int kBoxes = 4;                 // boxes per epilogue warp
constexpr uint32_t kBoxBytes = 32 * 64;   // 32 rows x 32 features
constexpr int kBarFull = 0;               // (even CTA) both CTAs' copies landed
constexpr int kBarEmpty = kStages;        // the pair's MMAs read the stage
constexpr int kBarAccFull = 2 * kStages;
constexpr int kBarAccEmpty = kBarAccFull + 2;  // (even CTA) both epilogues read it
constexpr int kBarDrain = kBarAccEmpty + 2;
constexpr int kBarRes = kBarDrain + 1;  // residual box landed, per warp and box
constexpr int kNumBars = kBarRes + 4 * kBoxes;
constexpr uint32_t kOffBox = kStages * kStageBytes;
constexpr uint32_t kOffBar = kOffBox + 4 * kBoxes * kBoxBytes;
constexpr uint32_t kOffTmemSlot = kOffBar + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmemSlot + 8;
constexpr uint32_t kSmemBytes = kOffAbort + 8 + 1024;  // + slack for 1024-byte alignment
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
constexpr uint16_t kPairMask = 0x3;

struct PairShape {
  int64_t S, N;
  int tn, nk1, nk;            // tile width; stages of x; stages in all
  int n_sb, n_rb, n_ft, n_tiles;  // row blocks per batch element, in all; feature tiles
};

struct PairMaps {
  CUtensorMap x, x2, w, w2, out, res;
};

// Tile t of the walk -> feature tile and row block.
__device__ __forceinline__ void tile_at(const PairShape &p, int t, int &ft, int &rb) {
  const int per = kGroup * p.n_ft;
  const int g = t / per;
  const int first = g * kGroup;
  const int size = p.n_rb - first < kGroup ? p.n_rb - first : kGroup;
  const int rem = t - g * per;
  ft = rem / size;
  rb = first + rem - ft * size;
}

__device__ __forceinline__ void bounded(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < kWaitBudgetCycles) {
  }
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairMaps maps, const PairShape p,
                       const LinearEpilogue epi, const int has_res, int *__restrict__ status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(base);
  auto bar = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + kOffTmemSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + kOffAbort);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t crank = cluster_ctarank();  // 0: issues the MMAs
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  const int feats = kGlu ? p.tn / 2 : p.tn;  // output features per tile

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(kBarAccFull + b), 1);
      mbar_init(bar(kBarAccEmpty + b), 8);  // four epilogue warps of each CTA
    }
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < 4 * kBoxes; ++i) mbar_init(bar(kBarRes + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(tmem_slot), 2 * kMaxTn);
    tmem_relinquish_pair();
  }
  // both CTAs' barriers are initialised before either signals the other's
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------- TMA producer
    const uint32_t bytes = kABytes + static_cast<uint32_t>(p.tn / 2) * kK * 2;
    int it = 0;  // stages filled so far
    bool ok = true;
    for (int t = cid; ok && t < p.n_tiles; t += ncl) {
      int ft, rb;
      tile_at(p, t, ft, rb);
      const int b = rb / p.n_sb;
      const int s0 = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows;
      // the even CTA's W rows: the tile's first half, or its gate features;
      // the odd CTA's: the second half, or the linear features
      const int64_t f0 = static_cast<int64_t>(ft) * feats;
      const int rw = static_cast<int>(crank == 0 ? f0 : kGlu ? p.N + f0 : f0 + p.tn / 2);
      for (int ks = 0; ks < p.nk; ++ks, ++it) {
        const int s = it % kStages;
        const uint32_t use = static_cast<uint32_t>(it / kStages);
        if (!(ok = mbar_wait_cluster(bar(kBarEmpty + s), (use & 1u) ^ 1u, abort_flag))) break;
        const uint32_t dst = sbase + s * kStageBytes;
        // both CTAs' copies complete on the even CTA's stage barrier
        if (crank == 0) mbar_arrive_expect_tx(bar(kBarFull + s), 2 * bytes);
        const uint32_t full0 = mapa_shared(bar(kBarFull + s), 0);
        const bool first = ks < p.nk1;
        const int c = (first ? ks : ks - p.nk1) * kK;
        tma_load_3d_pair(dst, first ? &maps.x : &maps.x2, full0, c, s0, b);
        tma_load_3d_pair(dst + kABytes, first ? &maps.w : &maps.w2, full0, c, rw, 0);
      }
    }
    // every copy of the pair has landed before the CTAs exit (the even CTA's
    // stage barriers count both CTAs' copies; the final cluster barrier
    // keeps the odd CTA until then)
    if (crank == 0)
      for (int j = (it > kStages ? it - kStages : 0); j < it; ++j)
        bounded(bar(kBarFull + j % kStages), static_cast<uint32_t>(j / kStages) & 1u);
  } else if (warp == 1 && crank == 0) {
    // ------------------------------------------------ MMA issuer (even CTA)
    const uint32_t idesc = idesc_bf16_f32(2 * kRows, p.tn, 0, 0);
    int it = 0;
    int lt = 0;
    bool ok = true;
    for (int t = cid; ok && t < p.n_tiles; t += ncl, ++lt) {
      const int buf = lt & 1;
      const uint32_t acc_par = ((static_cast<uint32_t>(lt) >> 1) & 1u) ^ 1u;
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait_cluster(bar(kBarAccEmpty + buf), acc_par, abort_flag))))
        break;
      tc_fence_after_sync();
      const uint32_t d = tmem + static_cast<uint32_t>(buf * kMaxTn);
      for (int ks = 0; ks < p.nk; ++ks, ++it) {
        const int s = it % kStages;
        const uint32_t par = static_cast<uint32_t>(it / kStages) & 1u;
        if (!(ok = __all_sync(0xffffffffu,
                              mbar_wait_cluster(bar(kBarFull + s), par, abort_flag))))
          break;
        tc_fence_after_sync();
        const uint64_t da = sdesc_sw128(sbase + s * kStageBytes, 16, 1024);
        const uint64_t db = sdesc_sw128(sbase + s * kStageBytes + kABytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kK / 16; ++kk)
          mma_ss_pair_elect(d, desc_advance(da, kk * 32), desc_advance(db, kk * 32), idesc,
                            (ks | kk) != 0 ? 1u : 0u);
        mma_commit_pair_elect(bar(kBarEmpty + s), kPairMask);  // both CTAs may refill
      }
      if (!ok) break;
      mma_commit_pair_elect(bar(kBarAccFull + buf), kPairMask);  // both accumulators complete
    }
    // every MMA issued above has finished before TMEM is released
    mma_commit_pair_elect(bar(kBarDrain), 0x1);
    bounded(bar(kBarDrain), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int wq = warp & 3;  // TMEM lane quadrant
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t acc_empty0 = mapa_shared(bar(kBarAccEmpty), 0);
    const uint32_t boxes = sbase + kOffBox + static_cast<uint32_t>(wq) * kBoxes * kBoxBytes;
    const int bar_res = kBarRes + wq * kBoxes;
    uint32_t n_loaded = 0, n_stored = 0;  // boxes of this warp whose residual was asked for / staged
    int lt = 0;
    bool ok = true;
    for (int t = cid; ok && t < p.n_tiles; t += ncl, ++lt) {
      int ft, rb;
      tile_at(p, t, ft, rb);
      const int b = rb / p.n_sb;
      const int s0 = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows + wq * 32;
      const int64_t f0 = static_cast<int64_t>(ft) * feats;
      const int64_t left = p.N - f0;
      // boxes of this tile that hold anything to write
      const int n_box = s0 >= p.S ? 0
                                  : static_cast<int>(left < feats ? (left + 31) / 32 : feats / 32);
      const int64_t row = static_cast<int64_t>(b) * p.S + (s0 + lane < p.S ? s0 + lane : p.S - 1);
      const int64_t gate_row = epi.gate != nullptr ? row / epi.gate_rows : 0;
      // the residual of box c: its buffer was last stored from kBoxes boxes
      // ago, at most one later store may still be reading
      auto load_residual = [&](int c) {
        const uint32_t slot = n_loaded % kBoxes;
        if (lane == 0) {
          bulk_wait_read_1();
          mbar_arrive_expect_tx(bar(bar_res + slot), kBoxBytes);
          tma_load_3d(boxes + slot * kBoxBytes, &maps.res, bar(bar_res + slot),
                      static_cast<int>(f0) + c * 32, s0, b);
        }
        ++n_loaded;
      };
      if (has_res)
        for (int c = 0; c < 2 && c < n_box; ++c) load_residual(c);
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait_cluster(bar(kBarAccFull + (lt & 1)),
                                              (static_cast<uint32_t>(lt) >> 1) & 1u, abort_flag))))
        break;
      tc_fence_after_sync();
      const uint32_t tacc = tmem + static_cast<uint32_t>((lt & 1) * kMaxTn) + lane_off;
#pragma unroll 1
      for (int c = 0; c < n_box; ++c) {
        const uint32_t slot = n_stored % kBoxes;
        const uint32_t box = boxes + slot * kBoxBytes;
        uint32_t a[32], u[32];
        tmem_ld32(tacc + c * 32, a);
        if constexpr (kGlu) tmem_ld32(tacc + feats + c * 32, u);
        if (has_res) {
          if (c + 2 < n_box) load_residual(c + 2);
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(bar_res + slot),
                                                       (n_stored / kBoxes) & 1u, abort_flag))))
            break;
        } else {
          if (lane == 0) bulk_wait_read_3();
          __syncwarp();
        }
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t f = f0 + c * 32 + g * 8;
          const uint32_t at = box + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4);
          if (f < p.N) {
            float av[8], uv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              av[i] = __uint_as_float(a[g * 8 + i]);
              uv[i] = kGlu ? __uint_as_float(u[g * 8 + i]) : 0.f;
            }
            uint4 res = make_uint4(0, 0, 0, 0);
            if (has_res) res = ld_shared_v4(at);
            st_shared_v4(at, finish8<kAct>(epi, p.N, f, gate_row, av, uv, has_res != 0, res));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out, box, static_cast<int>(f0) + c * 32, s0, b);
          bulk_commit();
        }
        ++n_stored;
      }
      if (!ok) break;
      // this warp's TMEM reads are complete: the accumulator may be reused
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8u * static_cast<uint32_t>((lt & 1)));
    }
    if (lane == 0) {
      // residual copies still in flight after an abort, then every output store
      for (uint32_t j = n_stored; j < n_loaded; ++j)
        bounded(bar(bar_res + j % kBoxes), (j / kBoxes) & 1u);
      bulk_wait_all();
    }
  }

  // neither CTA leaves while the other may still signal its barriers or
  // read its shared memory
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();
  if (warp == 2) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 2 * kMaxTn);
  }
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

// Tile width: the accumulator columns of a tile, a multiple of 32 (64 for
// SwiGLU). A stage of 64 channels keeps a pair busy for about 256 + tn cycles
// (its 128 token rows and tn/2 W rows per CTA have to arrive from L2; at
// tn = 256 the MMAs take the same 512), so a wave of tiles costs 256 + tn and
// the width with the cheapest sum of waves is taken, the widest among equals.
int pick_tile(int64_t n_rb, int64_t N, bool glu, int pairs) {
  const int step = glu ? 64 : 32;
  int best = kMaxTn;
  int64_t best_cost = INT64_MAX;
  for (int tn = kMaxTn; tn >= step; tn -= step) {
    const int64_t feats = glu ? tn / 2 : tn;
    const int64_t tiles = n_rb * ((N + feats - 1) / feats);
    const int64_t cost = (tiles + pairs - 1) / pairs * (256 + tn);
    if (cost < best_cost) best_cost = cost, best = tn;
  }
  return best;
}

template <int kAct>
cudaError_t launch(const LinearProblem &q, const LinearEpilogue &epi, int *status,
                   cudaStream_t stream) {
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  static std::atomic<int> max_pairs[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = linear_pair_kernel<kAct>;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
  });
  if (attr_err[dev] != cudaSuccess) return attr_err[dev];
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int np = max_pairs[dev].load(std::memory_order_relaxed);
  if (np == 0) {
    cfg.gridDim = dim3(2, 1, 1);
    e = cudaOccupancyMaxActiveClusters(&np, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (np < 1) return cudaErrorInvalidConfiguration;
    max_pairs[dev].store(np, std::memory_order_relaxed);
  }
  const bool glu = kAct == FLUX_ACT_SWIGLU;
  PairShape p;
  p.S = q.S;
  p.N = q.N;
  const int64_t n_sb = (q.S + 2 * kRows - 1) / (2 * kRows);
  const int64_t n_rb = n_sb * q.B;
  p.tn = pick_tile(n_rb, q.N, glu, np);
  const int64_t feats = glu ? p.tn / 2 : p.tn;
  const int64_t n_ft = (q.N + feats - 1) / feats;
  if (n_rb * n_ft > 0x3FFFFFFFLL || n_ft * kGroup > 0x3FFFFFFFLL) return cudaErrorInvalidValue;
  p.n_sb = static_cast<int>(n_sb);
  p.n_rb = static_cast<int>(n_rb);
  p.n_ft = static_cast<int>(n_ft);
  p.n_tiles = static_cast<int>(n_rb * n_ft);
  p.nk1 = (q.K + kK - 1) / kK;
  p.nk = p.nk1 + (q.K2 + kK - 1) / kK;
  const int64_t wr = glu ? 2 * q.N : q.N;
  const uint32_t w_box = static_cast<uint32_t>(p.tn / 2);
  PairMaps maps;
  const uint16_t *w2 = static_cast<const uint16_t *>(q.w) + q.K;
  if (!make_row_map(&maps.x, q.x, q.K, q.S, q.B, q.x_rs, q.x_bs, kK, kRows, 1) ||
      !make_row_map(&maps.w, q.w, q.K, wr, 1, q.w_rs, q.w_rs * wr, kK, w_box, 1) ||
      !make_row_map(&maps.out, q.out, q.N, q.S, q.B, q.o_rs, q.o_bs, 32, 32, 1))
    return cudaErrorInvalidValue;
  maps.x2 = maps.x;
  maps.w2 = maps.w;
  maps.res = maps.out;
  if (q.K2 > 0 &&
      (!make_row_map(&maps.x2, q.x2, q.K2, q.S, q.B, q.x2_rs, q.x2_bs, kK, kRows, 1) ||
       !make_row_map(&maps.w2, w2, q.K2, wr, 1, q.w_rs, q.w_rs * wr, kK, w_box, 1)))
    return cudaErrorInvalidValue;
  if (q.residual != nullptr &&
      !make_row_map(&maps.res, q.residual, q.N, q.S, q.B, q.r_rs, q.r_bs, 32, 32, 1))
    return cudaErrorInvalidValue;
  const int64_t pairs = p.n_tiles < np ? p.n_tiles : np;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, epi, q.residual != nullptr ? 1 : 0, status);
}

}  // namespace

bool make_row_map(CUtensorMap *map, const void *base, int64_t cols, int64_t S, int64_t B,
                  int64_t row_stride, int64_t batch_stride, uint32_t box_cols, uint32_t box_rows,
                  uint32_t box_b) {
  auto fn = reinterpret_cast<CUresult (*)(
      CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
      const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)>(
      tensor_map_encode_entry());
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(S),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_stride) * 2,
                                 static_cast<cuuint64_t>(batch_stride) * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, box_b};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_linear_pair(const LinearProblem &q, const LinearEpilogue &epi, int act,
                               int *status, cudaStream_t stream) {
  switch (act) {
    case FLUX_ACT_NONE: return launch<FLUX_ACT_NONE>(q, epi, status, stream);
    case FLUX_ACT_SILU: return launch<FLUX_ACT_SILU>(q, epi, status, stream);
    case FLUX_ACT_GELU_TANH: return launch<FLUX_ACT_GELU_TANH>(q, epi, status, stream);
    default: return launch<FLUX_ACT_SWIGLU>(q, epi, status, stream);
  }
}

}  // namespace flux
