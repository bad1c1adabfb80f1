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
// its instruction descriptor), chosen by plan_pair.
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
// 12 warps per CTA:
//   warp 0: TMA producer (a ring of 192 KB: six stages of a 256-column tile, up
//   to ten of narrower ones: a copy takes about 1.5 us to land, so the bytes on
//   their way bound what a CTA draws);
//   warp 1: MMA issuer in the even CTA (whole warp, elect.sync issues);
//   warp 2: TMEM allocation (two 256-column accumulators, pair-wide);
//   warps 4-11: epilogue, one TMEM lane (token row) per thread, 32 features at
//   a time, two warps per lane quadrant taking turns. The tile's bias and gate
//   are staged in shared memory as fp32 while its MMAs run. A warp stages its
//   32 rows x 32 features in one of two 2 KB boxes (64-byte swizzle). With a
//   residual the box is first filled by a TMA copy of the residual, issued a
//   box ahead (the first two of a tile before its accumulator is waited for),
//   and updated in place; lane 0 stores the box with one TMA copy. Rows past S
//   and features past N are neither read nor written.
// The two accumulators let the epilogue of one tile overlap the next tile's
// MMAs; the last tile's is what a call pays for (4 us with the residual; with
// four warps, each reading bias and gate from global memory, it was 10 us).
//
// The launch overlaps its prologue with the end of the kernel before it in the
// stream (programmatic dependent launch): what reads or writes global memory
// waits for that kernel first. Every wait is bounded; a wait that runs out
// aborts the CTA and sets the status word to FLUX_ERR_DEVICE_TIMEOUT.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "linear_common.cuh"

namespace flux {
namespace {

constexpr int kRows = 128;  // token rows per CTA (256 per pair)
constexpr int kMaxTn = 256;
constexpr int kK = 64;  // channels per stage
constexpr uint32_t kRingBytes = 6 * 32768;  // of stages: 6 of the widest tile's, up to 10
constexpr int kMaxStages = 10;
constexpr int kGroup = 9;
constexpr uint32_t kABytes = kRows * kK * 2;  // 16 KB: this CTA's token rows
constexpr uint32_t kBRowBytes = kK * 2;       // a W row of its half of the tile
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kBoxes = 2;                 // boxes per epilogue warp
constexpr uint32_t kBoxBytes = 32 * 64;   // 32 rows x 32 features
constexpr int kBarFull = 0;               // (even CTA) both CTAs' copies landed
constexpr int kBarEmpty = kMaxStages;     // the pair's MMAs read the stage
constexpr int kBarAccFull = 2 * kMaxStages;
constexpr int kBarAccEmpty = kBarAccFull + 2;  // (even CTA) both epilogues read it
constexpr int kBarDrain = kBarAccEmpty + 2;
constexpr int kBarRes = kBarDrain + 1;  // residual box landed, per warp and box
constexpr int kBarVecReady = kBarRes + kEpiWarps * kBoxes;  // a tile's vectors are staged
constexpr int kBarVecFree = kBarVecReady + 1;               // every epilogue warp has read them
constexpr int kNumBars = kBarVecFree + 1;
constexpr uint32_t kOffBox = kRingBytes;
constexpr uint32_t kOffVec = kOffBox + kEpiWarps * kBoxes * kBoxBytes;  // a tile's bias, gate
constexpr uint32_t kOffBar = kOffVec + 2 * kMaxTn * 4;
constexpr uint32_t kOffTmemSlot = kOffBar + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmemSlot + 8;
constexpr uint32_t kSmemBytes = kOffAbort + 8;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
constexpr uint16_t kPairMask = 0x3;

struct PairShape {
  int64_t S, N;
  int tn, stages, nk1, nk;        // tile width; ring; stages of x, in all
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

__device__ __forceinline__ void read8(float (&v)[8], const float *p) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0];
  const float4 b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void add8(float (&v)[8], const float *p) {
  float w[8];
  read8(w, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += w[i];
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairMaps maps, const PairShape p,
                       const LinearEpilogue epi, const int has_res, int *__restrict__ status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  extern __shared__ __align__(1024) uint8_t base[];
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
  const uint32_t stage_bytes = kABytes + static_cast<uint32_t>(p.tn / 2) * kBRowBytes;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(kBarAccFull + b), 1);
      mbar_init(bar(kBarAccEmpty + b), 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < kEpiWarps * kBoxes; ++i) mbar_init(bar(kBarRes + i), 1);
    mbar_init(bar(kBarVecReady), kEpiWarps);
    mbar_init(bar(kBarVecFree), kEpiWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(tmem_slot), 2 * kMaxTn);
    tmem_relinquish_pair();
  }
  // both CTAs' barriers are initialised before either signals the other's
  tc_fence_before_sync();
  cluster_sync_relaxed();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch_dependents();

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------- TMA producer
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
    int s = 0;          // stage
    uint32_t turn = 0;  // times round the ring
    bool ok = true;
    // the even CTA's W rows: the tile's first half, or its gate features; the
    // odd CTA's: the second half, or the linear features
    auto w_row = [&](int ft) {
      const int64_t f0 = static_cast<int64_t>(ft) * feats;
      return static_cast<int>(crank == 0 ? f0 : kGlu ? p.N + f0 : f0 + p.tn / 2);
    };
    grid_dep_wait();
    for (int t = cid; ok && t < p.n_tiles; t += ncl) {
      int ft, rb;
      tile_at(p, t, ft, rb);
      const int b = rb / p.n_sb;
      const int s0 = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows;
      const int rw = w_row(ft);
      for (int ks = 0; ks < p.nk; ++ks) {
        if (!(ok = mbar_wait_cluster(bar(kBarEmpty + s), (turn & 1u) ^ 1u, abort_flag))) break;
        const uint32_t dst = sbase + s * stage_bytes;
        // both CTAs' copies complete on the even CTA's stage barrier
        if (crank == 0) mbar_arrive_expect_tx(bar(kBarFull + s), 2 * stage_bytes);
        const uint32_t full0 = mapa_shared(bar(kBarFull + s), 0);
        const bool first = ks < p.nk1;
        const int c = (first ? ks : ks - p.nk1) * kK;
        tma_load_3d_pair(dst, first ? &maps.x : &maps.x2, full0, c, s0, b);
        tma_load_3d_pair(dst + kABytes, first ? &maps.w : &maps.w2, full0, c, rw, 0);
        if (++s == p.stages) s = 0, ++turn;
      }
    }
    // every copy of the pair has landed before the CTAs exit (the even CTA's
    // stage barriers count both CTAs' copies; the final cluster barrier
    // keeps the odd CTA until then)
    if (crank == 0) {
      const long long until = clock64() + kWaitBudgetCycles;
      for (int i = 0; i < p.stages; ++i) {
        // the stage's last use, if any, was in this turn or the one before
        if (i < s)
          ok &= mbar_settled(bar(kBarFull + i), turn & 1u, until);
        else if (turn > 0)
          ok &= mbar_settled(bar(kBarFull + i), (turn - 1) & 1u, until);
      }
      if (!ok) *abort_flag = 1;
    }
  } else if (warp == 1 && crank == 0) {
    // ------------------------------------------------ MMA issuer (even CTA)
    const uint32_t idesc = idesc_bf16_f32(2 * kRows, p.tn, 0, 0);
    int s = 0;
    uint32_t turn = 0;
    int lt = 0;
    bool ok = true;
    grid_dep_wait();  // the budget of the first stage's wait begins with its copy
    for (int t = cid; ok && t < p.n_tiles; t += ncl, ++lt) {
      const int buf = lt & 1;
      const uint32_t acc_par = ((static_cast<uint32_t>(lt) >> 1) & 1u) ^ 1u;
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait_cluster(bar(kBarAccEmpty + buf), acc_par, abort_flag))))
        break;
      tc_fence_after_sync();
      const uint32_t d = tmem + static_cast<uint32_t>(buf * kMaxTn);
      for (int ks = 0; ks < p.nk; ++ks) {
        if (!(ok = __all_sync(0xffffffffu,
                              mbar_wait_cluster(bar(kBarFull + s), turn & 1u, abort_flag))))
          break;
        tc_fence_after_sync();
        const uint64_t da = sdesc_sw128(sbase + s * stage_bytes, 16, 1024);
        const uint64_t db = sdesc_sw128(sbase + s * stage_bytes + kABytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kK / 16; ++kk)
          mma_ss_pair_elect(d, desc_advance(da, kk * 32), desc_advance(db, kk * 32), idesc,
                            (ks | kk) != 0 ? 1u : 0u);
        mma_commit_pair_elect(bar(kBarEmpty + s), kPairMask);  // both CTAs may refill
        if (++s == p.stages) s = 0, ++turn;
      }
      if (!ok) break;
      mma_commit_pair_elect(bar(kBarAccFull + buf), kPairMask);  // both accumulators complete
    }
    // every MMA issued above has finished before TMEM is released
    mma_commit_pair_elect(bar(kBarDrain), 0x1);
    if (!mbar_settled(bar(kBarDrain), 0, clock64() + kWaitBudgetCycles)) *abort_flag = 1;
    __syncwarp();
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int wq = warp & 3;         // TMEM lane quadrant
    const int turn = (warp - 4) >> 2;  // takes the boxes of this parity
    const int et = tid - 128;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t acc_empty0 = mapa_shared(bar(kBarAccEmpty), 0);
    const uint32_t boxes = sbase + kOffBox + static_cast<uint32_t>(warp - 4) * kBoxes * kBoxBytes;
    const int bar_res = kBarRes + (warp - 4) * kBoxes;
    float *vec_bias = reinterpret_cast<float *>(base + kOffVec);
    float *vec_gate = vec_bias + kMaxTn;
    const bool vecs = epi.bias != nullptr || epi.gate != nullptr;
    uint32_t n_loaded = 0, n_stored = 0;  // this warp's boxes: residual asked for, staged
    int lt = 0;
    bool ok = true;
    grid_dep_wait();
    for (int t = cid; ok && t < p.n_tiles; t += ncl, ++lt) {
      int ft, rb;
      tile_at(p, t, ft, rb);
      const int b = rb / p.n_sb;
      const int sc = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows;
      const int s0 = sc + wq * 32;
      const int64_t f0 = static_cast<int64_t>(ft) * feats;
      const int64_t left = p.N - f0;
      // boxes of this tile that hold anything to write
      const int n_box = s0 >= p.S ? 0
                                  : static_cast<int>(left < feats ? (left + 31) / 32 : feats / 32);
      // the residual of box c goes to the buffer of this warp's box before
      // last, whose store has read it
      auto load_residual = [&](int c) {
        const uint32_t slot = n_loaded % kBoxes;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(bar_res + slot), kBoxBytes);
          tma_load_3d(boxes + slot * kBoxBytes, &maps.res, bar(bar_res + slot),
                      static_cast<int>(f0) + c * 32, s0, b);
        }
        ++n_loaded;
      };
      if (has_res) {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        for (int c = turn; c < n_box && c < turn + 2 * kBoxes; c += 2) load_residual(c);
      }
      // bias and gate of the tile, once every warp is done with the last one's
      // (a gate that changes inside the CTA's rows is read row by row instead)
      bool gate_rowwise = false;
      int64_t gate_row = 0;
      if (epi.gate != nullptr) {
        const int64_t r0 = static_cast<int64_t>(b) * p.S + (sc < p.S ? sc : p.S - 1);
        const int64_t r1 =
            static_cast<int64_t>(b) * p.S + (sc + kRows < p.S ? sc + kRows : p.S) - 1;
        gate_row = r0 / epi.gate_rows;
        gate_rowwise = r1 / epi.gate_rows != gate_row;
      }
      if (vecs) {
        // (barriers with bounded waits: an aborting warp leaves the others)
        if (lt > 0 && !(ok = __all_sync(0xffffffffu,
                                        mbar_wait(bar(kBarVecFree),
                                                  static_cast<uint32_t>(lt - 1) & 1u, abort_flag))))
          break;
        if (epi.bias != nullptr && et < p.tn) {
          const int64_t f = f0 + (kGlu && et >= feats ? et - feats : et);
          if (f < p.N)
            vec_bias[et] = load_vec1(epi.bias, kGlu && et >= feats ? p.N + f : f, epi.vec_f32);
        }
        if (epi.gate != nullptr && !gate_rowwise && et < feats && f0 + et < p.N)
          vec_gate[et] = load_vec1(epi.gate, gate_row * epi.gate_bs + f0 + et, epi.vec_f32);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarVecReady));
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarVecReady),
                                                     static_cast<uint32_t>(lt) & 1u, abort_flag))))
          break;
      }
      if (gate_rowwise) {
        const int64_t r = static_cast<int64_t>(b) * p.S + (s0 + lane < p.S ? s0 + lane : p.S - 1);
        gate_row = r / epi.gate_rows;
      }
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait_cluster(bar(kBarAccFull + (lt & 1)),
                                              (static_cast<uint32_t>(lt) >> 1) & 1u, abort_flag))))
        break;
      tc_fence_after_sync();
      const uint32_t tacc = tmem + static_cast<uint32_t>((lt & 1) * kMaxTn) + lane_off;
#pragma unroll 1
      for (int c = turn; c < n_box; c += 2) {
        const uint32_t slot = n_stored % kBoxes;
        const uint32_t box = boxes + slot * kBoxBytes;
        uint32_t a[32], u[32];
        tmem_ld32(tacc + c * 32, a);
        if constexpr (kGlu) tmem_ld32(tacc + feats + c * 32, u);
        if (has_res) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(bar_res + slot),
                                                       (n_stored / kBoxes) & 1u, abort_flag))))
            break;
        } else {
          if (lane == 0) bulk_wait_read_1();
          __syncwarp();
        }
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t f = f0 + c * 32 + g * 8;
          const uint32_t at = box + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4);
          if (f < p.N) {
            const int v0 = c * 32 + g * 8;  // in the tile's vectors
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(a[g * 8 + i]);
            if (epi.bias != nullptr) add8(y, vec_bias + v0);
            if constexpr (kGlu) {
              float w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(u[g * 8 + i]);
              if (epi.bias != nullptr) add8(w, vec_bias + feats + v0);
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = activate<FLUX_ACT_SILU>(y[i]) * w[i];
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = activate<kAct>(y[i]);
            }
            if (epi.gate != nullptr) {
              float w[8];
              if (gate_rowwise)
                load_vec8(epi.gate, gate_row * epi.gate_bs + f, epi.vec_f32, w);
              else
                read8(w, vec_gate + v0);
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] *= w[i];
            }
            if (has_res) {
              float w[8];
              unpack8(ld_shared_v4(at), w);
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] += w[i];
            }
            st_shared_v4(at, pack8(y));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out, box, static_cast<int>(f0) + c * 32, s0, b);
          bulk_commit();
        }
        ++n_stored;
        if (has_res && c + 2 * kBoxes < n_box) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
          load_residual(c + 2 * kBoxes);
        }
      }
      if (!ok) break;
      // this warp's TMEM reads are complete: the accumulator may be reused
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8u * static_cast<uint32_t>(lt & 1));
      if (vecs && lane == 0) mbar_arrive(bar(kBarVecFree));
    }
    if (lane == 0) {
      // residual copies still in flight after an abort, then every output store
      const long long until = clock64() + kWaitBudgetCycles;
      for (uint32_t j = n_stored; j < n_loaded; ++j)
        if (!mbar_settled(bar(bar_res + j % kBoxes), (j / kBoxes) & 1u, until)) *abort_flag = 1;
      bulk_wait_all();
    }
  }

  // neither CTA leaves while the other may still signal its barriers or read
  // its shared memory (signals under way count: a barrier with release)
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();
  if (warp == 2) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 2 * kMaxTn);
  }
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

template <int kAct>
cudaError_t launch(const LinearProblem &q, int tn, const LinearEpilogue &epi, int *status,
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
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
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
  p.tn = tn;
  const int64_t feats = glu ? p.tn / 2 : p.tn;
  const int64_t n_ft = (q.N + feats - 1) / feats;
  if (n_rb * n_ft > 0x3FFFFFFFLL || n_ft * kGroup > 0x3FFFFFFFLL) return cudaErrorInvalidValue;
  p.n_sb = static_cast<int>(n_sb);
  p.n_rb = static_cast<int>(n_rb);
  p.n_ft = static_cast<int>(n_ft);
  p.n_tiles = static_cast<int>(n_rb * n_ft);
  p.stages = static_cast<int>(std::min<uint32_t>(
      kMaxStages, kRingBytes / (kABytes + static_cast<uint32_t>(p.tn / 2) * kBRowBytes)));
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
  cfg.numAttrs = 2;
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

// The tile's width: a multiple of 32 accumulator columns (64 for SwiGLU). A
// wave of tiles costs its stages, so the width decides both how long a wave is
// and how full the last one: 4096 x 4096 outputs are four full waves of 224
// columns (79.8 us with 4096 channels), or 3.4 of 256 (81.6 us).
PairPlan plan_pair(const LinearProblem &q, int act, int sms) {
  const bool glu = act == FLUX_ACT_SWIGLU;
  const int64_t n_rb = q.B * ((q.S + 2 * kRows - 1) / (2 * kRows));
  const double nk = static_cast<double>((q.K + kK - 1) / kK + (q.K2 + kK - 1) / kK);
  const int64_t pairs = std::max(1, sms / 2);
  PairPlan best{kMaxTn, 1e30};
  const int step = glu ? 64 : 32;
  for (int tn = kMaxTn; tn >= step; tn -= step) {
    const int64_t feats = glu ? tn / 2 : tn;
    const int64_t tiles = n_rb * ((q.N + feats - 1) / feats);
    const double waves = static_cast<double>((tiles + pairs - 1) / pairs);
    const double ns = waves * (nk * stage_ns(kABytes + tn / 2 * kBRowBytes, tn) + 66.0) +
                      3640.0 + 9.7 * tn;
    if (ns < best.ns) best = PairPlan{tn, ns};
  }
  return best;
}

cudaError_t launch_linear_pair(const LinearProblem &q, const PairPlan &plan,
                               const LinearEpilogue &epi, int act, int *status,
                               cudaStream_t stream) {
  switch (act) {
    case FLUX_ACT_NONE: return launch<FLUX_ACT_NONE>(q, plan.tn, epi, status, stream);
    case FLUX_ACT_SILU: return launch<FLUX_ACT_SILU>(q, plan.tn, epi, status, stream);
    case FLUX_ACT_GELU_TANH: return launch<FLUX_ACT_GELU_TANH>(q, plan.tn, epi, status, stream);
    default: return launch<FLUX_ACT_SWIGLU>(q, plan.tn, epi, status, stream);
  }
}

}  // namespace flux
