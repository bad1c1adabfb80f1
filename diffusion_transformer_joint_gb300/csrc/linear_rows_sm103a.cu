// flux_linear for few rows, on sm_103a (GB300): the weights stream once
// through tcgen05 as the M operand, the token rows are its N operand.
//
//   out[b, s, :] = residual[b, s, :] + gate[b, :] * act([x | x2][b, s, :] W^T + bias)
//
// With few rows the call is bound by reading W (2 bytes per weight), so a CTA
// takes a tile of 128 W rows against all tokens at once (T = B * roundup(S, 8)
// <= 256 accumulator columns) and every weight is read once. One W tile per
// CTA is too few CTAs to draw the memory's bandwidth when N is small, so the
// channels are split over a cluster of up to eight CTAs that work on the same
// W tile: each writes its fp32 partial sums to its shared memory, and after a
// cluster barrier every CTA adds the partials of its share of the tokens in
// rank order (the same order in every run) through distributed shared memory
// and writes the finished rows. No workspace, no atomics, one launch.
//
// For SwiGLU the 128 W rows of a tile are 64 gate rows and the 64 linear rows
// of the same outputs.
//
// 8 warps: warp 0 TMA producer, warp 1 MMA issuer (one M128 N=T K16 MMA per
// 16 channels), warp 2 TMEM allocation; then all eight move the accumulator
// to shared memory (one TMEM lane, i.e. W row, per thread: consecutive lanes
// write consecutive words) over the drained stages and finish it. A stage is
// 64 channels: 16 KB of W and T rows of x.
#include <algorithm>
#include <mutex>

#include "linear_common.cuh"

namespace flux {
namespace {

constexpr int kWRows = 128;
constexpr int kK = 64;
constexpr uint32_t kWBytes = kWRows * kK * 2;
constexpr int kMaxStages = 12;
constexpr int kThreads = 256;
constexpr uint32_t kSmemAll = 232448;       // one CTA per SM
constexpr uint32_t kSmemHalf = 114688;      // two CTAs per SM
constexpr uint32_t kTailBytes = 256 + 1024;  // barriers and flags, alignment slack

struct RowsShape {
  int64_t N, o_bs, o_rs, r_bs, r_rs;
  int S, Sp, T;     // tokens per batch element, rounded up to 8; accumulator columns
  int n_tok;        // B * Sp
  int nk1, nk;      // stages of x, in all
  int stages, tmem_cols;
};

struct RowsMaps {
  CUtensorMap x, x2, w, w2;
};

__device__ __forceinline__ void bounded(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < kWaitBudgetCycles) {
  }
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 2)
    linear_rows_kernel(const __grid_constant__ RowsMaps maps, const RowsShape p,
                       const LinearEpilogue epi, const uint16_t *__restrict__ residual,
                       uint16_t *__restrict__ out, int *__restrict__ status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  constexpr int kFeats = kGlu ? kWRows / 2 : kWRows;  // output features per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(base);
  const uint32_t stage_bytes = kWBytes + static_cast<uint32_t>(p.T) * kK * 2;
  const uint32_t tail = static_cast<uint32_t>(p.stages) * stage_bytes;
  auto bar_full = [&](int s) { return sbase + tail + 16u * static_cast<uint32_t>(s); };
  auto bar_empty = [&](int s) { return sbase + tail + 16u * static_cast<uint32_t>(s) + 8u; };
  const uint32_t bar_acc = sbase + tail + 16u * kMaxStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + tail + 16 * kMaxStages + 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + tail + 16 * kMaxStages + 16);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int C = static_cast<int>(cluster_size());
  const int64_t f0 = static_cast<int64_t>(cluster_id_x()) * kFeats;
  // this CTA's channels: an even share of the stages (at least one: C <= nk)
  const int k_lo = static_cast<int>(static_cast<int64_t>(p.nk) * rank / C);
  const int k_hi = static_cast<int>(static_cast<int64_t>(p.nk) * (rank + 1) / C);

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_acc, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_addr(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    const uint32_t bytes = kWBytes + static_cast<uint32_t>(p.n_tok) * kK * 2;
    bool ok = true;
    int it = 0;
    for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
      const int s = it % p.stages;
      if (!(ok = mbar_wait(bar_empty(s), (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u,
                           abort_flag)))
        break;
      const uint32_t dst = sbase + static_cast<uint32_t>(s) * stage_bytes;
      mbar_arrive_expect_tx(bar_full(s), bytes);
      const bool first = ks < p.nk1;
      const int c = (first ? ks : ks - p.nk1) * kK;
      const void *wm = first ? &maps.w : &maps.w2;
      if constexpr (kGlu) {
        tma_load_3d(dst, wm, bar_full(s), c, static_cast<int>(f0), 0);
        tma_load_3d(dst + kWBytes / 2, wm, bar_full(s), c, static_cast<int>(p.N + f0), 0);
      } else {
        tma_load_3d(dst, wm, bar_full(s), c, static_cast<int>(f0), 0);
      }
      tma_load_3d(dst + kWBytes, first ? &maps.x : &maps.x2, bar_full(s), c, 0, 0);
    }
    // every copy has landed before the stages are written over or released
    for (int j = (it > p.stages ? it - p.stages : 0); j < it; ++j)
      bounded(bar_full(j % p.stages), static_cast<uint32_t>(j / p.stages) & 1u);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(kWRows, p.T, 0, 0);
    const uint64_t d0 = sdesc_sw128(sbase, 16, 1024);
    const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
    bool ok = true;
    int it = 0;
    for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
      const int s = it % p.stages;
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait(bar_full(s), static_cast<uint32_t>(it / p.stages) & 1u,
                                      abort_flag))))
        break;
      tc_fence_after_sync();
      const uint32_t st = sbase + static_cast<uint32_t>(s) * stage_bytes;
      const uint32_t da = static_cast<uint32_t>(sdesc_sw128(st, 16, 1024));
      const uint32_t db = static_cast<uint32_t>(sdesc_sw128(st + kWBytes, 16, 1024));
#pragma unroll
      for (int kk = 0; kk < kK / 16; ++kk)
        mma_ss_elect(tmem, da + kk * 2, db + kk * 2, hi, idesc, (it | kk) != 0 ? 1u : 0u);
      mma_commit_elect(bar_empty(s));
    }
    mma_commit_elect(bar_acc);
  }
  __syncwarp();
  // every MMA has finished: the accumulator is complete and the stages free
  // (every thread waits; an aborted CTA's MMAs in flight are waited for too)
  bounded(bar_acc, 0);
  tc_fence_after_sync();
  __syncthreads();  // the producer has seen its last copies land
  {
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t col = static_cast<uint32_t>((warp & 3) * 32 + lane) * 4;
    for (int c = warp >> 2; c < p.T / 16; c += 2) {
      uint32_t r[16];
      tmem_ld16(tmem + lane_off + c * 16, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        st_shared_b32(sbase + static_cast<uint32_t>(c * 16 + i) * (kWRows * 4) + col, r[i]);
    }
  }
  tc_fence_before_sync();
  if (C > 1)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 2) tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));

  // tokens rank, rank + C, ...: eight features per thread
  constexpr int kOct = kFeats / 8;
  const int n_mine = (p.n_tok - rank + C - 1) / C;
  for (int i = tid; i < n_mine * kOct; i += kThreads) {
    const int tok = rank + (i / kOct) * C;
    const int o = i % kOct;
    const int b = tok / p.Sp;
    const int s = tok - b * p.Sp;
    const int64_t f = f0 + o * 8;
    if (s >= p.S || f >= p.N) continue;
    uint4 res = make_uint4(0, 0, 0, 0);
    if (residual != nullptr)
      res = *reinterpret_cast<const uint4 *>(residual + b * p.r_bs + s * p.r_rs + f);
    float a[8] = {}, u[8] = {};
    const uint32_t at = sbase + static_cast<uint32_t>(tok) * (kWRows * 4) + o * 32;
    for (int r = 0; r < C; ++r) {
      const uint32_t pr = mapa_shared(at, static_cast<uint32_t>(r));
      const float4 v0 = ld_cluster_f4(pr), v1 = ld_cluster_f4(pr + 16);
      a[0] += v0.x, a[1] += v0.y, a[2] += v0.z, a[3] += v0.w;
      a[4] += v1.x, a[5] += v1.y, a[6] += v1.z, a[7] += v1.w;
      if constexpr (kGlu) {
        const float4 w0 = ld_cluster_f4(pr + kFeats * 4), w1 = ld_cluster_f4(pr + kFeats * 4 + 16);
        u[0] += w0.x, u[1] += w0.y, u[2] += w0.z, u[3] += w0.w;
        u[4] += w1.x, u[5] += w1.y, u[6] += w1.z, u[7] += w1.w;
      }
    }
    const int64_t gate_row =
        epi.gate != nullptr ? (static_cast<int64_t>(b) * p.S + s) / epi.gate_rows : 0;
    const uint4 y = finish8<kAct>(epi, p.N, f, gate_row, a, u, residual != nullptr, res);
    *reinterpret_cast<uint4 *>(out + b * p.o_bs + s * p.o_rs + f) = y;
  }
  if (C > 1) cluster_sync_all();  // no CTA leaves while another reads its partials
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

// CTAs that split the channels of one W tile: enough of them that about two
// CTAs per SM stream W, each with at least four stages to itself.
int pick_split(int64_t tiles, int nk, int sms) {
  int c = 1;
  while (c < 8 && tiles * c < sms && nk / (2 * c) >= 4) c *= 2;
  return c;
}

template <int kAct>
cudaError_t launch(const LinearProblem &q, const LinearEpilogue &epi, int *status,
                   cudaStream_t stream) {
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = linear_rows_kernel<kAct>;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemAll));
  });
  if (attr_err[dev] != cudaSuccess) return attr_err[dev];
  const bool glu = kAct == FLUX_ACT_SWIGLU;
  RowsShape p;
  p.N = q.N;
  p.o_bs = q.o_bs, p.o_rs = q.o_rs, p.r_bs = q.r_bs, p.r_rs = q.r_rs;
  p.S = static_cast<int>(q.S);
  p.Sp = (p.S + 7) / 8 * 8;
  const int64_t n_tok = q.B * p.Sp;
  if (n_tok > kLinearRowsMax) return cudaErrorInvalidValue;
  p.n_tok = static_cast<int>(n_tok);
  p.T = (p.n_tok + 15) / 16 * 16;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.T) p.tmem_cols *= 2;
  p.nk1 = (q.K + kK - 1) / kK;
  p.nk = p.nk1 + (q.K2 + kK - 1) / kK;
  const uint32_t stage = kWBytes + static_cast<uint32_t>(p.T) * kK * 2;
  // the partial sums (512 bytes per token) take the stages' place
  const uint32_t budget = (p.T <= 64 ? kSmemHalf : kSmemAll) - kTailBytes;
  p.stages = static_cast<int>(std::min<uint32_t>(kMaxStages, budget / stage));
  const int64_t feats = glu ? kWRows / 2 : kWRows;
  const int64_t tiles = (q.N + feats - 1) / feats;
  const int C = pick_split(tiles, p.nk, sm_count_current_device());
  const int64_t wr = glu ? 2 * q.N : q.N;
  const uint32_t w_box = glu ? kWRows / 2 : kWRows;
  RowsMaps maps;
  const uint16_t *w2 = static_cast<const uint16_t *>(q.w) + q.K;
  if (!make_row_map(&maps.x, q.x, q.K, q.S, q.B, q.x_rs, q.x_bs, kK, p.Sp,
                    static_cast<uint32_t>(q.B)) ||
      !make_row_map(&maps.w, q.w, q.K, wr, 1, q.w_rs, q.w_rs * wr, kK, w_box, 1))
    return cudaErrorInvalidValue;
  maps.x2 = maps.x;
  maps.w2 = maps.w;
  if (q.K2 > 0 &&
      (!make_row_map(&maps.x2, q.x2, q.K2, q.S, q.B, q.x2_rs, q.x2_bs, kK, p.Sp,
                     static_cast<uint32_t>(q.B)) ||
       !make_row_map(&maps.w2, w2, q.K2, wr, 1, q.w_rs, q.w_rs * wr, kK, w_box, 1)))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * C), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<uint32_t>(p.stages) * stage + kTailBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, epi,
                            static_cast<const uint16_t *>(q.residual),
                            static_cast<uint16_t *>(q.out), status);
}

}  // namespace

cudaError_t launch_linear_rows(const LinearProblem &q, const LinearEpilogue &epi, int act,
                               int *status, cudaStream_t stream) {
  switch (act) {
    case FLUX_ACT_NONE: return launch<FLUX_ACT_NONE>(q, epi, status, stream);
    case FLUX_ACT_SILU: return launch<FLUX_ACT_SILU>(q, epi, status, stream);
    case FLUX_ACT_GELU_TANH: return launch<FLUX_ACT_GELU_TANH>(q, epi, status, stream);
    default: return launch<FLUX_ACT_SWIGLU>(q, epi, status, stream);
  }
}

}  // namespace flux
