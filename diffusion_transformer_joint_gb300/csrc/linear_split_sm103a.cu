// flux_linear where whole 256-row tiles would leave SMs idle (few rows, or few
// features), on sm_103a (GB300): tiles of 256 rows of one operand against up
// to 256 rows of the other, the channels split over a cluster.
//
//   out[b, s, :] = residual[b, s, :] + gate[b, :] * act([x | x2][b, s, :] W^T + bias)
//
// A tile is 256 x Q accumulators of a CTA pair: 256 rows of the operand P (128
// per CTA, the MMA's M) against Q <= 256 rows of the operand Q (half of them in
// each CTA's shared memory, the MMA's N). With few token rows P is W and Q
// holds every token (kTokensP false), so that the weights, which bound such a
// call, are read once. Otherwise P is token rows and Q features (kTokensP).
//
// Tiles alone are too few to draw the memory's bandwidth, and narrower ones
// are no help: an SM takes in about 110 GB/s, and a stage of 64 channels brings
// 128 bytes for each of its 128 + Q / 2 rows whatever the tile computes with
// them. So the channels of a tile are split over C = 1 to 4 pairs of a
// cluster: each CTA writes its fp32 partial sums to its shared memory and
// sends every other pair that pair's share of the tokens (bulk copies between
// the CTAs' shared memories, about 30 bytes per ns and SM); each then adds the
// partials of its own share in the pairs' order (the same in every run) and
// writes the finished rows. No workspace, no atomics, one launch.
//
// For SwiGLU the W rows of a tile are the gate rows of its outputs and their
// linear rows: side by side in each CTA as P, one CTA's each as Q.
//
// 16 warps: warp 0 TMA producer, warp 1 MMA issuer (in the pair's even CTA, one
// M256 N=Q K16 MMA per 16 channels), warp 2 TMEM allocation; then all of them
// move the CTA's 128 accumulator rows to shared memory over the drained stages
// and finish them. The prologue overlaps the end of the kernel before it
// (programmatic dependent launch). Every wait is bounded; a wait that runs out
// aborts the CTA and sets the status word to FLUX_ERR_DEVICE_TIMEOUT.
#include <algorithm>
#include <mutex>

#include "linear_common.cuh"

namespace flux {
namespace {

constexpr int kP = 128;  // rows of P per CTA
constexpr int kK = 64;
constexpr uint32_t kRowBytes = kK * 2;
constexpr uint32_t kPBytes = kP * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kMaxC = 4;  // pairs that split a tile's channels
constexpr int kThreads = 512;
constexpr uint32_t kSmemAll = 232448;   // one CTA per SM
constexpr uint32_t kSmemHalf = 114688;  // two CTAs per SM
constexpr uint32_t kTailBytes = 256;    // barriers and flags
// A ring that sums may have a place of their own beside: with less on its way
// than about 1.5 us of what an SM takes in, the stages wait for the memory.
constexpr uint32_t kEarlyRing = 176 * 1024;

struct SplitShape {
  int64_t N, o_bs, o_rs, r_bs, r_rs;
  int S;           // tokens per batch element of the launch
  int Q;           // tile columns
  int q_rows;      // rows of Q that each CTA copies
  int Sh;          // tokens as Q: half a batch element's tokens, rounded up to 8
  int n_sb;        // tokens as P: 256-row blocks per batch element
  int n_ft;        // feature tiles
  int feats;       // output features per tile (of a CTA, with W as P)
  int nk1, nk;     // stages of x, in all
  int stages, tmem_cols;
  int early;       // sums have a place of their own to arrive at
  uint32_t pitch;  // bytes per token of the partial sums
  uint32_t recv;   // where the other pairs' partial sums arrive
  uint32_t tail;   // barriers, behind the stages and the sums
};

struct SplitMaps {
  CUtensorMap x, x2, w, w2;
};

__device__ __forceinline__ void bounded(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait_cluster(bar, parity) && clock64() - t0 < kWaitBudgetCycles) {
  }
}

__device__ __forceinline__ void add4(float4 &v, float4 a) {
  v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
}

template <int kAct, bool kTokensP, int kC>
__global__ void __launch_bounds__(kThreads, 2)
    linear_split_kernel(const __grid_constant__ SplitMaps maps, const SplitShape p,
                        const LinearEpilogue epi, const uint16_t *residual, uint16_t *out,
                        int *status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t sbase = smem_addr(base);
  const uint32_t stage_bytes = kPBytes + static_cast<uint32_t>(p.Q / 2) * kRowBytes;
  const uint32_t tail = p.tail;
  auto bar_full = [&](int s) { return sbase + tail + 16u * static_cast<uint32_t>(s); };
  auto bar_empty = [&](int s) { return sbase + tail + 16u * static_cast<uint32_t>(s) + 8u; };
  const uint32_t bar_acc = sbase + tail + 16u * kMaxStages;
  const uint32_t bar_recv = bar_acc + 8u;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + tail + 16 * kMaxStages + 16);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + tail + 16 * kMaxStages + 24);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t even = rank & ~1u;            // the pair's even CTA: issues its MMAs
  const int side = static_cast<int>(rank & 1u);
  const int part = static_cast<int>(rank >> 1);  // of the channels
  // the tile: its first feature, and with tokens as P its batch element and
  // this CTA's first token
  const int tile = static_cast<int>(cluster_id_x());
  const int tb = tile / p.n_ft;
  const int ft = tile - tb * p.n_ft;
  const int64_t f0 = static_cast<int64_t>(kTokensP ? ft : 2 * ft + side) * p.feats;
  const int b0 = kTokensP ? tb / p.n_sb : 0;
  const int s0 = kTokensP ? ((tb - b0 * p.n_sb) * 2 + side) * kP : 0;
  // the tokens (rows of the partial sums) that this CTA finishes
  const int n_rows = kTokensP ? kP : p.Q;
  auto row_of = [&](int r) { return n_rows * r / kC; };
  const int row_lo = row_of(part), row_hi = row_of(part + 1);
  // the pair's channels: an even share of the stages (at least one: kC <= nk)
  const int k_lo = static_cast<int>(static_cast<int64_t>(p.nk) * part / kC);
  const int k_hi = static_cast<int>(static_cast<int64_t>(p.nk) * (part + 1) / kC);

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_acc, 1);
    mbar_init(bar_recv, 1);
    if (kC > 1)
      mbar_arrive_expect_tx(bar_recv,
                            static_cast<uint32_t>((kC - 1) * (row_hi - row_lo)) * p.pitch);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
  }
  // both CTAs' barriers are initialised before either signals the other's
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch_dependents();
  // first rows of this CTA's share of W
  const int w0 =
      static_cast<int>(kTokensP ? (side == 0 ? f0 : kGlu ? p.N + f0 : f0 + p.Q / 2) : f0);
  // everything up to here overlaps the end of the kernel before this one
  grid_dep_wait();

  if (warp == 0 && lane == 0) {
    const uint32_t bytes = kPBytes + static_cast<uint32_t>(p.q_rows) * kRowBytes;
    const int x0 = kTokensP ? s0 : side * p.Sh;
    bool ok = true;
    int s = 0;
    uint32_t turn = 0;
    for (int ks = k_lo; ks < k_hi; ++ks) {
      if (!(ok = mbar_wait_cluster(bar_empty(s), (turn & 1u) ^ 1u, abort_flag))) break;
      const uint32_t dst = sbase + static_cast<uint32_t>(s) * stage_bytes;
      const uint32_t dst_w = kTokensP ? dst + kPBytes : dst;
      const uint32_t dst_x = kTokensP ? dst : dst + kPBytes;
      // both CTAs' copies complete on the even CTA's stage barrier
      if (side == 0) mbar_arrive_expect_tx(bar_full(s), 2 * bytes);
      const uint32_t full = mapa_shared(bar_full(s), even);
      const bool first = ks < p.nk1;
      const int c = (first ? ks : ks - p.nk1) * kK;
      const void *wm = first ? &maps.w : &maps.w2;
      tma_load_3d_pair(dst_w, wm, full, c, w0, 0);
      if constexpr (kGlu && !kTokensP)
        tma_load_3d_pair(dst_w + kPBytes / 2, wm, full, c, static_cast<int>(p.N) + w0, 0);
      tma_load_3d_pair(dst_x, first ? &maps.x : &maps.x2, full, c, x0, b0);
      if (++s == p.stages) s = 0, ++turn;
    }
    // every copy of the pair has landed before the CTAs exit (the final cluster
    // barrier keeps the odd CTA until then)
    if (side == 0)
      for (int i = 0; i < p.stages; ++i) {
        // the stage's last use, if any, was in this turn or the one before
        if (i < s)
          bounded(bar_full(i), turn & 1u);
        else if (turn > 0)
          bounded(bar_full(i), (turn - 1) & 1u);
      }
  } else if (warp == 1 && side == 0) {
    const uint32_t idesc = idesc_bf16_f32(2 * kP, p.Q, 0, 0);
    const uint16_t mask = static_cast<uint16_t>(0x3u << even);
    bool ok = true;
    int s = 0;
    uint32_t turn = 0;
    for (int ks = k_lo; ks < k_hi; ++ks) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar_full(s), turn & 1u, abort_flag))))
        break;
      tc_fence_after_sync();
      const uint32_t st = sbase + static_cast<uint32_t>(s) * stage_bytes;
      const uint64_t da = sdesc_sw128(st, 16, 1024);
      const uint64_t db = sdesc_sw128(st + kPBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < kK / 16; ++kk)
        mma_ss_pair_elect(tmem, desc_advance(da, kk * 32), desc_advance(db, kk * 32), idesc,
                          (ks != k_lo || kk != 0) ? 1u : 0u);
      mma_commit_pair_elect(bar_empty(s), mask);
      if (++s == p.stages) s = 0, ++turn;
    }
    mma_commit_pair_elect(bar_acc, mask);
  }
  // Row r of the partial sums: its token, if it has one.
  auto token_of = [&](int r, int &b, int &s) {
    if constexpr (kTokensP) {
      b = b0;
      s = s0 + r;
      return s < p.S;
    } else {
      // columns: the even CTA's tokens (the first half of every batch element),
      // then the odd CTA's
      const int hi = r >= p.Q / 2 ? 1 : 0;
      const int t = r - hi * (p.Q / 2);
      b = p.q_rows == p.Sh ? 0 : t / p.Sh;
      s = hi * p.Sh + t - b * p.Sh;
      return t < p.q_rows && s < p.S;
    }
  };
  if (warp >= 4 && residual != nullptr) {
    // the residual's lines, wanted at the end, come to L2 meanwhile
    const int lines = (p.feats + 63) / 64;
    for (int i = tid - 128; i < (row_hi - row_lo) * lines; i += kThreads - 128) {
      int b, s;
      const int r = i / lines;
      const int64_t f = f0 + (i - r * lines) * 64;
      if (token_of(row_lo + r, b, s) && f < p.N)
        prefetch_l2(residual + b * p.r_bs + s * p.r_rs + f);
    }
  }
  __syncwarp();
  // every MMA of the pair has finished: the accumulator is complete and the
  // stages free (an aborted pair's MMAs in flight are waited for too)
  bounded(bar_acc, 0);
  tc_fence_after_sync();
  __syncthreads();
  {
    // one TMEM lane, i.e. row of P, per thread; 16 rows of Q at a time
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t row = static_cast<uint32_t>((warp & 3) * 32 + lane);
#pragma unroll 1
    for (int c = warp >> 2; c < p.Q / 16; c += kThreads / 128) {
      uint32_t r[16];
      tmem_ld16(tmem + lane_off + c * 16, r);
      tmem_ld_wait();
      if constexpr (kTokensP) {
        // the pitch is 16 bytes past a multiple of 128: eight lanes' 16-byte
        // stores lie in different banks
        const uint32_t at = sbase + row * p.pitch + c * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(at + i * 16, make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]));
      } else {
        // consecutive lanes write consecutive words
#pragma unroll
        for (int i = 0; i < 16; ++i)
          st_shared_b32(sbase + static_cast<uint32_t>(c * 16 + i) * p.pitch + row * 4, r[i]);
      }
    }
  }
  fence_proxy_async_smem();
  tc_fence_before_sync();
  // where sums arrive over the ring, every CTA of the cluster is done with its
  if (kC > 1 && !p.early)
    cluster_sync_all();
  else
    __syncthreads();
  // A thread finishes four features of tokens `per` apart. The loop is short
  // and its latencies are left to the 16 warps: this code runs once, and
  // unrolled it cost more in instruction misses than it saved.
  const int n_quad = p.feats / 4;
  const int per = kThreads / n_quad;
  const int o = tid % n_quad;
  const int64_t f = f0 + o * 4;
  const bool mine = tid < per * n_quad && f < p.N;
  float4 bias = make_float4(0.f, 0.f, 0.f, 0.f), bias_u = bias;
  if (mine && epi.bias != nullptr) {
    bias = load_vec4(epi.bias, f, epi.vec_f32);
    if constexpr (kGlu) bias_u = load_vec4(epi.bias, p.N + f, epi.vec_f32);
  }
  // the first token's residual and gate come while the sums arrive
  float4 gate = bias;
  uint32_t gate_row = 0xFFFFFFFFu;  // of `gate`
  auto load_gate = [&](int b, int s) {
    // joined batch elements (at most 2^30 tokens) are found by division
    const uint32_t row = epi.gate_rows == p.S
                             ? static_cast<uint32_t>(b)
                             : static_cast<uint32_t>(s) / static_cast<uint32_t>(epi.gate_rows);
    if (row != gate_row) gate = load_vec4(epi.gate, row * epi.gate_bs + f, epi.vec_f32);
    gate_row = row;
  };
  int r = row_lo + tid / n_quad;
  int b, s;
  bool in = mine && r < row_hi && token_of(r, b, s);
  uint2 res;
  if (in && residual != nullptr)
    res = *reinterpret_cast<const uint2 *>(residual + b * p.r_bs + s * p.r_rs + f);
  if (in && epi.gate != nullptr) load_gate(b, s);
  // where row row_lo of every pair's partial sums lies: this one's own, or
  // where the others' arrive
  uint32_t sums[kC];
#pragma unroll
  for (int r = 0; r < kC; ++r)
    sums[r] = sbase + o * 16 +
              (r == part ? static_cast<uint32_t>(row_lo) * p.pitch
                         : p.recv + static_cast<uint32_t>((r < part ? r : r - 1) *
                                                          (row_hi - row_lo)) * p.pitch);
  if constexpr (kC > 1) {
    if (tid < kC && tid != part) {
      // the rows of pair tid, to the place for this pair's among the others
      const int lo = row_of(tid), n = row_of(tid + 1) - lo;
      const uint32_t to = static_cast<uint32_t>(2 * tid + side);
      bulk_copy_cluster(
          mapa_shared(sbase + p.recv + static_cast<uint32_t>((part < tid ? part : part - 1) * n) *
                                           p.pitch, to),
          sbase + static_cast<uint32_t>(lo) * p.pitch, static_cast<uint32_t>(n) * p.pitch,
          mapa_shared(bar_recv, to));
    }
    __syncwarp();
    if (!mbar_wait_cluster(bar_recv, 0, abort_flag)) *abort_flag = 1;
  }
  __syncwarp();
  cluster_arrive();  // what was sent to this CTA has arrived

  if (mine) {
    const uint32_t half = static_cast<uint32_t>(p.feats) * 4;  // SwiGLU: to the linear sums
#pragma unroll 1
    for (; r < row_hi; r += per) {
      // the next row's residual is on its way while this one is finished
      int b_next, s_next;
      const bool in_next = r + per < row_hi && token_of(r + per, b_next, s_next);
      uint2 res_next;
      if (in_next && residual != nullptr)
        res_next = *reinterpret_cast<const uint2 *>(residual + b_next * p.r_bs +
                                                    s_next * p.r_rs + f);
      if (in) {
        const uint32_t at = static_cast<uint32_t>(r - row_lo) * p.pitch;
        float4 y = bias, w = bias_u;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          add4(y, ld_shared_f4(sums[c] + at));
          if constexpr (kGlu) add4(w, ld_shared_f4(sums[c] + at + half));
        }
        if constexpr (kGlu)
          y = make_float4(activate<FLUX_ACT_SILU>(y.x) * w.x, activate<FLUX_ACT_SILU>(y.y) * w.y,
                          activate<FLUX_ACT_SILU>(y.z) * w.z, activate<FLUX_ACT_SILU>(y.w) * w.w);
        else
          y = make_float4(activate<kAct>(y.x), activate<kAct>(y.y), activate<kAct>(y.z),
                          activate<kAct>(y.w));
        if (epi.gate != nullptr) {
          load_gate(b, s);
          y.x *= gate.x, y.y *= gate.y, y.z *= gate.z, y.w *= gate.w;
        }
        if (residual != nullptr)
          add4(y, make_float4(bf16lo_to_f32(res.x), bf16hi_to_f32(res.x), bf16lo_to_f32(res.y),
                              bf16hi_to_f32(res.y)));
        *reinterpret_cast<uint2 *>(out + b * p.o_bs + s * p.o_rs + f) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      }
      in = in_next, b = b_next, s = s_next, res = res_next;
    }
  }
  __syncwarp();
  cluster_wait();  // what this CTA sent has arrived: its shared memory may go
  if (warp == 2) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

// Shared memory of the partial sums of a CTA's rows; of those that arrive.
uint32_t own_bytes(bool tokens_p, int Q) {
  return static_cast<uint32_t>(tokens_p ? kP * (Q * 4 + 16) : Q * kP * 4);
}
uint32_t recv_bytes(bool tokens_p, int Q, int C) {
  const uint32_t rows = static_cast<uint32_t>(tokens_p ? kP : Q);
  const uint32_t pitch = static_cast<uint32_t>(tokens_p ? Q * 4 + 16 : kP * 4);
  return static_cast<uint32_t>(C - 1) * ((rows + C - 1) / C) * pitch;
}

template <int kAct, bool kTokensP, int kC>
cudaError_t launch(const LinearProblem &q, const SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = linear_split_kernel<kAct, kTokensP, kC>;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemAll));
  });
  if (attr_err[dev] != cudaSuccess) return attr_err[dev];
  const bool glu = kAct == FLUX_ACT_SWIGLU;
  const int64_t wr = glu ? 2 * q.N : q.N;
  SplitShape p;
  p.N = q.N;
  p.o_bs = q.o_bs, p.o_rs = q.o_rs, p.r_bs = q.r_bs, p.r_rs = q.r_rs;
  p.S = static_cast<int>(q.S);
  p.Q = plan.Q;
  p.Sh = (p.S + 15) / 16 * 8;
  p.q_rows = kTokensP ? p.Q / 2 : static_cast<int>(q.B) * p.Sh;
  p.feats = (kTokensP ? p.Q : kP) / (glu ? 2 : 1);
  p.n_sb = (p.S + 2 * kP - 1) / (2 * kP);
  const int64_t per_tile = kTokensP ? p.feats : 2 * p.feats;  // features of a pair's tile
  const int64_t n_ft = (q.N + per_tile - 1) / per_tile;
  const int64_t tiles = n_ft * (kTokensP ? q.B * p.n_sb : 1);
  if (tiles > 0x7FFFFFF || p.q_rows > p.Q / 2) return cudaErrorInvalidValue;
  p.n_ft = static_cast<int>(n_ft);
  p.tmem_cols = 32;
  while (p.tmem_cols < p.Q) p.tmem_cols *= 2;
  p.nk1 = (q.K + kK - 1) / kK;
  p.nk = p.nk1 + (q.K2 + kK - 1) / kK;
  p.pitch = static_cast<uint32_t>(kTokensP ? p.Q * 4 + 16 : kP * 4);
  p.stages = plan.stages;
  const uint32_t stage = kPBytes + static_cast<uint32_t>(p.Q / 2) * kRowBytes;
  // the CTA's own partial sums over the drained ring, the others' behind them
  const uint32_t ring = static_cast<uint32_t>(p.stages) * stage;
  const uint32_t own = own_bytes(kTokensP, p.Q);
  p.early = plan.early ? 1 : 0;
  p.recv = plan.early ? std::max(ring, own) : own;
  p.tail = std::max(ring, p.recv + recv_bytes(kTokensP, p.Q, kC));
  const uint32_t smem = p.tail + kTailBytes;
  if (smem > kSmemAll) return cudaErrorInvalidValue;
  const uint32_t w_box = static_cast<uint32_t>(kTokensP ? p.Q / 2 : p.feats);
  const uint32_t x_box = static_cast<uint32_t>(kTokensP ? kP : p.Sh);
  const uint32_t x_box_b = kTokensP ? 1 : static_cast<uint32_t>(q.B);
  SplitMaps maps;
  const uint16_t *w2 = static_cast<const uint16_t *>(q.w) + q.K;
  if (!make_row_map(&maps.x, q.x, q.K, q.S, q.B, q.x_rs, q.x_bs, kK, x_box, x_box_b) ||
      !make_row_map(&maps.w, q.w, q.K, wr, 1, q.w_rs, q.w_rs * wr, kK, w_box, 1))
    return cudaErrorInvalidValue;
  maps.x2 = maps.x;
  maps.w2 = maps.w;
  if (q.K2 > 0 &&
      (!make_row_map(&maps.x2, q.x2, q.K2, q.S, q.B, q.x2_rs, q.x2_bs, kK, x_box, x_box_b) ||
       !make_row_map(&maps.w2, w2, q.K2, wr, 1, q.w_rs, q.w_rs * wr, kK, w_box, 1)))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * kC;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * 2 * kC), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, epi,
                            static_cast<const uint16_t *>(q.residual),
                            static_cast<uint16_t *>(q.out), status);
}

template <int kAct, bool kTokensP>
cudaError_t launch(const LinearProblem &q, const SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  switch (plan.C) {
    case 1: return launch<kAct, kTokensP, 1>(q, plan, epi, status, stream);
    case 2: return launch<kAct, kTokensP, 2>(q, plan, epi, status, stream);
    case 3: return launch<kAct, kTokensP, 3>(q, plan, epi, status, stream);
    default: return launch<kAct, kTokensP, 4>(q, plan, epi, status, stream);
  }
}

template <int kAct>
cudaError_t launch(const LinearProblem &q, const SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  return plan.tokens_p ? launch<kAct, true>(q, plan, epi, status, stream)
                       : launch<kAct, false>(q, plan, epi, status, stream);
}

}  // namespace

// The tile, the split of the channels and the ring. A launch has so many CTAs
// resident: with all of an SM's shared memory each (clusters of 4, 6 and 8 do
// not fill every SM), or with half of it. Half leaves room for the next
// kernel's prologue, and for a second CTA, which helps where one wave of whole
// SMs is not enough; but then two CTAs share what the SM takes in, and a ring
// of half the bytes is refilled only every 1.1 us.
SplitPlan plan_split(const LinearProblem &q, int act, int sms) {
  const bool glu = act == FLUX_ACT_SWIGLU;
  const int64_t nk = (q.K + kK - 1) / kK + (q.K2 + kK - 1) / kK;
  const int64_t wr = glu ? 2 * q.N : q.N;
  const double bytes = 2.0 * (static_cast<double>(q.B * q.S + wr) * (q.K + q.K2) +
                              static_cast<double>(q.B * q.S) * q.N *
                                  (q.residual != nullptr ? 2 : 1));
  static constexpr int kWhole[kMaxC] = {152, 144, 138, 120}, kHalf[kMaxC] = {304, 296, 276, 288};
  SplitPlan best{false, false, 32, 1, 2, 1e30};
  auto consider = [&](bool tokens_p, int Q) {
    const int64_t feats = (tokens_p ? Q : 2 * kP) / (glu ? 2 : 1);  // of a tile
    const int64_t tiles =
        (q.N + feats - 1) / feats * (tokens_p ? q.B * ((q.S + 2 * kP - 1) / (2 * kP)) : 1);
    const uint32_t stage = kPBytes + static_cast<uint32_t>(Q / 2) * kRowBytes;
    const int rows = tokens_p ? kP : Q;
    const int cta_feats = (tokens_p ? Q : kP) / (glu ? 2 : 1);
    const double pitch = tokens_p ? Q * 4 + 16 : kP * 4;
    for (int C = 1; C <= kMaxC && C <= nk; ++C) {
      const uint32_t recv = recv_bytes(tokens_p, Q, C);
      const int64_t ctas = tiles * 2 * C;
      const int64_t whole = kWhole[C - 1] * static_cast<int64_t>(sms) / 152;
      for (int half = 0; half < 2; ++half) {
        const uint32_t room = (half ? kSmemHalf : kSmemAll) - kTailBytes;
        if (own_bytes(tokens_p, Q) + recv > room || 3 * stage > room) continue;
        int stages = static_cast<int>(std::min<uint32_t>(kMaxStages, room / stage));
        // a place of their own for the sums saves a cluster barrier, unless the
        // ring gets short for it
        const bool early = recv + kEarlyRing <= room;
        if (early)
          stages = static_cast<int>(std::min<uint32_t>(kMaxStages, (room - recv) / stage));
        const int64_t slots = half ? kHalf[C - 1] * static_cast<int64_t>(sms) / 152 : whole;
        const double waves = static_cast<double>((ctas + slots - 1) / slots);
        const double shared =
            !half ? 1.0 : std::min(ctas, slots) > sms ? 2.0 : ctas > whole ? 1.4 : 1.0;
        const double per_stage =
            std::max(stage_ns(stage, Q) * shared, 1090.0 / static_cast<double>(stages));
        const double ns =
            std::max(waves * static_cast<double>((nk + C - 1) / C) * per_stage, bytes / 9000.0) +
            waves * 2130.0 + 2100.0 - (half && ctas <= whole ? 260.0 : 0.0) +
            (C > 1 ? 520.0 + (C - 1) * (rows / static_cast<double>(C)) * pitch / 65.0 : 0.0) +
            0.17 * rows / C * cta_feats;
        if (ns < best.ns) best = SplitPlan{tokens_p, early, Q, C, stages, ns};
      }
    }
  };
  const int64_t rows_q = q.B * ((q.S + 15) / 16 * 16);
  if (rows_q <= 256) consider(false, static_cast<int>((rows_q + 31) / 32 * 32));
  if (q.B * q.S >= 64)  // fewer tokens would fill less than a quarter of P
    for (int Q = 32; Q <= 256; Q += 32) consider(true, Q);
  return best;
}

cudaError_t launch_linear_split(const LinearProblem &q, const SplitPlan &plan,
                                const LinearEpilogue &epi, int act, int *status,
                                cudaStream_t stream) {
  switch (act) {
    case FLUX_ACT_NONE: return launch<FLUX_ACT_NONE>(q, plan, epi, status, stream);
    case FLUX_ACT_SILU: return launch<FLUX_ACT_SILU>(q, plan, epi, status, stream);
    case FLUX_ACT_GELU_TANH: return launch<FLUX_ACT_GELU_TANH>(q, plan, epi, status, stream);
    default: return launch<FLUX_ACT_SWIGLU>(q, plan, epi, status, stream);
  }
}

}  // namespace flux
