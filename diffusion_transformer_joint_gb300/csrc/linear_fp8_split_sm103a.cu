// flux_linear_fp8 where whole 256-row tiles would leave SMs idle (few tokens, or
// few features), on sm_103a (GB300): tiles of 128 rows of W against up to 128
// tokens, the channels split over a cluster.
//
//   y[t, n] = sum_g xs[t, g] ws[n / 128, g] sum_{k in g} x[t, k] w[n, k]
//   out = residual + gate * act(y + bias)
//
// W's rows are the MMA's M and the tokens its N, so that the weights, which
// bound a call with few tokens, are read once and no row of the tile is empty.
// A pipeline stage is one group of 128 channels. Its four K32 MMAs start a
// fresh accumulator; eight warps read it, multiply each token's column with
// xs[t, g] * ws[.., g] and add it to fp32 sums in registers, while the MMAs of
// the next groups fill the other three accumulators: the products inside a group
// are summed by the tensor core, 32 at a time, to an fp32 accumulator (which aligns and
// truncates them: at most 2^-21 of the magnitudes' sum a step), the groups by fp32
// FMAs in the order of the channels.
//
// As linear_split, the groups of a tile are split over the C CTAs of a cluster
// (an SM takes in about 110 bytes per ns, whatever the tile computes), which send
// each other their partial sums by bulk copies; each adds the partials of its
// share of the tokens in the CTAs' order and writes the finished rows. No
// workspace, no atomics, one launch. CTAs allocate TMEM for their own SM only; up
// to 64 tokens two share an SM.
//
// 12 warps: warp 0 TMA producer, warp 1 MMA issuer, warp 2 TMEM allocation,
// warp 3 the scales: it multiplies each token's with the tile's (for SwiGLU the
// gate rows' and the linear rows') and hands them over four groups at a time (a
// wait costs the sums' warps some 100 cycles). Warps 4-11 sums: one TMEM lane (a row of W) per
// thread, 16 tokens at a time, the two warps of a lane quadrant taking turns.
// Then all of them finish. Every wait is bounded, as in linear_split.
//
// Measured (GB300, in a graph): one token 4096 -> 4096 with bias 7.0 us (start 1, the bytes 2.6
// at 6.4 TB/s, sums exchanged and finished 1.3, the rest the launch before), 96
// tokens 9.2, 96 tokens 12288 -> 4096 14.7 (3.4 TB/s of W: a group of 96 tokens
// takes an SM 0.28 us, its 28 KB come in 0.26).
#include <algorithm>
#include <cmath>
#include <mutex>

#include "linear_fp8_common.cuh"

namespace flux {
namespace {

constexpr int kP = 128;
constexpr uint32_t kPBytes = kP * kGroupK;
constexpr int kMaxStages = 8;
constexpr int kMaxUnits = 8;
constexpr int kThreads = 384;
constexpr int kSumWarps = 8;
constexpr int kScaleSlots = 2, kScaleBatch = 4;  // slots of the scales' ring, of so many groups
// Shared memory: of a CTA that shares its SM with another one; of one that does
// not. CTAs take no less than kSmemLeast: beside a CTA pair of linear_split (144
// KB or more) an SM has no room for another that allocates TMEM.
constexpr uint32_t kSmemHalf = 114688, kSmemAll = 232448, kSmemLeast = 98304;
constexpr uint32_t kPitch = kP * 4;  // bytes per token of the partial sums

// A kernel for up to 32 kChunks tokens a tile: a sums' warp has every other 16 of
// them.
template <int kChunks>
struct Split {
  static constexpr bool kShared = kChunks <= 2;  // two CTAs an SM
  static constexpr int kQ = 32 * kChunks;
  static constexpr int kBufs = 4;  // accumulators
  static constexpr uint32_t kScaleBytes = 2 * kQ * 4;  // a group: per token, twice for SwiGLU
  static constexpr int kFull = 0, kEmpty = kMaxStages, kAccFull = 2 * kMaxStages;
  static constexpr int kAccEmpty = kAccFull + kBufs, kScFull = kAccEmpty + kBufs;
  static constexpr int kScEmpty = kScFull + kScaleSlots, kDone = kScEmpty + kScaleSlots;
  static constexpr int kRecv = kDone + 1, kNumBars = kRecv + 1;
  static constexpr uint32_t kOffBar = kScaleSlots * kScaleBatch * kScaleBytes;  // of the tail
  static constexpr uint32_t kOffSlot = kOffBar + 8 * kNumBars;
  static constexpr uint32_t kOffAbort = kOffSlot + 8;
  static constexpr uint32_t kTailBytes = kOffAbort + 8;
  static constexpr uint32_t kSmemMax = kShared ? kSmemHalf : kSmemAll;
};

struct SplitShape {
  int64_t N, o_bs, o_rs, r_bs, r_rs, xs_bs, xs_rs, xs_ks, ws_rs, ws_ks;
  const float *xs, *ws;
  int S;              // tokens per batch element of the launch
  int Q, C;           // tokens of a tile; parts of the channels
  int n_sb, n_tb;     // token tiles per batch element, in all
  int feats;          // output features of a tile
  int nk, stages, tmem_cols;
  int early;          // sums have a place of their own to arrive at
  uint32_t recv, tail;
};

struct SplitMaps {
  CUtensorMap x, w;
};

__device__ __forceinline__ void add4(float4 &v, float4 a) {
  v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
}

template <int kAct, int kChunks>
__global__ void __launch_bounds__(kThreads, Split<kChunks>::kShared ? 2 : 1)
    linear_fp8_split_kernel(const __grid_constant__ SplitMaps maps, const SplitShape p,
                            const LinearEpilogue epi, const uint16_t *residual, uint16_t *out,
                            int *status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  using T = Split<kChunks>;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t sbase = smem_addr(base);
  const uint32_t stage_bytes = kPBytes + static_cast<uint32_t>(p.Q) * kGroupK;
  const uint32_t tail = sbase + p.tail;
  auto bar = [&](int i) { return tail + T::kOffBar + 8u * static_cast<uint32_t>(i); };
  auto scales_at = [&](int i) {  // group i of the ring's slots
    return tail + T::kScaleBytes * static_cast<uint32_t>(i);
  };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + p.tail + T::kOffSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + p.tail + T::kOffAbort);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int part = static_cast<int>(cluster_ctarank());  // of the channels
  const int tile = static_cast<int>(cluster_id_x());
  const int ft = tile / p.n_tb, tb = tile - ft * p.n_tb;
  const int64_t f0 = static_cast<int64_t>(ft) * p.feats;
  const int b0 = tb / p.n_sb;
  const int s0 = (tb - b0 * p.n_sb) * p.Q;
  // the tile's tokens that this CTA finishes, and the groups that it sums
  auto row_of = [&](int r) { return p.Q * r / p.C; };
  const int row_lo = row_of(part), row_hi = row_of(part + 1);
  const int k_lo = static_cast<int>(static_cast<int64_t>(p.nk) * part / p.C);
  const int k_hi = static_cast<int>(static_cast<int64_t>(p.nk) * (part + 1) / p.C);

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(T::kFull + s), 1);
      mbar_init(bar(T::kEmpty + s), 1);
    }
    for (int i = 0; i < T::kBufs; ++i) {
      mbar_init(bar(T::kAccFull + i), 1);
      mbar_init(bar(T::kAccEmpty + i), kSumWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(bar(T::kScFull + i), 1);
      mbar_init(bar(T::kScEmpty + i), kSumWarps);
    }
    mbar_init(bar(T::kDone), 1);
    mbar_init(bar(T::kRecv), 1);
    if (p.C > 1)
      mbar_arrive_expect_tx(bar(T::kRecv),
                            static_cast<uint32_t>((p.C - 1) * (row_hi - row_lo)) * kPitch);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_addr(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
  }
  // every CTA's barriers are initialised before another signals them
  tc_fence_before_sync();
  cluster_sync_relaxed();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch_dependents();
  // everything up to here overlaps the end of the kernel before this one
  grid_dep_wait();

  // A thread finishes four features of tokens `per` apart.
  const int n_quad = p.feats / 4;
  const int per = kThreads / n_quad;
  const int o = tid % n_quad;
  const int64_t f = f0 + o * 4;
  const bool mine = f < p.N;
  int r = row_lo + tid / n_quad;
  uint4 bias_raw = make_uint4(0u, 0u, 0u, 0u), bias_u_raw = bias_raw, gate_raw = bias_raw;
  uint32_t gate_row = 0xFFFFFFFFu;  // of gate_raw
  auto load_gate = [&](int s) {     // of token s of batch element b0
    const uint32_t row = epi.gate_rows == p.S
                             ? static_cast<uint32_t>(b0)
                             : static_cast<uint32_t>(s) / static_cast<uint32_t>(epi.gate_rows);
    if (row != gate_row) gate_raw = load_raw4(epi.gate, row * epi.gate_bs + f, epi.vec_f32);
    gate_row = row;
  };
  auto load_vectors = [&] {
    if (mine && epi.bias != nullptr) {
      bias_raw = load_raw4(epi.bias, f, epi.vec_f32);
      if constexpr (kGlu) bias_u_raw = load_raw4(epi.bias, p.N + f, epi.vec_f32);
    }
    if (mine && epi.gate != nullptr && r < row_hi && s0 + r < p.S) load_gate(s0 + r);
  };
  // (the sums of larger tiles leave no registers for them)
  if constexpr (T::kShared) load_vectors();

  uint64_t acc[kChunks][8];  // pairs of sums
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0;

  if (warp == 0 && lane == 0) {
    bool ok = true;
    int s = 0;
    uint32_t turn = 0;
    for (int g = k_lo; g < k_hi; ++g) {
      if (!(ok = mbar_wait(bar(T::kEmpty + s), (turn & 1u) ^ 1u, abort_flag))) break;
      const uint32_t dst = sbase + static_cast<uint32_t>(s) * stage_bytes;
      mbar_arrive_expect_tx(bar(T::kFull + s), stage_bytes);
      tma_load_3d(dst, &maps.w, bar(T::kFull + s), g * kGroupK, static_cast<int>(f0), 0);
      if constexpr (kGlu)
        tma_load_3d(dst + kPBytes / 2, &maps.w, bar(T::kFull + s), g * kGroupK,
                    static_cast<int>(p.N + f0), 0);
      tma_load_3d(dst + kPBytes, &maps.x, bar(T::kFull + s), g * kGroupK, s0, b0);
      if (++s == p.stages) s = 0, ++turn;
    }
    // every copy has landed before the ring is used for the sums
    const long long until = clock64() + kWaitBudgetCycles;
    for (int i = 0; i < p.stages; ++i) {
      // the stage's last use, if any, was in this turn or the one before
      if (i < s)
        ok &= mbar_settled(bar(T::kFull + i), turn & 1u, until);
      else if (turn > 0)
        ok &= mbar_settled(bar(T::kFull + i), (turn - 1) & 1u, until);
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == 1) {
    const uint32_t idesc = idesc_e4m3_f32(kP, p.Q);
    int s = 0, buf = 0;
    uint32_t turn = 0, use = 0;  // times round the stages, the accumulators
    for (int g = k_lo; g < k_hi; ++g) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(T::kAccEmpty + buf), (use & 1u) ^ 1u, abort_flag)))
        break;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(T::kFull + s), turn & 1u, abort_flag))) break;
      tc_fence_after_sync();
      const uint32_t st = sbase + static_cast<uint32_t>(s) * stage_bytes;
      const uint64_t da = sdesc_sw128(st, 16, 1024);
      const uint64_t db = sdesc_sw128(st + kPBytes, 16, 1024);
      const uint32_t d = tmem + static_cast<uint32_t>(buf * p.Q);
#pragma unroll
      for (int kk = 0; kk < kGroupK / 32; ++kk)
        mma_f8_elect(d, desc_advance(da, kk * 32), desc_advance(db, kk * 32), idesc,
                     kk != 0 ? 1u : 0u);
      mma_commit_elect(bar(T::kEmpty + s));
      mma_commit_elect(bar(T::kAccFull + buf));
      if (++s == p.stages) s = 0, ++turn;
      if (++buf == T::kBufs) buf = 0, ++use;
    }
    mma_commit_elect(bar(T::kDone));
  } else if (warp == 3) {
    // lanes take the tokens lane, lane + 32, ...; rows of W: one block of 128
    // (for SwiGLU one of the gate rows and one of the linear rows)
    const float *ws0 = p.ws + (f0 / 128) * p.ws_rs;
    const float *ws1 = p.ws + ((p.N + f0) / 128) * p.ws_rs;
    const float *xs = p.xs + b0 * p.xs_bs;
    bool ok = true;
    int slot = 0;
    uint32_t use = 0;
    for (int g0 = k_lo; ok && g0 < k_hi; g0 += kScaleBatch) {
      float x[kScaleBatch][kChunks], w0[kScaleBatch], w1[kScaleBatch];
#pragma unroll
      for (int i = 0; i < kScaleBatch; ++i) {
        const int g = g0 + i < k_hi ? g0 + i : k_hi - 1;
        w0[i] = ws0[g * p.ws_ks];
        if constexpr (kGlu) w1[i] = ws1[g * p.ws_ks];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          const int t = j * 32 + lane;
          x[i][j] = t < p.Q && s0 + t < p.S ? xs[(s0 + t) * p.xs_rs + g * p.xs_ks] : 0.f;
        }
      }
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait(bar(T::kScEmpty + slot), (use & 1u) ^ 1u, abort_flag))))
        break;
#pragma unroll
      for (int i = 0; i < kScaleBatch; ++i) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          const uint32_t at = scales_at(slot * kScaleBatch + i) + static_cast<uint32_t>(j * 32 + lane) * 4;
          st_shared_b32(at, __float_as_uint(x[i][j] * w0[i]));
          if constexpr (kGlu) st_shared_b32(at + T::kQ * 4, __float_as_uint(x[i][j] * w1[i]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(T::kScFull + slot));
      if (++slot == kScaleSlots) slot = 0, ++use;
    }
  } else if (warp >= 4) {
    const int turn = (warp - 4) >> 2;  // takes the 16-token columns of this parity
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // the linear rows of a SwiGLU tile are its rows from 64 on
    const uint32_t sc_off = kGlu && (warp & 3) >= 2 ? T::kQ * 4 : 0;
    int buf = 0, slot = 0;
    uint32_t use = 0, sc_use = 0;
    bool ready = false;  // the next accumulator was complete when last looked at
    for (int g = k_lo; g < k_hi; ++g) {
      const int in_slot = (g - k_lo) % kScaleBatch;
      if (in_slot == 0 && !__all_sync(0xffffffffu, mbar_wait(bar(T::kScFull + slot), sc_use & 1u,
                                                             abort_flag)))
        break;
      if (!__all_sync(0xffffffffu, ready) &&
          !__all_sync(0xffffffffu, mbar_wait(bar(T::kAccFull + buf), use & 1u, abort_flag)))
        break;
      const uint32_t scales = scales_at(slot * kScaleBatch + in_slot) + sc_off;
      const int next = buf + 1 == T::kBufs ? 0 : buf + 1;
      const uint32_t next_use = next == 0 ? use + 1 : use;
      tc_fence_after_sync();
      const uint32_t from = tmem + static_cast<uint32_t>(buf * p.Q) + lane_off;
      if (turn * 16 < p.Q) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint32_t c = static_cast<uint32_t>((2 * i + turn) * 16);
          uint64_t v[8];
          tmem_ld16_pairs(from + c, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 sc = ld_shared_v4(scales + c * 4 + j * 16);
            const uint64_t s0 = f2_pack(__uint_as_float(sc.x), __uint_as_float(sc.y));
            const uint64_t s1 = f2_pack(__uint_as_float(sc.z), __uint_as_float(sc.w));
            acc[i][2 * j] = f2_fma(v[2 * j], s0, acc[i][2 * j]);
            acc[i][2 * j + 1] = f2_fma(v[2 * j + 1], s1, acc[i][2 * j + 1]);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(T::kAccEmpty + buf));
      ready = mbar_test_wait(bar(T::kAccFull + next), next_use & 1u);
      if (in_slot == kScaleBatch - 1 || g == k_hi - 1) {
        if (lane == 0) mbar_arrive(bar(T::kScEmpty + slot));
        if (++slot == kScaleSlots) slot = 0, ++sc_use;
      }
      buf = next, use = next_use;
    }
  }
  __syncwarp();
  // The MMAs have read the ring, an aborted CTA's too: its issuer commits them
  // when its own wait has run out, so that this one is longer.
  if (!mbar_settled(bar(T::kDone), 0, clock64() + 3 * kWaitBudgetCycles)) *abort_flag = 1;
  __syncthreads();
  if (warp >= 4) {
    // one row of W per thread: consecutive lanes write consecutive words
    const int turn = (warp - 4) >> 2;
    const uint32_t row = static_cast<uint32_t>((warp & 3) * 32 + lane);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (turn * 16 >= p.Q) break;
      const uint32_t at = sbase + static_cast<uint32_t>((2 * i + turn) * 16) * kPitch + row * 4;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a, b;
        f2_unpack(acc[i][j], a, b);
        st_shared_b32(at + (2 * j) * kPitch, __float_as_uint(a));
        st_shared_b32(at + (2 * j + 1) * kPitch, __float_as_uint(b));
      }
    }
  }
  fence_proxy_async_smem();
  // where sums arrive over the ring, every CTA of the cluster is done with its
  if (p.C > 1 && !p.early)
    cluster_sync_relaxed();
  else
    __syncthreads();
  // the residual of the first tokens comes while the sums arrive
  auto fetch = [&](int row) {
    uint2 v = make_uint2(0u, 0u);
    if (mine && residual != nullptr && row < row_hi && s0 + row < p.S)
      v = *reinterpret_cast<const uint2 *>(residual + b0 * p.r_bs + (s0 + row) * p.r_rs + f);
    return v;
  };
  if constexpr (!T::kShared) load_vectors();
  uint2 res = fetch(r), res1 = fetch(r + per);
  if (p.C > 1) {
    // a warp per other CTA sends that one's rows, in four copies
    if (warp < p.C && warp != part && lane < 4) {
      const int lo = row_of(warp), n = row_of(warp + 1) - lo;
      const int q_lo = n * lane / 4, q_n = n * (lane + 1) / 4 - q_lo;
      const uint32_t to = static_cast<uint32_t>(warp);
      if (q_n > 0)
        bulk_copy_cluster(
            mapa_shared(sbase + p.recv + static_cast<uint32_t>(
                            (part < warp ? part : part - 1) * n + q_lo) * kPitch, to),
            sbase + static_cast<uint32_t>(lo + q_lo) * kPitch,
            static_cast<uint32_t>(q_n) * kPitch, mapa_shared(bar(T::kRecv), to));
    }
    __syncwarp();
    // An abort does not end this wait: every CTA sends its rows, an aborted one
    // too, and they must have arrived before this one lets the cluster go. The
    // last may have waited for its MMAs for three budgets since this one was done.
    if (!mbar_try_wait_cluster(bar(T::kRecv), 0) &&
        !mbar_settled(bar(T::kRecv), 0, clock64() + 4 * kWaitBudgetCycles))
      *abort_flag = 1;
  }
  __syncwarp();
  cluster_arrive_relaxed();  // what was sent to this CTA has arrived

  if (mine) {
    const float4 bias = raw4_values(bias_raw, epi.vec_f32);
    const float4 bias_u = raw4_values(bias_u_raw, epi.vec_f32);
    const uint32_t half = static_cast<uint32_t>(p.feats) * 4;  // SwiGLU: to the linear sums
    const uint32_t own = sbase + o * 16 + static_cast<uint32_t>(row_lo) * kPitch;
    const uint32_t theirs = sbase + o * 16 + p.recv;
    const uint32_t block = static_cast<uint32_t>(row_hi - row_lo) * kPitch;
#pragma unroll 1
    for (; r < row_hi && s0 + r < p.S; r += per) {
      const uint2 res_next = fetch(r + 2 * per);
      const uint32_t at = static_cast<uint32_t>(r - row_lo) * kPitch;
      float4 y = bias, w = bias_u;
#pragma unroll 1
      for (int c = 0; c < p.C; ++c) {  // the parts in the channels' order
        const uint32_t from =
            at + (c == part ? own : theirs + static_cast<uint32_t>(c < part ? c : c - 1) * block);
        add4(y, ld_shared_f4(from));
        if constexpr (kGlu) add4(w, ld_shared_f4(from + half));
      }
      if constexpr (kGlu)
        y = make_float4(activate<FLUX_ACT_SILU>(y.x) * w.x, activate<FLUX_ACT_SILU>(y.y) * w.y,
                        activate<FLUX_ACT_SILU>(y.z) * w.z, activate<FLUX_ACT_SILU>(y.w) * w.w);
      else
        y = make_float4(activate<kAct>(y.x), activate<kAct>(y.y), activate<kAct>(y.z),
                        activate<kAct>(y.w));
      if (epi.gate != nullptr) {
        load_gate(s0 + r);
        const float4 gate = raw4_values(gate_raw, epi.vec_f32);
        y.x *= gate.x, y.y *= gate.y, y.z *= gate.z, y.w *= gate.w;
      }
      if (residual != nullptr)
        add4(y, make_float4(bf16lo_to_f32(res.x), bf16hi_to_f32(res.x), bf16lo_to_f32(res.y),
                            bf16hi_to_f32(res.y)));
      *reinterpret_cast<uint2 *>(out + b0 * p.o_bs + (s0 + r) * p.o_rs + f) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      res = res1, res1 = res_next;
    }
  }
  __syncwarp();
  cluster_wait();  // what this CTA sent has arrived: its shared memory may go
  if (warp == 2) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

uint32_t stage_size(int Q) { return kPBytes + static_cast<uint32_t>(Q) * kGroupK; }
uint32_t own_bytes(int Q) { return static_cast<uint32_t>(Q) * kPitch; }
uint32_t recv_bytes(int Q, int C) {
  return static_cast<uint32_t>((C - 1) * ((Q + C - 1) / C)) * kPitch;
}

// A tile's tokens: 16, 32, 64, 96 or 128.
int chunks_of(int Q) { return (Q + 31) / 32; }

template <int kAct, int kChunks>
cudaError_t launch(const LinearFp8Problem &q, const Fp8SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  using T = Split<kChunks>;
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = linear_fp8_split_kernel<kAct, kChunks>;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(T::kSmemMax));
  });
  if (attr_err[dev] != cudaSuccess) return attr_err[dev];
  constexpr bool glu = kAct == FLUX_ACT_SWIGLU;
  SplitShape p;
  p.N = q.N;
  p.o_bs = q.o_bs, p.o_rs = q.o_rs, p.r_bs = q.r_bs, p.r_rs = q.r_rs;
  p.xs_bs = q.xs_bs, p.xs_rs = q.xs_rs, p.xs_ks = q.xs_ks, p.ws_rs = q.ws_rs, p.ws_ks = q.ws_ks;
  p.xs = q.xs, p.ws = q.ws;
  p.S = static_cast<int>(q.S);
  p.Q = plan.Q, p.C = plan.C, p.stages = plan.stages;
  p.feats = glu ? kP / 2 : kP;
  const int64_t n_sb = (q.S + plan.Q - 1) / plan.Q;
  const int64_t n_ft = (q.N + p.feats - 1) / p.feats;
  if (n_sb > 0x7FFFFFF / q.B || n_ft > 0x7FFFFFF / (n_sb * q.B)) return cudaErrorInvalidValue;
  p.n_sb = static_cast<int>(n_sb);
  p.n_tb = static_cast<int>(n_sb * q.B);
  p.nk = (q.K + kGroupK - 1) / kGroupK;
  p.tmem_cols = 32;
  while (p.tmem_cols < T::kBufs * p.Q) p.tmem_cols *= 2;
  // the CTA's own partial sums over the drained ring, the others' behind them
  const uint32_t ring = static_cast<uint32_t>(p.stages) * stage_size(p.Q);
  const uint32_t own = own_bytes(p.Q), recv = recv_bytes(p.Q, p.C);
  p.early = plan.early ? 1 : 0;
  p.recv = plan.early ? std::max(ring, own) : own;
  p.tail = (std::max(ring, p.recv + recv) + 127) & ~127u;
  const uint32_t smem = std::max(p.tail + T::kTailBytes, kSmemLeast);
  if (smem > T::kSmemMax || p.C > p.nk || p.C > kMaxUnits || chunks_of(p.Q) != kChunks)
    return cudaErrorInvalidValue;
  const int64_t wr = glu ? 2 * q.N : q.N;
  SplitMaps maps;
  if (!make_byte_map(&maps.x, q.x, q.K, q.S, q.B, q.x_rs, q.x_bs, static_cast<uint32_t>(p.Q)) ||
      !make_byte_map(&maps.w, q.w, q.K, wr, 1, q.w_rs, q.w_rs * wr,
                     static_cast<uint32_t>(p.feats)))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(n_ft * p.n_tb * p.C), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, epi,
                            static_cast<const uint16_t *>(q.residual),
                            static_cast<uint16_t *>(q.out), status);
}

template <int kAct>
cudaError_t launch(const LinearFp8Problem &q, const Fp8SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  switch (chunks_of(plan.Q)) {
    case 1: return launch<kAct, 1>(q, plan, epi, status, stream);
    case 2: return launch<kAct, 2>(q, plan, epi, status, stream);
    case 3: return launch<kAct, 3>(q, plan, epi, status, stream);
    case 4: return launch<kAct, 4>(q, plan, epi, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

uint32_t tail_bytes(int Q) {
  const int c = chunks_of(Q);
  return c == 1 ? Split<1>::kTailBytes : c == 2 ? Split<2>::kTailBytes
         : c == 3 ? Split<3>::kTailBytes : Split<4>::kTailBytes;
}

}  // namespace

Fp8SplitPlan plan_fp8_split(const LinearFp8Problem &q, int act, int sms) {
  const bool glu = act == FLUX_ACT_SWIGLU;
  const int nk = (q.K + kGroupK - 1) / kGroupK;
  const int64_t feats = glu ? kP / 2 : kP, n_ft = (q.N + feats - 1) / feats;
  Fp8SplitPlan best{0, 0, 0, false, 1e30};
  // Estimates in ns, fitted to the times of these forms at 38 problems of 1 to 512
  // tokens (with linear_fp8_pair's, the pick takes 1.02 times the best form's time,
  // geometric mean, 1.2 at most): per wave, group and its column, bytes per ns that
  // a CTA's stages and sums come at (a CTA that shares its SM at half that), what a
  // late place for the sums costs, finishing a row.
  struct Costs {
    double wave, group, column, bytes, send, late, row;
  };
  static constexpr Costs kShared = {3110.0, 148.0, 7.5, 69.0, 14.7, 113.0, 0.0};
  static constexpr Costs kWhole = {4480.0, 0.0, 3.95, 100.0, 44.0, 0.0, 6.5};
  static constexpr int kTokens[] = {16, 32, 64, 96, 128};
  static constexpr int kResident[9] = {0, 152, 152, 147, 144, 140, 138, 0, 120};  // an SM each
  const int64_t wr = glu ? 2 * q.N : q.N;
  const double bytes = static_cast<double>(q.B * q.S + wr) * q.K +
                       2.0 * static_cast<double>(q.B * q.S) * q.N * (q.residual != nullptr ? 2 : 1);
  for (int Q : kTokens) {
    const int64_t n_tb = q.B * ((q.S + Q - 1) / Q);
    const bool shared = chunks_of(Q) <= 2;
    const Costs &t = shared ? kShared : kWhole;
    const uint32_t room = (shared ? kSmemHalf : kSmemAll) - tail_bytes(Q) - 128;
    for (int C = 1; C <= kMaxUnits && C <= nk; C += C == 6 ? 2 : 1) {
      const int64_t slots = shared ? 2 * sms : kResident[C] * static_cast<int64_t>(sms) / 152;
      const uint32_t stage = stage_size(Q), recv = recv_bytes(Q, C);
      if (slots < C || own_bytes(Q) + recv > room || 3 * stage > room) continue;
      // a place of their own for the sums saves a cluster barrier, unless the ring
      // gets short for it
      const bool early = C > 1 && recv <= 16 * 1024 && recv + 3 * stage <= room;
      const int stages = static_cast<int>(std::min<uint32_t>(
          kMaxStages, (early ? room - recv : room) / stage));
      const double ctas = static_cast<double>(n_ft) * static_cast<double>(n_tb) * C;
      const double waves = std::ceil(ctas / static_cast<double>(slots));
      const double share = !shared || ctas <= sms ? 1.0 : std::min(2.0, ctas / sms);
      const double per = std::max(stage / t.bytes * share, t.group + t.column * Q);
      const double ns =
          std::max(waves * (t.wave + std::ceil(static_cast<double>(nk) / C) * per),
                   bytes / 6690.0 + t.wave) +
          (C > 1 ? recv / t.send + (early ? 0.0 : t.late) : 0.0) + t.row * Q / C;
      if (ns < best.ns) best = Fp8SplitPlan{Q, C, stages, early, ns};
    }
    if (Q >= q.S) break;
  }
  return best;
}

cudaError_t launch_fp8_split(const LinearFp8Problem &q, const Fp8SplitPlan &plan,
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
