// flux_linear where whole 256-row tiles would leave SMs idle (few rows, or few
// features), on sm_103a (GB300): tiles of 128 or 256 rows of one operand
// against up to 256 rows of the other, the channels split over a cluster.
//
//   out[b, s, :] = residual[b, s, :] + gate[b, :] * act([x | x2][b, s, :] W^T + bias)
//
// A unit is a CTA, or a CTA pair, that computes P x Q accumulators: 128 rows of
// the operand P per CTA (the MMA's M) against Q <= 256 rows of the operand Q
// (its N; in a pair each CTA's shared memory holds half of them). Three forms:
//   kSingle  P is W, Q holds every token (64 at most), a unit is one CTA with
//            half an SM's shared memory;
//   kPairW   P is W, Q holds every token (256 at most), a unit is a pair;
//   kPairX   P is token rows, Q features, a unit is a pair.
// With W as P the weights, which bound a call with few tokens, are read once.
//
// Tiles alone are too few to draw the memory's bandwidth, and narrower ones
// are no help: an SM takes in about 110 GB/s, and a stage of 64 channels brings
// 128 bytes for each of its rows whatever the tile computes with them. So the
// channels of a tile are split over the units of a cluster (kC of them): each
// CTA writes its fp32 partial sums to its shared memory and sends every other
// unit that unit's share of the tokens (bulk copies between the CTAs' shared
// memories, about 30 bytes per ns and SM); each then adds the partials of its
// own share in the units' order (the same in every run) and writes the
// finished rows. No workspace, no atomics, one launch.
//
// For SwiGLU the W rows of a tile are the gate rows of its outputs and their
// linear rows: side by side in each CTA as P, one CTA's each as Q.
//
// A CTA pair has its two SMs to itself. Two pairs on the same SMs would
// allocate TMEM for both SMs at the same time, and an SM lets one CTA allocate
// until that one is done: each pair could hold one SM and wait for the other
// for ever (pairs with half an SM's memory each did hang, once in some 10^5
// calls). Two CTAs share an SM only where each allocates for itself.
//
// 16 warps: warp 0 TMA producer, warp 1 MMA issuer (of the pair's even CTA; one
// K16 MMA per 16 channels), warp 2 TMEM allocation; then all of them move the
// CTA's 128 accumulator rows to shared memory over the drained stages and
// finish them. The prologue overlaps the end of the kernel before it
// (programmatic dependent launch). Every wait on an mbarrier is bounded; a wait
// that runs out aborts the CTA and sets the status word to
// FLUX_ERR_DEVICE_TIMEOUT.
//
// Measured on a GB300 (us, in a graph), the best of each form and of
// linear_pair, 4096 channels to 4096 features: 16 tokens 7.6 single, 9.0
// kPairW (17 where one unit takes all channels); 128 tokens 10.6 kPairW, 12.1
// kPairX, 19.9 linear_pair; 512 tokens 17.2 kPairX, 21.0 linear_pair; 1200
// tokens 44.7 kPairX, 39.0 linear_pair. Two rows of 4096 channels to 24576
// features 34.5 (5.8 TB/s; kPairW 40.4); 2 x 77 tokens of 12288 channels to
// 4096 24.9, of which the stages are 16 (what 96 SMs take in) and sending sums
// and finishing them 5; 4056 tokens of 4096 channels to 128 features 10.7
// (linear_pair 19.6); one row of 256 channels 3.55.
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
constexpr int kSingle = 0, kPairW = 1, kPairX = 2;
// units that split a tile's channels: clusters have up to eight CTAs
constexpr int kMaxUnits = 8;
constexpr int max_units(int form) { return form == kSingle ? kMaxUnits : kMaxUnits / 2; }
constexpr int kThreads = 512;
constexpr uint32_t kSmemAll = 232448;   // a pair's CTAs: one per SM
constexpr uint32_t kSmemHalf = 114688;  // single CTAs: two per SM
// CTAs take no less, whatever their plan needs: beside a pair's CTA an SM (228 KB,
// of which the system takes 1 KB per CTA) has no room for another that allocates
// TMEM.
constexpr uint32_t kSmemPair = 147456, kSmemSingle = 98304;
constexpr uint32_t kSmemSm = 233472 - 2 * 1024;  // for two CTAs
static_assert(2 * kSmemPair > kSmemSm && kSmemPair + kSmemSingle > kSmemSm, "a pair's SM");
constexpr uint32_t kTailBytes = 256;    // barriers and flags
// A ring that sums may have a place of their own beside: with less on its way
// than about 1.5 us of what an SM takes in, the stages wait for the memory.
constexpr uint32_t kEarlyRing = 176 * 1024;

struct SplitShape {
  int64_t N, o_bs, o_rs, r_bs, r_rs;
  int S;           // tokens per batch element of the launch
  int Q;           // tile columns
  int q_rows;      // rows of Q that each CTA copies
  int Sh;          // tokens as Q: a batch element's in one CTA, rounded up to 8
  int n_sb;        // tokens as P: 256-row blocks per batch element
  int n_tb;        // tokens as P: 256-row blocks; those of one feature tile are
                   // neighbours and read its W from L2
  int feats;       // output features of a CTA's tile
  int nk1, nk;     // stages of x, in all
  int stages, tmem_cols;
  int early;       // sums have a place of their own to arrive at
  uint32_t pitch;  // bytes per token of the partial sums
  uint32_t recv;   // where the other units' partial sums arrive
  uint32_t tail;   // barriers, behind the stages and the sums
};

struct SplitMaps {
  CUtensorMap x, x2, w, w2;
};

// After an abort the even CTA of a pair counts no further copies, but the odd
// one may still have issued some into stages that were free; they complete on
// the even CTA's barriers in a phase that nobody ends, and the odd CTA, whose
// accumulators are committed all the same, would not stay for them. The even
// CTA's producer stays a millisecond (a copy lands within some microseconds, and
// none is issued later: the MMAs that free stages stop with the abort), and with
// it the cluster, which no CTA leaves before all have arrived at its last barrier.
constexpr long long kHoldCycles = 2000000;
__device__ __forceinline__ void hold_after_abort() {
  const long long t0 = clock64();
  while (clock64() - t0 < kHoldCycles) {
  }
}

__device__ __forceinline__ void add4(float4 &v, float4 a) {
  v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
}

template <int kAct, int kForm, int kC>
__global__ void __launch_bounds__(kThreads, kForm == kSingle ? 2 : 1)
    linear_split_kernel(const __grid_constant__ SplitMaps maps, const SplitShape p,
                        const LinearEpilogue epi, const uint16_t *residual, uint16_t *out,
                        int *status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  constexpr bool kPair = kForm != kSingle, kTokensP = kForm == kPairX;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t sbase = smem_addr(base);
  const int q_cta = kPair ? p.Q / 2 : p.Q;  // rows of Q in this CTA
  const uint32_t stage_bytes = kPBytes + static_cast<uint32_t>(q_cta) * kRowBytes;
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
  const uint32_t even = kPair ? rank & ~1u : rank;  // the CTA that issues the unit's MMAs
  const int side = static_cast<int>(rank - even);
  const int part = static_cast<int>(kPair ? rank >> 1 : rank);  // of the channels
  auto rank_of = [&](int unit) {  // the CTA with this one's rows of P in another unit
    return static_cast<uint32_t>(kPair ? 2 * unit + side : unit);
  };
  // the tile: its first feature, and with tokens as P its batch element and
  // this CTA's first token
  const int tile = static_cast<int>(cluster_id_x());
  const int ft = kTokensP ? tile / p.n_tb : tile;
  const int tb = tile - ft * p.n_tb;  // (tokens as P)
  const int64_t f0 = static_cast<int64_t>(kForm == kPairW ? 2 * ft + side : ft) * p.feats;
  const int b0 = kTokensP ? tb / p.n_sb : 0;
  const int s0 = kTokensP ? ((tb - b0 * p.n_sb) * 2 + side) * kP : 0;
  // the tokens (rows of the partial sums) that this CTA finishes
  const int n_rows = kTokensP ? kP : p.Q;
  auto row_of = [&](int r) { return n_rows * r / kC; };
  const int row_lo = row_of(part), row_hi = row_of(part + 1);
  // the unit's channels: an even share of the stages (at least one: kC <= nk)
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
    if constexpr (kPair) {
      tmem_alloc_pair(smem_addr(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
      tmem_relinquish();
    }
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
  // first rows of this CTA's share of W
  const int w0 =
      static_cast<int>(kTokensP ? (side == 0 ? f0 : kGlu ? p.N + f0 : f0 + p.Q / 2) : f0);
  // everything up to here overlaps the end of the kernel before this one
  grid_dep_wait();

  // Row r of the partial sums: its token, if it has one.
  auto token_of = [&](int r, int &b, int &s) {
    if constexpr (kTokensP) {
      b = b0;
      s = s0 + r;
      return s < p.S;
    } else {
      // columns: the even CTA's tokens (of a pair the first half of every batch
      // element), then the odd CTA's
      const int hi = r >= q_cta ? 1 : 0;
      const int t = r - hi * q_cta;
      b = p.q_rows == p.Sh ? 0 : t / p.Sh;
      s = hi * p.Sh + t - b * p.Sh;
      return t < p.q_rows && s < p.S;
    }
  };
  // A thread finishes four features of tokens `per` apart, from row r of the
  // partial sums on. Their bias and the first one's gate come while the tile
  // is computed (loaded at its end they cost 0.3 to 0.6 us of a call).
  const int n_quad = p.feats / 4;
  const int per = kThreads / n_quad;
  const int o = tid % n_quad;
  const int64_t f = f0 + o * 4;
  const bool mine = tid < per * n_quad && f < p.N;
  int r = row_lo + tid / n_quad;
  int b, s;
  uint4 bias_raw = make_uint4(0u, 0u, 0u, 0u), bias_u_raw = bias_raw, gate_raw = bias_raw;
  uint32_t gate_row = 0xFFFFFFFFu;  // of gate_raw
  auto load_gate = [&] {            // of token (b, s)
    // joined batch elements (at most 2^30 tokens) are found by division
    const uint32_t row = epi.gate_rows == p.S
                             ? static_cast<uint32_t>(b)
                             : static_cast<uint32_t>(s) / static_cast<uint32_t>(epi.gate_rows);
    if (row != gate_row) gate_raw = load_raw4(epi.gate, row * epi.gate_bs + f, epi.vec_f32);
    gate_row = row;
  };
  if (mine && epi.bias != nullptr) {
    bias_raw = load_raw4(epi.bias, f, epi.vec_f32);
    if constexpr (kGlu) bias_u_raw = load_raw4(epi.bias, p.N + f, epi.vec_f32);
  }
  if (mine && epi.gate != nullptr && r < row_hi && token_of(r, b, s)) load_gate();

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
      // the unit's copies complete on its even CTA's stage barrier
      if (side == 0) mbar_arrive_expect_tx(bar_full(s), (kPair ? 2 : 1) * bytes);
      const uint32_t full = kPair ? mapa_shared(bar_full(s), even) : bar_full(s);
      auto load = [&](uint32_t to, const void *map, int c0, int c1, int c2) {
        if constexpr (kPair)
          tma_load_3d_pair(to, map, full, c0, c1, c2);
        else
          tma_load_3d(to, map, full, c0, c1, c2);
      };
      const bool first = ks < p.nk1;
      const int c = (first ? ks : ks - p.nk1) * kK;
      const void *wm = first ? &maps.w : &maps.w2;
      load(dst_w, wm, c, w0, 0);
      if constexpr (kGlu && !kTokensP)
        load(dst_w + kPBytes / 2, wm, c, static_cast<int>(p.N) + w0, 0);
      load(dst_x, first ? &maps.x : &maps.x2, c, x0, b0);
      if (++s == p.stages) s = 0, ++turn;
    }
    // every copy of the unit has landed before its CTAs exit (the final cluster
    // barrier keeps the odd CTA until then)
    if (side == 0) {
      const long long until = clock64() + kWaitBudgetCycles;
      for (int i = 0; i < p.stages; ++i) {
        // the stage's last use, if any, was in this turn or the one before
        if (i < s)
          ok &= mbar_settled(bar_full(i), turn & 1u, until);
        else if (turn > 0)
          ok &= mbar_settled(bar_full(i), (turn - 1) & 1u, until);
      }
      if (!ok) {
        *abort_flag = 1;
        if constexpr (kPair) hold_after_abort();
      }
    }
  } else if (warp == 1 && side == 0) {
    const uint32_t idesc = idesc_bf16_f32(kPair ? 2 * kP : kP, p.Q, 0, 0);
    auto commit = [&](uint32_t bar) {  // arrives in every CTA of the unit
      if constexpr (kPair)
        mma_commit_pair_elect(bar, static_cast<uint16_t>(0x3u << even));
      else
        mma_commit_elect(bar);
    };
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
      for (int kk = 0; kk < kK / 16; ++kk) {
        const uint64_t ak = desc_advance(da, kk * 32), bk = desc_advance(db, kk * 32);
        const uint32_t more = (ks != k_lo || kk != 0) ? 1u : 0u;
        if constexpr (kPair)
          mma_ss_pair_elect(tmem, ak, bk, idesc, more);
        else
          mma_ss_elect(tmem, static_cast<uint32_t>(ak), static_cast<uint32_t>(bk),
                       static_cast<uint32_t>(ak >> 32), idesc, more);
      }
      commit(bar_empty(s));
      if (++s == p.stages) s = 0, ++turn;
    }
    commit(bar_acc);
  }
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
  // every MMA of the unit has finished: the accumulator is complete and the
  // stages free. An aborted unit's MMAs in flight are waited for too: its issuer
  // commits them when its own wait has run out, so that this one is longer.
  if (!mbar_settled(bar_acc, 0, clock64() + 3 * kWaitBudgetCycles)) *abort_flag = 1;
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
    cluster_sync_relaxed();
  else
    __syncthreads();
  // the residual of the first tokens comes while the sums arrive
  auto fetch = [&](int row) {  // row's residual: three are on their way at a time
    uint2 v = make_uint2(0u, 0u);
    if (mine && residual != nullptr && row < row_hi && token_of(row, b, s))
      v = *reinterpret_cast<const uint2 *>(residual + b * p.r_bs + s * p.r_rs + f);
    return v;
  };
  uint2 res = fetch(r), res1 = fetch(r + per), res2 = fetch(r + 2 * per);
  // where row row_lo of every unit's partial sums lies: this one's own, or
  // where the others' arrive
  uint32_t sums[kC];
#pragma unroll
  for (int r = 0; r < kC; ++r)
    sums[r] = sbase + o * 16 +
              (r == part ? static_cast<uint32_t>(row_lo) * p.pitch
                         : p.recv + static_cast<uint32_t>((r < part ? r : r - 1) *
                                                          (row_hi - row_lo)) * p.pitch);
  if constexpr (kC > 1) {
    // a warp per other unit sends that one's rows, four copies of a quarter
    // each (one copy, or all from one warp, took 0.2 to 0.4 us more), to the
    // place for this unit's among the others
    if (warp < kC && warp != part && lane < 4) {
      const int lo = row_of(warp), n = row_of(warp + 1) - lo;
      const int q_lo = n * lane / 4, q_n = n * (lane + 1) / 4 - q_lo;
      const uint32_t to = rank_of(warp);
      if (q_n > 0)
        bulk_copy_cluster(
            mapa_shared(sbase + p.recv + static_cast<uint32_t>(
                            (part < warp ? part : part - 1) * n + q_lo) * p.pitch, to),
            sbase + static_cast<uint32_t>(lo + q_lo) * p.pitch,
            static_cast<uint32_t>(q_n) * p.pitch, mapa_shared(bar_recv, to));
    }
    __syncwarp();
    // An abort does not end this wait: every unit sends its rows, an aborted one
    // too, and they must have arrived before this CTA lets the cluster go. The
    // last unit may have waited for its accumulators for three budgets since this
    // one was done.
    if (!mbar_try_wait_cluster(bar_recv, 0) &&
        !mbar_settled(bar_recv, 0, clock64() + 4 * kWaitBudgetCycles))
      *abort_flag = 1;
  }
  __syncwarp();
  cluster_arrive_relaxed();  // what was sent to this CTA has arrived

  if (mine) {
    const float4 bias = raw4_values(bias_raw, epi.vec_f32);
    const float4 bias_u = raw4_values(bias_u_raw, epi.vec_f32);
    const uint32_t half = static_cast<uint32_t>(p.feats) * 4;  // SwiGLU: to the linear sums
    // a short loop, its latencies left to the 16 warps: this code runs once, and
    // unrolled it cost more in instruction misses than it saved
#pragma unroll 1
    for (; r < row_hi; r += per) {
      const uint2 res_next = fetch(r + 3 * per);
      if (token_of(r, b, s)) {
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
          load_gate();
          const float4 gate = raw4_values(gate_raw, epi.vec_f32);
          y.x *= gate.x, y.y *= gate.y, y.z *= gate.z, y.w *= gate.w;
        }
        if (residual != nullptr)
          add4(y, make_float4(bf16lo_to_f32(res.x), bf16hi_to_f32(res.x), bf16lo_to_f32(res.y),
                              bf16hi_to_f32(res.y)));
        *reinterpret_cast<uint2 *>(out + b * p.o_bs + s * p.o_rs + f) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      }
      res = res1, res1 = res2, res2 = res_next;
    }
  }
  __syncwarp();
  cluster_wait();  // what this CTA sent has arrived: its shared memory may go
  if (warp == 2) {
    tc_fence_after_sync();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, static_cast<uint32_t>(p.tmem_cols));
    else
      tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

// Rows of a CTA's partial sums and bytes per row.
int sum_rows(int form, int Q) { return form == kPairX ? kP : Q; }
uint32_t sum_pitch(int form, int Q) {
  return static_cast<uint32_t>(form == kPairX ? Q * 4 + 16 : kP * 4);
}
// Shared memory of the partial sums of a CTA's rows; of those that arrive.
uint32_t own_bytes(int form, int Q) {
  return static_cast<uint32_t>(sum_rows(form, Q)) * sum_pitch(form, Q);
}
uint32_t recv_bytes(int form, int Q, int C) {
  const int rows = sum_rows(form, Q);
  return static_cast<uint32_t>((C - 1) * ((rows + C - 1) / C)) * sum_pitch(form, Q);
}
uint32_t stage_size(int form, int Q) {
  return kPBytes + static_cast<uint32_t>(form == kSingle ? Q : Q / 2) * kRowBytes;
}

template <int kAct, int kForm, int kC>
cudaError_t launch(const LinearProblem &q, const SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = linear_split_kernel<kAct, kForm, kC>;
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
  p.Sh = kForm == kSingle ? (p.S + 7) / 8 * 8 : (p.S + 15) / 16 * 8;
  const int q_cta = kForm == kSingle ? p.Q : p.Q / 2;
  p.q_rows = kForm == kPairX ? q_cta : static_cast<int>(q.B) * p.Sh;
  p.feats = (kForm == kPairX ? p.Q : kP) / (glu ? 2 : 1);
  p.n_sb = (p.S + 2 * kP - 1) / (2 * kP);
  const int64_t per_tile = kForm == kPairW ? 2 * p.feats : p.feats;  // features of a unit's tile
  const int64_t n_ft = (q.N + per_tile - 1) / per_tile;
  const int64_t tiles = n_ft * (kForm == kPairX ? q.B * p.n_sb : 1);
  if (tiles > 0x7FFFFFF || p.q_rows > q_cta) return cudaErrorInvalidValue;
  p.n_tb = static_cast<int>(kForm == kPairX ? q.B * p.n_sb : 1);
  p.tmem_cols = 32;
  while (p.tmem_cols < p.Q) p.tmem_cols *= 2;
  p.nk1 = (q.K + kK - 1) / kK;
  p.nk = p.nk1 + (q.K2 + kK - 1) / kK;
  p.pitch = sum_pitch(kForm, p.Q);
  p.stages = plan.stages;
  // the CTA's own partial sums over the drained ring, the others' behind them
  const uint32_t ring = static_cast<uint32_t>(p.stages) * stage_size(kForm, p.Q);
  const uint32_t own = own_bytes(kForm, p.Q);
  p.early = plan.early ? 1 : 0;
  p.recv = plan.early ? std::max(ring, own) : own;
  p.tail = std::max(ring, p.recv + recv_bytes(kForm, p.Q, kC));
  const uint32_t need = p.tail + kTailBytes;
  const uint32_t smem = std::max(need, kForm == kSingle ? kSmemSingle : kSmemPair);
  if (smem > (kForm == kSingle ? kSmemHalf : kSmemAll)) return cudaErrorInvalidValue;
  const uint32_t w_box = static_cast<uint32_t>(kForm == kPairX ? p.Q / 2 : p.feats);
  const uint32_t x_box = static_cast<uint32_t>(kForm == kPairX ? kP : p.Sh);
  const uint32_t x_box_b = kForm == kPairX ? 1 : static_cast<uint32_t>(q.B);
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
  attr[0].val.clusterDim.x = kForm == kSingle ? kC : 2 * kC;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * attr[0].val.clusterDim.x, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, epi,
                            static_cast<const uint16_t *>(q.residual),
                            static_cast<uint16_t *>(q.out), status);
}

template <int kAct, int kForm>
cudaError_t launch(const LinearProblem &q, const SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  switch (plan.C) {
    case 1: return launch<kAct, kForm, 1>(q, plan, epi, status, stream);
    case 2: return launch<kAct, kForm, 2>(q, plan, epi, status, stream);
    case 3: return launch<kAct, kForm, 3>(q, plan, epi, status, stream);
    case 4: return launch<kAct, kForm, 4>(q, plan, epi, status, stream);
    default: break;
  }
  if constexpr (kForm == kSingle) {
    if (plan.C == 6) return launch<kAct, kForm, 6>(q, plan, epi, status, stream);
    if (plan.C == 8) return launch<kAct, kForm, 8>(q, plan, epi, status, stream);
  }
  return cudaErrorInvalidValue;
}

template <int kAct>
cudaError_t launch(const LinearProblem &q, const SplitPlan &plan, const LinearEpilogue &epi,
                   int *status, cudaStream_t stream) {
  switch (plan.form) {
    case kSingle: return launch<kAct, kSingle>(q, plan, epi, status, stream);
    case kPairW: return launch<kAct, kPairW>(q, plan, epi, status, stream);
    case kPairX: return launch<kAct, kPairX>(q, plan, epi, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// The form, the split of the channels and the ring. A launch has so many CTAs
// resident, by the CTAs of a cluster: those of pairs have an SM each (clusters
// of 4, 6 and 8 do not fill every SM), single ones half an SM. Half an SM
// leaves room for the next kernel's prologue and for a second CTA; but then
// the two share what the SM takes in, and a ring of half the bytes is refilled
// only every 1.3 us.
SplitPlan plan_split(const LinearProblem &q, int act, int sms) {
  const bool glu = act == FLUX_ACT_SWIGLU;
  const int64_t nk = (q.K + kK - 1) / kK + (q.K2 + kK - 1) / kK;
  const int64_t wr = glu ? 2 * q.N : q.N;
  const double bytes = 2.0 * (static_cast<double>(q.B * q.S + wr) * (q.K + q.K2) +
                              static_cast<double>(q.B * q.S) * q.N *
                                  (q.residual != nullptr ? 2 : 1));
  static constexpr int kResident[2][9] = {{0, 152, 152, 0, 144, 0, 138, 0, 120},    // an SM each
                                          {0, 304, 304, 291, 296, 0, 276, 0, 288}};  // half an SM
  // Coefficients of a regression over the 103 problems, each named for what its
  // term grows with; they make up for one another and are no measurements. In ns:
  // per refill of a ring (what a pair's ring brings hides it), wave, call, row of
  // Q, joining of sums, sum finished. In bytes per ns: hbm for all bytes (the
  // memory has 6770; a pair's stages, waves and sums account for its times without
  // that bound), send for the sums sent (bulk copies reach about 30 per SM).
  struct Costs {
    double refill, wave, call, row, join, finish, hbm, send;
  };
  static constexpr Costs kPairCosts = {0.0, 4100.0, 240.0, 0.0, 330.0, 0.056, 23000.0, 123.0};
  static constexpr Costs kSingleCosts = {1275.0, 4720.0, -2210.0, 16.0, 158.0, 0.046, 7860.0, 92.0};
  SplitPlan best{-1, false, 0, 0, 0, 1e30};  // no form yet
  auto consider = [&](int form, int Q) {
    const bool single = form == kSingle;
    const int64_t feats = (form == kPairX ? Q : single ? kP : 2 * kP) / (glu ? 2 : 1);
    const int64_t tiles = (q.N + feats - 1) / feats *
                          (form == kPairX ? q.B * ((q.S + 2 * kP - 1) / (2 * kP)) : 1);
    const int rows = sum_rows(form, Q);
    const int cta_feats = (form == kPairX ? Q : kP) / (glu ? 2 : 1);
    const uint32_t stage = stage_size(form, Q);
    const uint32_t room = (single ? kSmemHalf : kSmemAll) - kTailBytes;
    for (int C = 1; C <= max_units(form) && C <= nk; ++C) {
      const int size = single ? C : 2 * C;  // CTAs of a cluster
      const int64_t slots = kResident[single ? 1 : 0][size] * static_cast<int64_t>(sms) / 152;
      const uint32_t recv = recv_bytes(form, Q, C);
      if (slots < size || own_bytes(form, Q) + recv > room || 3 * stage > room) continue;
      int stages = static_cast<int>(std::min<uint32_t>(kMaxStages, room / stage));
      // a place of their own for the sums saves a cluster barrier, unless the
      // ring gets short for it
      const bool early = recv + kEarlyRing <= room;
      if (early) stages = static_cast<int>(std::min<uint32_t>(kMaxStages, (room - recv) / stage));
      const int64_t ctas = tiles * size;
      const double waves = static_cast<double>((ctas + slots - 1) / slots);
      const double shared = !single || ctas <= sms ? 1.0 : std::min(2.0, ctas / (0.59 * sms));
      const Costs &t = single ? kSingleCosts : kPairCosts;
      const double per_stage =
          std::max(stage_ns(stage, single ? Q / 2 : Q) * shared, t.refill / stages);
      const double ns =
          std::max(waves * static_cast<double>((nk + C - 1) / C) * per_stage, bytes / t.hbm) +
          waves * t.wave + t.call + t.row * Q +
          (C > 1 ? t.join + (C - 1) * (rows / static_cast<double>(C)) * sum_pitch(form, Q) / t.send
                 : 0.0) +
          t.finish * rows / C * cta_feats;
      if (ns < best.ns) best = SplitPlan{form, early, Q, C, stages, ns};
    }
  };
  const int64_t rows8 = q.B * ((q.S + 7) / 8 * 8), rows16 = q.B * ((q.S + 15) / 16 * 16);
  if (rows8 <= 64) consider(kSingle, static_cast<int>((rows8 + 15) / 16 * 16));
  if (rows16 <= 256) consider(kPairW, static_cast<int>((rows16 + 31) / 32 * 32));
  // Fewer tokens would fill less than a quarter of P; but of many batch elements
  // that do not follow one another, each rounded up, the tokens may be too many
  // columns for either form above.
  if (q.B * q.S >= 64 || best.form < 0)
    for (int Q = 32; Q <= 256; Q += 32) consider(kPairX, Q);
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
