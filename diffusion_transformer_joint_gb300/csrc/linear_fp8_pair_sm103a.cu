// flux_linear_fp8 for many rows, on sm_103a (GB300): a GEMM of e4m3 operands on
// tcgen05 CTA pairs whose sums leave the tensor core after every group of 128
// channels, to be scaled and added in registers.
//
//   y[t, n] = sum_g xs[t, g] ws[n / 128, g] sum_{k in g} x[t, k] w[n, k]
//   out = residual + gate * act(y + bias)
//
// Tiles: 256 token rows of one batch element x tn accumulator columns, 128
// channels (one group, 128 bytes) per pipeline stage. The columns are two halves
// of tn / 2, an MMA of N = tn / 2 each, which TMEM holds twice over or more: the
// MMAs of a group start both halves afresh, while the groups' sums before are read. The
// scales do not fit the tensor core's own block scaling, whose factors are
// powers of two.
//
// What that costs: a group's 128 x tn sums per SM are read from TMEM (128 KB at
// tn = 256) and take as many FMAs, in the 512 cycles that the group's MMAs last.
// So one warpgroup adds a half: thread = TMEM lane = token row, its up to 128
// running sums in registers (setmaxnreg). A half of a group is read while the
// other half's MMAs run, and has three halves' time (768 cycles) from its last MMA
// until its columns are wanted again. Its hand-back to the even CTA's issuer is an
// arrival without a release, which waits for the thread's stores: with one, a
// group took 1.3 us instead of 0.7 (0.43 with all that follows).
//
// Warp 3 of each CTA brings the scales, four groups at a time, to a ring in shared
// memory: every other way took the sums' warps longer, which set the pace (a
// barrier's wait per group, some 100 cycles; copies of their own, 130).
//
// SwiGLU: a half's columns are gate features and the linear features of the same
// outputs, so that a thread has both factors of what it writes.
//
// CTA pairs, the walk over the tiles, the residual through boxes in shared
// memory, the vectors of a tile and the bounded waits are as in linear_pair. The
// epilogue takes its values from registers; the MMAs meanwhile run on for two
// groups. A residual's boxes are fetched while the tile's groups are added: three
// boxes a warp with one, else two. The ring has the rest of the shared memory: five
// stages of 256 columns either way, 6, 7 and 8 (9 without a residual) of 192, 128 and 64.
//
// 12 warps per CTA: warp 0 TMA producer, warps 1 and 2 MMA issuers of a half each
// (even CTA; one warp for both took longer to issue a group's MMAs, between waits
// of some 100 cycles, than they run), warp 2 TMEM allocation, warps 4-7 and 8-11
// the sums of the two halves.
//
// Measured (GB300, in a graph of 2 ms; in brackets calls for a second or more, at the
// power limit): 4096 tokens 4096 -> 4096 with gate and residual 79 us, 1745 TFLOP/s
// (79), 4056 tokens 4096 -> SwiGLU 12288 373, 2190 (381), 12800 tokens 18432 -> 6144
// 1110, 2610 (1240, 2340). A group takes 0.43 us at 256 columns (its MMAs 0.26, its copies
// 0.29): a half's columns go from MMAs to sums and back, and TMEM holds two of them.
// At 64 and 128 columns it takes 0.28, and still 0.26 to 0.27 without its MMAs,
// W's copies or its additions: a chain of hand-offs, none of which is alone the bound.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "linear_fp8_common.cuh"

namespace flux {
namespace {

constexpr int kRows = 128;  // token rows per CTA (256 per pair)
constexpr int kMaxTn = 256;
constexpr int kGroup = 9;  // row blocks of a group of tiles (the walk)
constexpr uint32_t kABytes = kRows * kGroupK;  // 16 KB: this CTA's token rows
constexpr int kMaxStages = 10;
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kMaxBoxes = 3;             // boxes per epilogue warp
constexpr uint32_t kBoxBytes = 32 * 64;  // 32 rows x 32 features
constexpr int kScaleSlots = 2, kScaleBatch = 4;  // slots, of so many groups
constexpr uint32_t kScaleBytes = kRows * 4 + 16;  // a group: the rows', two of W's per half
constexpr int kBarFull = 0;                    // (even CTA) both CTAs' copies landed
constexpr int kBarEmpty = kMaxStages;          // the pair's MMAs read the stage
constexpr int kMaxBufs = 8;
constexpr int kBarAccFull = 2 * kMaxStages;               // + 2 * buffer + half
constexpr int kBarAccEmpty = kBarAccFull + 2 * kMaxBufs;  // (even CTA) both CTAs read it
constexpr int kBarDrain = kBarAccEmpty + 2 * kMaxBufs;
constexpr int kBarScFull = kBarDrain + 2;
constexpr int kBarScEmpty = kBarScFull + kScaleSlots;
constexpr int kBarRes = kBarScEmpty + kScaleSlots;  // residual box landed, per warp and box
constexpr int kBarVecReady = kBarRes + kEpiWarps * kMaxBoxes;
constexpr int kBarVecFree = kBarVecReady + 1;
constexpr int kNumBars = kBarVecFree + 1;
// shared memory from here on is behind the ring and the boxes
constexpr uint32_t kOffScale = 0;
constexpr uint32_t kOffVec = kScaleSlots * kScaleBatch * kScaleBytes;  // a tile's bias, gate
constexpr uint32_t kOffBar = kOffVec + 2 * kMaxTn * 4;
constexpr uint32_t kOffTmemSlot = kOffBar + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmemSlot + 8;
constexpr uint32_t kTailBytes = kOffAbort + 8;
constexpr uint32_t kSmemMax = 232448;
constexpr uint16_t kPairMask = 0x3;
// Registers: 384 threads x 168 at launch. (Sums in pieces of 32 columns spilled at
// any split, and a spill inside the loop is dear: 12800 x 18432 -> 6144 took 1.09
// to 1.27 ms.)
constexpr uint32_t kSumRegs = 216, kRestRegs = 72;
static_assert(2 * kSumRegs + kRestRegs == 3 * 168, "warpgroups' shares of the registers");

struct PairShape {
  int64_t S, N, xs_bs, xs_rs, xs_ks, ws_rs, ws_ks;
  const float *xs, *ws;
  int stages, boxes, nk;
  int n_sb, n_rb, n_ft, n_tiles;  // row blocks per batch element, in all; feature tiles
  uint32_t off_box, off_tail;
};

struct PairMaps {
  CUtensorMap x, w, out, res;
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

// y += v, y *= v: 32 entries in shared memory, the same for all lanes.
template <bool kMul>
__device__ __forceinline__ void join32(float (&y)[32], const float *v) {
#pragma unroll
  for (int k = 0; k < 32; k += 16) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const float4 *>(v + k)[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[k + 4 * i + e] = kMul ? y[k + 4 * i + e] * u[e] : y[k + 4 * i + e] + u[e];
    }
  }
}

// acc += s * (16 sums as loaded from TMEM)
__device__ __forceinline__ void add_scaled(uint64_t *acc, const uint64_t (&v)[8], float s) {
  const uint64_t s2 = f2_pack(s, s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i]) : "l"(v[i]), "l"(s2));
}

// kPieces: 32-column pieces of a half, tn = 64 kPieces. (As a launch parameter it
// cost a third more time: running sums were moved between registers.)
template <int kAct, int kPieces>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp8_pair_kernel(const __grid_constant__ PairMaps maps, const PairShape p,
                           const LinearEpilogue epi, const int has_res, int *__restrict__ status) {
  constexpr bool kGlu = kAct == FLUX_ACT_SWIGLU;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t sbase = smem_addr(base);
  const uint32_t tail = sbase + p.off_tail;
  auto bar = [&](int i) { return tail + kOffBar + 8u * static_cast<uint32_t>(i); };
  auto scales_at = [&](int i) {  // group i of the ring's slots
    return tail + kOffScale + kScaleBytes * static_cast<uint32_t>(i);
  };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + p.off_tail + kOffTmemSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + p.off_tail + kOffAbort);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t crank = cluster_ctarank();  // 0: issues the MMAs
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  constexpr int tn = 64 * kPieces;           // accumulator columns
  constexpr int hw = tn / 2;                 // columns of a half
  // accumulators that TMEM holds: a power of two
  constexpr uint32_t bufs = tn == 64 ? 8 : tn == 128 ? 4 : 2;
  constexpr int feats = kGlu ? hw : tn;      // output features per tile
  constexpr int hfeats = feats / 2;          // of a half
  // 16-column pieces that the sums' warps load at once (with two, the tile of 192
  // columns spills)
  constexpr int kStep = kPieces == 3 ? 1 : 2;
  constexpr uint32_t half_bytes = static_cast<uint32_t>(hw / 2) * kGroupK;  // W rows of this CTA
  constexpr uint32_t stage_bytes = kABytes + 2 * half_bytes;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 2);  // both halves' MMAs
    }
    for (uint32_t b = 0; b < 2 * bufs; ++b) {
      mbar_init(bar(kBarAccFull + b), 1);
      mbar_init(bar(kBarAccEmpty + b), kEpiWarps);  // a half's four warps of both CTAs
    }
    for (int h = 0; h < 2; ++h) mbar_init(bar(kBarDrain + h), 1);
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(bar(kBarScFull + i), 1);
      mbar_init(bar(kBarScEmpty + i), kEpiWarps);
    }
    for (int i = 0; i < kEpiWarps * kMaxBoxes; ++i) mbar_init(bar(kBarRes + i), 1);
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

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- TMA producer
      tma_prefetch_desc(&maps.x);
      tma_prefetch_desc(&maps.w);
      int s = 0;          // stage
      uint32_t turn = 0;  // times round the ring
      bool ok = true;
      // this CTA's W rows of a half: the first or second part of the half's
      // features, or its gate or linear features
      auto w_row = [&](int ft, int h) {
        const int64_t f = static_cast<int64_t>(ft) * feats + h * hfeats;
        return static_cast<int>(crank == 0 ? f : kGlu ? p.N + f : f + hw / 2);
      };
      grid_dep_wait();
      for (int t = cid; ok && t < p.n_tiles; t += ncl) {
        int ft, rb;
        tile_at(p, t, ft, rb);
        const int b = rb / p.n_sb;
        const int s0 = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows;
        const int w0 = w_row(ft, 0), w1 = w_row(ft, 1);
        for (int g = 0; g < p.nk; ++g) {
          if (!(ok = mbar_wait(bar(kBarEmpty + s), (turn & 1u) ^ 1u, abort_flag))) break;
          const uint32_t dst = sbase + s * stage_bytes;
          // both CTAs' copies complete on the even CTA's stage barrier
          if (crank == 0) mbar_arrive_expect_tx(bar(kBarFull + s), 2 * stage_bytes);
          const uint32_t full0 = mapa_shared(bar(kBarFull + s), 0);
          const int c = g * kGroupK;
          tma_load_3d_pair(dst, &maps.x, full0, c, s0, b);
          tma_load_3d_pair(dst + kABytes, &maps.w, full0, c, w0, 0);
          tma_load_3d_pair(dst + kABytes + half_bytes, &maps.w, full0, c, w1, 0);
          if (++s == p.stages) s = 0, ++turn;
        }
      }
      // every copy of the pair has landed before the CTAs exit (as linear_pair)
      if (crank == 0) {
        const long long until = clock64() + kWaitBudgetCycles;
        for (int i = 0; i < p.stages; ++i) {
          // the stage's last use, if any, was in this turn or the one before
          if (i < s)
            ok &= mbar_settled(bar(kBarFull + i), turn & 1u, until);
          else if (turn > 0)
            ok &= mbar_settled(bar(kBarFull + i), (turn - 1) & 1u, until);
        }
        if (!ok) {
          *abort_flag = 1;
          hold_after_abort();
        }
      }
    } else if ((warp == 1 || warp == 2) && crank == 0) {
      // ------------------------------ MMA issuers (even CTA), one for each half
      const uint32_t h = static_cast<uint32_t>(warp - 1);
      const uint32_t idesc = idesc_e4m3_f32(2 * kRows, hw);
      int s = 0;
      uint32_t turn = 0, n = 0;  // n: groups so far
      bool ok = true;
      grid_dep_wait();  // the budget of the first stage's wait begins with its copy
      for (int t = cid; ok && t < p.n_tiles; t += ncl) {
        for (int g = 0; g < p.nk; ++g, ++n) {
          const uint32_t a = 2 * (n % bufs) + h, par = (n / bufs & 1u) ^ 1u;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarFull + s), turn & 1u, abort_flag) &&
                                                 mbar_wait(bar(kBarAccEmpty + a), par, abort_flag))))
            break;
          tc_fence_after_sync();
          const uint32_t st = sbase + s * stage_bytes;
          const uint64_t da = sdesc_sw128(st, 16, 1024);
          const uint64_t db = sdesc_sw128(st + kABytes + h * half_bytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kGroupK / 32; ++kk)
            mma_f8_pair_elect(tmem + a * hw, desc_advance(da, kk * 32),
                              desc_advance(db, kk * 32), idesc, kk != 0 ? 1u : 0u);
          mma_commit_pair_elect(bar(kBarAccFull + a), kPairMask);
          mma_commit_pair_elect(bar(kBarEmpty + s), kPairMask);  // (and the other half's)
          if (++s == p.stages) s = 0, ++turn;
        }
      }
      // every MMA issued above has finished before TMEM is released
      mma_commit_pair_elect(bar(kBarDrain + static_cast<int>(h)), 0x1);
      if (!mbar_settled(bar(kBarDrain + static_cast<int>(h)), 0, clock64() + kWaitBudgetCycles))
        *abort_flag = 1;
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------------- scales
      // Rows lane, lane + 32, ...; lane 2 h + i: W's block i of half h, the first
      // and the last one of its features (SwiGLU: of its gate and linear ones).
      int slot = 0;
      uint32_t use = 0;
      bool ok = true;
      const int N = static_cast<int>(p.N);
      grid_dep_wait();
      for (int t = cid; ok && t < p.n_tiles; t += ncl) {
        int ft, rb;
        tile_at(p, t, ft, rb);
        const int b = rb / p.n_sb;
        const int s0 = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows;
        const int rows = static_cast<int>(p.S) - s0 - lane;  // from this lane's first one on
        const float *xs = p.xs + b * p.xs_bs + (s0 + lane) * p.xs_rs;
        int f = ft * feats + ((lane >> 1) & 1) * hfeats;
        if (lane & 1) f += kGlu ? N : hw - 1;
        const int last = (kGlu ? 2 * N : N) - 1;
        const float *ws = p.ws + ((f < last ? f : last) / 128) * p.ws_rs;
        for (int g0 = 0; g0 < p.nk; g0 += kScaleBatch) {
          float x[kScaleBatch][4], w[kScaleBatch];
#pragma unroll
          for (int i = 0; i < kScaleBatch; ++i) {
            w[i] = lane < 4 ? *ws : 0.f;
            const float *at = xs;
#pragma unroll
            for (int j = 0; j < 4; ++j, at += 32 * p.xs_rs) x[i][j] = 32 * j < rows ? *at : 0.f;
            if (g0 + i + 1 < p.nk) xs += p.xs_ks, ws += p.ws_ks;  // (past the end: the last again)
          }
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarScEmpty + slot), (use & 1u) ^ 1u,
                                                       abort_flag))))
            break;
#pragma unroll
          for (int i = 0; i < kScaleBatch; ++i) {
            const uint32_t at = scales_at(slot * kScaleBatch + i) + static_cast<uint32_t>(lane) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) st_shared_b32(at + j * 128, __float_as_uint(x[i][j]));
            if (lane < 4) st_shared_b32(at + kRows * 4, __float_as_uint(w[i]));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarScFull + slot));
          if (++slot == kScaleSlots) slot = 0, ++use;
        }
      }
    }
  } else {
    // ------------------------------------------------------ sums and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int wq = warp & 3;            // TMEM lane quadrant
    const int h = (warp - 4) >> 2;      // half of the columns
    const int et = tid - 128;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t acc_empty0 = mapa_shared(bar(kBarAccEmpty), 0);
    const uint32_t boxes =
        sbase + p.off_box + static_cast<uint32_t>((warp - 4) * p.boxes) * kBoxBytes;
    const int bar_res = kBarRes + (warp - 4) * kMaxBoxes;
    float *vec_bias = reinterpret_cast<float *>(base + p.off_tail + kOffVec);
    float *vec_gate = vec_bias + kMaxTn;
    const bool vecs = epi.bias != nullptr || epi.gate != nullptr;
    int load_slot = 0, store_slot = 0;  // this warp's boxes: residual asked for, staged
    uint32_t res_par = 0;               // bit i: parity of box i's next residual
    int loads_ahead = 0;
    int slot = 0;         // of the scales
    uint32_t sc_use = 0;
    bool ready = false;   // the next accumulator was complete when last looked at
    uint32_t n = 0;
    int lt = 0;
    bool ok = true;
    grid_dep_wait();
    for (int t = cid; ok && t < p.n_tiles; t += ncl, ++lt) {
      int ft, rb;
      tile_at(p, t, ft, rb);
      const int b = rb / p.n_sb;
      const int sc = (rb - b * p.n_sb) * (2 * kRows) + static_cast<int>(crank) * kRows;
      const int s0 = sc + wq * 32;
      const int N = static_cast<int>(p.N);  // (at most 2^28, and tiles end below 2^29)
      const int f0 = ft * feats;            // of the tile
      const int fh = f0 + h * hfeats;       // of the half
      const int left = N - fh;
      // boxes of this tile that hold anything to write
      const int n_box = s0 >= p.S || left <= 0
                            ? 0
                            : left < hfeats ? (left + 31) / 32 : hfeats / 32;
      // Pieces whose columns have W's first block of the half (128, 64 or 32
      // columns from a multiple of their number on lie in one block).
      const int in_first = ((fh / 128 + 1) * 128 - fh) / 32;
      auto load_residual = [&](int c) {  // a box whose store has read it
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(bar_res + load_slot), kBoxBytes);
          tma_load_3d(boxes + load_slot * kBoxBytes, &maps.res, bar(bar_res + load_slot),
                      fh + c * 32, s0, b);
        }
        if (++load_slot == p.boxes) load_slot = 0;
        ++loads_ahead;
      };
      if (has_res) {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        for (int c = 0; c < n_box && c < p.boxes; ++c) load_residual(c);
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
        if (lt > 0 && !(ok = __all_sync(0xffffffffu,
                                        mbar_wait(bar(kBarVecFree),
                                                  static_cast<uint32_t>(lt - 1) & 1u, abort_flag))))
          break;
        if (epi.bias != nullptr && et < tn) {
          const int f = f0 + (kGlu && et >= feats ? et - feats : et);
          if (f < N)
            vec_bias[et] = load_vec1(epi.bias, kGlu && et >= feats ? N + f : f, epi.vec_f32);
        }
        if (epi.gate != nullptr && !gate_rowwise && et < feats && f0 + et < N)
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

      uint64_t acc[16 * kPieces];  // pairs of sums
#pragma unroll
      for (int i = 0; i < 16 * kPieces; ++i) acc[i] = 0;
#pragma unroll 1
      for (int g = 0; g < p.nk; ++g, ++n) {
        const uint32_t a = 2 * (n % bufs) + static_cast<uint32_t>(h);
        const int in_slot = g % kScaleBatch;
        if (in_slot == 0 &&
            !(ok = __all_sync(0xffffffffu,
                              mbar_wait(bar(kBarScFull + slot), sc_use & 1u, abort_flag))))
          break;
        const uint32_t scales = scales_at(slot * kScaleBatch + in_slot);
        const float xs = ld_shared_f32(scales + static_cast<uint32_t>(wq * 32 + lane) * 4);
        const uint2 ws = ld_shared_v2(scales + kRows * 4 + 8 * h);
        if (!__all_sync(0xffffffffu, ready) &&
            !(ok = __all_sync(0xffffffffu,
                              mbar_wait(bar(kBarAccFull + a), n / bufs & 1u, abort_flag))))
          break;
        const float sa = xs * __uint_as_float(ws.x), sb = xs * __uint_as_float(ws.y);
        tc_fence_after_sync();
        const uint32_t from = tmem + a * hw + lane_off;
        // kStep pieces at a time through the same registers: the FMAs take 290 cycles
        // a group for the two warps of a scheduler, a load some more. (One piece at a
        // time: 12288 -> 4096 channels of 4096 tokens 187.9 us, two 185.4; two whose
        // registers take turns: half as long again.)
        uint64_t v[8], v1[8];
#pragma unroll
        for (int k = 0; k < 2 * kPieces; k += kStep) {
          if constexpr (kStep == 2)
            tmem_ld16_pairs2(from + k * 16, from + k * 16 + 16, v, v1);
          else
            tmem_ld16_pairs(from + k * 16, v);
          if (k == 2 * kPieces - kStep) {
            // this warp's TMEM reads are complete: the columns may be reused
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + 8u * a);
            // a look at the next group's, whose answer comes while these are added
            ready = mbar_test_wait(
                bar(kBarAccFull + static_cast<int>(2 * ((n + 1) % bufs)) + h), (n + 1) / bufs & 1u);
          }
          // (both pieces lie in one block of W)
          const float s = (kGlu ? k < kPieces : kPieces != 3 || k < 2 * in_first) ? sa : sb;
          add_scaled(acc + k * 8, v, s);
          if constexpr (kStep == 2) add_scaled(acc + (k + 1) * 8, v1, s);
        }
        if (in_slot == kScaleBatch - 1 || g == p.nk - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarScEmpty + slot));
          if (++slot == kScaleSlots) slot = 0, ++sc_use;
        }
      }
      if (!ok) break;

      // 32 features at a time: the rows' values into a box, which one copy stores
#pragma unroll
      for (int c = 0; c < hfeats / 32; ++c) {
        if (c >= n_box) break;
        const uint32_t box = boxes + store_slot * kBoxBytes;
        if (has_res) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(bar_res + store_slot),
                                                       (res_par >> store_slot) & 1u, abort_flag))))
            break;
          res_par ^= 1u << store_slot;
          --loads_ahead;
        } else {
          if (lane == 0) bulk_wait_read_1();
          __syncwarp();
        }
        // One operand at a time for all 32 features, its loads on their way together.
        // (Features past N: whatever lies there, never stored by the copy.)
        const uint32_t row = box + lane * 64, turn = static_cast<uint32_t>(lane >> 1) & 3u;
        const int v0 = h * hfeats + c * 32;  // in the tile's vectors
        float y[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) f2_unpack(acc[c * 16 + i], y[2 * i], y[2 * i + 1]);
        if (epi.bias != nullptr) join32<false>(y, vec_bias + v0);
        if constexpr (kGlu) {
          float w[32];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            f2_unpack(acc[8 * kPieces + c * 16 + i], w[2 * i], w[2 * i + 1]);
          if (epi.bias != nullptr) join32<false>(w, vec_bias + feats + v0);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = activate<FLUX_ACT_SILU>(y[i]) * w[i];
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = activate<kAct>(y[i]);
        }
        if (epi.gate != nullptr) {
          if (gate_rowwise) {
            for (int q = 0; q < 4; ++q) {
              if (c * 32 + q * 8 >= left) break;
              float w[8];
              load_vec8(epi.gate, gate_row * epi.gate_bs + fh + c * 32 + q * 8, epi.vec_f32, w);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >> 3 == q) y[i] *= w[i & 7];
            }
          } else {
            join32<true>(y, vec_gate + v0);
          }
        }
        if (has_res) {
          uint4 r[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) r[q] = ld_shared_v4(row + ((q ^ turn) << 4));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float w[8];
            unpack8(r[q], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[q * 8 + i] += w[i];
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_shared_v4(row + ((q ^ turn) << 4),
                       make_uint4(pack_bf16x2(y[q * 8], y[q * 8 + 1]),
                                  pack_bf16x2(y[q * 8 + 2], y[q * 8 + 3]),
                                  pack_bf16x2(y[q * 8 + 4], y[q * 8 + 5]),
                                  pack_bf16x2(y[q * 8 + 6], y[q * 8 + 7])));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out, box, fh + c * 32, s0, b);
          bulk_commit();
        }
        if (++store_slot == p.boxes) store_slot = 0;
        if (has_res && c + p.boxes < n_box) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
          load_residual(c + p.boxes);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (vecs && lane == 0) mbar_arrive(bar(kBarVecFree));
    }
    if (lane == 0) {
      // residual copies still in flight after an abort, then every output store
      const long long until = clock64() + kWaitBudgetCycles;
      for (int j = 0; j < loads_ahead; ++j) {
        const int i = (store_slot + j) % p.boxes;
        if (!mbar_settled(bar(bar_res + i), (res_par >> i) & 1u, until)) *abort_flag = 1;
      }
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

template <int kAct, int kPieces>
cudaError_t launch(const LinearFp8Problem &q, const LinearEpilogue &epi, int *status,
                   cudaStream_t stream) {
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  static std::atomic<int> max_pairs[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = linear_fp8_pair_kernel<kAct, kPieces>;
  constexpr int tn = 64 * kPieces;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemMax));
  });
  if (attr_err[dev] != cudaSuccess) return attr_err[dev];
  constexpr bool glu = kAct == FLUX_ACT_SWIGLU;
  PairShape p;
  p.S = q.S, p.N = q.N;
  p.xs_bs = q.xs_bs, p.xs_rs = q.xs_rs, p.xs_ks = q.xs_ks, p.ws_rs = q.ws_rs, p.ws_ks = q.ws_ks;
  p.xs = q.xs, p.ws = q.ws;
  p.boxes = q.residual != nullptr ? kMaxBoxes : 2;
  const uint32_t stage = kABytes + static_cast<uint32_t>(tn / 2) * kGroupK;
  const uint32_t box_bytes = static_cast<uint32_t>(kEpiWarps * p.boxes) * kBoxBytes;
  p.stages = static_cast<int>(std::min<uint32_t>(
      kMaxStages, (kSmemMax - kTailBytes - box_bytes) / stage));
  p.off_box = static_cast<uint32_t>(p.stages) * stage;
  p.off_tail = p.off_box + box_bytes;
  const uint32_t smem = p.off_tail + kTailBytes;
  const int64_t n_sb = (q.S + 2 * kRows - 1) / (2 * kRows);
  const int64_t n_rb = n_sb * q.B;
  const int64_t feats = glu ? tn / 2 : tn;
  const int64_t n_ft = (q.N + feats - 1) / feats;
  if (n_rb * n_ft > 0x3FFFFFFFLL || n_ft * kGroup > 0x3FFFFFFFLL) return cudaErrorInvalidValue;
  p.n_sb = static_cast<int>(n_sb);
  p.n_rb = static_cast<int>(n_rb);
  p.n_ft = static_cast<int>(n_ft);
  p.n_tiles = static_cast<int>(n_rb * n_ft);
  p.nk = (q.K + kGroupK - 1) / kGroupK;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
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
  const int64_t wr = glu ? 2 * q.N : q.N;
  PairMaps maps;
  if (!make_byte_map(&maps.x, q.x, q.K, q.S, q.B, q.x_rs, q.x_bs, kRows) ||
      !make_byte_map(&maps.w, q.w, q.K, wr, 1, q.w_rs, q.w_rs * wr,
                     static_cast<uint32_t>(tn / 4)) ||
      !make_row_map(&maps.out, q.out, q.N, q.S, q.B, q.o_rs, q.o_bs, 32, 32, 1))
    return cudaErrorInvalidValue;
  maps.res = maps.out;
  if (q.residual != nullptr &&
      !make_row_map(&maps.res, q.residual, q.N, q.S, q.B, q.r_rs, q.r_bs, 32, 32, 1))
    return cudaErrorInvalidValue;
  const int64_t pairs = p.n_tiles < np ? p.n_tiles : np;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, epi, q.residual != nullptr ? 1 : 0, status);
}

template <int kAct>
cudaError_t launch(const LinearFp8Problem &q, int tn, const LinearEpilogue &epi, int *status,
                   cudaStream_t stream) {
  if (tn == 256) return launch<kAct, 4>(q, epi, status, stream);
  if (tn == 128) return launch<kAct, 2>(q, epi, status, stream);
  if constexpr (kAct != FLUX_ACT_SWIGLU) {
    if (tn == 192) return launch<kAct, 3>(q, epi, status, stream);
    if (tn == 64) return launch<kAct, 1>(q, epi, status, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// The tile's width: 64, 128, 192 or 256 accumulator columns (SwiGLU: 128 or 256).
// Its estimate in ns: what a group of channels takes, the end of a tile that the
// next one's MMAs do not hide, and a call; fitted to 194 times at 42 problems of 32
// to 4608 tokens.
Fp8PairPlan plan_fp8_pair(const LinearFp8Problem &q, int act, int sms) {
  struct Costs {
    int tn;
    double group, tile, call;
  };
  static constexpr Costs kCosts[] = {{256, 432.0, 4500.0, 400.0}, {192, 397.0, 2870.0, 1330.0},
                                     {128, 278.0, 1900.0, 2100.0}, {64, 283.0, 220.0, 3700.0}};
  const bool glu = act == FLUX_ACT_SWIGLU;
  const int64_t n_rb = q.B * ((q.S + 2 * kRows - 1) / (2 * kRows));
  const double nk = static_cast<double>((q.K + kGroupK - 1) / kGroupK);
  const int64_t pairs = std::max(1, sms / 2);
  const int64_t wr = glu ? 2 * q.N : q.N;
  const double bytes = static_cast<double>(q.B * q.S + wr) * q.K +
                       2.0 * static_cast<double>(q.B * q.S) * q.N * (q.residual != nullptr ? 2 : 1);
  Fp8PairPlan best{kMaxTn, 1e30};
  for (const Costs &t : kCosts) {
    if (glu && t.tn % 128 != 0) continue;
    const int64_t feats = glu ? t.tn / 2 : t.tn;
    const int64_t tiles = n_rb * ((q.N + feats - 1) / feats);
    const double waves = static_cast<double>((tiles + pairs - 1) / pairs);
    const double ns = std::max(t.call + waves * (nk * t.group + t.tile), bytes / 6690.0 + 4000.0);
    if (ns < best.ns) best = Fp8PairPlan{t.tn, ns};
  }
  return best;
}

cudaError_t launch_fp8_pair(const LinearFp8Problem &q, const Fp8PairPlan &plan,
                            const LinearEpilogue &epi, int act, int *status, cudaStream_t stream) {
  switch (act) {
    case FLUX_ACT_NONE: return launch<FLUX_ACT_NONE>(q, plan.tn, epi, status, stream);
    case FLUX_ACT_SILU: return launch<FLUX_ACT_SILU>(q, plan.tn, epi, status, stream);
    case FLUX_ACT_GELU_TANH: return launch<FLUX_ACT_GELU_TANH>(q, plan.tn, epi, status, stream);
    default: return launch<FLUX_ACT_SWIGLU>(q, plan.tn, epi, status, stream);
  }
}

}  // namespace flux
