// flux_cross_attention on sm_103a (GB300): queries over the keys and values of
// another sequence (an encoder's states), tcgen05 MMAs accumulating in TMEM.
//
//   out[b, i, h, :] = sum_j softmax_j(scale q[b, i, h] . k[b, j, h / G]) v[b, j, h / G, :]
//
// over the keys j below the batch element's length whose mask is set; a row that
// no key is left for is zero. G query heads share a key head: a tile's 128 rows
// are 128 / G queries x G heads, so that keys and values are read once for all
// of them (a single query of a group fills G rows instead of one of G tiles).
//
// Softmax in the log2 domain, one pass: per row a running maximum m and sum l in
// fp32, p = 2^(s scale log2(e) - m) rounded to bf16 for the second product, O and
// l rescaled only when m grows by more than 8 (a factor of 256), exact after the
// final division by l (where |m| passes 2^24 the score's product is rounded like m's
// before m is taken off: see kFar). A key that does not take part has p = 0: its score is
// replaced before the maximum, and its row of V, which may hold anything, is
// zeroed in shared memory, for 0 times infinity or NaN is NaN.
//
// Two forms, chosen by plan_cross (sizes alone):
//   wide    (many queries) a CTA owns two tiles of queries and walks every key
//           tile for both; persistent, items round robin. Where keys are few (a
//           prompt's one to four tiles) items are short: so Q tiles are loaded,
//           multiplied and stored on their own, and the next item's first products
//           are issued before this one's last values are read, without a break at
//           its end.
//   narrow  (few queries) a CTA owns one tile of queries and a range of the keys,
//           whose tiles go in turn to two streams with a softmax and an O each;
//           C CTAs of a cluster split the keys. The parts are joined through
//           distributed shared memory, every CTA finishing a share of the values;
//           no workspace, no second launch, the same order in every run.
//
// 16 warps: warp 0 TMA producer of Q and K, warp 1 MMA issuer, warp 2 TMEM
// allocation, V rows that take no part zeroed (masks),
// warp 3 TMA producer of V; warps 4-7 and 8-11 the softmax of stream 0 and 1
// (thread = TMEM lane = row), warps 12-15 the epilogue, so that a stream's softmax
// goes on with the next item while its O is read.
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512); P_t is
// written as packed bf16 over the first 64 columns of S_t.
//
// The launch overlaps its prologue with the end of the kernel before it. Every
// wait is bounded (one for a whole item's work from the last tile on); one that
// runs out aborts the CTA and sets the status word to
// FLUX_ERR_DEVICE_TIMEOUT.
//
// Measured (GB300, in a graph of 2 ms; heads of 128 channels, and of 64): 12800 queries
// x 4096 keys, 48 heads 751 to 765 us (1700 TFLOP/s; 825 in calls for a second, at the
// power limit), 684; 2 x 4056 queries over prompts padded to 512, 32 heads, with lengths
// 50 to 52 (an item's chain S, softmax of 0.6 us, PV; tensor cores 45% active), 42, with a
// mask for the same padding 67, 56; 12800 over 512, 32 heads 81, 71, with a random mask
// 118, 112; 64 queries over 2 x 4096 keys, 32 heads 27.8 (4.8 TB/s), 19.7; one query over
// 12800 masked keys, 32 heads over 8 17.7 (3.0 TB/s: 96 CTAs, and what an SM takes in),
// 14.8. -Xptxas -v reports spills of 24 to 36 bytes a thread in the wide form at 128
// channels and 16 in the narrow one with a mask.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "flux_internal.h"
#include "ptx_sm103a.cuh"

namespace flux {
namespace {

constexpr int kTile = 128;  // rows of a query tile, keys of a key tile
constexpr int kThreads = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLowest = -3.0e38f;        // a maximum no key has been counted in
constexpr float kFar = 16777216.f;         // 2^24: maxima from here on are multiples of 2
constexpr uint32_t kBlockBytes = 16384;    // 128 rows x 64 channels, one swizzle block
constexpr uint32_t kBoxBytes = 32 * 128;   // epilogue: 32 rows x 64 channels
constexpr uint32_t kTmemCols = 512;
constexpr int kAll = 0, kLengths = 1, kMask = 2;
constexpr int kMaxParts = 16;  // of the keys: CTAs of a cluster
// registers: 512 threads x 128 at launch
constexpr uint32_t kRegsSoftmax = 168, kRegsCopyMma = 72, kRegsEpilogue = 104;
static_assert(2 * kRegsSoftmax + kRegsCopyMma + kRegsEpilogue == 4 * 128, "register shares");

template <int kD, bool kNarrow>
struct Layout {
  static constexpr uint32_t kTileBytes = (kD / 64) * kBlockBytes;
  static constexpr int kQTiles = kNarrow ? 1 : 2;
  static constexpr int kStages = (kNarrow ? 3 : 2) * (128 / kD);
  static constexpr uint32_t kOffK = kQTiles * kTileBytes;
  static constexpr uint32_t kOffV = kOffK + kStages * kTileBytes;
  static constexpr uint32_t kOffBox = kOffV + kStages * kTileBytes;
  static constexpr uint32_t kOffRow = kOffBox + (kNarrow ? 0 : 4 * (kD / 64) * kBoxBytes);
  static constexpr uint32_t kOffBar = kOffRow + 2 * 2 * kTile * 4;  // (m and l of a stream's rows)
  // barriers
  static constexpr int kQFull = 0, kQFree = 2, kKFull = 4, kKEmpty = kKFull + kStages;
  static constexpr int kVRaw = kKEmpty + kStages, kVFull = kVRaw + kStages;
  static constexpr int kVEmpty = kVFull + kStages, kSFull = kVEmpty + kStages;
  static constexpr int kPFull = kSFull + 2, kODone = kPFull + 2, kOFree = kODone + 2;
  static constexpr int kRowFull = kOFree + 2, kRowFree = kRowFull + 2, kDrain = kRowFree + 2;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr uint32_t kOffTmemSlot = kOffBar + 8 * kNumBars;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
  static constexpr uint32_t kOffProgress = kOffAbort + 4;
  static constexpr uint32_t kSmemBytes = kOffProgress + 4;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  // the parts of a narrow item: fp32 O of 128 rows over the drained K and V
  static constexpr uint32_t kPitch = kD * 4 + 16;
  static_assert(!kNarrow || kTile * kPitch <= 2 * kStages * kTileBytes, "a part's O");
};

struct Maps {
  CUtensorMap q, k, v, out;
};

struct Shape {
  const int32_t *lengths;  // [B], or null
  const uint8_t *mask;     // [B, Sk] at stride mask_bs, or null
  uint16_t *out;
  int64_t mask_bs, o_bs, o_rs;
  int Sq, Sk, Hk, G;
  int n_s;                // queries of a tile: 128 / G
  int n_rb, n_items;      // row blocks per key head; items
  int parts;              // of the keys (narrow)
  int boxed;              // 32 rows of a box are whole queries: stored by TMA
  float scale_log2;
};

// An item: a batch element, a key head, the first query; and how many key tiles
// it has, from tile lo on.
struct Item {
  int b, h, s0, lo, n, keys;
};

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}
// A wait for what takes a whole item's time, or several items': keys are not
// limited, so that its budget begins anew whenever the producer of V has gone on.
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          volatile const uint32_t *progress) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    uint32_t seen = *progress;
    long long t0 = clock64();
    while (!(ok = mbar_try_wait(bar, parity)) && !*abort_flag) {
      const uint32_t now = *progress;
      if (now != seen) {
        seen = now;
        t0 = clock64();
      } else if (clock64() - t0 > kWaitBudgetCycles) {
        *abort_flag = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
// Whether a row's maximum is so far from 0 that its rounding shows in p.
__device__ __forceinline__ bool is_far(float m) {
  return fabsf(m) >= kFar && m != kLowest;
}
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Five-dimensional tile copies: channels, heads of a group, key heads, tokens,
// batch elements.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, uint32_t bar, int c0,
                                            int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
__device__ __forceinline__ void tma_store_5d(const void *tmap, uint32_t src, int c0, int c1, int c2,
                                             int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(tmap)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// kKeys: all keys take part, or those below a length, or those of a mask too.
template <int kD, bool kNarrow, int kKeys>
__global__ void __launch_bounds__(kThreads, 1)
    cross_attention_kernel(const __grid_constant__ Maps maps, const Shape p, int *status) {
  using L = Layout<kD, kNarrow>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t sbase = smem_addr(base);
  auto bar = [&](int i) { return sbase + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + L::kOffTmemSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + L::kOffAbort);
  // tiles of V asked for so far
  volatile uint32_t *progress = reinterpret_cast<volatile uint32_t *>(base + L::kOffProgress);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int part = kNarrow && p.parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = kNarrow && p.parts > 1 ? static_cast<int>(cluster_id_x())
                                           : static_cast<int>(blockIdx.x);
  const int step = kNarrow && p.parts > 1 ? p.n_items : static_cast<int>(gridDim.x);
  // rows of the keys' row ranges: m, then l of a stream
  auto row_at = [&](int t, int what, int row) {
    return sbase + L::kOffRow + static_cast<uint32_t>(((t * 2 + what) * kTile + row) * 4);
  };

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::kQFull + t), 1);
      mbar_init(bar(L::kQFree + t), 1);
      mbar_init(bar(L::kSFull + t), 1);
      mbar_init(bar(L::kPFull + t), 4);
      mbar_init(bar(L::kODone + t), 1);
      mbar_init(bar(L::kOFree + t), 4);
      mbar_init(bar(L::kRowFull + t), 4);
      mbar_init(bar(L::kRowFree + t), 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(L::kKFull + s), 1);
      mbar_init(bar(L::kKEmpty + s), 1);
      mbar_init(bar(L::kVRaw + s), 1);
      mbar_init(bar(L::kVFull + s), 1);
      mbar_init(bar(L::kVEmpty + s), 1);
    }
    mbar_init(bar(L::kDrain), 1);
    *abort_flag = 0;
    *progress = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // Rows of a Q tile that no copy reaches (groups that do not divide 128): what
  // another kernel left there would have a say in when their warp rescales.
  const int q_rows = p.n_s * p.G;
  if (q_rows < kTile) {
    const int chunks = (kTile - q_rows) * 8;
    for (int u = tid; u < L::kQTiles * (kD / 64) * chunks; u += kThreads)
      st_shared_v4(sbase + static_cast<uint32_t>(u / chunks) * kBlockBytes +
                       static_cast<uint32_t>(q_rows * 128 + u % chunks * 16),
                   make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async_smem();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch_dependents();
  // everything up to here overlaps the end of the kernel before this one
  grid_dep_wait();

  int len_b = -1, len_keys = 0;  // the batch element looked up last
  auto item_at = [&](int i) {
    Item it;
    const int rb = i % p.n_rb, bh = i / p.n_rb;
    it.h = bh % p.Hk;
    it.b = bh / p.Hk;
    it.s0 = rb * p.n_s * L::kQTiles;
    it.keys = p.Sk;
    if constexpr (kKeys != kAll) {
      if (p.lengths != nullptr) {
        if (it.b != len_b) {
          len_b = it.b;
          len_keys = p.lengths[it.b];
          len_keys = len_keys < 0 ? 0 : len_keys < p.Sk ? len_keys : p.Sk;
        }
        it.keys = len_keys;
      }
    }
    const int n = (it.keys + kTile - 1) / kTile;
    it.lo = kNarrow ? static_cast<int>(static_cast<int64_t>(n) * part / p.parts) : 0;
    it.n = (kNarrow ? static_cast<int>(static_cast<int64_t>(n) * (part + 1) / p.parts) : n) - it.lo;
    return it;
  };

  // Which keys of tile j take part, 32 a word, all of a warp's lanes together.
  auto key_bits = [&](const Item &it, int j, uint32_t (&bits)[4]) {
    const int valid = it.keys - (it.lo + j) * kTile;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int n = valid - 32 * w;
      bits[w] = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    }
    if constexpr (kKeys == kMask) {
      const uint8_t *row = p.mask + it.b * p.mask_bs + (it.lo + j) * kTile + lane;
      uint8_t in[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) in[w] = (bits[w] >> lane) & 1u ? row[32 * w] : 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) bits[w] = __ballot_sync(0xffffffffu, in[w] != 0);
    }
  };
  // A tile of V some of whose rows may have to be zeroed lands on V-raw and is
  // passed on to V-full by the mask warp, other ones land on V-full.
  auto v_raw = [&](const Item &it, int j) {
    return kKeys == kMask || (kKeys == kLengths && it.keys - (it.lo + j) * kTile < kTile);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCopyMma));
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------- producer: Q and K
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      const uint32_t q_bytes = static_cast<uint32_t>(p.n_s * p.G) * kD * 2;
      int s = 0;
      uint32_t turn = 0, k = 0;  // times round the ring; items with keys so far
      bool ok = true;
      for (int i = first; ok && i < p.n_items; i += step) {
        const Item it = item_at(i);
        if (it.n == 0) continue;
        for (int j = 0; j < it.n; ++j) {
          if (!(ok = mbar_wait(bar(L::kKEmpty + s), (turn & 1u) ^ 1u, abort_flag))) break;
          const uint32_t dst = sbase + L::kOffK + static_cast<uint32_t>(s) * L::kTileBytes;
          mbar_arrive_expect_tx(bar(L::kKFull + s), L::kTileBytes);
          for (int c = 0; c < kD / 64; ++c)
            tma_load_4d(dst + c * kBlockBytes, &maps.k, bar(L::kKFull + s), c * 64, it.h,
                        (it.lo + j) * kTile, it.b);
          if (++s == kStages) s = 0, ++turn;
          // Q behind the first K tile, whose stage is free before the last
          // item's products have read its Q
          for (int t = 0; ok && j == 0 && t < L::kQTiles; ++t) {
            if (!(ok = mbar_wait(bar(L::kQFree + t), (k & 1u) ^ 1u, abort_flag))) break;
            const uint32_t to = sbase + static_cast<uint32_t>(t) * L::kTileBytes;
            mbar_arrive_expect_tx(bar(L::kQFull + t), q_bytes);
            for (int c = 0; c < kD / 64; ++c)
              tma_load_5d(to + c * kBlockBytes, &maps.q, bar(L::kQFull + t), c * 64, 0, it.h,
                          it.s0 + t * p.n_s, it.b);
          }
          if (!ok) break;
        }
        ++k;
      }
      // every copy issued above has landed before the CTA exits (a no-op unless
      // an abort left some unconsumed)
      if (!ok) {
        const long long until = clock64() + kWaitBudgetCycles;
        for (int i = 0; i < kStages; ++i) {
          // the stage's last use, if any, was in this turn or the one before
          if (i < s)
            (void)mbar_settled(bar(L::kKFull + i), turn & 1u, until);
          else if (turn > 0)
            (void)mbar_settled(bar(L::kKFull + i), (turn - 1) & 1u, until);
        }
        // a Q tile is waited for twice over: its last copy, or the one before
        const long long q_until = clock64() + kWaitBudgetCycles / 4;
        for (int t = 0; t < L::kQTiles; ++t) (void)mbar_settled(bar(L::kQFull + t), k & 1u, q_until);
      }
    } else if (warp == 3 && lane == 0) {
      // ------------------------------------------------------- producer: V
      tma_prefetch_desc(&maps.v);
      int s = 0;
      uint32_t turn = 0;
      uint32_t asked = 0;                  // tiles so far
      uint32_t raw_par = 0, last_raw = 0;  // bit s: V-raw's next parity; the last copy's barrier
      bool ok = true;
      for (int i = first; ok && i < p.n_items; i += step) {
        const Item it = item_at(i);
        for (int j = 0; j < it.n; ++j) {
          if (!(ok = mbar_wait(bar(L::kVEmpty + s), (turn & 1u) ^ 1u, abort_flag))) break;
          const uint32_t dst = sbase + L::kOffV + static_cast<uint32_t>(s) * L::kTileBytes;
          const bool raw = v_raw(it, j);
          const uint32_t landed = bar((raw ? L::kVRaw : L::kVFull) + s);
          last_raw = (last_raw & ~(1u << s)) | (raw ? 1u << s : 0u);
          if (raw) raw_par ^= 1u << s;
          mbar_arrive_expect_tx(landed, L::kTileBytes);
          for (int c = 0; c < kD / 64; ++c)
            tma_load_4d(dst + c * kBlockBytes, &maps.v, landed, c * 64, it.h, (it.lo + j) * kTile,
                        it.b);
          *progress = ++asked;
          if (++s == kStages) s = 0, ++turn;
        }
      }
      if (!ok) {
        const long long until = clock64() + kWaitBudgetCycles;
        for (int i = 0; i < kStages; ++i) {
          if (i >= s && turn == 0) continue;
          if ((last_raw >> i) & 1u)
            (void)mbar_settled(bar(L::kVRaw + i), ((raw_par >> i) & 1u) ^ 1u, until);
          else
            (void)mbar_settled(bar(L::kVFull + i), (i < s ? turn : turn - 1) & 1u, until);
        }
      }
    } else if (kKeys != kAll && warp == 2) {
      // ------------------------------------------------------------- masks
      int s = 0;
      uint32_t raw_par = 0;
      bool ok = true;
      for (int i = first; ok && i < p.n_items; i += step) {
        const Item it = item_at(i);
        for (int j = 0; j < it.n; ++j, s = s + 1 == kStages ? 0 : s + 1) {
          if (!v_raw(it, j)) continue;
          uint32_t bits[4];
          key_bits(it, j, bits);
          if (!(ok = wait_long(bar(L::kVRaw + s), (raw_par >> s) & 1u, abort_flag, progress))) break;
          raw_par ^= 1u << s;
          // the V rows that take no part, one per lane, its chunks in an order that
          // keeps eight lanes in different banks
          const uint32_t tile = sbase + L::kOffV + static_cast<uint32_t>(s) * L::kTileBytes;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (bits[w] == 0xffffffffu) continue;
            if ((bits[w] >> lane) & 1u) continue;
#pragma unroll
            for (int c = 0; c < kD / 8; ++c)
              st_shared_v4(tile + (c >> 3) * kBlockBytes + static_cast<uint32_t>(32 * w + lane) * 128 +
                               static_cast<uint32_t>((c ^ lane) & 7) * 16,
                           make_uint4(0u, 0u, 0u, 0u));
          }
          if ((bits[0] & bits[1] & bits[2] & bits[3]) != 0xffffffffu) fence_proxy_async_smem();
          warp_arrive(bar(L::kVFull + s), lane);
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t idesc_qk = idesc_bf16_f32(kTile, kTile, 0, 0);
      const uint32_t idesc_pv = idesc_bf16_f32(kTile, kD, 0, 1);
      const uint32_t desc_hi = static_cast<uint32_t>(sdesc_sw128(sbase, 16, 1024) >> 32);
      auto issue_s = [&](int t, int s) {
        const uint32_t q_at = sbase + (kNarrow ? 0u : static_cast<uint32_t>(t) * L::kTileBytes);
        const uint32_t da = static_cast<uint32_t>(sdesc_sw128(q_at, 16, 1024));
        const uint32_t db = static_cast<uint32_t>(sdesc_sw128(
            sbase + L::kOffK + static_cast<uint32_t>(s) * L::kTileBytes, 16, 1024));
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4;
          mma_ss_elect(tmem + t * 128, da + off, db + off, desc_hi, idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit_elect(bar(L::kSFull + t));
      };
      auto issue_pv = [&](int t, int s, bool add) {
        const uint32_t dv = static_cast<uint32_t>(
            sdesc_sw128(sbase + L::kOffV + static_cast<uint32_t>(s) * L::kTileBytes, kBlockBytes, 1024));
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts_elect(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, dv + ((kk * 2048) >> 4),
                       desc_hi, idesc_pv, add || kk > 0 ? 1u : 0u);
      };
      // the ring position of a walk over all key tiles of the CTA's items
      struct Ring {
        int s = 0;
        uint32_t turn = 0;
        __device__ void next() {
          if (++s == kStages) s = 0, ++turn;
        }
      };
      bool ok = true;
      if constexpr (!kNarrow) {
        // PV0(j) S0(j + 1) PV1(j) S1(j + 1): MMAs run in order, so S_t(j + 1)
        // follows the read of P_t(j), and its commit covers PV_t(j)
        struct At {  // a tile: the item's number among those with keys, its place
          int i, n, j;
          uint32_t k;
        };
        auto from = [&](int i, uint32_t k) {  // the first tile of item i or after
          At a{i, 0, 0, k};
          for (; a.i < p.n_items; a.i += step) {
            a.n = item_at(a.i).n;
            if (a.n > 0) break;
          }
          return a;
        };
        At at = from(first, 0);
        Ring kr, vr;
        uint32_t g = 0;  // tiles so far: parity of the hand-offs with the softmax
        if (at.i < p.n_items) {
          for (int t = 0; ok && t < 2; ++t) {
            ok = (t > 0 || wait_warp(bar(L::kKFull), 0, abort_flag)) &&
                 wait_warp(bar(L::kQFull + t), 0, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
            issue_s(t, 0);
            if (at.n == 1) mma_commit_elect(bar(L::kQFree + t));
          }
          if (ok) mma_commit_elect(bar(L::kKEmpty));
          kr.next();
        }
        // the tile after, found while the products run
        auto after = [&](At a) { return ++a.j < a.n ? a : from(a.i + step, a.k + 1); };
        At nx = at.i < p.n_items ? after(at) : at;
        while (ok && at.i < p.n_items) {
          const bool more = nx.i < p.n_items, last = at.j == at.n - 1;
          if (!(ok = wait_warp(bar(L::kVFull + vr.s), vr.turn & 1u, abort_flag))) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!(ok = wait_warp(bar(L::kPFull + t), g & 1u, abort_flag))) break;
            // the epilogue has read the O that is overwritten
            if (at.j == 0 &&
                !(ok = wait_warp(bar(L::kOFree + t), (at.k & 1u) ^ 1u, abort_flag)))
              break;
            tc_fence_after_sync();
            issue_pv(t, vr.s, at.j > 0);
            if (last) mma_commit_elect(bar(L::kODone + t));
            if (t == 1) mma_commit_elect(bar(L::kVEmpty + vr.s));
            if (!more) continue;
            if (t == 0 && !(ok = wait_warp(bar(L::kKFull + kr.s), kr.turn & 1u, abort_flag))) break;
            if (nx.j == 0 && !(ok = wait_warp(bar(L::kQFull + t), nx.k & 1u, abort_flag))) break;
            tc_fence_after_sync();
            issue_s(t, kr.s);
            if (nx.j == nx.n - 1) mma_commit_elect(bar(L::kQFree + t));
            if (t == 1) mma_commit_elect(bar(L::kKEmpty + kr.s));
          }
          if (!ok) break;
          vr.next();
          if (more) kr.next();
          at = nx;
          if (more) nx = after(nx);
          ++g;
        }
      } else {
        // tile j belongs to stream j & 1: S of tile j + 2 follows PV of tile j
        Ring kr, vr;
        uint32_t n_s[2] = {0, 0}, k_o[2] = {0, 0};  // a stream's tiles, its items so far
        uint32_t k = 0;
        for (int i = first; ok && i < p.n_items; i += step) {
          const Item it = item_at(i);
          if (it.n == 0) continue;
          if (!(ok = wait_warp(bar(L::kQFull), k & 1u, abort_flag))) break;
          auto scores = [&](int j) {
            if (!(ok = wait_warp(bar(L::kKFull + kr.s), kr.turn & 1u, abort_flag))) return;
            tc_fence_after_sync();
            issue_s(j & 1, kr.s);
            mma_commit_elect(bar(L::kKEmpty + kr.s));
            if (j == it.n - 1) mma_commit_elect(bar(L::kQFree));
            kr.next();
          };
          for (int j = 0; ok && j < 2 && j < it.n; ++j) scores(j);
          for (int j = 0; ok && j < it.n; ++j) {
            const int t = j & 1;
            if (!(ok = wait_warp(bar(L::kPFull + t), n_s[t] & 1u, abort_flag) &&
                       wait_warp(bar(L::kVFull + vr.s), vr.turn & 1u, abort_flag)))
              break;
            if (j < 2 && !(ok = wait_warp(bar(L::kOFree + t), (k_o[t] & 1u) ^ 1u, abort_flag))) break;
            tc_fence_after_sync();
            issue_pv(t, vr.s, j >= 2);
            if (j + 2 >= it.n) mma_commit_elect(bar(L::kODone + t));
            mma_commit_elect(bar(L::kVEmpty + vr.s));
            vr.next();
            ++n_s[t];
            if (j < 2) ++k_o[t];
            if (j + 2 < it.n) scores(j + 2);
          }
          ++k;
        }
      }
      // every MMA issued above has finished before TMEM is released
      mma_commit_elect(bar(L::kDrain));
      if (!mbar_settled(bar(L::kDrain), 0, clock64() + kWaitBudgetCycles)) *abort_flag = 1;
      __syncwarp();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = (warp - 4) >> 2;  // stream
    const int wq = warp & 3;        // TMEM lane quadrant
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lane_off;
    const uint32_t tO = tmem + 256 + t * 128 + lane_off;
    const float scale_log2 = p.scale_log2;
    bool ok = true;
    uint32_t g = 0, k = 0;  // the stream's tiles and items so far
    for (int i = first; ok && i < p.n_items; i += step) {
      const Item it = item_at(i);
      float m_run = kLowest, l_run = 0.f;
      bool fresh = true, far = false;  // far: the maximum of a row of the warp is
      // a warp without rows of the tensor takes part in the hand-offs only (its P
      // is whatever was there, for rows that nobody reads)
      const int s_tile = it.s0 + (kNarrow ? 0 : t * p.n_s);
      const bool idle = wq * 32 >= (p.Sq - s_tile < p.n_s ? p.Sq - s_tile : p.n_s) * p.G;
      for (int j = 0; j < it.n; ++j) {
        if (kNarrow && (j & 1) != t) continue;
        uint32_t bits[4];  // (a mask's, while the scores are on their way)
        if constexpr (kKeys == kMask) key_bits(it, j, bits);
        if (!(ok = wait_warp(bar(L::kSFull + t), g & 1u, abort_flag))) break;
        tc_fence_after_sync();
        if (idle) {
          ++g;
          tc_fence_before_sync();
          warp_arrive(bar(L::kPFull + t), lane);
          continue;
        }
        // The row's maximum so far and how O and l have to be scaled for it.
        float alpha = 1.f, m_use = m_run;
        auto rise = [&](float mx) {
          mx = fmaxf(mx * scale_log2, kLowest);  // (no key so far: p is 2^-inf below)
          const bool any = __any_sync(0xffffffffu, fresh ? is_far(mx) : mx > m_run + kRescaleThreshold);
          if (fresh) {
            m_use = mx;
            far = any;
          } else if (any) {
            m_use = fmaxf(m_run, mx);
            far = __any_sync(0xffffffffu, is_far(m_use));
            alpha = ex2_approx(m_run - m_use);
            // S_t of this tile is complete, hence so is PV_t before it: O_t is stable
#pragma unroll 1
            for (int c = 0; c < kD / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(tO + c * 16, o);
            }
          }
        };
        // Scores of keys left out, of 32, become -infinity; the largest of the others.
        auto leave_out = [&](uint32_t *sc, uint32_t kept) {
          float a = -INFINITY, b = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            if (!(kept & (1u << e))) sc[e] = 0xff800000u;
            if (!(kept & (2u << e))) sc[e + 1] = 0xff800000u;
            if (e & 2)
              a = fmax3(a, __uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
            else
              b = fmax3(b, __uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
          }
          return fmaxf(a, b);
        };
        // Far from 0 the maximum's own rounding, half an ulp, is what the largest key's
        // exponent comes out as (100 and more at 2^32, where p would overflow or vanish).
        // There scores are scaled, and rounded, like the maximum before it is taken off:
        // times pre here, times factor in weigh. For the warp's other rows pre is 1.
        auto scale_first = [&](uint32_t *sc) {
          const float pre = is_far(m_use) ? scale_log2 : 1.f;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            sc[e] = __float_as_uint(__fmul_rn(__uint_as_float(sc[e]), pre));
          return is_far(m_use) ? 1.f : scale_log2;
        };
        // p of 32 scores, packed to bf16, and its sums
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        auto weigh = [&](const uint32_t *sc, uint32_t (&pk)[16], float factor) {
          const uint64_t scale2 = f2_pack(factor, factor);
          const uint64_t negm2 = f2_pack(-m_use, -m_use);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x2 = f2_pack(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
            float y0, y1;
            f2_unpack(f2_fma(x2, scale2, negm2), y0, y1);
            const float p0 = ex2_approx(y0);
            const float p1 = ex2_approx(y1);
            acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(p0, p1));
            pk[e / 2] = pack_bf16x2(p0, p1);
          }
        };
        const bool whole = kKeys == kMask
                               ? (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu
                               : it.keys - (it.lo + j) * kTile >= kTile;
        // Few queries' masks leave out some keys of every tile, say: their code stays
        // at hand, and replacing scores in registers is the faster way (one query over
        // 12800 masked keys 19.3 us in clusters of eight, 23.1 with the short loops below).
        constexpr bool kInPlace = kNarrow && kKeys == kMask;
        if (whole || kInPlace) {
          uint32_t sr[kTile];
          float mr[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tmem_ld32_max(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]), mr[c]);
          tmem_ld_wait();
          if (kInPlace && !whole) {
#pragma unroll
            for (int w = 0; w < 4; ++w) mr[w] = leave_out(&sr[w * 32], bits[w]);
          }
          rise(fmax3(mr[0], mr[1], fmaxf(mr[2], mr[3])));
          if (!far) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[16];
              weigh(&sr[c * 32], pk, scale_log2);
              tmem_st16(tS + c * 16, pk);
            }
          } else {  // (rare: read once more, so that this needs no registers above)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t sc[32], pk[16];
              tmem_ld32(tS + c * 32, sc);
              tmem_ld_wait();
              if (kInPlace && !whole)
                (void)leave_out(sc, c == 0 ? bits[0] : c == 1 ? bits[1] : c == 2 ? bits[2] : bits[3]);
              const float factor = scale_first(sc);
              weigh(sc, pk, factor);
              tmem_st16(tS + c * 16, pk);
            }
          }
        } else {
          // Some keys take no part: 32 keys at a time in short loops, for this code,
          // met once an item, has to be fetched (unrolled for all 128 it took twice
          // as long). Scores of keys left out are replaced in TMEM; words without
          // any other key are passed over.
          if constexpr (kKeys != kMask) key_bits(it, j, bits);
          uint32_t word[4] = {bits[0], bits[1], bits[2], bits[3]};
          auto rotate = [&] {
            const uint32_t w = word[0];
            word[0] = word[1], word[1] = word[2], word[2] = word[3], word[3] = w;
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c, rotate()) {
            if (word[0] == 0) continue;
            uint32_t sc[32];
            float m;
            tmem_ld32_max(tS + c * 32, sc, m);
            tmem_ld_wait();
            if (word[0] != 0xffffffffu) {
              m = leave_out(sc, word[0]);
              tmem_st32(tS + c * 32, sc);
            }
            mx = fmaxf(mx, m);
          }
          tmem_st_wait();
          rise(mx);
#pragma unroll 1
          for (int c = 0; c < 4; ++c, rotate()) {
            // (P of these keys goes over scores that have been read)
            uint32_t pk[16];
            if (word[0] == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0;
            } else {
              uint32_t sc[32];
              tmem_ld32(tS + c * 32, sc);
              tmem_ld_wait();
              const float factor = far ? scale_first(sc) : scale_log2;
              weigh(sc, pk, factor);
            }
            tmem_st16(tS + c * 16, pk);
          }
        }
        float sum;
        {
          float a0, a1, b0, b1;
          f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
          f2_unpack(f2_add(acc[2], acc[3]), b0, b1);
          sum = (a0 + a1) + (b0 + b1);
        }
        fresh = false;
        tmem_st_wait();
        l_run = l_run * alpha + sum;
        m_run = m_use;
        ++g;
        tc_fence_before_sync();
        warp_arrive(bar(L::kPFull + t), lane);
      }
      if (!ok) break;
      if (it.n == 0) continue;
      // the row's m and l for the epilogue, once it has read the last item's
      if (!(ok = wait_warp(bar(L::kRowFree + t), (k & 1u) ^ 1u, abort_flag))) break;
      st_shared_f32(row_at(t, 0, wq * 32 + lane), m_run);
      st_shared_f32(row_at(t, 1, wq * 32 + lane), l_run);
      warp_arrive(bar(L::kRowFull + t), lane);
      ++k;
    }
  } else {
    // ----------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const int qs = row / p.G;                    // the row's query of the tile, its head
    const int qh = row - qs * p.G;
    bool ok = true;
    uint32_t k = 0, k_o[2] = {0, 0};             // items with keys, with keys of a stream
    for (int i = first; ok && i < p.n_items; i += step) {
      const Item it = item_at(i);
      if constexpr (!kNarrow) {
        for (int t = 0; t < 2; ++t) {
          const int s_tile = it.s0 + t * p.n_s, s = s_tile + qs;
          const bool row_ok = qs < p.n_s && s < p.Sq;
          auto row_to = [&] {
            return p.out + it.b * p.o_bs + static_cast<int64_t>(s) * p.o_rs +
                   static_cast<int64_t>(it.h * p.G + qh) * kD;
          };
          if (it.n <= 0) {  // no keys
            if (row_ok)
              for (int q = 0; q < kD / 8; ++q)
                st_global_v4(row_to() + q * 8, make_uint4(0u, 0u, 0u, 0u));
            continue;
          }
          if (!(ok = wait_long(bar(L::kRowFull + t), k & 1u, abort_flag, progress))) break;
          const float l = ld_shared_f32(row_at(t, 1, row));
          const float inv_l = l == 0.f ? 0.f : 1.f / l;
          warp_arrive(bar(L::kRowFree + t), lane);
          if (!(ok = wait_warp(bar(L::kODone + t), k & 1u, abort_flag))) break;
          tc_fence_after_sync();
          // the row's values to registers as bf16, and O is free for the next item
          const uint32_t tO = tmem + 256 + t * 128 + lane_off;
          const uint64_t inv2 = f2_pack(inv_l, inv_l);
          uint32_t w[kD / 2];
#pragma unroll
          for (int c = 0; c < kD / 16; ++c) {
            uint64_t o[8];
            tmem_ld16_pairs(tO + c * 16, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float x, y;
              f2_unpack(f2_mul(o[e], inv2), x, y);
              w[c * 8 + e] = pack_bf16x2(x, y);
            }
          }
          tc_fence_before_sync();
          warp_arrive(bar(L::kOFree + t), lane);
          if (p.boxed) {
            // boxes of 64 channels, a row's 16-byte chunks swizzled over 128 bytes
            const uint32_t boxes = sbase + L::kOffBox +
                                   static_cast<uint32_t>((warp - 12) * (kD / 64)) * kBoxBytes;
            const int box_s = s_tile + wq * 32 / p.G;  // first query of the warp's boxes
            if (lane == 0) bulk_wait_read_all();  // the copies before have read the boxes
            __syncwarp();
#pragma unroll
            for (int q = 0; q < kD / 8; ++q)
              st_shared_v4(boxes + (q >> 3) * kBoxBytes + lane * 128 + (((q ^ lane) & 7) << 4),
                           make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && box_s < p.Sq) {
              for (int c = 0; c < kD / 64; ++c)
                tma_store_5d(&maps.out, boxes + c * kBoxBytes, c * 64, 0, it.h, box_s, it.b);
              bulk_commit();
            }
          } else if (row_ok) {
            uint16_t *to = row_to();
#pragma unroll
            for (int q = 0; q < kD / 8; ++q)
              st_global_v4(to + q * 8, make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]));
          }
        }
        if (!ok) break;
        if (it.n > 0) ++k;
      } else {
        // join the two streams (the second has none of a single tile)
        const int s = it.s0 + qs;
        const bool row_ok = qs < p.n_s && s < p.Sq;
        float m[2] = {kLowest, kLowest}, l[2] = {0.f, 0.f};
        for (int t = 0; t < 2; ++t) {
          if (it.n == 0) break;
          if (!(ok = wait_long(bar(L::kRowFull + t), k & 1u, abort_flag, progress))) break;
          m[t] = ld_shared_f32(row_at(t, 0, row));
          l[t] = ld_shared_f32(row_at(t, 1, row));
          warp_arrive(bar(L::kRowFree + t), lane);
          if (it.n > t && !(ok = wait_warp(bar(L::kODone + t), k_o[t] & 1u, abort_flag))) break;
        }
        if (!ok) break;
        tc_fence_after_sync();
        const float mm = fmaxf(m[0], m[1]);
        float w0 = ex2_approx(m[0] - mm), w1 = ex2_approx(m[1] - mm);
        const float ll = w0 * l[0] + w1 * l[1];
        if (p.parts == 1) {
          const float inv_l = ll == 0.f ? 0.f : 1.f / ll;
          w0 *= inv_l, w1 *= inv_l;
        }
        const uint32_t tO = tmem + 256 + lane_off;
        uint16_t *to = p.out + it.b * p.o_bs + static_cast<int64_t>(s) * p.o_rs +
                       static_cast<int64_t>(it.h * p.G + qh) * kD;
        const uint32_t part_o = sbase + L::kOffK + static_cast<uint32_t>(row) * L::kPitch;
#pragma unroll 1
        for (int c = 0; c < kD / 16; ++c) {
          uint32_t a[16], b[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) a[e] = b[e] = 0;
          if (it.n > 0) tmem_ld16(tO + c * 16, a);
          if (it.n > 1) tmem_ld16(tO + 128 + c * 16, b);
          tmem_ld_wait();
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = fmaf(__uint_as_float(b[e]), w1, __uint_as_float(a[e]) * w0);
          if (p.parts > 1) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_shared_v4(part_o + c * 64 + q * 16,
                           make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                      __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])));
          } else if (row_ok) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              st_global_v4(to + c * 16 + q * 8,
                           make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]),
                                      pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                      pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                                      pack_bf16x2(v[8 * q + 6], v[8 * q + 7])));
          }
        }
        if (p.parts > 1) {  // (the softmax writes its rows' once: one item a cluster)
          st_shared_f32(row_at(0, 0, row), mm);
          st_shared_f32(row_at(0, 1, row), ll);
        }
        tc_fence_before_sync();
        for (int t = 0; t < 2; ++t) {
          if (it.n > t) {
            warp_arrive(bar(L::kOFree + t), lane);
            ++k_o[t];
          }
        }
        if (it.n > 0) ++k;
      }
    }
    if (lane == 0) bulk_wait_all();  // every output store is complete
  }

  tc_fence_before_sync();
  __syncwarp();
  if (kNarrow && p.parts > 1) {
    // Join the parts: every CTA finishes a share of the item's values, four
    // channels a thread, adding the parts in their order.
    cluster_sync_all();
    const Item it = item_at(first);
    int rows = (p.Sq - it.s0 < p.n_s ? p.Sq - it.s0 : p.n_s) * p.G;
    const int units = rows * (kD / 4);
    const int lo = static_cast<int>(static_cast<int64_t>(units) * part / p.parts);
    const int hi = static_cast<int>(static_cast<int64_t>(units) * (part + 1) / p.parts);
    for (int u = lo + tid; u < hi; u += kThreads) {
      const int row = u / (kD / 4), c = u - row * (kD / 4);
      float top = kLowest;
#pragma unroll 4
      for (int r = 0; r < p.parts; ++r)
        top = fmaxf(top, ld_cluster_f32(mapa_shared(row_at(0, 0, row), r)));
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int r = 0; r < p.parts; ++r) {
        const float w = ex2_approx(ld_cluster_f32(mapa_shared(row_at(0, 0, row), r)) - top);
        const float4 o = ld_cluster_f4(mapa_shared(
            sbase + L::kOffK + static_cast<uint32_t>(row) * L::kPitch + c * 16, r));
        sum = fmaf(w, ld_cluster_f32(mapa_shared(row_at(0, 1, row), r)), sum);
        v.x = fmaf(w, o.x, v.x), v.y = fmaf(w, o.y, v.y);
        v.z = fmaf(w, o.z, v.z), v.w = fmaf(w, o.w, v.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int qs = row / p.G, qh = row - qs * p.G;
      uint16_t *to = p.out + it.b * p.o_bs + static_cast<int64_t>(it.s0 + qs) * p.o_rs +
                     static_cast<int64_t>(it.h * p.G + qh) * kD + c * 4;
      *reinterpret_cast<uint2 *>(to) =
          make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    }
    __syncwarp();
    cluster_sync_all();  // the others have read this CTA's part
  } else {
    __syncthreads();
  }
  if (warp == 2) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Heads [B, S, Hk, G, D] as (D, G, Hk, S, B), or [B, S, Hk, D] as (D, Hk, S, B)
// with G = 0; a box is 64 channels (a swizzled row of 128 bytes) of the G heads of
// box_s tokens.
bool make_map(CUtensorMap *map, const void *x, int D, int G, int Hk, int64_t S, int64_t B,
              int64_t rs, int64_t bs, uint32_t box_s) {
  auto fn = reinterpret_cast<EncodeFn>(tensor_map_encode_entry());
  if (fn == nullptr) return false;
  cuuint64_t dims[5], strides[4];
  cuuint32_t box[5], estr[5] = {1, 1, 1, 1, 1};
  int n = 0;
  auto axis = [&](int64_t size, int64_t step, uint32_t b) {
    dims[n] = static_cast<cuuint64_t>(size);
    if (n > 0) strides[n - 1] = static_cast<cuuint64_t>(step) * 2;
    box[n++] = b;
  };
  axis(D, 1, 64);
  if (G > 0) axis(G, D, static_cast<uint32_t>(G));
  axis(Hk, static_cast<int64_t>(G > 0 ? G : 1) * D, 1);
  axis(S, rs, box_s);
  axis(B, bs, 1);
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(n), const_cast<void *>(x),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, bool kNarrow, int kKeys>
cudaError_t launch(const CrossAttention &a, const CrossPlan &plan, int sms, int *status,
                   cudaStream_t stream) {
  using L = Layout<kD, kNarrow>;
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = cross_attention_kernel<kD, kNarrow, kKeys>;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(L::kSmemBytes));
    if (kNarrow && attr_err[dev] == cudaSuccess)  // clusters of more than eight
      attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (attr_err[dev] != cudaSuccess) return attr_err[dev];
  Shape p;
  p.lengths = a.lengths, p.mask = a.mask, p.mask_bs = a.mask_bs;
  p.out = static_cast<uint16_t *>(a.out), p.o_bs = a.o_bs, p.o_rs = a.o_rs;
  p.Sq = static_cast<int>(a.Sq), p.Sk = static_cast<int>(a.Sk), p.Hk = a.Hk, p.G = a.H / a.Hk;
  p.n_s = kTile / p.G;
  const int64_t per = static_cast<int64_t>(p.n_s) * L::kQTiles;
  const int64_t n_rb = (a.Sq + per - 1) / per;
  const int64_t items = n_rb * a.Hk * a.B;
  if (items > 0x7FFFFFF) return cudaErrorInvalidValue;
  p.n_rb = static_cast<int>(n_rb);
  p.n_items = static_cast<int>(items);
  p.parts = plan.parts;
  p.boxed = 32 % p.G == 0 ? 1 : 0;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  Maps maps;
  if (!make_map(&maps.q, a.q, kD, p.G, a.Hk, a.Sq, a.B, a.q_rs, a.q_bs,
                static_cast<uint32_t>(p.n_s)) ||
      !make_map(&maps.k, a.k, kD, 0, a.Hk, a.Sk, a.B, a.k_rs, a.k_bs, kTile) ||
      !make_map(&maps.v, a.v, kD, 0, a.Hk, a.Sk, a.B, a.v_rs, a.v_bs, kTile))
    return cudaErrorInvalidValue;
  maps.out = maps.q;  // (not looked at where rows are stored one by one)
  if (!kNarrow && p.boxed &&
      !make_map(&maps.out, a.out, kD, p.G, a.Hk, a.Sq, a.B, a.o_rs, a.o_bs,
                static_cast<uint32_t>(32 / p.G)))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.parts);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  const int64_t grid = p.parts > 1 ? items * p.parts : std::min<int64_t>(items, sms);
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = L::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, status);
}

template <int kD, bool kNarrow>
cudaError_t launch(const CrossAttention &a, const CrossPlan &plan, int sms, int *status,
                   cudaStream_t stream) {
  if (a.mask != nullptr) return launch<kD, kNarrow, kMask>(a, plan, sms, status, stream);
  if (a.lengths != nullptr) return launch<kD, kNarrow, kLengths>(a, plan, sms, status, stream);
  return launch<kD, kNarrow, kAll>(a, plan, sms, status, stream);
}

}  // namespace

CrossPlan plan_cross(const CrossAttention &a, int sms) {
  const int64_t n_s = kTile / (a.H / a.Hk), bh = a.B * a.Hk;
  const int64_t tiles = (a.Sk + kTile - 1) / kTile;
  const int64_t wide = bh * ((a.Sq + 2 * n_s - 1) / (2 * n_s));
  const int64_t narrow = bh * ((a.Sq + n_s - 1) / n_s);
  auto waves = [&](int64_t n, int64_t slots) { return static_cast<double>((n + slots - 1) / slots); };
  CrossPlan best{false, 1, 2500.0 + waves(wide, sms) * (1100.0 * tiles + 1000.0)};
  // CTAs of clusters that fit 152 SMs at once: four and more do not fill every SM.
  // (Eight key heads' 12800 keys, one query, the one size that the row of twelve was
  // measured for: 17.2 us in clusters of twelve, 19.3 of eight, 29.9 of sixteen, for
  // which the eighth has to wait.)
  struct Split {
    int parts, ctas;
    double join;
  };
  static constexpr Split kSplits[] = {{1, 152, 0.0},     {2, 152, 4500.0},  {4, 144, 4500.0},
                                      {8, 120, 4500.0}, {12, 96, 4900.0}, {kMaxParts, 112, 5300.0}};
  for (const auto &[parts, ctas, join] : kSplits) {
    if (parts > tiles) break;
    const int64_t slots = sms * ctas / 152 / parts;
    const double own = std::ceil(static_cast<double>(tiles) / parts);
    const double per = 600.0 * own + 1400.0 + join;
    const double ns = 2500.0 + waves(narrow, std::max<int64_t>(1, slots)) * per;
    if (ns < best.ns) best = CrossPlan{true, parts, ns};
  }
  return best;
}

cudaError_t launch_cross_attention(const CrossAttention &a, const CrossPlan &plan, int *status,
                                   cudaStream_t stream) {
  const int sms = sm_count_current_device();
  if (sms < 1) return cudaErrorInvalidDevice;
  if (a.D == 64)
    return plan.narrow ? launch<64, true>(a, plan, sms, status, stream)
                       : launch<64, false>(a, plan, sms, status, stream);
  return plan.narrow ? launch<128, true>(a, plan, sms, status, stream)
                     : launch<128, false>(a, plan, sms, status, stream);
}

}  // namespace flux
