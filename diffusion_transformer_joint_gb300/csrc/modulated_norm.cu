// flux_modulated_norm: the modulated norm in front of a block's products,
// fused with the gated residual of the product before it.
//
//   x_out = x + gate * y
//   h     = norm(x_out) * (1 + scale) + shift
// norm(v) = (v - mean v) / sqrt(mean (v - mean v)^2 + eps), or, for RMS,
// v / sqrt(mean v^2 + eps), over the channels of a token.
//
// Bound by memory: x and y are read once, x_out and h written once. A row is
// held in registers by a group of W warps (kVec x 256 channels per warp), so
// the variance is taken about the mean in a second pass over registers, not
// from a difference of sums; both sums are fp32, by warp shuffles and, for
// W > 1, one exchange through shared memory. The norm is taken of the fp32
// sum x + gate * y, before x_out is rounded to its type.
//
// Persistent, one block per SM: a group walks the rows round robin and keeps
// its next rows of x and y on their way into shared memory (cp.async, `depth`
// rows ahead), so that memory stays busy while a row is reduced. A warp
// copies and reads its own channels only: the ring needs no block barrier.
//
// Next to memory, what costs is instruction issue. gate, scale and shift are
// the same for every token of a batch element: a thread keeps those of its
// channels in registers (as stored, bf16 or fp32; read from L1 for every row
// instead, 4096 rows of 4096 channels took 19.5 us) and loads them when the
// batch element changes. A thread's channels lie at constant distances, so
// that loads and stores need no address arithmetic; rows that fill their warps
// exactly (kFull: the hidden widths in use) need no predicates; arithmetic is
// on fp32 pairs. A thread holds 16 channels beside a residual's gate, else 32
// (in a row of over 8192 channels with a residual 32 as well, and spills).
//
// The launch overlaps its prologue with the end of the kernel before it in the
// stream (programmatic dependent launch); no tensor is touched before that
// kernel has ended.
//
// Measured on a GB300, several inputs in turn: 4096 rows of 4096 channels bf16
// 12.9 us, 5.2 TB/s (a kernel that only copies the rows takes 12.8); two times
// 4608 rows of 4096 with an fp32 stream and the gated residual 71.5 us, 6.3
// TB/s; 12800 rows of 6144 bf16 with the gated residual 92.6 us, 6.8 TB/s, as
// fast as memory copies; one row 2.1 us.
#include <algorithm>

#include "linear_common.cuh"

namespace flux {
namespace {

constexpr int kMaxGroupWarps = 16;
constexpr uint32_t kRing = 200 * 1024;

// Warps of a block, by the registers its threads need.
template <int kVec, bool kY>
constexpr int kBlockWarps = kVec <= 2 && !kY ? 24 : 16;

// Rows that a block has in hand. Without a residual 16 or 24 warps' worth (four
// rows of 4096 channels: 13.0 us for 4096 of them, against 15.2 with two). With
// one there is twice the work per byte of latency and four streams of rows in
// memory, and fewer rows at a time keep each of them in longer runs: 12 warps
// (one row of 4096 or 6144 channels: 92.5 us for 12800 rows of 6144, against
// 110 us with two).
template <bool kY>
constexpr int kRowWarps = kY ? 12 : 24;

// A tensor's walk: bytes from a row to the group's next one, and the
// correction when that passes the end of a batch element.
struct Walk {
  int64_t step, wrap;
};

struct NormPlan {
  int S, step_s;         // tokens per batch element; a group's step within one
  int rows, step;        // rows in all, between a group's rows
  int W, groups, depth;  // warps per row, rows per block, ring (2 or 4 rows)
  Walk x, y, xo, h;
};

__device__ __forceinline__ void copy_async_16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight channels as four fp32 pairs.
struct Eight {
  uint64_t p[4];
};
__device__ __forceinline__ void two_from_bf16(uint2 w, uint64_t *p) {
  p[0] = f2_pack(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x));
  p[1] = f2_pack(bf16lo_to_f32(w.y), bf16hi_to_f32(w.y));
}
__device__ __forceinline__ uint32_t round_pair(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint64_t both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ ulonglong2 as_pairs(uint4 w) {
  return make_ulonglong2(static_cast<uint64_t>(w.y) << 32 | w.x,
                         static_cast<uint64_t>(w.w) << 32 | w.z);
}

// A thread's eight channels of a 256-channel block: the lane's eight
// neighbours, or (kQuad) the lane's four of each half of the block. Where a
// tensor is fp32, 16 bytes hold four channels, and only quads let a warp's
// access be contiguous.
template <bool kQuad>
constexpr int kHalfStep = kQuad ? 128 : 4;  // channels from the first four to the others
template <bool kQuad>
__device__ __forceinline__ int first_channel(int lane) {
  return lane * (kQuad ? 4 : 8);
}

// Loads, by load16 / load8 of that many bytes at a distance. hi_in: whether
// the second half lies inside the row; if not the first is read twice.
template <bool kF32, bool kQuad, typename Load16, typename Load8>
__device__ __forceinline__ Eight get8(Load16 load16, Load8 load8, bool hi_in) {
  Eight v;
  const int step = hi_in ? kHalfStep<kQuad> : 0;
  if constexpr (kF32) {
    const ulonglong2 lo = as_pairs(load16(0)), hi = as_pairs(load16(step * 4));
    v = {{lo.x, lo.y, hi.x, hi.y}};
  } else if constexpr (kQuad) {
    two_from_bf16(load8(0), v.p);
    two_from_bf16(load8(step * 2), v.p + 2);
  } else {
    const uint4 w = load16(0);
    two_from_bf16(make_uint2(w.x, w.y), v.p);
    two_from_bf16(make_uint2(w.z, w.w), v.p + 2);
  }
  return v;
}
template <bool kF32, bool kQuad>
__device__ __forceinline__ Eight get8_shared(uint32_t at) {
  return get8<kF32, kQuad>([&](int d) { return ld_shared_v4(at + d); },
                           [&](int d) { return ld_shared_v2(at + d); }, true);
}
// Eight entries of a modulation vector, as a thread keeps them: fp32 pairs, or
// bf16 as it is stored.
template <bool kF32>
struct Kept {
  uint32_t w[kF32 ? 8 : 4];
};
template <bool kF32, bool kQuad>
__device__ __forceinline__ Kept<kF32> get_kept(const void *base, int64_t off, bool hi_in) {
  const char *at = static_cast<const char *>(base) + off * (kF32 ? 4 : 2);
  const int step = (hi_in ? kHalfStep<kQuad> : 0) * (kF32 ? 4 : 2);
  if constexpr (kF32) {
    const uint4 a = *reinterpret_cast<const uint4 *>(at);
    const uint4 b = *reinterpret_cast<const uint4 *>(at + step);
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  } else if constexpr (kQuad) {
    const uint2 a = *reinterpret_cast<const uint2 *>(at);
    const uint2 b = *reinterpret_cast<const uint2 *>(at + step);
    return {{a.x, a.y, b.x, b.y}};
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(at);
    return {{a.x, a.y, a.z, a.w}};
  }
}
template <bool kF32>
__device__ __forceinline__ Kept<kF32> keep_constant(float v) {
  Kept<kF32> k;
#pragma unroll
  for (int i = 0; i < (kF32 ? 8 : 4); ++i) k.w[i] = kF32 ? __float_as_uint(v) : pack_bf16x2(v, v);
  return k;
}
template <bool kF32>
__device__ __forceinline__ Eight widen(const Kept<kF32> &k) {
  Eight v;
  if constexpr (kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.p[i] = f2_pack(__uint_as_float(k.w[2 * i]), __uint_as_float(k.w[2 * i + 1]));
  } else {
    two_from_bf16(make_uint2(k.w[0], k.w[1]), v.p);
    two_from_bf16(make_uint2(k.w[2], k.w[3]), v.p + 2);
  }
  return v;
}
// Stores; `lo` and `hi` say which half lies inside the row.
template <bool kF32, bool kQuad>
__device__ __forceinline__ void put8(char *at, const Eight &v, bool lo, bool hi) {
  if constexpr (kF32) {
    if (lo) *reinterpret_cast<ulonglong2 *>(at) = make_ulonglong2(v.p[0], v.p[1]);
    if (hi)
      *reinterpret_cast<ulonglong2 *>(at + kHalfStep<kQuad> * 4) = make_ulonglong2(v.p[2], v.p[3]);
  } else {
    const uint2 a = make_uint2(round_pair(v.p[0]), round_pair(v.p[1]));
    const uint2 b = make_uint2(round_pair(v.p[2]), round_pair(v.p[3]));
    if constexpr (kQuad) {
      if (lo) *reinterpret_cast<uint2 *>(at) = a;
      if (hi) *reinterpret_cast<uint2 *>(at + kHalfStep<kQuad> * 2) = b;
    } else {
      if (lo) *reinterpret_cast<uint4 *>(at) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// Sum over the W warps of a row's group; every thread gets it. `part` holds a
// slot per warp, zeros behind the last; it is written again only after a later
// barrier of the group that follows its last read.
__device__ __forceinline__ float group_sum(uint64_t v2, float4 *part, int W, int gwarp, int group) {
  float v, hi;
  f2_unpack(v2, v, hi);
  v += hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W > 1) {
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float *>(part)[gwarp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
    const float4 a = part[0];
    v = (a.x + a.y) + (a.z + a.w);
    if (W > 4) {
      const float4 b = part[1];
      v += (b.x + b.y) + (b.z + b.w);
      if (W > 8) {
        const float4 c = part[2], d = part[3];
        v += ((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w));
      }
    }
  }
  return v;
}

// kF32: type of x; kY: with the residual; kVecF32: type of the modulation;
// kFull: dim = W * kVec * 256.
template <int kVec, bool kF32, bool kY, bool kVecF32, bool kFull>
__global__ void __launch_bounds__(kBlockWarps<kVec, kY> * 32, 1)
    modulated_norm_kernel(const ModulatedNorm q, const NormPlan p) {
  constexpr bool kQuad = kF32;
  constexpr int kXs = kF32 ? 4 : 2;  // bytes per channel
  constexpr int kSeg = kVec * 256;   // channels per warp
  constexpr uint32_t kXSeg = kSeg * kXs, kSlot = kXSeg + (kY ? kSeg * 2 : 0);
  __shared__ float4 parts[kBlockWarps<kVec, kY>][3][kMaxGroupWarps / 4];
  extern __shared__ __align__(16) uint8_t ring[];
  const int W = p.W;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const int group = warp / W, gwarp = warp - group * W;
  float4(*part)[kMaxGroupWarps / 4] = parts[group];
  const int row0 = static_cast<int>(blockIdx.x) * p.groups + group;
  if (row0 >= p.rows) return;  // whole groups leave; each has its own barrier
  if (W > 1 && gwarp == 0 && lane < 3 * kMaxGroupWarps / 4)
    part[0][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
  int64_t b = row0 / p.S;
  int s = row0 - static_cast<int>(b) * p.S;
  int row = row0, row_ahead = row0, s_ahead = s;

  // this thread's first channel, and how many channels from there to the end
  const int c0 = gwarp * kSeg + first_channel<kQuad>(lane);
  const int left = q.dim - c0;
  auto lo_in = [&](int j) { return kFull || j * 256 < left; };
  auto hi_in = [&](int j) { return kFull || j * 256 + kHalfStep<kQuad> < left; };
  // copies are 16-byte words of the warp's channels, consecutive lanes
  // side by side
  const int copy_left = q.dim - gwarp * kSeg;
  const char *xa = static_cast<const char *>(q.x) +
                   (b * q.x_bs + s * q.x_rs + gwarp * kSeg) * kXs + lane * 16;
  const char *ya = static_cast<const char *>(q.y) +
                   (b * q.y_bs + s * q.y_rs + gwarp * kSeg) * 2 + lane * 16;
  char *xo = static_cast<char *>(q.x_out) + (b * q.xo_bs + s * q.xo_rs + c0) * kXs;
  char *h = static_cast<char *>(q.h) + (b * q.h_bs + s * q.h_rs + c0) * 2;
  const uint64_t one = both(1.f);
  // gate, scale and shift of this thread's channels for the batch element
  Kept<kVecF32> gate[kVec], scale[kVec], shift[kVec];
  auto keep_mods = [&]() {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int64_t c = c0 + j * 256;
      if constexpr (kY)
        gate[j] = q.gate == nullptr || !lo_in(j)
                      ? keep_constant<kVecF32>(1.f)
                      : get_kept<kVecF32, kQuad>(q.gate, b * q.gate_bs + c, hi_in(j));
      scale[j] = q.scale == nullptr || !lo_in(j)
                     ? keep_constant<kVecF32>(0.f)
                     : get_kept<kVecF32, kQuad>(q.scale, b * q.scale_bs + c, hi_in(j));
      shift[j] = q.shift == nullptr || !lo_in(j)
                     ? keep_constant<kVecF32>(0.f)
                     : get_kept<kVecF32, kQuad>(q.shift, b * q.shift_bs + c, hi_in(j));
      if constexpr (kVecF32) {  // 1 + scale once; a bf16 scale has no room for it
#pragma unroll
        for (int i = 0; i < 8; ++i)
          scale[j].w[i] = __float_as_uint(1.f + __uint_as_float(scale[j].w[i]));
      }
    }
  };

  // the warp's ring: `depth` rows of its channels of x, then of y
  const uint32_t slots = smem_addr(ring) + static_cast<uint32_t>(warp * p.depth) * kSlot;
  auto fetch = [&](uint32_t slot) {
    if (row_ahead < p.rows) {
      const uint32_t to = slot + lane * 16;
#pragma unroll
      for (int j = 0; j < kVec * kXs / 2; ++j)
        if (kFull || (j * 32 + lane) * (16 / kXs) < copy_left)
          copy_async_16(to + j * 512, xa + j * 512);
      if constexpr (kY) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (kFull || (j * 32 + lane) * 8 < copy_left)
            copy_async_16(to + kXSeg + j * 512, ya + j * 512);
      }
      row_ahead += p.step;
      s_ahead += p.step_s;
      xa += p.x.step;
      if constexpr (kY) ya += p.y.step;
      if (s_ahead >= p.S) {
        s_ahead -= p.S;
        xa += p.x.wrap;
        if constexpr (kY) ya += p.y.wrap;
      }
    }
    copy_async_commit();
  };
  // everything up to here overlaps the end of the kernel before this one
  grid_dep_launch_dependents();
  grid_dep_wait();
  const uint32_t slots_end = slots + static_cast<uint32_t>(p.depth) * kSlot;
  for (uint32_t slot = slots; slot < slots_end; slot += kSlot) fetch(slot);

  keep_mods();
  const float inv_dim = 1.f / static_cast<float>(q.dim);
  uint32_t slot = slots;
  int parity = 0;
  for (;;) {
    if (p.depth == 4)
      copy_async_wait<3>();
    else
      copy_async_wait<1>();
    __syncwarp();
    Eight v[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const uint32_t from = slot + first_channel<kQuad>(lane) * kXs + j * 256 * kXs;
      v[j] = get8_shared<kF32, kQuad>(from);
      if constexpr (kY) {
        const Eight y =
            get8_shared<false, kQuad>(slot + kXSeg + first_channel<kQuad>(lane) * 2 + j * 512);
        const Eight g = widen<kVecF32>(gate[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j].p[i] = f2_fma(g.p[i], y.p[i], v[j].p[i]);
      }
      if (!kFull) {  // what lies past the end counts nothing
        if (!lo_in(j)) v[j].p[0] = v[j].p[1] = 0;
        if (!hi_in(j)) v[j].p[2] = v[j].p[3] = 0;
      }
    }
    __syncwarp();
    // the warp has read its slot: the row `depth` further on may land there
    fetch(slot);
    slot = slot + kSlot == slots_end ? slots : slot + kSlot;

    if constexpr (kY) {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        put8<kF32, kQuad>(xo + j * 256 * kXs, v[j], lo_in(j), hi_in(j));
    }

    if (!q.rms) {
      uint64_t sum = 0;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = f2_add(sum, v[j].p[i]);
      const uint64_t m = both(-group_sum(sum, part[2], W, gwarp, group) * inv_dim);
#pragma unroll
      for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < 2 ? lo_in(j) : hi_in(j)) v[j].p[i] = f2_add(v[j].p[i], m);
    }
    uint64_t sq = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = f2_fma(v[j].p[i], v[j].p[i], sq);
    const float var = group_sum(sq, part[parity], W, gwarp, group) * inv_dim;
    parity ^= 1;
    const uint64_t r = both(rsqrtf(var + q.eps));

#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (!lo_in(j)) continue;
      const Eight m = widen<kVecF32>(scale[j]), n = widen<kVecF32>(shift[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t u = f2_mul(v[j].p[i], r);
        // u (1 + scale) + shift
        v[j].p[i] = kVecF32 ? f2_fma(u, m.p[i], n.p[i])
                            : f2_add(f2_fma(u, m.p[i], u), n.p[i]);
      }
      put8<false, kQuad>(h + j * 512, v[j], true, hi_in(j));
    }

    row += p.step;
    if (row >= p.rows) break;
    s += p.step_s;
    h += p.h.step;
    if constexpr (kY) xo += p.xo.step;
    bool other = p.step >= p.S;  // (the step may pass whole batch elements)
    if (s >= p.S) {
      s -= p.S;
      other = true;
      h += p.h.wrap;
      if constexpr (kY) xo += p.xo.wrap;
    }
    if (other) {
      b = row / p.S;
      keep_mods();
    }
  }
}

template <int kVec, bool kF32, bool kY, bool kVecF32>
cudaError_t launch(const ModulatedNorm &q, int W, int sms, cudaStream_t stream) {
  auto kernel = q.dim == W * kVec * 256 ? modulated_norm_kernel<kVec, kF32, kY, kVecF32, true>
                                        : modulated_norm_kernel<kVec, kF32, kY, kVecF32, false>;
  NormPlan p;
  p.S = static_cast<int>(q.S);
  p.rows = static_cast<int>(q.B * q.S);
  p.W = W;
  const uint32_t row = static_cast<uint32_t>(kVec * 256 * ((kF32 ? 4 : 2) + (kY ? 2 : 0)) * W);
  const int warps = std::min(kBlockWarps<kVec, kY>, kRowWarps<kY>);
  p.groups = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({warps / W, kRing / (2 * row), (p.rows + sms - 1) / sms})));
  const int blocks = std::min((p.rows + p.groups - 1) / p.groups, sms);
  p.step = blocks * p.groups;
  p.step_s = p.step % p.S;
  const int64_t step_b = p.step / p.S;
  p.depth = kY && 4 * p.groups * row <= kRing ? 4 : 2;
  const int xs = kF32 ? 4 : 2;
  auto walk = [&](int64_t bs, int64_t rs, int size) {
    return Walk{(step_b * bs + p.step_s * rs) * size, (bs - q.S * rs) * size};
  };
  p.x = walk(q.x_bs, q.x_rs, xs);
  p.y = walk(q.y_bs, q.y_rs, 2);
  p.xo = walk(q.xo_bs, q.xo_rs, xs);
  p.h = walk(q.h_bs, q.h_rs, 2);
  const uint32_t smem = static_cast<uint32_t>(p.depth * p.groups) * row;
  if (smem > 32 * 1024) {  // 48 KB need no attribute, the sums' slots among them
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kRing));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(p.groups * W * 32), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, q, p);
}

template <int kVec>
cudaError_t launch(const ModulatedNorm &q, int W, int sms, cudaStream_t stream) {
  switch ((q.stream_f32 ? 4 : 0) | (q.y != nullptr ? 2 : 0) | (q.vec_f32 ? 1 : 0)) {
    case 0: return launch<kVec, false, false, false>(q, W, sms, stream);
    case 1: return launch<kVec, false, false, true>(q, W, sms, stream);
    case 2: return launch<kVec, false, true, false>(q, W, sms, stream);
    case 3: return launch<kVec, false, true, true>(q, W, sms, stream);
    case 4: return launch<kVec, true, false, false>(q, W, sms, stream);
    case 5: return launch<kVec, true, false, true>(q, W, sms, stream);
    case 6: return launch<kVec, true, true, false>(q, W, sms, stream);
    default: return launch<kVec, true, true, true>(q, W, sms, stream);
  }
}

}  // namespace

cudaError_t launch_modulated_norm(const ModulatedNorm &q, cudaStream_t stream) {
  const int sms = sm_count_current_device();
  if (sms < 1) return cudaErrorInvalidDevice;
  // blocks of 256 channels per warp: one while there are SMs without a row;
  // two beside a residual's gate, four without, as registers allow
  const int blocks = (q.dim + 255) / 256;
  int vec = q.B * q.S <= sms ? 1 : blocks == 1 ? 1 : blocks <= 4 || q.y != nullptr ? 2 : 4;
  while (vec * kMaxGroupWarps < blocks) vec *= 2;
  const int W = (blocks + vec - 1) / vec;
  switch (vec) {
    case 1: return launch<1>(q, W, sms, stream);
    case 2: return launch<2>(q, W, sms, stream);
    default: return launch<4>(q, W, sms, stream);
  }
}

}  // namespace flux
