// flux_quantize_fp8 on sm_103a (GB300): token rows or a weight to e4m3, with an
// fp32 scale per group of 128 channels of a row, or per 128 x 128 block.
//
//   t = max(max |x| over the group, 2^-100),  scale = t / 448,
//   q = e4m3(x * (448 / t)),  each operation fp32, to nearest even.
//
// The maximum is taken of the magnitudes' bits as integers: the order is that of
// the values, and a NaN stays the largest, so that its whole group comes out
// NaN (an infinity gives a scale of infinity and the factor 0). The floor of
// 2^-100 keeps 448 / t finite.
//
// Bound by memory: 3 bytes per element of bf16. A thread holds 16 channels (32
// or 64 bytes read, 16 written), eight neighbouring threads a row's group.
// Rows: a block takes 32 tokens x kU groups, so that a warp's threads read 256
// (512) consecutive bytes per token, and the scales of one group, which lie
// beside one another for consecutive tokens, leave as whole 128-byte lines.
// kU groups have their loads in flight together: four where that still gives
// every SM two blocks, else one. Blocks: a CTA's 256 threads hold one 128 x 128 block.
//
// Measured (GB300, in a graph): rows 4096 x 4096 9.4 us (5.4 TB/s, of which start and
// end take about 1 us), 154 x 4096 1.9 us (a launch), blocks 12288 x 4096 22.6 us
// (6.7 TB/s).
#include <cuda_runtime.h>

#include "flux_internal.h"
#include "ptx_sm103a.cuh"

namespace flux {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 32;  // tokens per block of rows
constexpr float kTop = 448.f;
constexpr uint32_t kLeastBits = 0x0D800000u;  // 2^-100

// 16 channels as loaded: bf16 pairs, or fp32.
template <bool kF32>
struct Sixteen {
  uint4 w[kF32 ? 4 : 2];
};

template <bool kF32>
__device__ __forceinline__ Sixteen<kF32> load16(const void *x, int64_t at) {
  Sixteen<kF32> v;
  const uint4 *p = kF32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + at)
                        : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) v.w[i] = p[i];
  return v;
}

template <bool kF32>
__device__ __forceinline__ Sixteen<kF32> zero16() {
  Sixteen<kF32> v;
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) v.w[i] = make_uint4(0u, 0u, 0u, 0u);
  return v;
}

// The largest magnitude's bits, as an fp32 value's.
template <bool kF32>
__device__ __forceinline__ uint32_t top_bits(const Sixteen<kF32> &v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
    const uint32_t w[4] = {v.w[i].x, v.w[i].y, v.w[i].z, v.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = kF32 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
  }
  return kF32 ? m : max(m << 16, m & 0xFFFF0000u);
}

// Four values times f, rounded to e4m3: `a` in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d, float f) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a * f), "f"(b * f), "f"(c * f), "f"(d * f));
  return r;
}

template <bool kF32>
__device__ __forceinline__ uint4 scaled16(const Sixteen<kF32> &v, float f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kF32) {
      const uint4 w = v.w[i];
      r[i] = pack_e4m3x4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                         __uint_as_float(w.w), f);
    } else {
      const uint4 w = v.w[i >> 1];
      const uint32_t a = i & 1 ? w.z : w.x, b = i & 1 ? w.w : w.y;
      r[i] = pack_e4m3x4(bf16lo_to_f32(a), bf16hi_to_f32(a), bf16lo_to_f32(b), bf16hi_to_f32(b), f);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint32_t group_max(uint32_t m) {  // of eight neighbouring lanes
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

template <bool kF32, int kU>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantizeFp8 q, int n_kb) {
  grid_dep_launch_dependents();
  const int part = static_cast<int>(threadIdx.x) & 7;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + (threadIdx.x >> 3);
  const bool in = t < q.B * q.S;
  const int64_t b = in ? t / q.S : 0, s = in ? t - b * q.S : 0;
  const int kb0 = static_cast<int>(blockIdx.y) * kU;
  const int64_t xat = b * q.x_bs + s * q.x_rs + part * 16;
  uint8_t *to = static_cast<uint8_t *>(q.q) + b * q.q_bs + s * q.q_rs + part * 16;
  float *scale = q.scale + b * q.s_bs + s * q.s_rs;
  grid_dep_wait();
  Sixteen<kF32> v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int c = (kb0 + u) * 128;
    v[u] = in && c + part * 16 < q.K ? load16<kF32>(q.x, xat + c) : zero16<kF32>();
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const float top = __uint_as_float(max(group_max(top_bits(v[u])), kLeastBits));
    const int c = (kb0 + u) * 128;
    if (!in || kb0 + u >= n_kb) continue;
    if (c + part * 16 < q.K)
      *reinterpret_cast<uint4 *>(to + c) = scaled16(v[u], __fdiv_rn(kTop, top));
    if (part == 0) scale[(kb0 + u) * q.s_ks] = __fdiv_rn(top, kTop);
  }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const QuantizeFp8 q) {
  grid_dep_launch_dependents();
  __shared__ uint32_t tops[kThreads / 32];
  const int part = static_cast<int>(threadIdx.x) & 7;
  const int64_t kb = blockIdx.x, rb = blockIdx.y;
  const int64_t c = kb * 128 + part * 16, r0 = rb * 128 + (threadIdx.x >> 3);
  grid_dep_wait();
  Sixteen<kF32> v[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = r0 + 32 * i < q.S && c < q.K ? load16<kF32>(q.x, (r0 + 32 * i) * q.x_rs + c)
                                        : zero16<kF32>();
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, top_bits(v[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = m;
  __syncthreads();
  m = kLeastBits;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max(m, tops[i]);
  const float top = __uint_as_float(m), f = __fdiv_rn(kTop, top);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + 32 * i < q.S && c < q.K)
      *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(q.q) + (r0 + 32 * i) * q.q_rs + c) =
          scaled16(v[i], f);
  if (threadIdx.x == 0) q.scale[rb * q.s_rs + kb * q.s_ks] = __fdiv_rn(top, kTop);
}

}  // namespace

cudaError_t launch_quantize_fp8(const QuantizeFp8 &q, cudaStream_t stream) {
  const int sms = sm_count_current_device();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int n_kb = (q.K + 127) / 128;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (q.rows > 1) {
    const int64_t n_rb = (q.S + 127) / 128;
    if (n_rb > 65535) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(static_cast<unsigned>(n_kb), static_cast<unsigned>(n_rb), 1);
    return q.x_f32 ? cudaLaunchKernelEx(&cfg, quantize_blocks_kernel<true>, q)
                   : cudaLaunchKernelEx(&cfg, quantize_blocks_kernel<false>, q);
  }
  const int64_t n_tb = (q.B * q.S + kTokens - 1) / kTokens;
  const bool four = n_tb * ((n_kb + 3) / 4) >= 2 * sms;
  const int u = four ? 4 : 1;
  if ((n_kb + u - 1) / u > 65535) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(static_cast<unsigned>(n_tb), static_cast<unsigned>((n_kb + u - 1) / u), 1);
  if (q.x_f32)
    return four ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<true, 4>, q, n_kb)
                : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<true, 1>, q, n_kb);
  return four ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<false, 4>, q, n_kb)
              : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<false, 1>, q, n_kb);
}

}  // namespace flux
