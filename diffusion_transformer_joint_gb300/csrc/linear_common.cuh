// What the two kernels behind flux_linear share: the problem's description,
// the activations and the loads of the per-feature vectors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "flux_attn.h"
#include "flux_internal.h"
#include "ptx_sm103a.cuh"

namespace flux {

// The epilogue's operands: out = residual + gate * act(acc + bias). bias,
// gate and residual may be NULL. Token (b, s) of the launch reads gate row
// (b * S + s) / gate_rows: a launch may join the batch elements into one run
// of rows, while the gate still changes every gate_rows of them.
struct LinearEpilogue {
  const void *bias, *gate;
  int64_t gate_bs;    // elements from one gate row to the next
  int64_t gate_rows;  // rows that share a gate row
  int vec_f32;        // bias and gate: 1 fp32, 0 bf16
};

// act(y) in fp32. SiLU y / (1 + e^-y); GELU in its tanh form, of which
// 0.5 (1 + tanh u) = 1 / (1 + e^-2u) needs one exponential. The fast division
// is off by two fp32 steps, and gives 0 where the divisor passes 2^126: SiLU is
// 0 below y of about -87.3, GELU below -10, where their values, some of which
// bf16 could still hold, are under 1.1e-36 and 1.2e-37 in magnitude. An epilogue
// with the exact division took twice as long.
template <int kAct>
__device__ __forceinline__ float activate(float y) {
  if constexpr (kAct == FLUX_ACT_SILU) {
    return __fdividef(y, 1.f + __expf(-y));
  } else if constexpr (kAct == FLUX_ACT_GELU_TANH) {
    const float u2 = 1.5957691216057308f * (y + 0.044715f * y * y * y);  // 2 sqrt(2/pi) (...)
    return __fdividef(y, 1.f + __expf(-u2));
  } else {
    return y;
  }
}

// Eight consecutive entries of a bf16 or fp32 vector, 16-byte aligned. (Plain
// loads: a launch that overlaps the end of the kernel before it must not take
// the read-only path to what that kernel may have written.)
__device__ __forceinline__ void load_vec8(const void *base, int64_t off, int f32, float (&v)[8]) {
  if (f32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off);
    v[0] = bf16lo_to_f32(w.x), v[1] = bf16hi_to_f32(w.x);
    v[2] = bf16lo_to_f32(w.y), v[3] = bf16hi_to_f32(w.y);
    v[4] = bf16lo_to_f32(w.z), v[5] = bf16hi_to_f32(w.z);
    v[6] = bf16lo_to_f32(w.w), v[7] = bf16hi_to_f32(w.w);
  }
}

// Four entries, 8-byte (bf16) or 16-byte (fp32) aligned, as stored; and their
// values, for when they have arrived.
__device__ __forceinline__ uint4 load_raw4(const void *base, int64_t off, int f32) {
  if (f32) return *reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off);
  const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + off);
  return make_uint4(w.x, w.y, 0u, 0u);
}
__device__ __forceinline__ float4 raw4_values(uint4 v, int f32) {
  if (f32)
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                       __uint_as_float(v.w));
  return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y),
                     bf16hi_to_f32(v.y));
}

__device__ __forceinline__ float load_vec1(const void *base, int64_t off, int f32) {
  if (f32) return static_cast<const float *>(base)[off];
  return bf16lo_to_f32(static_cast<const uint16_t *>(base)[off]);
}

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  v[0] = bf16lo_to_f32(w.x), v[1] = bf16hi_to_f32(w.x);
  v[2] = bf16lo_to_f32(w.y), v[3] = bf16hi_to_f32(w.y);
  v[4] = bf16lo_to_f32(w.z), v[5] = bf16hi_to_f32(w.z);
  v[6] = bf16lo_to_f32(w.w), v[7] = bf16hi_to_f32(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// What the plans' estimates (ns) share: an SM takes in about 112 bytes per ns;
// a stage's 64 channels are four MMAs of N / 2 cycles, about N ns. Fitted, like
// the constants beside them, to the times of every form at 103 problems of 1 to
// 4608 rows, 256 to 16384 channels and 128 to 24576 features: the form that the
// estimates pick takes 1.006 times the best one's time there (geometric mean; at
// most 1.17). Beyond those sizes the estimates only extrapolate.
constexpr double kBytesPerNs = 112.0;
inline double stage_ns(double bytes, int n) {
  return bytes / kBytesPerNs > n ? bytes / kBytesPerNs : n;
}

// A 3-D tensor map over bf16 rows [B, S, cols] with the given element
// strides; one box = box_cols columns x box_rows tokens x box_b batch
// elements, swizzled over its row (128 bytes for 64 columns, 64 for 32).
// Elements outside the tensor read as zero and are not written.
bool make_row_map(CUtensorMap *map, const void *base, int64_t cols, int64_t S, int64_t B,
                  int64_t row_stride, int64_t batch_stride, uint32_t box_cols, uint32_t box_rows,
                  uint32_t box_b);

}  // namespace flux
