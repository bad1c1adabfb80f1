// flux_modulated_norm: the modulated norm in front of a block's products,
// fused with the gated residual of the product before it.
//
//   x_out = x + gate * y
//   h     = norm(x_out) * (1 + scale) + shift
// norm(v) = (v - mean v) / sqrt(mean (v - mean v)^2 + eps), or, for RMS,
// v / sqrt(mean v^2 + eps), over the channels of a token.
//
// Bound by memory: x and y are read once, x_out and h written once. A row is
// held in registers by a group of threads (kVec 16-byte vectors of 8 channels
// each), so the variance is taken about the mean in a second pass over
// registers, not from a difference of sums; both sums are fp32, by warp
// shuffles and one exchange through shared memory. The norm is taken of the
// fp32 sum x + gate * y, before x_out is rounded to its type. gate, scale and
// shift are the same for every token of a batch element and come from L1 / L2.
#include "linear_common.cuh"

namespace flux {
namespace {

constexpr int kBlock = 256;

struct NormShape {
  int64_t rows, S;
  int nvec;  // 16-byte vectors of 8 channels in a row
};

// Sum over the kT threads of a row's group; every thread gets it. `part` has
// kT / 32 slots of the group, used for one sum only.
template <int kT>
__device__ __forceinline__ float group_sum(float v, float *part, int group, int lane, int gwarp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kT > 32) {
    if (lane == 0) part[gwarp] = v;
    if constexpr (kT >= kBlock)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kT) : "memory");
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kT / 32; ++i) v += part[i];
  }
  return v;
}

template <int kT, int kVec, bool kF32>
__global__ void __launch_bounds__(kT > kBlock ? kT : kBlock)
    modulated_norm_kernel(const ModulatedNorm q, const NormShape p) {
  constexpr int kThreads = kT > kBlock ? kT : kBlock;
  constexpr int kGroups = kThreads / kT;  // rows per block
  __shared__ float part[kGroups][2][kT / 32];
  const int group = static_cast<int>(threadIdx.x) / kT;
  const int gt = static_cast<int>(threadIdx.x) % kT;
  const int lane = gt & 31, gwarp = gt >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  if (row >= p.rows) return;  // whole groups leave; each has its own barrier
  const int64_t b = row / p.S, s = row - b * p.S;

  float v[kVec][8];
  {
    const char *x = static_cast<const char *>(q.x) + (b * q.x_bs + s * q.x_rs) * (kF32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = gt + j * kT;
      if (c < p.nvec) {
        if constexpr (kF32) {
          const uint4 lo = ld_global_stream_v4(x + c * 32), hi = ld_global_stream_v4(x + c * 32 + 16);
          v[j][0] = __uint_as_float(lo.x), v[j][1] = __uint_as_float(lo.y);
          v[j][2] = __uint_as_float(lo.z), v[j][3] = __uint_as_float(lo.w);
          v[j][4] = __uint_as_float(hi.x), v[j][5] = __uint_as_float(hi.y);
          v[j][6] = __uint_as_float(hi.z), v[j][7] = __uint_as_float(hi.w);
        } else {
          unpack8(ld_global_stream_v4(x + c * 16), v[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      }
    }
  }
  if (q.y != nullptr) {
    const uint16_t *y = static_cast<const uint16_t *>(q.y) + b * q.y_bs + s * q.y_rs;
    char *xo = static_cast<char *>(q.x_out) + (b * q.xo_bs + s * q.xo_rs) * (kF32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = gt + j * kT;
      if (c >= p.nvec) continue;
      float w[8];
      unpack8(ld_global_stream_v4(y + c * 8), w);
      if (q.gate != nullptr) {
        float g[8];
        load_vec8(q.gate, b * q.gate_bs + c * 8, q.vec_f32, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = fmaf(g[i], w[i], v[j][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += w[i];
      }
      if constexpr (kF32) {
        *reinterpret_cast<float4 *>(xo + c * 32) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
        *reinterpret_cast<float4 *>(xo + c * 32 + 16) =
            make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
      } else {
        *reinterpret_cast<uint4 *>(xo + c * 16) = pack8(v[j]);
      }
    }
  }

  const float inv_dim = 1.f / static_cast<float>(q.dim);
  float mean = 0.f;
  if (!q.rms) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[j][i];
    mean = group_sum<kT>(sum, part[group][0], group, lane, gwarp) * inv_dim;
  }
  float sq = 0.f;
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    if (gt + j * kT < p.nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] -= mean;
        sq = fmaf(v[j][i], v[j][i], sq);
      }
    }
  const float var = group_sum<kT>(sq, part[group][1], group, lane, gwarp) * inv_dim;
  const float r = 1.f / sqrtf(var + q.eps);

  uint16_t *h = static_cast<uint16_t *>(q.h) + b * q.h_bs + s * q.h_rs;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int c = gt + j * kT;
    if (c >= p.nvec) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] *= r;
    if (q.scale != nullptr) {
      float m[8];
      load_vec8(q.scale, b * q.scale_bs + c * 8, q.vec_f32, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= 1.f + m[i];
    }
    if (q.shift != nullptr) {
      float m[8];
      load_vec8(q.shift, b * q.shift_bs + c * 8, q.vec_f32, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += m[i];
    }
    *reinterpret_cast<uint4 *>(h + c * 8) = pack8(v[j]);
  }
}

template <int kT, int kVec>
cudaError_t launch(const ModulatedNorm &q, cudaStream_t stream) {
  constexpr int kThreads = kT > kBlock ? kT : kBlock;
  NormShape p{q.B * q.S, q.S, q.dim / 8};
  const int64_t blocks = (p.rows + kThreads / kT - 1) / (kThreads / kT);
  if (q.stream_f32)
    modulated_norm_kernel<kT, kVec, true><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(q, p);
  else
    modulated_norm_kernel<kT, kVec, false><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(q, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_modulated_norm(const ModulatedNorm &q, cudaStream_t stream) {
  const int nvec = q.dim / 8;
  if (nvec <= 32) return launch<32, 1>(q, stream);
  if (nvec <= 64) return launch<32, 2>(q, stream);
  if (nvec <= 128) return launch<64, 2>(q, stream);
  if (nvec <= 256) return launch<128, 2>(q, stream);
  if (nvec <= 512) return launch<256, 2>(q, stream);
  if (nvec <= 768) return launch<256, 3>(q, stream);
  if (nvec <= 1024) return launch<512, 2>(q, stream);
  return launch<512, 4>(q, stream);
}

}  // namespace flux
