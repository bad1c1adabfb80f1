// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "flux_attn.h"

namespace flux {

// FLUX_OK if the current device is an sm_103 part (cached per device),
// FLUX_ERR_UNSUPPORTED if not, FLUX_ERR_CUDA if the runtime cannot tell.
int check_device();

// Number of SMs of the current device (cached per device ordinal, atomically);
// 0 if the runtime cannot tell.
int sm_count_current_device();

// Largest rotation-pair count of one head (head width 512).
constexpr int kMaxPairs = 256;

// Per-pair RoPE parameters handed to the table kernel by value: the axis a
// pair belongs to, and its frequency in turns per unit of position id,
// theta^(-2j/d_a) / (2 pi) (j the pair's index inside its axis of width
// d_a), as an unsigned 0.64 fixed-point fraction of a turn (it is < 1).
struct RopePairs {
  int n_pairs;
  int n_axes;
  uint8_t axis[kMaxPairs];
  uint64_t turns_q64[kMaxPairs];
};

// Fills `pp` from host axes_dims; returns FLUX_OK or FLUX_ERR_AXES.
int make_rope_pairs(const int32_t *axes_dims, int n_axes, double theta, RopePairs *pp);

// Output formats of the table kernel.
enum class TableFormat {
  kF32Pair,    // cos [S, P] and sin [S, P] fp32 (flux_rope_tables)
  kPackedF16,  // one uint32 per (token, pair): fp16 cos in bits 0-15, fp16 sin in 16-31
};

// Enqueues the table kernel over the joint id sequence [seg0 ; seg1]. For
// kPackedF16 the table goes to `packed` ([S, P] uint32) and cos/sin are unused.
// `clear` (nullable): a device int the kernel sets to 0 (a call's status
// word). The kernel lets a programmatically dependent launch (an attention
// kernel launched with pdl) begin as soon as it starts.
cudaError_t launch_rope_tables(const int32_t *ids0, int64_t S0, const int32_t *ids1, int64_t S1,
                               const RopePairs &pp, TableFormat fmt, float *cos_out,
                               float *sin_out, uint32_t *packed, cudaStream_t stream,
                               int *clear = nullptr);

// Workspace layout of flux_joint_rope_attention: a 256-byte status block,
// then the packed table [S, D/2] uint32, padded to 256 bytes.
constexpr size_t kStatusBytes = 256;
inline size_t packed_table_bytes(int64_t S, int D) {
  size_t b = static_cast<size_t>(S) * static_cast<size_t>(D / 2) * sizeof(uint32_t);
  return (b + 255) & ~static_cast<size_t>(255);
}

// Exchange buffer of the attention kernel for [B, S, H, D] inputs: one 8-byte
// flag per (batch, head, key tile, RoPE warp), padded to 256 bytes, then a
// [B, S, H, D] bf16 copy of K after RoPE, then one of Q after RoPE. 0 if D is
// not 128 or the shape is empty.
inline size_t krot_flag_bytes(int B, int64_t S, int H) {
  const size_t tiles = static_cast<size_t>((S + 127) / 128);
  size_t b = static_cast<size_t>(B) * static_cast<size_t>(H) * tiles * 4 * sizeof(uint64_t);
  return (b + 255) & ~static_cast<size_t>(255);
}
inline size_t krot_scratch_bytes(int B, int64_t S, int H, int D) {
  if (D != 128 || B < 1 || H < 1 || S < 1) return 0;
  return krot_flag_bytes(B, S, H) +
         2 * static_cast<size_t>(B) * static_cast<size_t>(S) * static_cast<size_t>(H) * 128 * 2;
}

// Optional QK RMS normalisation for launch_joint_attention: fp32 [128] device
// weight vectors for the queries and keys of text tokens (the first s_txt
// tokens) and of the other tokens, and eps.
struct QkNormArgs {
  const float *q_txt, *k_txt, *q_img, *k_img;
  int64_t s_txt;
  float eps;
};

// One segment of a launch: queries [q_lo, q_hi) (rows of Q / out) attend to
// keys [k_lo, k_hi) (rows of K / V). Segments with the same key_range
// (0 .. kMaxSegments-1) must have the same key range and share its
// exchange-buffer flags.
constexpr int kMaxSegments = 3;
struct AttnSegment {
  int64_t q_lo, q_hi, k_lo, k_hi;
  int key_range;
  int64_t n_pre;  // rows [0, n_pre) of the pre-rotated K / V join the key range
};

// Keys that arrive rotated already (a reference-image cache) and their
// values: bf16 [B, S, H, 128]; they skip RoPE.
struct PreRotatedKV {
  const void *k, *v;
  int64_t S;
};

// Bytes of the exchange buffer of launch_attention_segments: the flags of
// each key range, padded to 256 bytes, then bf16 [B, S_k, H, D] rotated K
// and [B, S_q, H, D] rotated Q.
size_t exchange_bytes(int B, int64_t S_q, int64_t S_k, int H, const AttnSegment *segs,
                      int n_segs);

// Enqueues the attention kernel over segments: Q / out [B, S_q, H, 128] and
// K / V [B, S_k, H, 128] bf16; table_q [S_q, 64] and table_k [S_k, 64]
// packed tables for the rows of Q and of K; xbuf (nullable) the exchange
// buffer of exchange_bytes(...) bytes, 256-byte aligned.
// pdl: launch with programmatic stream serialization, so that the kernel's
// prologue and first Q / K / V copies overlap the table kernel enqueued just
// before it on `stream` (which must be the previous kernel in the stream);
// everything that reads the table or the status word waits for it first.
// h0, Hl: attend only heads h0 .. h0 + Hl - 1 of the H heads of Q / K / V /
// out (Hl 0: all H heads); the exchange buffer is laid out for the Hl heads
// (exchange_bytes with H = Hl).
cudaError_t launch_attention_segments(const void *q, const void *k, const void *v, void *out,
                                      const uint32_t *table_q, const uint32_t *table_k,
                                      int *status, int B, int64_t S_q, int64_t S_k, int H,
                                      const AttnSegment *segs, int n_segs,
                                      const PreRotatedKV *pre, void *xbuf,
                                      const QkNormArgs *norm, cudaStream_t stream,
                                      bool pdl = false, int h0 = 0, int Hl = 0);

// The driver's cuTensorMapEncodeTiled for the projection's tensor maps,
// fetched once through the runtime (no -lcuda); NULL when unavailable.
void *tensor_map_encode_entry();

// Enqueues the fused single-stream input projection: x [M, dim] and W
// [3 * H * 128 + 2 * mlp, dim] bf16 row-major; q, k, v [M, H, 128] and act
// [M, mlp] bf16 written. dim a multiple of 64, mlp a multiple of 128.
cudaError_t launch_qkv_mlp_proj(const void *x, const void *w, int64_t M, int dim, int H,
                                int64_t mlp, void *q, void *k, void *v, void *act, int *status,
                                cudaStream_t stream);

// out = residual + gate * act([x | x2] W^T + bias) over tokens [B, S]. Strides
// are in elements: _bs between batch elements, _rs between token rows (w_rs
// between W's rows), every one a multiple of 8. K, K2, N multiples of 8.
struct LinearProblem {
  const void *x, *x2, *w, *residual;
  void *out;
  int64_t x_bs, x_rs, x2_bs, x2_rs, w_rs, r_bs, r_rs, o_bs, o_rs;
  int64_t B, S, N;
  int K, K2;
};
struct LinearEpilogue;

// How linear_split runs a problem: its form, the tile's width, the units that
// split its channels, whether their sums arrive early, the ring; how
// linear_pair does: the tile's width. Both with an estimate of the time in ns.
struct SplitPlan {
  int form;
  bool early;
  int Q, C, stages;
  double ns;
};
struct PairPlan {
  int tn;
  double ns;
};
SplitPlan plan_split(const LinearProblem &q, int act, int sms);
PairPlan plan_pair(const LinearProblem &q, int act, int sms);

// The form with the smaller estimate: split, or else pair.
struct LinearPlan {
  bool use_split;
  SplitPlan split;
  PairPlan pair;
};
LinearPlan plan_linear(const LinearProblem &q, int act, int sms);

// The two kernels behind flux_linear (act: a flux_activation).
cudaError_t launch_linear_pair(const LinearProblem &q, const PairPlan &plan,
                               const LinearEpilogue &epi, int act, int *status,
                               cudaStream_t stream);
cudaError_t launch_linear_split(const LinearProblem &q, const SplitPlan &plan,
                                const LinearEpilogue &epi, int act, int *status,
                                cudaStream_t stream);

// x [B, S, K] (bf16, or fp32 with x_f32) to e4m3 q and fp32 scales per `rows`
// rows (1, or 128 with B = 1) and 128 channels. K a multiple of 16; strides in
// elements: x_*, q_* as the token tensors of LinearFp8Problem, s_bs, s_rs, s_ks
// between the scales of batch elements, rows (of blocks) and groups.
struct QuantizeFp8 {
  const void *x;
  void *q;
  float *scale;
  int64_t x_bs, x_rs, q_bs, q_rs, s_bs, s_rs, s_ks;
  int64_t B, S;
  int K, rows, x_f32;
};
cudaError_t launch_quantize_fp8(const QuantizeFp8 &q, cudaStream_t stream);

// out = residual + gate * act(x W^T + bias) over tokens [B, S]: x and W e4m3
// with fp32 scales per 128 channels of a token (xs) and per 128 x 128 block of W
// (ws). Strides in elements: x_* and w_rs multiples of 16, r_* and o_* of 8, the
// scales' any that are not negative (_ks from one group of channels to the next).
struct LinearFp8Problem {
  const void *x, *w, *residual;
  void *out;
  const float *xs, *ws;
  int64_t x_bs, x_rs, w_rs, r_bs, r_rs, o_bs, o_rs, xs_bs, xs_rs, xs_ks, ws_rs, ws_ks;
  int64_t B, S, N;
  int K;
};

// How a problem runs: split (units of one CTA over Q tokens, the channels in C
// parts) or else pairs of CTAs (tiles of tn accumulator columns), each with an
// estimate of its time in ns.
struct Fp8SplitPlan {
  int Q, C, stages;
  bool early;
  double ns;
};
struct Fp8PairPlan {
  int tn;
  double ns;
};
struct Fp8Plan {
  bool use_split;
  Fp8SplitPlan split;
  Fp8PairPlan pair;
};
Fp8SplitPlan plan_fp8_split(const LinearFp8Problem &q, int act, int sms);
Fp8PairPlan plan_fp8_pair(const LinearFp8Problem &q, int act, int sms);
Fp8Plan plan_linear_fp8(const LinearFp8Problem &q, int act, int sms);
cudaError_t launch_fp8_split(const LinearFp8Problem &q, const Fp8SplitPlan &plan,
                             const LinearEpilogue &epi, int act, int *status, cudaStream_t stream);
cudaError_t launch_fp8_pair(const LinearFp8Problem &q, const Fp8PairPlan &plan,
                            const LinearEpilogue &epi, int act, int *status, cudaStream_t stream);

// out = softmax(scale q k^T) v, bf16 q and out [B, Sq, H, D], k and v [B, Sk, Hk,
// D], D 64 or 128, Hk a divisor of H and H / Hk at most 128. Strides in elements,
// heads adjacent. lengths (int32 [B]) and mask (bytes [B, Sk] at stride mask_bs),
// each nullable, say which keys take part.
struct CrossAttention {
  const void *q, *k, *v;
  void *out;
  const int32_t *lengths;
  const uint8_t *mask;
  int64_t q_bs, q_rs, k_bs, k_rs, v_bs, v_rs, o_bs, o_rs, mask_bs;
  int64_t B, Sq, Sk;
  int H, Hk, D;
  float scale;
};
// The form that runs: narrow, with the keys in `parts` parts, or else wide; and
// an estimate of its time in ns.
struct CrossPlan {
  bool narrow;
  int parts;
  double ns;
};
CrossPlan plan_cross(const CrossAttention &a, int sms);
cudaError_t launch_cross_attention(const CrossAttention &a, const CrossPlan &plan, int *status,
                                   cudaStream_t stream);

// x_out = x + gate * y, h = norm(x_out) * (1 + scale) + shift over tokens
// [B, S] of `dim` channels. x and x_out are bf16, or fp32 with stream_f32; y
// and h bf16; gate, scale and shift bf16, or fp32 with vec_f32. y NULL: no
// residual (x_out and gate unused); scale, shift and gate may be NULL.
// Strides in elements, multiples of 8 (the vectors' may be 0).
struct ModulatedNorm {
  const void *x, *y, *gate, *scale, *shift;
  void *x_out, *h;
  int64_t x_bs, x_rs, y_bs, y_rs, gate_bs, scale_bs, shift_bs, xo_bs, xo_rs, h_bs, h_rs;
  int64_t B, S;
  int dim, rms, stream_f32, vec_f32;
  float eps;
};
constexpr int kNormMaxDim = 16384;
cudaError_t launch_modulated_norm(const ModulatedNorm &q, cudaStream_t stream);

// Enqueues the attention kernel. q/k/v/out are [B, S, H, 128] bf16; `table`
// is the packed table of the joint sequence; status is the device status word.
// `krot_scratch` (256-byte aligned, krot_scratch_bytes long) lets the CTAs
// that work on one head share rotated K tiles; NULL makes every CTA rotate
// every K tile it loads. `norm` (nullable) normalises Q and K before RoPE.
cudaError_t launch_joint_attention(const void *q, const void *k, const void *v, void *out,
                                   const uint32_t *table, int *status, int B, int64_t S, int H,
                                   void *krot_scratch, const QkNormArgs *norm,
                                   cudaStream_t stream, bool pdl = false, int h0 = 0,
                                   int Hl = 0);

}  // namespace flux
