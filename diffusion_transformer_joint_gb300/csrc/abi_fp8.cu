// C-ABI entry points of the products in 8-bit floating point, declared in
// include/flux_attn.h: argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "abi_rows.h"
#include "flux_internal.h"
#include "linear_common.cuh"

using namespace flux;

namespace {

// Scales [B, R, G] (batch elements, rows or blocks of rows, groups of
// channels), any strides in elements that are not negative.
struct Scales {
  const float *p;
  int64_t B, R, G, bs, rs, ks;
};

bool scale_strides_ok(const Scales &s) {
  if (s.bs < 0 || s.rs < 0 || s.ks < 0) return false;
  return s.bs <= kMaxSpan / s.B && s.rs <= kMaxSpan / s.R && s.ks <= kMaxSpan / s.G;
}

// No two of an output's scales share their place: each stride passes the whole
// extent of those below it.
bool scales_disjoint(const Scales &s) {
  struct Axis {
    int64_t n, step;
  } a[3] = {{s.B, s.bs}, {s.R, s.rs}, {s.G, s.ks}};
  std::sort(a, a + 3, [](const Axis &x, const Axis &y) { return x.step < y.step; });
  int64_t extent = 1;
  for (const Axis &x : a) {
    if (x.n == 1) continue;
    if (x.step < extent) return false;
    extent = x.step * (x.n - 1) + extent;
  }
  return true;
}

// The scales as one run of memory, for share().
Rows scale_rows(const Scales &s) {
  const int64_t n = (s.B - 1) * s.bs + (s.R - 1) * s.rs + (s.G - 1) * s.ks + 1;
  return Rows{s.p, 1, 1, n, n, n, 4};
}

// 8-bit rows are copied in 16-byte pieces.
bool byte_strides_ok(const Rows &t) { return t.rs % 16 == 0 && t.bs % 16 == 0; }

constexpr int kMaxChannels = 1 << 22;

}  // namespace

flux::Fp8Plan flux::plan_linear_fp8(const LinearFp8Problem &q, int act, int sms) {
  Fp8Plan p{true, plan_fp8_split(q, act, sms), plan_fp8_pair(q, act, sms)};
  p.use_split = p.split.ns < p.pair.ns;
  return p;
}

extern "C" {

int flux_quantize_fp8(const void *x, int64_t x_bs, int64_t x_rs, int x_f32, int B, int64_t S, int K,
                      int rows, void *q, int64_t q_bs, int64_t q_rs, float *scale, int64_t s_bs,
                      int64_t s_rs, int64_t s_ks, void *stream) {
  if (x == nullptr || q == nullptr || scale == nullptr) return FLUX_ERR_NULL;
  if (B < 1 || S < 1 || S > kMaxTokens / B || K < 16 || K % 16 != 0 || K > kMaxChannels ||
      (rows != 1 && rows != 128) || (x_f32 != 0 && x_f32 != 1))
    return FLUX_ERR_SHAPE;
  if (rows == 128 && (B != 1 || S > kMaxChannels)) return FLUX_ERR_SHAPE;
  Rows rx{x, B, S, K, x_bs, x_rs, x_f32 ? 4 : 2}, rq{q, B, S, K, q_bs, q_rs, 1};
  for (Rows *t : {&rx, &rq}) {
    settle(*t);
    if (!strides_ok(*t)) return FLUX_ERR_SHAPE;
  }
  if (!byte_strides_ok(rq) || !rows_disjoint(rq)) return FLUX_ERR_SHAPE;
  const Scales sc{scale, B, (S + rows - 1) / rows, (K + 127) / 128, B > 1 ? s_bs : 0,
                  S > rows ? s_rs : 0, K > 128 ? s_ks : 0};
  if (!scale_strides_ok(sc) || !scales_disjoint(sc)) return FLUX_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scale) & 3u))
    return FLUX_ERR_ALIGN;
  const Rows rs = scale_rows(sc);
  if (share(rq, rx) || share(rs, rx) || share(rs, rq)) return FLUX_ERR_ALIAS;
  const int dc = check_device();
  if (dc != FLUX_OK) return dc;
  const QuantizeFp8 p{x,     q,     scale, rx.bs, rx.rs, rq.bs, rq.rs, sc.bs,
                      sc.rs, sc.ks, B,     S,     K,     rows,  x_f32};
  return launch_quantize_fp8(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FLUX_OK
                                                                                 : FLUX_ERR_CUDA;
}

int flux_linear_fp8(const void *x, int64_t x_bs, int64_t x_rs, const float *x_scale, int64_t xs_bs,
                    int64_t xs_rs, int64_t xs_ks, const void *w, int64_t w_rs,
                    const float *w_scale, int64_t ws_rs, int64_t ws_ks, int B, int64_t S, int K,
                    int64_t N, int act, const void *bias, const void *gate, int64_t gate_bs,
                    int vec_f32, const void *residual, int64_t r_bs, int64_t r_rs, void *out,
                    int64_t o_bs, int64_t o_rs, int32_t *status, void *stream) {
  if (x == nullptr || x_scale == nullptr || w == nullptr || w_scale == nullptr ||
      out == nullptr || status == nullptr)
    return FLUX_ERR_NULL;
  if (B < 1 || S < 1 || S > kMaxTokens / B || K < 16 || K % 16 != 0 || K > kMaxChannels ||
      N < 8 || N % 8 != 0 || N > (1 << 28))
    return FLUX_ERR_SHAPE;
  if (act < FLUX_ACT_NONE || act > FLUX_ACT_SWIGLU || (vec_f32 != 0 && vec_f32 != 1))
    return FLUX_ERR_SHAPE;
  if (act == FLUX_ACT_SWIGLU && N % 128 != 0) return FLUX_ERR_SHAPE;
  const int64_t wr = act == FLUX_ACT_SWIGLU ? 2 * N : N;
  Rows rx{x, B, S, K, x_bs, x_rs, 1}, rw{w, 1, wr, K, 0, w_rs, 1};
  Rows rr{residual, B, S, N, r_bs, r_rs, 2}, ro{out, B, S, N, o_bs, o_rs, 2};
  for (Rows *t : {&rx, &rw, &rr, &ro}) {
    if (t->p == nullptr) continue;
    settle(*t);
    if (!strides_ok(*t)) return FLUX_ERR_SHAPE;
  }
  if (!byte_strides_ok(rx) || !byte_strides_ok(rw) || !rows_disjoint(ro)) return FLUX_ERR_SHAPE;
  const int64_t kb = (K + 127) / 128;
  const Scales sx{x_scale, B, S, kb, xs_bs, xs_rs, xs_ks};
  const Scales sw{w_scale, 1, (wr + 127) / 128, kb, 0, ws_rs, ws_ks};
  if (!scale_strides_ok(sx) || !scale_strides_ok(sw)) return FLUX_ERR_SHAPE;
  if (gate != nullptr && !vec_stride_ok(gate_bs, B)) return FLUX_ERR_SHAPE;
  for (const void *p : {x, w, static_cast<const void *>(out), bias, gate, residual})
    if (!aligned16(p)) return FLUX_ERR_ALIGN;
  for (const void *p : {static_cast<const void *>(x_scale), static_cast<const void *>(w_scale),
                        static_cast<const void *>(status)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return FLUX_ERR_ALIGN;
  const Rows rb = vec_rows(bias, 1, wr, 0, vec_f32), rg = vec_rows(gate, B, N, gate_bs, vec_f32);
  const Rows rs{status, 1, 1, 1, 1, 1, 4};
  for (const Rows &t : {rx, rw, scale_rows(sx), scale_rows(sw), rb, rg, rs})
    if (share(ro, t)) return FLUX_ERR_ALIAS;
  // the residual may be the output itself, element for element
  const bool in_place = residual == out && rr.rs == ro.rs && rr.bs == ro.bs;
  if (!in_place && share(ro, rr)) return FLUX_ERR_ALIAS;
  const int dc = check_device();
  if (dc != FLUX_OK) return dc;

  const LinearEpilogue epi{bias, gate, B > 1 ? gate_bs : 0, S, vec_f32};
  LinearFp8Problem q{x,     w,     residual, out,   x_scale, w_scale, rx.bs, rx.rs,
                     rw.rs, rr.bs, rr.rs,    ro.bs, ro.rs,   xs_bs,   xs_rs, xs_ks,
                     ws_rs, ws_ks, B,        S,     N,       K};
  if (S == 1) {  // batch elements of one token: tokens at the batch stride
    q.x_rs = rx.bs, q.r_rs = rr.bs, q.o_rs = ro.bs, q.xs_rs = xs_bs;
    q.B = 1, q.S = B;
  } else if (joins(rx) && joins(rr) && joins(ro) && (B == 1 || xs_bs == S * xs_rs)) {
    q.B = 1, q.S = B * S;
  }
  if (q.B == 1)  // (a batch stride that nothing looks at, but the tensor maps take)
    q.x_bs = q.x_rs * q.S, q.r_bs = q.r_rs * q.S, q.o_bs = q.o_rs * q.S, q.xs_bs = 0;
  const int sms = sm_count_current_device();
  if (sms < 1) return FLUX_ERR_CUDA;
  const Fp8Plan plan = plan_linear_fp8(q, act, sms);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = plan.use_split ? launch_fp8_split(q, plan.split, epi, act, status, st)
                                       : launch_fp8_pair(q, plan.pair, epi, act, status, st);
  return e == cudaSuccess ? FLUX_OK : FLUX_ERR_CUDA;
}

}  // extern "C"
