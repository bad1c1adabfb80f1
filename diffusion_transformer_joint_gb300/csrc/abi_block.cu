// C-ABI entry points of the operators around the attention in a block,
// declared in include/flux_attn.h: argument checks and launches.
#include <cuda_runtime.h>

#include <atomic>

#include "flux_internal.h"
#include "linear_common.cuh"

namespace {

// Rows [B, S] of `width` elements of `size` bytes, strides in elements.
struct Rows {
  const void *p;
  int64_t B, S, width, bs, rs;
  int size;
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Largest extent in elements of one tensor (a tensor map's strides stay below
// 2^40 bytes).
constexpr int64_t kMaxSpan = int64_t{1} << 38;

// Strides that no size looks at get those of contiguous rows.
void settle(Rows &t) {
  if (t.S == 1) t.rs = (t.width + 7) / 8 * 8;
  if (t.B == 1) t.bs = t.rs <= kMaxSpan / t.S ? t.S * t.rs : t.rs;
}

// Strides are multiples of 8 elements, no smaller than a row, and the rows fit
// the span.
bool strides_ok(const Rows &t) {
  if (t.rs <= 0 || t.bs <= 0 || t.rs % 8 != 0 || t.bs % 8 != 0) return false;
  if (t.rs > kMaxSpan / t.S || t.bs > kMaxSpan / t.B) return false;
  return (t.S == 1 || t.rs >= t.width) && (t.B == 1 || t.bs >= t.width);
}

// No two rows of the tensor share an element (an output's condition): batch
// elements follow one another, or interleave between the tokens of the first.
bool rows_disjoint(const Rows &t) {
  if (t.S > 1 && t.rs < t.width) return false;
  if (t.B > 1 && t.bs < t.width) return false;
  if (t.S == 1 || t.B == 1) return true;
  return t.bs >= (t.S - 1) * t.rs + t.width || t.rs >= (t.B - 1) * t.bs + t.width;
}

int64_t span_bytes(const Rows &t) {
  return ((t.B - 1) * t.bs + (t.S - 1) * t.rs + t.width) * t.size;
}

bool ranges_meet(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(nb) && b0 < a0 + static_cast<uintptr_t>(na);
}

// Whether two tensors share a byte. Tensors with the same strides (views of
// one buffer: two streams of a joint sequence, two blocks of its columns) are
// decided row by row; others by the address ranges they span.
bool share(const Rows &a, const Rows &b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  if (!ranges_meet(a.p, span_bytes(a), b.p, span_bytes(b))) return false;
  if (a.bs * a.size != b.bs * b.size && a.B > 1 && b.B > 1) return true;
  if (a.rs * a.size != b.rs * b.size && a.S > 1 && b.S > 1) return true;
  // row (i, j) of b starts `off` + i * big + j * small bytes after row (i', j')
  // of a, differences i - i' and j - j' within the sizes
  struct Axis {
    int64_t step, lo, hi;
  };
  Axis big{(a.B > 1 ? a.bs * a.size : b.bs * b.size), -(a.B - 1), b.B - 1};
  Axis small{(a.S > 1 ? a.rs * a.size : b.rs * b.size), -(a.S - 1), b.S - 1};
  if (big.step < small.step) {
    const Axis t = big;
    big = small;
    small = t;
  }
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p)) -
                      static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p));
  const int64_t wa = a.width * a.size, wb = b.width * b.size;
  // rows meet when -wb < distance < wa; the long axis leaves few candidates
  const int64_t reach = (small.hi > -small.lo ? small.hi : -small.lo) * small.step + wa + wb;
  int64_t i0 = (-off - reach) / big.step - 1, i1 = (-off + reach) / big.step + 1;
  if (i0 < big.lo) i0 = big.lo;
  if (i1 > big.hi) i1 = big.hi;
  if (i1 - i0 > 4096) return true;
  for (int64_t i = i0; i <= i1; ++i) {
    const int64_t d = off + i * big.step;
    int64_t j0 = (-wb - d) / small.step - 1, j1 = (wa - d) / small.step + 1;
    if (j0 < small.lo) j0 = small.lo;
    if (j1 > small.hi) j1 = small.hi;
    for (int64_t j = j0; j <= j1; ++j) {
      const int64_t e = d + j * small.step;
      if (e > -wb && e < wa) return true;
    }
  }
  return false;
}

// A vector per batch element (gate, scale, shift): [B, width] at stride bs,
// which may be 0 (one vector for all).
bool vec_stride_ok(int64_t bs, int64_t B) {
  return bs >= 0 && bs % 8 == 0 && bs <= kMaxSpan / B;
}
Rows vec_rows(const void *p, int64_t B, int64_t width, int64_t bs, int f32) {
  if (bs == 0 || B == 1) return Rows{p, 1, 1, width, width, width, f32 ? 4 : 2};
  return Rows{p, B, 1, width, bs, width, f32 ? 4 : 2};
}

constexpr int64_t kMaxTokens = int64_t{1} << 30;

// The library's own status word, one per device that loads the library. The
// host's name for it is no device address: own_status_word looks that up.
static __device__ int32_t g_status;

int32_t *own_status_word() {
  static std::atomic<void *> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  void *p = cached[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) {
      (void)cudaGetLastError();  // not to surface in a later call
      return nullptr;
    }
    cached[dev].store(p, std::memory_order_relaxed);
  }
  return static_cast<int32_t *>(p);
}

// Batch elements that follow one another at the token stride are one run of
// tokens.
bool joins(const Rows &t) { return t.p == nullptr || t.B == 1 || t.bs == t.S * t.rs; }

}  // namespace

// With few tokens most rows of linear_pair's tiles would be empty, and its
// estimate is not fitted there.
flux::LinearPlan flux::plan_linear(const LinearProblem &q, int act, int sms) {
  LinearPlan p{true, plan_split(q, act, sms), {0, 2e30}};
  if (q.B * q.S >= 128) p.pair = plan_pair(q, act, sms);
  p.use_split = p.split.ns < p.pair.ns;
  return p;
}

extern "C" {

int flux_linear(const void *x, int64_t x_bs, int64_t x_rs, int K, const void *x2, int64_t x2_bs,
                int64_t x2_rs, int K2, const void *w, int64_t w_rs, int B, int64_t S, int64_t N,
                int act, const void *bias, const void *gate, int64_t gate_bs, int vec_f32,
                const void *residual, int64_t r_bs, int64_t r_rs, void *out, int64_t o_bs,
                int64_t o_rs, int32_t *status, void *stream) {
  if (x == nullptr || w == nullptr || out == nullptr || status == nullptr ||
      (K2 > 0 && x2 == nullptr))
    return FLUX_ERR_NULL;
  if (B < 1 || S < 1 || S > kMaxTokens / B || K < 8 || K % 8 != 0 || K2 < 0 || K2 % 8 != 0 ||
      N < 8 || N % 8 != 0 || N > (1 << 28) || K > (1 << 28) || K2 > (1 << 28))
    return FLUX_ERR_SHAPE;
  if (act < FLUX_ACT_NONE || act > FLUX_ACT_SWIGLU || (vec_f32 != 0 && vec_f32 != 1))
    return FLUX_ERR_SHAPE;
  const int64_t wr = act == FLUX_ACT_SWIGLU ? 2 * N : N;
  Rows rx{x, B, S, K, x_bs, x_rs, 2}, rx2{K2 > 0 ? x2 : nullptr, B, S, K2, x2_bs, x2_rs, 2};
  Rows rr{residual, B, S, N, r_bs, r_rs, 2}, ro{out, B, S, N, o_bs, o_rs, 2};
  Rows rw{w, 1, wr, K + static_cast<int64_t>(K2), 0, w_rs, 2};
  for (Rows *t : {&rx, &rx2, &rr, &ro, &rw}) {
    if (t->p == nullptr) continue;
    settle(*t);
    if (!strides_ok(*t)) return FLUX_ERR_SHAPE;
  }
  if (!rows_disjoint(ro)) return FLUX_ERR_SHAPE;
  if (gate != nullptr && !vec_stride_ok(gate_bs, B)) return FLUX_ERR_SHAPE;
  for (const void *p : {x, w, static_cast<const void *>(out), rx2.p, bias, gate, residual})
    if (!aligned16(p)) return FLUX_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(status) & 3u) return FLUX_ERR_ALIGN;
  const Rows rb = vec_rows(bias, 1, wr, 0, vec_f32), rg = vec_rows(gate, B, N, gate_bs, vec_f32);
  const Rows rs{status, 1, 1, 1, 1, 1, 4};
  for (const Rows &t : {rx, rx2, rw, rb, rg, rs})
    if (share(ro, t)) return FLUX_ERR_ALIAS;
  // the residual may be the output itself, element for element
  const bool in_place = residual == out && rr.rs == ro.rs && rr.bs == ro.bs;
  if (!in_place && share(ro, rr)) return FLUX_ERR_ALIAS;
  const int dc = flux::check_device();
  if (dc != FLUX_OK) return dc;

  const flux::LinearEpilogue epi{bias, gate, B > 1 ? gate_bs : 0, S, vec_f32};
  flux::LinearProblem q{x,     rx2.p, w,     residual, out,   rx.bs, rx.rs, rx2.bs, rx2.rs, rw.rs,
                        rr.bs, rr.rs, ro.bs, ro.rs,    B,     S,     N,     K,      K2};
  if (S == 1) {  // batch elements of one token: tokens at the batch stride
    q.x_rs = rx.bs, q.x2_rs = rx2.bs, q.r_rs = rr.bs, q.o_rs = ro.bs;
    q.B = 1, q.S = B;
  } else if (joins(rx) && joins(rx2) && joins(rr) && joins(ro)) {
    q.B = 1, q.S = B * S;
  }
  if (q.B == 1) {  // (a batch stride that nothing looks at, but the tensor maps take)
    q.x_bs = q.x_rs * q.S, q.x2_bs = q.x2_rs * q.S, q.r_bs = q.r_rs * q.S, q.o_bs = q.o_rs * q.S;
  }
  const int sms = flux::sm_count_current_device();
  if (sms < 1) return FLUX_ERR_CUDA;
  const flux::LinearPlan plan = flux::plan_linear(q, act, sms);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = plan.use_split
                            ? flux::launch_linear_split(q, plan.split, epi, act, status, st)
                            : flux::launch_linear_pair(q, plan.pair, epi, act, status, st);
  return e == cudaSuccess ? FLUX_OK : FLUX_ERR_CUDA;
}

int flux_modulated_norm(const void *x, int64_t x_bs, int64_t x_rs, int stream_f32, const void *y,
                        int64_t y_bs, int64_t y_rs, const void *gate, int64_t gate_bs,
                        const void *scale, int64_t scale_bs, const void *shift, int64_t shift_bs,
                        int vec_f32, int B, int64_t S, int dim, int norm, float eps, void *x_out,
                        int64_t xo_bs, int64_t xo_rs, void *h, int64_t h_bs, int64_t h_rs,
                        void *stream) {
  if (x == nullptr || h == nullptr || (y != nullptr && x_out == nullptr)) return FLUX_ERR_NULL;
  if (B < 1 || S < 1 || S > kMaxTokens / B || dim < 8 || dim % 8 != 0 || dim > flux::kNormMaxDim)
    return FLUX_ERR_SHAPE;
  if ((norm != FLUX_NORM_LAYER && norm != FLUX_NORM_RMS) || !(eps >= 0.f) || !(eps < 3.0e38f) ||
      (vec_f32 != 0 && vec_f32 != 1) || (stream_f32 != 0 && stream_f32 != 1))
    return FLUX_ERR_SHAPE;
  if (y == nullptr) x_out = nullptr, gate = nullptr;
  const int xs = stream_f32 ? 4 : 2;
  Rows rx{x, B, S, dim, x_bs, x_rs, xs}, ry{y, B, S, dim, y_bs, y_rs, 2};
  Rows ro{x_out, B, S, dim, xo_bs, xo_rs, xs}, rh{h, B, S, dim, h_bs, h_rs, 2};
  for (Rows *t : {&rx, &ry, &ro, &rh}) {
    if (t->p == nullptr) continue;
    settle(*t);
    if (!strides_ok(*t)) return FLUX_ERR_SHAPE;
  }
  if (!rows_disjoint(rh) || (x_out != nullptr && !rows_disjoint(ro))) return FLUX_ERR_SHAPE;
  if ((gate != nullptr && !vec_stride_ok(gate_bs, B)) ||
      (scale != nullptr && !vec_stride_ok(scale_bs, B)) ||
      (shift != nullptr && !vec_stride_ok(shift_bs, B)))
    return FLUX_ERR_SHAPE;
  for (const void *p : {x, y, gate, scale, shift, static_cast<const void *>(x_out),
                        static_cast<const void *>(h)})
    if (!aligned16(p)) return FLUX_ERR_ALIGN;
  const Rows rg = vec_rows(gate, B, dim, gate_bs, vec_f32),
             rs = vec_rows(scale, B, dim, scale_bs, vec_f32),
             rf = vec_rows(shift, B, dim, shift_bs, vec_f32);
  for (const Rows &t : {rx, ry, rg, rs, rf, ro})
    if (share(rh, t)) return FLUX_ERR_ALIAS;
  if (x_out != nullptr) {
    // the stream may be updated in place, element for element
    const bool in_place = x_out == x && ro.rs == rx.rs && ro.bs == rx.bs;
    for (const Rows &t : {ry, rg, rs, rf})
      if (share(ro, t)) return FLUX_ERR_ALIAS;
    if (!in_place && share(ro, rx)) return FLUX_ERR_ALIAS;
  }
  const int dc = flux::check_device();
  if (dc != FLUX_OK) return dc;
  const int64_t keep = B > 1 ? 1 : 0;  // one batch element: no stride is looked at
  const flux::ModulatedNorm q{x,     y,     gate,  scale, shift, x_out, h,     rx.bs, rx.rs, ry.bs,
                              ry.rs, keep * gate_bs, keep * scale_bs, keep * shift_bs,
                              ro.bs, ro.rs, rh.bs, rh.rs, B, S, dim,
                              norm == FLUX_NORM_RMS ? 1 : 0, stream_f32, vec_f32, eps};
  return flux::launch_modulated_norm(q, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLUX_OK
             : FLUX_ERR_CUDA;
}

int flux_status_word(int32_t **status) {
  if (status == nullptr) return FLUX_ERR_NULL;
  const int dc = flux::check_device();
  if (dc != FLUX_OK) return dc;
  *status = own_status_word();
  return *status != nullptr ? FLUX_OK : FLUX_ERR_CUDA;
}

int flux_take_status(void *stream) {
  int32_t *word = nullptr;
  const int rc = flux_status_word(&word);
  if (rc != FLUX_OK) return rc;
  const int status = flux_query_status(word, stream);
  if (status == FLUX_OK) return status;
  // cleared before a later call of the stream can report again
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(word, 0, sizeof(*word), st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return FLUX_ERR_CUDA;
  return status;
}

}  // extern "C"
