// C-ABI entry point of the cross-attention, declared in include/flux_attn.h:
// argument checks and the launch.
#include <cuda_runtime.h>

#include <cmath>

#include "abi_rows.h"
#include "flux_internal.h"

using namespace flux;

extern "C" int flux_cross_attention(const void *q, int64_t q_bs, int64_t q_rs, const void *k,
                                    int64_t k_bs, int64_t k_rs, const void *v, int64_t v_bs,
                                    int64_t v_rs, const int32_t *lengths, const uint8_t *mask,
                                    int64_t mask_bs, int B, int64_t Sq, int64_t Sk, int H, int Hk,
                                    int D, float scale, void *out, int64_t o_bs, int64_t o_rs,
                                    int32_t *status, void *stream) {
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || status == nullptr)
    return FLUX_ERR_NULL;
  if (B < 1 || Sq < 1 || Sk < 1 || Sq > kMaxTokens / B || Sk > kMaxTokens / B || H < 1 || Hk < 1 ||
      H > 65536 || H % Hk != 0 || H / Hk > 128 || (D != 64 && D != 128))
    return FLUX_ERR_SHAPE;
  // times log2(e) it has to be finite (and is not where it is no number)
  if (!(scale >= 0.f) || !(scale <= 0x1p127f)) return FLUX_ERR_SHAPE;
  // batch elements, key heads and blocks of at least 128 H / Hk rows: an item each
  const int64_t n_s = 128 / (H / Hk);
  if ((Sq + n_s - 1) / n_s > (int64_t{1} << 24) / Hk / B) return FLUX_ERR_SHAPE;
  const int64_t wq = static_cast<int64_t>(H) * D, wk = static_cast<int64_t>(Hk) * D;
  Rows rq{q, B, Sq, wq, q_bs, q_rs, 2}, rk{k, B, Sk, wk, k_bs, k_rs, 2};
  Rows rv{v, B, Sk, wk, v_bs, v_rs, 2}, ro{out, B, Sq, wq, o_bs, o_rs, 2};
  for (Rows *t : {&rq, &rk, &rv, &ro}) {
    settle(*t);
    if (!strides_ok(*t)) return FLUX_ERR_SHAPE;
  }
  if (!rows_disjoint(ro)) return FLUX_ERR_SHAPE;
  if (mask != nullptr && (mask_bs < 0 || mask_bs > kMaxSpan / B)) return FLUX_ERR_SHAPE;
  for (const void *p : {q, k, v, static_cast<const void *>(out)})
    if (!aligned16(p)) return FLUX_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(status) & 3u) || (reinterpret_cast<uintptr_t>(lengths) & 3u))
    return FLUX_ERR_ALIGN;
  const Rows rl{lengths, 1, 1, B, B, B, 4}, rs{status, 1, 1, 1, 1, 1, 4};
  const Rows rm{mask, 1, 1, (B - 1) * (mask != nullptr ? mask_bs : 0) + Sk, 1, 1, 1};
  for (const Rows &t : {rq, rk, rv, rl, rm, rs})
    if (share(ro, t)) return FLUX_ERR_ALIAS;
  const int dc = check_device();
  if (dc != FLUX_OK) return dc;
  const int sms = sm_count_current_device();
  if (sms < 1) return FLUX_ERR_CUDA;
  const CrossAttention a{q,     k,     v,     out,   lengths, mask,    rq.bs, rq.rs, rk.bs, rk.rs,
                         rv.bs, rv.rs, ro.bs, ro.rs, mask_bs, B,       Sq,    Sk,    H,     Hk,
                         D,     scale > 0.f ? scale : 1.f / std::sqrt(static_cast<float>(D))};
  return launch_cross_attention(a, plan_cross(a, sms), status, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FLUX_OK
             : FLUX_ERR_CUDA;
}
