// Prints what flux_linear_fp8 and flux_cross_attention take, on a GPU with 152 SMs,
// for each line of the standard input (sizes as the kernels get them, batch
// elements joined where they can be):
//   "linear B S K N act residual" -> "split Q C ns" or "pair tn 1 ns",
//   "cross B Sq Sk H Hk D" -> "narrow parts 0 ns" or "wide 1 0 ns".
#include <cstdio>
#include <cstring>

#include "flux_internal.h"

int main() {
  char kind[16];
  long long a, b, c, d, e, f;
  while (std::scanf("%15s %lld %lld %lld %lld %lld %lld", kind, &a, &b, &c, &d, &e, &f) == 7) {
    if (std::strcmp(kind, "linear") == 0) {
      flux::LinearFp8Problem q{};
      q.B = a, q.S = b, q.K = static_cast<int>(c), q.N = d;
      if (f != 0) q.residual = &q;
      const flux::Fp8Plan p = flux::plan_linear_fp8(q, static_cast<int>(e), 152);
      if (p.use_split)
        std::printf("split %d %d %.0f\n", p.split.Q, p.split.C, p.split.ns);
      else
        std::printf("pair %d 1 %.0f\n", p.pair.tn, p.pair.ns);
    } else {
      flux::CrossAttention q{};
      q.B = a, q.Sq = b, q.Sk = c;
      q.H = static_cast<int>(d), q.Hk = static_cast<int>(e), q.D = static_cast<int>(f);
      const flux::CrossPlan p = flux::plan_cross(q, 152);
      std::printf("%s %d 0 %.0f\n", p.narrow ? "narrow" : "wide", p.parts, p.ns);
    }
  }
  return 0;
}
