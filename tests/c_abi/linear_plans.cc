// Prints which kernel, form and tile flux_linear takes: for each line
// "B S K K2 N act residual" of the standard input (sizes as the kernels get
// them, batch elements joined where they can be) a line "kernel form tile parts
// ns", of a GPU with 152 SMs.
#include <cstdio>

#include "flux_internal.h"

int main() {
  long long B, S, N;
  int K, K2, act, residual;
  while (std::scanf("%lld %lld %d %d %lld %d %d", &B, &S, &K, &K2, &N, &act, &residual) == 7) {
    flux::LinearProblem q{};
    q.B = B, q.S = S, q.K = K, q.K2 = K2, q.N = N;
    if (residual != 0) q.residual = &q;
    const flux::LinearPlan p = flux::plan_linear(q, act, 152);
    if (p.use_split)
      std::printf("split %d %d %d %.0f\n", p.split.form, p.split.Q, p.split.C, p.split.ns);
    else
      std::printf("pair 0 %d 1 %.0f\n", p.pair.tn, p.pair.ns);
  }
  return 0;
}
