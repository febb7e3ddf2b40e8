// Prints the norm join's launches for each "T C" read: threads, forward workgroups, backward rows at a
// time and workgroups.
#include <cstdio>

#include "../../blockwise_fp8_zero_fold_amd/csrc/norm_plan.h"

int main() {
  long long T, C;
  while (std::scanf("%lld %lld", &T, &C) == 2) {
    const fp8z1::NormGroups b = fp8z1::norm_bwd_groups(T, C);
    std::printf("%d %lld %lld %lld\n", fp8z1::norm_threads(C), static_cast<long long>(fp8z1::norm_fwd_groups(T, C)),
                static_cast<long long>(b.rows), static_cast<long long>(b.count));
  }
  return 0;
}
