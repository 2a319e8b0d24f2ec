// Prints the form of 8-bit products: a number per line of "rows experts n_out fast".
#include <cstdio>

#include "mlora_fp8_plan.h"

int main() {
  long long rows, experts, n;
  int fast;
  while (std::scanf("%lld %lld %lld %d", &rows, &experts, &n, &fast) == 4)
    std::printf("%d\n", mlora::plan_fp8(rows, experts, n, fast != 0));
  return 0;
}
