// The prefill's cut of a total weight into shares, on the host: for each line
// "total min_weight long_total grid" of the input, the number of shares.
#include <cstdio>

#include "prefill_plan.cuh"

int main() {
  long long total, long_total;
  int min_weight;
  unsigned grid;
  while (std::scanf("%lld %d %lld %u", &total, &min_weight, &long_total, &grid) == 4)
    std::printf("%u\n", vt::pf_share_count(total, min_weight, long_total, grid));
  return 0;
}
