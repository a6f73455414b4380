// The prefill's cut of a total weight into shares, on the host: for each line
// "total min_weight long_total grid" of the input, the number of shares and
// what each but the last weighs.
#include <cstdio>

#include "prefill_plan.cuh"

int main() {
  long long total, long_total;
  int min_weight;
  unsigned grid;
  while (std::scanf("%lld %d %lld %u", &total, &min_weight, &long_total, &grid) == 4) {
    const unsigned ctas = vt::pf_share_count(total, min_weight, long_total, grid);
    std::printf("%u %lld\n", ctas, vt::pf_share_weight(total, ctas));
  }
  return 0;
}
