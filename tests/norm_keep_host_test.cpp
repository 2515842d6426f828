// norm_keep_host_test.cpp - runs norm_keep_from (precision_state_amd/csrc/norm_keep.h)
// on lists from stdin: "chunk keep n", then n times "elements bytes"; prints one
// result a line.
#include <cstdio>
#include <utility>
#include <vector>

#include "norm_keep.h"

int main() {
  long long chunk, keep;
  int n;
  while (scanf("%lld %lld %d", &chunk, &keep, &n) == 3) {
    std::vector<std::pair<int64_t, int64_t>> t(n);
    for (auto& x : t) {
      long long a, b;
      if (scanf("%lld %lld", &a, &b) != 2) return 1;
      x = {a, b};
    }
    printf("%llu\n", (unsigned long long)ps::norm_keep_from(t, [](const auto& x) { return x; }, chunk, keep));
  }
  return 0;
}
