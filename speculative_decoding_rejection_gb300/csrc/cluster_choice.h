// Choice of a cluster size for a persistent kernel (host, plain C++).
#pragma once

#include <atomic>

namespace sv {

struct ClusterChoice {
  int size, count;   // CTAs of a cluster, clusters that run at a time; 0, 0: none
};

// Of the sizes 1 .. most that fit, the one that runs on the most SMs, the smaller
// of equals. counts[C]: what ask(C) said, the clusters of C CTAs that run at a time,
// 0 before it was asked (once per size; the callers' threads share it). A size that
// the device cannot run (ask gives 0 or less) is passed over.
template <class Fits, class Ask>
ClusterChoice choose_cluster(std::atomic<int> *counts, int most, Fits fits, Ask ask) {
  ClusterChoice best{0, 0};
  for (int C = 1; C <= most; ++C) {
    if (!fits(C)) continue;
    int n = counts[C].load(std::memory_order_relaxed);
    if (n == 0) {
      n = ask(C);
      if (n <= 0) n = -1;
      counts[C].store(n, std::memory_order_relaxed);
    }
    if (n > 0 && n * C > best.count * best.size) best = ClusterChoice{C, n};
  }
  return best;
}

}  // namespace sv
