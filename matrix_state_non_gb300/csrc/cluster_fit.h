// How many clusters of each size a GPU runs at once, as each GPU answered before.
// Host code alone, without CUDA's headers.
#pragma once

#include <atomic>

namespace m2rnn {

constexpr int kMaxCluster = 8;

class ClusterFit {
 public:
  // For clusters of `size` blocks, 2 to kMaxCluster, on `device`.  `query` asks
  // the GPU; an answer below 1 is none: then `otherwise` serves, this once.
  template <typename Query>
  int get(int device, int size, int otherwise, Query&& query) {
    std::atomic<int>* kept = device >= 0 && device < kDevices ? &of_[device][size] : nullptr;
    int n = kept != nullptr ? kept->load(std::memory_order_relaxed) : 0;
    if (n < 1) {
      n = query();
      if (n < 1) return otherwise;
      if (kept != nullptr) kept->store(n, std::memory_order_relaxed);
    }
    return n;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> of_[kDevices][kMaxCluster + 1] = {};
};

}  // namespace m2rnn
