// Numbers that every device answers for itself, each asked for once. Plain C++, for
// the host's tests too.
#pragma once
#include <atomic>

namespace bws {

template <int kDevices, int kIndexes>
class DeviceCounts {
 public:
  // ask(): the number, below 0 where the question failed, which counts as none and is
  // asked again by the next call. Static storage only: it starts as zeros.
  template <class Ask>
  int get(int device, int index, Ask ask) {
    std::atomic<int>& known = known_[device][index];   // and one
    const int k = known.load(std::memory_order_relaxed);
    if (k > 0) return k - 1;
    const int n = ask();
    if (n < 0) return 0;
    known.store(n + 1, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<int> known_[kDevices][kIndexes];
};

}  // namespace bws
