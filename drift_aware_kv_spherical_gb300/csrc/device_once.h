// What a process does once a GPU, whichever of its threads comes first.  Host only.
#pragma once

#include <atomic>
#include <cstdint>

namespace ps {

class DeviceOnce {
 public:
  constexpr DeviceOnce() = default;
  bool done(int device) const {
    return known(device) && (bits_.load(std::memory_order_acquire) >> device & 1) != 0;
  }
  void set(int device) {
    if (known(device)) bits_.fetch_or(uint64_t{1} << device, std::memory_order_release);
  }

 private:
  // (others have it done again every time)
  static constexpr bool known(int device) { return device >= 0 && device < 64; }
  std::atomic<uint64_t> bits_{0};
};

}  // namespace ps
