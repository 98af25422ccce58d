// Host code: something done once for each device (an attribute of a kernel, say).  What failed is not remembered,
// so a later call tries it again.
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>

namespace dit6 {

class OncePerDevice {
 public:
  // attempt() returns 0 (cudaSuccess) if it worked; so does this where it has worked on `device` before.
  template <typename F>
  auto run(int device, F attempt) -> decltype(attempt()) {
    if (device < 0 || device >= DEVICES) return attempt();
    const uint64_t bit = uint64_t(1) << device;
    if (done_.load(std::memory_order_acquire) & bit) return decltype(attempt())(0);
    std::lock_guard<std::mutex> hold(attempting_);
    if (done_.load(std::memory_order_relaxed) & bit) return decltype(attempt())(0);
    const auto status = attempt();
    if (status == decltype(attempt())(0)) done_.fetch_or(bit, std::memory_order_release);
    return status;
  }
  static constexpr int DEVICES = 64;

 private:
  std::atomic<uint64_t> done_{0};
  std::mutex attempting_;
};

}  // namespace dit6
