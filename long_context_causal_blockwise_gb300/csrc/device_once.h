// Host-side "once per device context" set-up flags.
//
// Settings such as a kernel's dynamic shared-memory limit
// (cudaFuncSetAttribute) belong to one device's context: a process that drives
// two GPUs must apply them on each, and a context torn down by
// cudaDeviceReset and created again has lost them. DeviceOnce keeps, per
// device ordinal, the id of the context in which the set-up last succeeded;
// run(dev, ctx_id, f) calls f unless that id equals ctx_id. Context ids are
// unique within a process and never 0; ctx_id 0 (no id known) runs f every
// time. A failed set-up is not remembered, so the next call retries it.
// DeviceCounts keeps, in the same way, numbers that a query about the device
// answers.
// Plain C++ (no CUDA), so that its logic can be checked on a machine without
// a GPU with made-up device ordinals and context ids.
#pragma once

#include <atomic>
#include <mutex>

namespace lcb {

constexpr int kMaxDeviceOrdinals = 64;

class DeviceOnce {
 public:
  // Returns f()'s status when it runs, 0 when the set-up is already done in
  // context ctx_id of device `dev`, and `bad_device` for an ordinal outside
  // [0, kMaxDeviceOrdinals).
  template <class F>
  int run(int dev, unsigned long long ctx_id, F&& f, int bad_device) {
    if (dev < 0 || dev >= kMaxDeviceOrdinals) return bad_device;
    if (ctx_id == 0) return f();
    if (key_[dev].load(std::memory_order_acquire) == ctx_id) return 0;
    std::lock_guard<std::mutex> lk(mu_);
    if (key_[dev].load(std::memory_order_relaxed) == ctx_id) return 0;
    const int rc = f();
    if (rc == 0) key_[dev].store(ctx_id, std::memory_order_release);
    return rc;
  }

  // True if the set-up succeeded in context ctx_id of device `dev`.
  bool done(int dev, unsigned long long ctx_id) const {
    return dev >= 0 && dev < kMaxDeviceOrdinals && ctx_id != 0 &&
           key_[dev].load(std::memory_order_acquire) == ctx_id;
  }

 private:
  std::mutex mu_;
  std::atomic<unsigned long long> key_[kMaxDeviceOrdinals] = {};
};

// Counts under keys [0, N) that belong to a device context (how many clusters
// of a size it holds at once), asked for once in each.
template <int N>
class DeviceCounts {
 public:
  // The count under `key` in context ctx_id of device `dev`: what ask() says,
  // kept if it is not negative. A negative answer means that the query failed:
  // 0 this time, and the next call asks again. Outside the table (an ordinal
  // or id too large, ctx_id 0) it asks every time.
  template <class F>
  int get(int dev, unsigned long long ctx_id, int key, F&& ask) {
    const bool kept = dev >= 0 && dev < kMaxDeviceOrdinals && ctx_id != 0 && ctx_id < (1ull << 48);
    if (kept) {
      const unsigned long long w = word_[dev][key].load(std::memory_order_relaxed);
      if (w >> 16 == ctx_id) return static_cast<int>(w & 0xffffu);
    }
    const int n = ask();
    if (n < 0) return 0;
    if (kept && n < (1 << 16))
      word_[dev][key].store(ctx_id << 16 | static_cast<unsigned long long>(n), std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<unsigned long long> word_[kMaxDeviceOrdinals][N] = {};  // context id, then 16 bits of count
};

}  // namespace lcb
