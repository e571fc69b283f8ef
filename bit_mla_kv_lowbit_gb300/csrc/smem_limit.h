// The dynamic shared-memory limits that kernels have been given.
//
// A kernel's limit is an attribute of the function on a device and stays as it was
// set last, so a call that set it to its own smaller size would take away what another
// thread's larger launch is about to use.  One entry a (device, kernel) holds the
// largest size, and only a larger one is set.  (Host code without CUDA headers: the
// caller passes the device and the function that sets a limit.)
#pragma once

#include <mutex>

namespace mlalb {

class SmemLimits {
 public:
  // Makes `kernel`'s limit on device `dev` at least `bytes`: set(bytes) when it is
  // not, whose result other than 0 is handed on and leaves the entry as it was.
  template <typename Set>
  int ensure(int dev, const void* kernel, int bytes, Set set) {
    std::lock_guard<std::mutex> lock(mu_);
    Entry* e = find(dev, kernel);
    if (e && e->bytes >= bytes) return 0;
    if (const int st = set(bytes)) return st;
    if (e)
      e->bytes = bytes;
    else if (count_ < kEntries)
      entries_[count_++] = Entry{dev, kernel, bytes};
    return 0;
  }

 private:
  struct Entry {
    int dev;
    const void* kernel;
    int bytes;
  };
  Entry* find(int dev, const void* kernel) {
    for (int i = 0; i < count_; ++i)
      if (entries_[i].dev == dev && entries_[i].kernel == kernel) return &entries_[i];
    return nullptr;
  }
  static constexpr int kEntries = 2048;  // a hundred and some kernels a device
  Entry entries_[kEntries];
  int count_ = 0;
  std::mutex mu_;
};

}  // namespace mlalb
