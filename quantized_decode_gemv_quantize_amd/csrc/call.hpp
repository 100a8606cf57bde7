// call.hpp - what the entry points around the mat-vecs share: limits, the
// alignment test and the device of a call's stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmv {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRow = int64_t(1) << 24;

// The stream's device current for the launch, as the kernels and their
// arguments belong to it.
class OnStreamDevice {
 public:
  explicit OnStreamDevice(hipStream_t st) {
    hipDevice_t dev;
    if (!st || hipStreamGetDevice(st, &dev) != hipSuccess) return;
    int now = 0;
    if (hipGetDevice(&now) != hipSuccess || now == dev) return;
    if (hipSetDevice(dev) == hipSuccess) back_ = now;
  }
  ~OnStreamDevice() {
    if (back_ >= 0) (void)hipSetDevice(back_);
  }
  OnStreamDevice(const OnStreamDevice&) = delete;
  OnStreamDevice& operator=(const OnStreamDevice&) = delete;

 private:
  int back_ = -1;
};

}  // namespace qmv
