// smem_table.h - which kernels have had their dynamic shared memory limit raised, per device. Plain C++: no CUDA.
#pragma once

namespace favor {

// The largest limit set so far for each (kernel, device). The library has some 60 kernels; a kernel takes one row
// whatever the number of devices, so that a process that uses them all still finds every one.
class SmemTable {
 public:
  static constexpr int kKernels = 128, kDevices = 64;
  bool known(const void* kernel, int dev, int bytes) const {
    if (dev < 0 || dev >= kDevices) return false;
    for (int i = 0; i < n_; ++i)
      if (rows_[i].kernel == kernel) return rows_[i].bytes[dev] >= bytes;
    return false;
  }
  void set(const void* kernel, int dev, int bytes) {
    if (dev < 0 || dev >= kDevices) return;
    int i = 0;
    while (i < n_ && rows_[i].kernel != kernel) ++i;
    if (i == kKernels) return;
    if (i == n_) rows_[n_++].kernel = kernel;
    rows_[i].bytes[dev] = bytes;
  }

 private:
  struct Row {
    const void* kernel = nullptr;
    int bytes[kDevices] = {};
  };
  Row rows_[kKernels];
  int n_ = 0;
};

}  // namespace favor
