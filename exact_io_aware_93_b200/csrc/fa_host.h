// fa_host.h -- host-side state and checks shared by the sources of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "../../include/fa.h"

namespace fa {

constexpr int kMaxDevices = 64;

// Per-device set-up.  The first call on a device fills `ok`, `sm_count` and `status` under
// device_mutex() and only then publishes `probed` (release); later calls read `probed`
// (acquire) without the lock.  The kernel-attribute flags are set under the same mutex, so
// first calls from several host threads at once are safe.
struct DeviceInfo {
  std::atomic<bool> probed{false};
  bool ok = false;
  int sm_count = 0;
  int* status = nullptr;
  bool fwd_attr[3][2][2] = {};  // [element type][d==128][causal]
  bool bwd_attr[2][2][2] = {};
  bool dec_attr[2][2][4] = {};  // [fp16][d==128][M = 128; M = 64 with 1, 2, 4 row copies]
  bool paged_attr[2][2][2][3] = {};  // [fp16][e4m3 pages][d==128][tiles; 8, 16 rows]
};

// Defined in fa_api.cu.
std::mutex& device_mutex();
fa_status current_device(DeviceInfo** out);

// Runs `setup` (which returns true on success) once per flag, under device_mutex().
template <typename F>
bool once_per_device(bool& flag, F setup) {
  std::lock_guard<std::mutex> lock(device_mutex());
  if (!flag) {
    if (!setup()) {
      cudaGetLastError();
      return false;
    }
    flag = true;
  }
  return true;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The warp-specialised kernels move registers between warpgroups with setmaxnreg; the
// split is computed for a launch at exactly fa::kLaunchRegs registers per thread.  The
// build script fails when ptxas reports another count; this check refuses to launch a
// library that was built some other way with a different count.
template <typename K>
bool launch_regs_ok(K kern, uint32_t expected) {
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, kern) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.numRegs == static_cast<int>(expected);
}

}  // namespace fa
