// Host helpers shared by libg4's translation units: CUDA error text, the device guard and
// kernel launches.
#pragma once
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <string>

#include "../../include/g4.h"

namespace g4 {

extern thread_local std::string g_last_cuda;  // g4_last_cuda_error's text

inline bool cuda_ok(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return true;
  char buf[512];
  snprintf(buf, sizeof buf, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  try {
    g_last_cuda = buf;
  } catch (...) {  // no memory for the text: no exception may leave a C entry
    g_last_cuda.clear();
  }
  return false;
}
#define CK(call)                                           \
  do {                                                     \
    if (!cuda_ok((call), #call)) return G4_ERR_CUDA;       \
  } while (0)
#define TRY(x)                          \
  do {                                  \
    g4_status s_ = (x);                 \
    if (s_ != G4_OK) return s_;         \
  } while (0)

// Makes `dev` current for the guard's lifetime and gives the caller's current device back
// afterwards, so no entry point changes the calling thread's device.
struct DeviceGuard {
  int prev = -1, dev = -1;
  cudaError_t err = cudaSuccess;
  explicit DeviceGuard(int d) : dev(d) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) err = cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  }
};
#define DEVICE_GUARD(d)   \
  DeviceGuard dg_guard_(d); \
  CK(dg_guard_.err)

inline int cdiv(int a, int b) { return (a + b - 1) / b; }

// Programmatic dependent launch for every kernel of the step (G4_PDL=0 disables it).
inline bool pdl_enabled() {
  static const bool on = [] {
    const char* e = getenv("G4_PDL");
    return !(e && e[0] == '0');
  }();
  return on;
}

template <typename... KArgs, typename... Args>
void launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kern, args...);
}

// Every kernel of a step prefers the largest shared-memory carve-out.  Under programmatic
// dependent launch the next kernel's CTAs become resident while the current kernel runs and
// stream their weights in; an SM configured for a smaller carve-out can take a CTA that needs
// more shared memory only after it drains, which delays that CTA (and its weight loads) to
// the end of the current kernel.  With one carve-out for all kernels any mix of CTAs fits.
template <typename... KArgs>
void carve_max(void (*k)(KArgs...)) {
  cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
}
// Opt every kernel into the full shared-memory carve-out once per process (never during a
// stream capture).
template <typename... KArgs>
void set_max_dyn(void (*k)(KArgs...), int optin) {
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, k) != cudaSuccess) return;
  cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - (int)fa.sharedSizeBytes);
  carve_max(k);
}

}  // namespace g4
