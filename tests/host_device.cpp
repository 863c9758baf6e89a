// Host-side helpers of pkv_internal.h against a CUDA runtime of two devices that
// is made up here: prints what they answer, one line each.
#include <cstdio>

#include "pkv_internal.h"

static int g_device = 0;
static cudaError_t g_get_device = cudaSuccess;

extern "C" cudaError_t cudaGetDevice(int* device) {
  *device = g_device;
  return g_get_device;
}

namespace pkv {
void record_cuda_error(cudaError_t e) { std::printf("recorded %d\n", static_cast<int>(e)); }
}  // namespace pkv

int main() {
  pkv_pool pool = {};
  for (pool.device = 0; pool.device < 2; ++pool.device)
    for (g_device = 0; g_device < 2; ++g_device)
      std::printf("pool on %d, current %d: %d\n", pool.device, g_device, pkv::check_pool_device(&pool));
  g_get_device = cudaErrorNoDevice;
  std::printf("no device: %d\n", pkv::check_pool_device(&pool));
  g_get_device = cudaSuccess;

  // a kernel's attributes are set once on each device, and again after a failure
  int calls[2] = {0, 0};
  cudaError_t answer = cudaErrorInvalidValue;
  pkv::DeviceSetup setup;
  for (int round = 0; round < 3; ++round, answer = cudaSuccess)
    for (g_device = 0; g_device < 2; ++g_device) {
      const int device = g_device;
      const cudaError_t e = setup([&] {
        ++calls[device];
        return answer;
      });
      std::printf("set-up %d on %d: %d, set %d times\n", round, device, static_cast<int>(e), calls[device]);
    }
}
