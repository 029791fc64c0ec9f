// csrc/launch.cuh's SmemLimits over fakes of the two CUDA calls it makes, for the tests.
#include <cstddef>

#include "launch.cuh"

// (linked with -Bsymbolic: a CUDA runtime may be in the process)
static int g_device, g_error, g_get_error, g_calls[128];

extern "C" {

cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return static_cast<cudaError_t>(g_get_error);
}

cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  ++g_calls[g_device];
  return static_cast<cudaError_t>(g_error);
}

// One call on `device` whose fakes return these errors; *calls: attributes set on that device since the start.
int raise_on(int device, int get_error, int set_error, int* calls) {
  static llama::SmemLimits limits;
  g_device = device;
  g_get_error = get_error;
  g_error = set_error;
  const int e = limits.raise({{&g_device, 1000}, {&g_error, 2000}});
  *calls = g_calls[device];
  return e;
}
}
