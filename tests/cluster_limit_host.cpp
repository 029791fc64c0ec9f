// csrc/launch.cuh's ClusterLimit over fakes of the two CUDA calls it makes, for the tests.
#include <cstddef>

#include "launch.cuh"

// (linked with -Bsymbolic: a CUDA runtime may be in the process)
static int g_device, g_get_error, g_error, g_answer, g_calls, g_ctas, g_threads;
static size_t g_smem;

extern "C" {

cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return static_cast<cudaError_t>(g_get_error);
}

cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* cfg) {
  ++g_calls;
  g_ctas = static_cast<int>(cfg->attrs[0].val.clusterDim.x);
  g_threads = static_cast<int>(cfg->blockDim.x);
  g_smem = cfg->dynamicSmemBytes;
  *n = g_answer;
  return static_cast<cudaError_t>(g_error);
}

// One call on `device` whose fakes return these errors and this answer; out: the answer given and the calls made since the start.
int ask(int device, int get_error, int error, int answer, int* out) {
  static llama::ClusterLimit limit;
  g_device = device;
  g_get_error = get_error;
  g_error = error;
  g_answer = answer;
  out[0] = -1;
  const int e = limit.get(&g_device, 4, 192, 1000, out);
  out[1] = g_calls;
  return g_calls && (g_ctas != 4 || g_threads != 192 || g_smem != 1000) ? -1 : e;
}
}
