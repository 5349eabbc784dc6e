// Compares the AdamW kernel's square root (minus_root2: an estimate and one
// Newton step) with the correctly rounded one for every fp32 value of a range
// of bit patterns, each in both places of the pair.  Built by
// tests/test_gpu_adamw_mixed.py.
#include <cuda_runtime.h>

#include "k_adamw_mixed.cuh"

using namespace muonb200;

__global__ void root_check(uint32_t first, uint32_t count, unsigned long long* bad) {
  const uint32_t stride = gridDim.x * blockDim.x;
  unsigned long long n = 0;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < count; i += stride) {
    const float v = __uint_as_float(first + i);
    const float2 r = minus_root2(make_float2(-v, -__uint_as_float(first + (count - 1 - i))));
    const float2 s = minus_root2(make_float2(-__uint_as_float(first + (count - 1 - i)), -v));
    const float want = -__fsqrt_rn(v);
    n += r.x != want;
    n += s.y != want;
  }
  if (n) atomicAdd(bad, n);
}

// Number of differing roots over patterns first .. first + count - 1, or -1.
extern "C" long long root_differences(uint32_t first, uint32_t count) {
  unsigned long long* bad = nullptr;
  unsigned long long host = 0;
  if (cudaMalloc(&bad, sizeof(host)) != cudaSuccess) return -1;
  cudaMemset(bad, 0, sizeof(host));
  root_check<<<148 * 8, 256>>>(first, count, bad);
  const bool ok =
      cudaMemcpy(&host, bad, sizeof(host), cudaMemcpyDeviceToHost) == cudaSuccess;
  cudaFree(bad);
  return ok ? static_cast<long long>(host) : -1;
}
