// K-NORM: the Euclidean norm of many gradient tensors taken together, and the
// coefficient that brings it to a maximum:
//
//   norm = sqrt(sum of all g^2);  c = min(1, max_norm / (norm + 1e-6)),
//   c = NaN when some gradient is not finite
//
// Squares are taken and added in 64 bits: no finite gradient overflows or
// vanishes, and the sum over 10^9 elements is good to more digits than the
// fp32 result holds.  Every block writes its sum to its own slot and the last
// one to finish (a ticket) adds the slots in a fixed order: the same bits on
// every run.  Tensors past one launch's table go into further launches, each
// adding its sum to the workspace's carry.
//
// Context: PR #1893 "Record: L_ParallelResiduals_UNetSkips_DepthRecur_Muon_
// 1.0901", table "Architecture and training stack"; the pages print no
// clipping rule, the formula is the usual one of clipping by a global norm.
#pragma once

#include <cstdint>

#include "k_adamw_mixed.cuh"

namespace muonb200 {

constexpr int kNormThreads = 256;
constexpr int kNormMaxSegs = 1300;    // 1300 x 24 bytes of kernel parameters
constexpr int kNormMaxGrid = 2048;

struct NormSeg {
  const void* g;
  long long numel;
  uint32_t ubeg;
  uint32_t flags;    // kMixGradBf16, kMixVec
};
static_assert(sizeof(NormSeg) == 24, "kNormMaxSegs counts on 24 bytes");

struct NormWorkspace {
  unsigned ticket;   // 0 between calls
  unsigned pad;
  double carry;
  double part[kNormMaxGrid];
};

template <int kSegs>
struct NormParams {
  NormSeg seg[kSegs];
  NormWorkspace* ws;
  float* out;               // norm, coefficient
  double max_norm;
  uint32_t n_seg, n_units;
  int32_t first, last;      // first / last launch of the call
};

__device__ __forceinline__ double block_sum(double x, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) x += sh[w];
  return x;
}

template <int kSegs>
__global__ void __launch_bounds__(kNormThreads)
grad_norm_kernel(const __grid_constant__ NormParams<kSegs> a) {
  __shared__ double sh[2][kNormThreads / 32];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31;
  const uint32_t stride = gridDim.x * (kNormThreads / 32);
  uint32_t u = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  double sum = 0.0;
  if (u < a.n_units) {
    uint32_t cur = find_seg(a.seg, a.n_seg, u);
    for (; u < a.n_units; u += stride) {
      while (cur + 1 < a.n_seg && u >= a.seg[cur + 1].ubeg) ++cur;
      const NormSeg& s = a.seg[cur];
      const long long i0 = static_cast<long long>(u - s.ubeg) * kA8Block;
      const long long left = s.numel - i0;
      const bool vec = (s.flags & kMixVec) && left >= kA8Block;
      const bool g16 = s.flags & kMixGradBf16;
      float g[8];
      if (vec) {
        const long long iv = i0 + lane * 8;
        if (g16) unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(
                                   static_cast<const uint16_t*>(s.g) + iv)), g);
        else load_f32x8(static_cast<const float*>(s.g) + iv, g);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = k * 32 + lane;
          g[k] = j >= left ? 0.f
                 : g16     ? __uint_as_float(static_cast<uint32_t>(
                             static_cast<const uint16_t*>(s.g)[i0 + j]) << 16)
                           : static_cast<const float*>(s.g)[i0 + j];
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fma(static_cast<double>(g[k]), static_cast<double>(g[k]), sum);
    }
  }
  sum = block_sum(sum, sh[0]);
  if (threadIdx.x == 0) {
    a.ws->part[blockIdx.x] = sum;
    __threadfence();
    s_last = atomicInc(&a.ws->ticket, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double t = 0.0;
  for (unsigned b = threadIdx.x; b < gridDim.x; b += kNormThreads) t += __ldcg(&a.ws->part[b]);
  t = block_sum(t, sh[1]);
  if (threadIdx.x == 0) {
    if (!a.first) t += a.ws->carry;
    if (!a.last) {
      a.ws->carry = t;
    } else {
      const double norm = sqrt(t);
      a.out[0] = static_cast<float>(norm);
      a.out[1] = isfinite(t) ? static_cast<float>(fmin(1.0, a.max_norm / (norm + 1e-6)))
                             : __uint_as_float(0x7fc00000u);
    }
  }
}

}  // namespace muonb200
