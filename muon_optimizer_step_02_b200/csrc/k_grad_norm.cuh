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
// Bound by memory: 4 or 2 bytes per element.  A thread block's loads are
// written four chunks of 2,048 elements ahead of their use (two: 77 us, eight:
// 60 us on the first figure below; small gradients come in more even shares
// with fewer).  For bf16 those are 16 registers of data, all in flight at once;
// for fp32 they would be 32, as many as a thread has here, so not all can
// be, and 8 bytes are spilled (4 thread blocks per SM, 64 registers: none).  The
// conversions to 64 bits fill 71 % of their pipe at that rate and the GPU's
// power limit lowers the clock when the call runs on end.  184 M bf16
// gradients: 60 us (6.1 TB/s, 0.94 of the measured copy bandwidth), 69 us on
// end; 67 M fp32: 43 us (6.2 TB/s).
//
// Context: PR #1893 "Record: L_ParallelResiduals_UNetSkips_DepthRecur_Muon_
// 1.0901", table "Architecture and training stack"; the pages print no
// clipping rule, the formula is the usual one of clipping by a global norm.
#pragma once

#include <cstdint>

#include "k_adamw_mixed.cuh"

namespace muonb200 {

constexpr int kNormThreads = 256;
constexpr int kNormChunk = kNormThreads * 8;
constexpr int kNormDeep = 4;          // chunks of a unit
constexpr int kNormUnit = kNormDeep * kNormChunk;
constexpr int kNormResident = 8;      // thread blocks per SM (32 registers, 8 bytes spilled)
constexpr int kNormMaxSegs = 1300;    // 1300 x 20 bytes of kernel parameters
constexpr int kNormMaxGrid = 2048;

// A tensor from its first 16-byte boundary on, and the up to 7 elements before
// it, which are taken apart (squares may be added in any order).
struct NormSeg {
  const void* g;
  unsigned long long numel;   // from g on; their number before g (kSegPlace), kSegBf16
};

struct NormWorkspace {
  unsigned ticket;   // 0 between calls
  unsigned pad;
  double carry;
  double part[kNormMaxGrid];
};

template <int kSegs>
struct NormParams {
  NormSeg seg[kSegs];
  uint32_t ubeg[kSegs + 1];  // first unit of each tensor in the launch, and the end
  uint32_t n_seg;
  NormWorkspace* ws;
  float* out;               // norm, coefficient
  double max_norm;
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

__device__ __forceinline__ void add_squares(const float2 (&g)[4], double (&sum)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const double x = static_cast<double>(g[k].x), y = static_cast<double>(g[k].y);
    sum[k] = fma(x, x, sum[k]);
    sum[k] = fma(y, y, sum[k]);
  }
}

// kCount whole chunks of a gradient from element i0 on, requested before the
// first is used as far as registers allow.
template <int kCount, bool kG16>
__device__ __forceinline__ void add_chunks(const void* g, long long i0, double (&sum)[4]) {
  float2 x[4];
  if (kG16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + i0) +
                     threadIdx.x;
    uint4 raw[kCount];
#pragma unroll
    for (int c = 0; c < kCount; ++c) raw[c] = __ldcs(p + c * kNormThreads);
#pragma unroll
    for (int c = 0; c < kCount; ++c) {
      unpack8(raw[c], x);
      add_squares(x, sum);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(g) + i0) +
                      threadIdx.x;
    float4 raw[2 * kCount];
#pragma unroll
    for (int c = 0; c < 2 * kCount; ++c) raw[c] = __ldcs(p + c * kNormThreads);
#pragma unroll
    for (int c = 0; c < kCount; ++c) {
      x[0] = make_float2(raw[2 * c].x, raw[2 * c].y);
      x[1] = make_float2(raw[2 * c].z, raw[2 * c].w);
      x[2] = make_float2(raw[2 * c + 1].x, raw[2 * c + 1].y);
      x[3] = make_float2(raw[2 * c + 1].z, raw[2 * c + 1].w);
      add_squares(x, sum);
    }
  }
}

template <int kSegs>
__global__ void __launch_bounds__(kNormThreads, kNormResident)
grad_norm_kernel(const __grid_constant__ NormParams<kSegs> a) {
  __shared__ double sh[2][kNormThreads / 32];
  __shared__ bool s_last;
  const uint32_t n_units = a.ubeg[a.n_seg];
  uint32_t cur = 0, end = 0;
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  grid_launch_dependents();
  grid_dependency_wait();
  for (uint32_t u = blockIdx.x; u < n_units; u += gridDim.x) {
    if (u >= end) {
      cur = find_seg(a.ubeg, a.n_seg, u);
      end = a.ubeg[cur + 1];
    }
    const NormSeg& s = a.seg[cur];
    long long i0 = static_cast<long long>(u - a.ubeg[cur]) * kNormUnit;
    long long left = static_cast<long long>(s.numel & kSegNumel) - i0;
    const bool g16 = (s.numel & kSegBf16) != 0;
    if (left >= kNormUnit) {
      if (g16) add_chunks<kNormDeep, true>(s.g, i0, sum);
      else add_chunks<kNormDeep, false>(s.g, i0, sum);
      continue;
    }
    // a tensor's last unit: chunk by chunk
    for (int c = 0; c < kNormDeep && left > 0; ++c, i0 += kNormChunk, left -= kNormChunk) {
      if (left >= kNormChunk) {
        if (g16) add_chunks<1, true>(s.g, i0, sum);
        else add_chunks<1, false>(s.g, i0, sum);
        continue;
      }
      float2 g[4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k * kNormThreads + threadIdx.x;
        at(g, k) = j >= left ? 0.f
                   : g16     ? bf16_at(s.g, i0 + j)
                             : static_cast<const float*>(s.g)[i0 + j];
      }
      add_squares(g, sum);
    }
  }
  double total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  for (uint32_t c = blockIdx.x; c < a.n_seg; c += gridDim.x) {
    const NormSeg& s = a.seg[c];
    const uint32_t before = static_cast<uint32_t>(s.numel >> kSegPlace) & 7u;
    if (threadIdx.x < before) {
      const long long i = static_cast<long long>(threadIdx.x) - before;
      const double x = static_cast<double>(
          s.numel & kSegBf16 ? bf16_at(s.g, i) : static_cast<const float*>(s.g)[i]);
      total = fma(x, x, total);
    }
  }
  total = block_sum(total, sh[0]);
  if (threadIdx.x == 0) {
    a.ws->part[blockIdx.x] = total;
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
