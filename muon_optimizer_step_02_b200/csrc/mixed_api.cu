// C ABI of the AdamW step with 32-bit or 8-bit moments, the global gradient
// norm and the conversions of the 8-bit states (include/muon_b200.h):
// argument validation and the launches.  Nothing is allocated and no call
// synchronises.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>

#include "muon_b200.h"

#include "k_adamw_mixed.cuh"
#include "k_grad_norm.cuh"

using namespace muonb200;

namespace {

constexpr int64_t kMaxElements = int64_t{1} << 39;   // of one call: blocks count in 32 bits
constexpr int kFewSegs = 16;   // launches of few tensors carry a short table

// The kernel's division takes a denominator below fp32's normal range for 0,
// which an eps down there would leave of elements without moments.
constexpr double kLeastEps = 0x1p-126;

// The kernels take settings in fp32.
inline bool finite32(double x) { return std::isfinite(static_cast<float>(x)); }

inline uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

inline uint32_t units_of(int64_t numel, int unit) {
  return static_cast<uint32_t>((numel + unit - 1) / unit);
}

inline unsigned long long flagged(int64_t numel, bool bf16, bool vec) {
  return static_cast<unsigned long long>(numel) | (bf16 ? kSegBf16 : 0) | (vec ? kSegVec : 0);
}

inline muon_status_t sm_count(int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MUON_ERR_CUDA;
  return MUON_OK;
}

// At least one thread block, so that an empty call still advances its counter
// or writes its norm.
inline unsigned grid_for(uint32_t units, int sms, int blocks_per_sm) {
  return std::max(1u, std::min(units, static_cast<unsigned>(blocks_per_sm * sms)));
}

inline float2 twice(double x) {
  return make_float2(static_cast<float>(x), static_cast<float>(x));
}

// Launched as a programmatic dependent of whatever runs before it on the
// stream: its thread blocks may be set up while that ends (the kernels wait for
// its completion before they touch memory).
template <class P>
muon_status_t launch(void (*kernel)(P), const P& params, unsigned grid, int threads,
                     cudaStream_t st) {
  void* args[] = {const_cast<P*>(&params)};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args) != cudaSuccess) {
    cudaGetLastError();
    return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

template <int kSegs>
muon_status_t mixed_launch(const adamw_mixed_tensor_t* x, int first, int n,
                           const adamw_mixed_hyper_t& h, int32_t step, int32_t* step_dev,
                           const float* lr_dev, const float* coef_dev, bool advance, int sms,
                           cudaStream_t st) {
  MixParams<kSegs> a;
  a.step_dev = step_dev;
  a.lr_dev = lr_dev;
  a.coef_dev = coef_dev;
  a.step = step;
  a.key = mix32(mix32(static_cast<uint32_t>(h.seed)) ^ static_cast<uint32_t>(h.seed >> 32));
  a.first_tensor = static_cast<uint32_t>(first);
  a.advance = advance ? 1 : 0;
  a.lr = static_cast<float>(h.lr);
  a.b1 = twice(h.beta1);
  a.omb1 = twice(1.0 - h.beta1);
  a.minus_b2 = twice(-h.beta2);
  a.minus_omb2 = twice(-(1.0 - h.beta2));
  a.eps = twice(h.eps);
  a.wd = static_cast<float>(h.weight_decay);
  a.d = twice(h.ema_decay);
  a.omd = twice(1.0 - h.ema_decay);
  a.one = 1.f;
  a.pow1[0] = h.beta1;
  a.pow2[0] = h.beta2;
  for (int j = 1; j < 31; ++j) {
    a.pow1[j] = a.pow1[j - 1] * a.pow1[j - 1];
    a.pow2[j] = a.pow2[j - 1] * a.pow2[j - 1];
  }
  uint32_t units = 0;
  int k = 0;
  for (int eight = 1; eight >= 0; --eight) {
    for (int i = 0; i < n; ++i) {
      const adamw_mixed_tensor_t& t = x[first + i];
      if ((t.scale != nullptr) != (eight == 1)) continue;
      const uintptr_t wide = bits(t.param) | bits(t.ema);
      const bool g16 = t.grad_dtype == MUON_BF16;
      const uintptr_t codes = bits(t.exp_avg) | bits(t.exp_avg_sq);
      const uintptr_t halves = bits(t.copy_bf16) | (g16 ? bits(t.grad) : 0);
      const bool vec = ((wide | (eight ? 0 : codes) | (g16 ? 0 : bits(t.grad))) & 31u) == 0 &&
                       (halves & 15u) == 0 && (codes & 7u) == 0 && (bits(t.scale) & 1u) == 0;
      a.seg[k] = MixSeg{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.scale, t.ema, t.copy_bf16,
                        flagged(t.numel, g16, vec) |
                            static_cast<unsigned long long>(i) << kSegPlace,
                        t.lr_scale, t.wd_scale};
      a.ubeg[k++] = units;
      units += units_of(t.numel, kMixUnit);
    }
    if (eight) a.units8 = units;
  }
  a.n_seg = static_cast<uint32_t>(n);
  a.ubeg[n] = units;
  const unsigned grid = grid_for(units, sms, kMixResident);
  return h.rounding == MUON_ROUND_STOCHASTIC
             ? launch(adamw_mixed_kernel<true, kSegs>, a, grid, kMixThreads, st)
             : launch(adamw_mixed_kernel<false, kSegs>, a, grid, kMixThreads, st);
}

template <int kSegs>
muon_status_t norm_launch(const grad_tensor_t* x, int n, double max_norm, NormWorkspace* ws,
                          float* out, bool first, bool last, int sms, cudaStream_t st) {
  NormParams<kSegs> a;
  a.ws = ws;
  a.out = out;
  a.max_norm = max_norm;
  a.first = first ? 1 : 0;
  a.last = last ? 1 : 0;
  uint32_t units = 0;
  for (int i = 0; i < n; ++i) {
    const bool g16 = x[i].dtype == MUON_BF16;
    const int size = g16 ? 2 : 4;
    const int64_t before = std::min<int64_t>(
        x[i].numel, static_cast<int64_t>((-bits(x[i].grad) & 15u) / size));
    const int64_t from = x[i].numel - before;
    a.seg[i] = NormSeg{static_cast<const char*>(x[i].grad) + before * size,
                       flagged(from, g16, false) |
                           static_cast<unsigned long long>(before) << kSegPlace};
    a.ubeg[i] = units;
    // (one unit at least, so that many small tensors spread over the grid)
    units += x[i].numel > 0 ? std::max(1u, units_of(from, kNormUnit)) : 0u;
  }
  a.n_seg = static_cast<uint32_t>(n);
  a.ubeg[n] = units;
  const unsigned grid = std::min<unsigned>(grid_for(units, sms, kNormResident), kNormMaxGrid);
  return launch(grad_norm_kernel<kSegs>, a, grid, kNormThreads, st);
}

template <int kSegs>
muon_status_t adam8_launch(const adam8_tensor_t* x, int n, int32_t dtype, bool write, int sms,
                           cudaStream_t st) {
  A8Params<kSegs> a;
  uint32_t units = 0;
  for (int i = 0; i < n; ++i) {
    const adam8_tensor_t& t = x[i];
    const bool vec =
        ((bits(t.exp_avg) | bits(t.second)) & (dtype == MUON_BF16 ? 15u : 31u)) == 0 &&
        ((bits(t.exp_avg8) | bits(t.root8)) & 7u) == 0;
    a.seg[i] = A8Seg{t.exp_avg8, t.root8, t.scale, t.exp_avg, t.second,
                     flagged(t.numel, dtype == MUON_BF16, vec)};
    a.ubeg[i] = units;
    units += units_of(t.numel, kMixUnit);
  }
  if (units == 0) return MUON_OK;
  a.n_seg = static_cast<uint32_t>(n);
  a.ubeg[n] = units;
  const unsigned grid = grid_for(units, sms, write ? kA8WriteResident : kA8ReadResident);
  return write ? launch(adam8_write_kernel<kSegs>, a, grid, kMixThreads, st)
               : launch(adam8_read_kernel<kSegs>, a, grid, kMixThreads, st);
}

muon_status_t adam8_convert(const adam8_tensor_t* tensors, int32_t n_tensors, int32_t dtype,
                            bool write, muon_stream_t stream) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return MUON_ERR_INVALID_ARG;
  if (dtype != MUON_F32 && dtype != MUON_BF16) return MUON_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const adam8_tensor_t& t = tensors[i];
    if (t.numel < 0) return MUON_ERR_INVALID_ARG;
    if (t.numel == 0) continue;
    if (!t.exp_avg8 || !t.root8 || !t.scale || !t.exp_avg || !t.second)
      return MUON_ERR_INVALID_ARG;
    if ((bits(t.exp_avg) | bits(t.second)) & (dtype == MUON_BF16 ? 1u : 3u))
      return MUON_ERR_ALIGNMENT;
    if (t.numel > kMaxElements - total) return MUON_ERR_UNSUPPORTED;
    total += t.numel;
  }
  if (total == 0) return MUON_OK;
  int sms = 0;
  if (sm_count(sms) != MUON_OK) return MUON_ERR_CUDA;
  nvtxRangePushA(write ? "muon.adam8_write" : "muon.adam8_read");
  muon_status_t rc = MUON_OK;
  for (int first = 0; first < n_tensors && rc == MUON_OK; first += kA8MaxSegs) {
    const int n = std::min(n_tensors - first, kA8MaxSegs);
    rc = n <= kFewSegs
             ? adam8_launch<kFewSegs>(tensors + first, n, dtype, write, sms,
                                      static_cast<cudaStream_t>(stream))
             : adam8_launch<kA8MaxSegs>(tensors + first, n, dtype, write, sms,
                                        static_cast<cudaStream_t>(stream));
  }
  nvtxRangePop();
  return rc;
}

}  // namespace

extern "C" {

muon_status_t adamw_mixed_batched(const adamw_mixed_tensor_t* tensors, int32_t n_tensors,
                                  const adamw_mixed_hyper_t* hyper, int32_t step,
                                  int32_t* step_dev, const float* lr_dev,
                                  const float* coef_dev, muon_stream_t stream) {
  if (n_tensors < 0 || !hyper || (n_tensors > 0 && !tensors)) return MUON_ERR_INVALID_ARG;
  const adamw_mixed_hyper_t& h = *hyper;
  if (!finite32(h.lr) || !finite32(h.weight_decay) || !std::isfinite(h.eps) ||
      !finite32(h.ema_decay) || !(h.beta1 >= 0.0 && h.beta1 < 1.0) ||
      !(h.beta2 >= 0.0 && h.beta2 < 1.0))
    return MUON_ERR_INVALID_ARG;
  if (h.eps != 0.0 && !(h.eps >= kLeastEps))
    return MUON_ERR_INVALID_ARG;
  if (h.rounding != MUON_ROUND_NEAREST && h.rounding != MUON_ROUND_STOCHASTIC)
    return MUON_ERR_INVALID_ARG;
  if (!step_dev && step < 1) return MUON_ERR_INVALID_ARG;
  if ((bits(step_dev) | bits(lr_dev) | bits(coef_dev)) & 3u) return MUON_ERR_ALIGNMENT;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const adamw_mixed_tensor_t& t = tensors[i];
    if (t.numel < 0 || (t.grad_dtype != MUON_F32 && t.grad_dtype != MUON_BF16) ||
        !std::isfinite(t.lr_scale) || !std::isfinite(t.wd_scale))
      return MUON_ERR_INVALID_ARG;
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return MUON_ERR_INVALID_ARG;
    if (((bits(t.param) | bits(t.ema)) & 3u) || (bits(t.copy_bf16) & 1u) ||
        (bits(t.grad) & (t.grad_dtype == MUON_BF16 ? 1u : 3u)) ||
        (!t.scale && ((bits(t.exp_avg) | bits(t.exp_avg_sq)) & 3u)))
      return MUON_ERR_ALIGNMENT;
    if (t.numel > kMaxElements - total) return MUON_ERR_UNSUPPORTED;
    total += t.numel;
  }
  if (total == 0 && !step_dev) return MUON_OK;
  int sms = 0;
  if (sm_count(sms) != MUON_OK) return MUON_ERR_CUDA;
  nvtxRangePushA("muon.adamw_mixed");
  muon_status_t rc = MUON_OK;
  int first = 0;
  do {
    const int n = std::min(n_tensors - first, kMixMaxSegs);
    const bool advance = step_dev && first + n == n_tensors;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = n <= kFewSegs ? mixed_launch<kFewSegs>(tensors, first, n, h, step, step_dev, lr_dev,
                                                coef_dev, advance, sms, st)
                       : mixed_launch<kMixMaxSegs>(tensors, first, n, h, step, step_dev, lr_dev,
                                                   coef_dev, advance, sms, st);
    first += n;
  } while (first < n_tensors && rc == MUON_OK);
  nvtxRangePop();
  return rc;
}

size_t grad_norm_workspace_bytes(void) { return sizeof(NormWorkspace); }

muon_status_t grad_norm_batched(const grad_tensor_t* tensors, int32_t n_tensors,
                                double max_norm, void* workspace, size_t workspace_bytes,
                                float* out, muon_stream_t stream) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !out || !(max_norm > 0.0))
    return MUON_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < sizeof(NormWorkspace) || (bits(workspace) & 15u))
    return MUON_ERR_WORKSPACE;
  if (bits(out) & 3u) return MUON_ERR_ALIGNMENT;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const grad_tensor_t& t = tensors[i];
    if (t.numel < 0 || (t.dtype != MUON_F32 && t.dtype != MUON_BF16)) return MUON_ERR_INVALID_ARG;
    if (t.numel == 0) continue;
    if (!t.grad) return MUON_ERR_INVALID_ARG;
    if (bits(t.grad) & (t.dtype == MUON_BF16 ? 1u : 3u)) return MUON_ERR_ALIGNMENT;
    if (t.numel > kMaxElements - total) return MUON_ERR_UNSUPPORTED;
    total += t.numel;
  }
  int sms = 0;
  if (sm_count(sms) != MUON_OK) return MUON_ERR_CUDA;
  nvtxRangePushA("muon.grad_norm");
  muon_status_t rc = MUON_OK;
  int first = 0;
  do {
    const int n = std::min(n_tensors - first, kNormMaxSegs);
    NormWorkspace* ws = static_cast<NormWorkspace*>(workspace);
    const bool last = first + n == n_tensors;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = n <= kFewSegs ? norm_launch<kFewSegs>(tensors + first, n, max_norm, ws, out, first == 0,
                                               last, sms, st)
                       : norm_launch<kNormMaxSegs>(tensors + first, n, max_norm, ws, out,
                                                   first == 0, last, sms, st);
    first += n;
  } while (first < n_tensors && rc == MUON_OK);
  nvtxRangePop();
  return rc;
}

muon_status_t adam8_write_batched(const adam8_tensor_t* tensors, int32_t n_tensors,
                                  int32_t dtype, muon_stream_t stream) {
  return adam8_convert(tensors, n_tensors, dtype, true, stream);
}

muon_status_t adam8_read_batched(const adam8_tensor_t* tensors, int32_t n_tensors,
                                 int32_t dtype, muon_stream_t stream) {
  return adam8_convert(tensors, n_tensors, dtype, false, stream);
}

static int32_t launches_of(int32_t n_tensors, int32_t per) {
  return n_tensors <= 0 ? 1 : (n_tensors - 1) / per + 1;
}

int32_t adamw_mixed_launches(int32_t n_tensors) { return launches_of(n_tensors, kMixMaxSegs); }
int32_t grad_norm_launches(int32_t n_tensors) { return launches_of(n_tensors, kNormMaxSegs); }
int32_t adam8_launches(int32_t n_tensors) {
  return n_tensors <= 0 ? 0 : launches_of(n_tensors, kA8MaxSegs);
}

}  // extern "C"
