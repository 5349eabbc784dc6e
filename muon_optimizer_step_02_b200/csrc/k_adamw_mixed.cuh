// K-MIXED: the AdamW step of many tensors with 32-bit or 8-bit moments, from
// fp32 or bf16 gradients, with the EMA and a bf16 copy of the new values:
//
//   g  = c G                         c: clip coefficient, or 1
//   m' = b1 m + (1 - b1) g;  v' = b2 v + (1 - b2) g^2;  r' = sqrt(v')
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (r' / sqrt(1 - b2^t) + eps)
//   e' = d e + (1 - d) p';   copy = bf16(p')
//
// The update uses the new moments before they are rounded to 8 bits (k_adam8.cuh
// has the codes), so that a step's own rounding reaches the weights only
// through the next step's state.  The operations that lead to m', v' and r'
// are rounded one by one in the order written (no fused multiply-add), so
// that the codes are a definite function of the inputs that a plain program
// in 32 bits reproduces bit for bit.
//
// A coefficient that is not finite (some gradient was not) skips the step:
// nothing is written and the device's step count stays.
//
// Source: PR #1893 "Record: L_ParallelResiduals_UNetSkips_DepthRecur_Muon_
// 1.0901", table "Architecture and training stack", rows "Optimizer" (AdamW
// on embeddings/scalars) and "EMA"; the page gives no setting and no state
// format.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "k_adam8.cuh"

namespace muonb200 {

constexpr int kMixThreads = 256;
constexpr int kMixMaxSegs = 400;      // 400 x 80 bytes of kernel parameters (limit 32,764)

constexpr uint32_t kMixGradBf16 = 1;  // gradient is bf16
constexpr uint32_t kMixVec = 2;       // every array is aligned for 8-element accesses

struct MixSeg {
  float* p;
  const void* g;
  void* m;           // fp32, or codes
  void* v;           // fp32, or codes of the root
  uint8_t* s;        // scale bytes (m, r) per block; null: fp32 moments
  float* e;          // null: no EMA
  uint16_t* c;       // null: no bf16 copy
  long long numel;
  uint32_t ubeg;     // first block of this tensor in the launch's block space
  uint32_t flags;
  float lr_scale, wd_scale;
};
static_assert(sizeof(MixSeg) == 80, "kMixMaxSegs counts on 80 bytes");

template <int kSegs>
struct MixParams {
  MixSeg seg[kSegs];
  int32_t* step_dev;        // [0] steps taken, [1] ticket; or null
  const float* lr_dev;      // or null
  const float* coef_dev;    // or null
  double beta1, beta2;
  int32_t step;             // t when step_dev is null
  uint32_t key;             // random key before the step number
  uint32_t n_seg, n_units, first_tensor;
  int32_t advance;          // this launch advances *step_dev
  float lr, b1, omb1, b2, omb2, eps, wd, d, omd;
};

// b^t by squaring: the same products on the host and on the device.
__host__ __device__ inline double pow_int(double b, uint32_t t) {
  double r = 1.0;
  for (; t; t >>= 1) {
    if (t & 1u) r *= b;
    b *= b;
  }
  return r;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load_f32x8(const float* p, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void store_f32x8(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  uint4 o;
  uint32_t* w = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return o;
}

constexpr float kMixRootLow = 0x1p-49f, kMixRootHigh = 0x1p63f;

__device__ __forceinline__ float scaled_root(float r, float g, float b2, float omb2, float up,
                                             float down) {
  const float rs = __fmul_rn(r, up), gs = __fmul_rn(g, up);
  const float v = __fadd_rn(__fmul_rn(__fmul_rn(rs, rs), b2),
                            __fmul_rn(__fmul_rn(gs, gs), omb2));
  return __fmul_rn(__fsqrt_rn(v), down);
}

// Last segment whose first block is at or before u.
template <class Seg>
__device__ __forceinline__ uint32_t find_seg(const Seg* seg, uint32_t n, uint32_t u) {
  uint32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if (seg[mid].ubeg <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One warp per block of 256 elements.  Full blocks of aligned tensors move 8
// consecutive elements per lane (16-byte accesses, 8-byte ones of codes);
// others element by element, lane l taking l, l + 32, ...
template <bool kStochastic, int kSegs>
__global__ void __launch_bounds__(kMixThreads)
adamw_mixed_kernel(const __grid_constant__ MixParams<kSegs> a) {
  __shared__ float s_bc[2];
  __shared__ uint32_t s_t;
  if (threadIdx.x < 32) {
    const uint32_t t = a.step_dev ? static_cast<uint32_t>(*a.step_dev) + 1u
                                  : static_cast<uint32_t>(a.step);
    const double pw = pow_int(threadIdx.x == 0 ? a.beta1 : a.beta2, t);
    const double bc = 1.0 / (1.0 - pw);
    if (threadIdx.x == 0) { s_bc[0] = static_cast<float>(bc); s_t = t; }
    if (threadIdx.x == 1) s_bc[1] = static_cast<float>(sqrt(bc));
  }
  const float coef = a.coef_dev ? *a.coef_dev : 1.f;
  const bool skip = !isfinite(coef);
  const float lr0 = a.lr_dev ? *a.lr_dev : a.lr;
  __syncthreads();
  if (a.advance && threadIdx.x == 0) {
    // The last block to have read the count moves it on.
    __threadfence();
    const unsigned last = gridDim.x - 1;
    if (atomicInc(reinterpret_cast<unsigned*>(a.step_dev + 1), last) == last && !skip)
      *a.step_dev = static_cast<int32_t>(s_t);
  }
  if (skip) return;
  const float bc1 = s_bc[0], rbc2 = s_bc[1];
  const uint32_t key = kStochastic ? mix32(a.key ^ s_t) : 0u;

  const int lane = threadIdx.x & 31;
  const uint32_t stride = gridDim.x * (kMixThreads / 32);
  uint32_t u = blockIdx.x * (kMixThreads / 32) + (threadIdx.x >> 5);
  if (u >= a.n_units) return;
  uint32_t cur = find_seg(a.seg, a.n_seg, u);
  for (; u < a.n_units; u += stride) {
    while (cur + 1 < a.n_seg && u >= a.seg[cur + 1].ubeg) ++cur;
    const MixSeg& s = a.seg[cur];
    const uint32_t blk = u - s.ubeg;
    const long long i0 = static_cast<long long>(blk) * kA8Block;
    const long long left = s.numel - i0;
    const bool vec = (s.flags & kMixVec) && left >= kA8Block;
    const bool g16 = s.flags & kMixGradBf16;
    const bool eight = s.s != nullptr;
    const long long iv = i0 + lane * 8;

    float p[8], g[8], m[8], v[8], e[8];
    uint32_t mbyte = 0, rbyte = 0;
    if (eight) {
      mbyte = s.s[2ll * blk];
      rbyte = s.s[2ll * blk + 1];
    }
    if (vec) {
      load_f32x8(s.p + iv, p);
      if (g16) unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(
                                 static_cast<const uint16_t*>(s.g) + iv)), g);
      else load_f32x8(static_cast<const float*>(s.g) + iv, g);
      if (s.e) load_f32x8(s.e + iv, e);
      if (eight) {
        const uint2 mw = __ldcs(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(s.m) + iv));
        const uint2 rw = __ldcs(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(s.v) + iv));
        const float mf = a8_factor(mbyte), rf = a8_factor(rbyte);
        a8_decode_m4(mw.x, mf, *reinterpret_cast<float(*)[4]>(m));
        a8_decode_m4(mw.y, mf, *reinterpret_cast<float(*)[4]>(m + 4));
        a8_decode_r4(rw.x, rf, *reinterpret_cast<float(*)[4]>(v));
        a8_decode_r4(rw.y, rf, *reinterpret_cast<float(*)[4]>(v + 4));
      } else {
        load_f32x8(static_cast<const float*>(s.m) + iv, m);
        load_f32x8(static_cast<const float*>(s.v) + iv, v);
      }
    } else {
      const float mf = a8_factor(mbyte), rf = a8_factor(rbyte);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k * 32 + lane;
        const bool in = j < left;
        const long long i = i0 + j;
        p[k] = in ? s.p[i] : 0.f;
        g[k] = !in ? 0.f
                   : g16 ? __uint_as_float(static_cast<uint32_t>(
                               static_cast<const uint16_t*>(s.g)[i]) << 16)
                         : static_cast<const float*>(s.g)[i];
        e[k] = in && s.e ? s.e[i] : 0.f;
        if (eight) {
          float x[4];
          a8_decode_m4(in ? static_cast<uint8_t*>(s.m)[i] : 0u, mf, x);
          m[k] = in ? x[0] : 0.f;
          a8_decode_r4(in ? static_cast<uint8_t*>(s.v)[i] : 0u, rf, x);
          v[k] = in ? x[0] : 0.f;
        } else {
          m[k] = in ? static_cast<const float*>(s.m)[i] : 0.f;
          v[k] = in ? static_cast<const float*>(s.v)[i] : 0.f;
        }
      }
    }

    const float lr = lr0 * s.lr_scale;
    const float keep = 1.f - lr * (a.wd * s.wd_scale);
    float r[8];
    float rmin = kMixRootLow, rmax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = __fmul_rn(g[k], coef);
      m[k] = __fadd_rn(__fmul_rn(m[k], a.b1), __fmul_rn(g[k], a.omb1));
      const float v0 = eight ? __fmul_rn(v[k], v[k]) : v[k];
      const float v1 = __fadd_rn(__fmul_rn(v0, a.b2), __fmul_rn(__fmul_rn(g[k], g[k]), a.omb2));
      r[k] = __fsqrt_rn(v1);
      rmin = fminf(rmin, r[k]);
      rmax = fmaxf(rmax, r[k]);
      if (!eight) v[k] = v1;
    }
    // An 8-bit state holds roots whose squares fp32 does not: where r' leaves
    // [2^-49, 2^63], it comes from inputs scaled by a power of two.
    if (eight && (rmin < kMixRootLow || rmax > kMixRootHigh)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (r[k] < kMixRootLow)
          r[k] = scaled_root(v[k], g[k], a.b2, a.omb2, 0x1p70f, 0x1p-70f);
        else if (r[k] > kMixRootHigh)
          r[k] = scaled_root(v[k], g[k], a.b2, a.omb2, 0x1p-70f, 0x1p70f);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float upd = __fdividef(m[k] * bc1, fmaf(r[k], rbc2, a.eps));
      p[k] = fmaf(p[k], keep, -lr * upd);
      e[k] = fmaf(a.d, e[k], a.omd * p[k]);
    }

    if (vec) {
      store_f32x8(s.p + iv, p);
      if (s.e) store_f32x8(s.e + iv, e);
      if (s.c) __stcs(reinterpret_cast<uint4*>(s.c + iv), pack_bf16x8(p));
      if (!eight) {
        store_f32x8(static_cast<float*>(s.m) + iv, m);
        store_f32x8(static_cast<float*>(s.v) + iv, v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k * 32 + lane;
        if (j >= left) continue;
        const long long i = i0 + j;
        s.p[i] = p[k];
        if (s.e) s.e[i] = e[k];
        if (s.c) s.c[i] = __bfloat16_as_ushort(__float2bfloat16_rn(p[k]));
        if (!eight) {
          static_cast<float*>(s.m)[i] = m[k];
          static_cast<float*>(s.v)[i] = v[k];
        }
      }
    }
    if (eight) {
      uint32_t word[8], m8[2], r8[2];
      if (kStochastic) {
        const uint32_t bkey = mix32(mix32(key ^ (a.first_tensor + cur)) ^ blk);
#pragma unroll
        for (int k = 0; k < 8; ++k) word[k] = mix32(bkey ^ (vec ? lane * 8 + k : k * 32 + lane));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) word[k] = 0u;
      }
      if (!vec) {
        // past the tensor's end nothing enters the block's largest
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k * 32 + lane >= left) m[k] = r[k] = 0.f;
      }
      a8_encode_block<kStochastic>(m, r, word, m8, r8, mbyte, rbyte);
      if (vec) {
        __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.m) + iv),
               make_uint2(m8[0], m8[1]));
        __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.v) + iv),
               make_uint2(r8[0], r8[1]));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = k * 32 + lane;
          if (j >= left) continue;
          static_cast<uint8_t*>(s.m)[i0 + j] = static_cast<uint8_t>(m8[k >> 2] >> (8 * (k & 3)));
          static_cast<uint8_t*>(s.v)[i0 + j] = static_cast<uint8_t>(r8[k >> 2] >> (8 * (k & 3)));
        }
      }
      if (lane == 0) {
        s.s[2ll * blk] = static_cast<uint8_t>(mbyte);
        s.s[2ll * blk + 1] = static_cast<uint8_t>(rbyte);
      }
    }
  }
}

// ---- 8-bit states from and to plain arrays --------------------------------

constexpr int kA8MaxSegs = 500;   // 500 x 56 bytes of kernel parameters

struct A8Seg {
  uint8_t *m8, *r8, *s;
  void* m;          // fp32 or bf16
  void* v;          // fp32: the second moment; bf16: its root
  long long numel;
  uint32_t ubeg;
  uint32_t flags;   // kMixGradBf16: the plain arrays are bf16; kMixVec
};
static_assert(sizeof(A8Seg) == 56, "kA8MaxSegs counts on 56 bytes");

template <int kSegs>
struct A8Params {
  A8Seg seg[kSegs];
  uint32_t n_seg, n_units;
};

// Plain moments -> codes (rounded to the nearest).
template <int kSegs>
__global__ void __launch_bounds__(kMixThreads)
adam8_write_kernel(const __grid_constant__ A8Params<kSegs> a) {
  const int lane = threadIdx.x & 31;
  const uint32_t stride = gridDim.x * (kMixThreads / 32);
  uint32_t u = blockIdx.x * (kMixThreads / 32) + (threadIdx.x >> 5);
  if (u >= a.n_units) return;
  uint32_t cur = find_seg(a.seg, a.n_seg, u);
  for (; u < a.n_units; u += stride) {
    while (cur + 1 < a.n_seg && u >= a.seg[cur + 1].ubeg) ++cur;
    const A8Seg& s = a.seg[cur];
    const uint32_t blk = u - s.ubeg;
    const long long i0 = static_cast<long long>(blk) * kA8Block;
    const long long left = s.numel - i0;
    const bool vec = (s.flags & kMixVec) && left >= kA8Block;
    const bool b16 = s.flags & kMixGradBf16;
    const long long iv = i0 + lane * 8;
    float m[8], r[8];
    if (vec) {
      if (b16) {
        unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(static_cast<uint16_t*>(s.m) + iv)), m);
        unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(static_cast<uint16_t*>(s.v) + iv)), r);
      } else {
        load_f32x8(static_cast<float*>(s.m) + iv, m);
        load_f32x8(static_cast<float*>(s.v) + iv, r);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k * 32 + lane;
        const long long i = i0 + j;
        m[k] = r[k] = 0.f;
        if (j < left) {
          if (b16) {
            m[k] = __uint_as_float(static_cast<uint32_t>(static_cast<uint16_t*>(s.m)[i]) << 16);
            r[k] = __uint_as_float(static_cast<uint32_t>(static_cast<uint16_t*>(s.v)[i]) << 16);
          } else {
            m[k] = static_cast<float*>(s.m)[i];
            r[k] = static_cast<float*>(s.v)[i];
          }
        }
      }
    }
    uint32_t word[8], m8[2], r8[2], mbyte, rbyte;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      word[k] = 0u;
      // a second moment (or root) below zero is not one: NaN, like sqrt's
      r[k] = b16 ? (r[k] < 0.f ? __uint_as_float(0x7fc00000u) : fabsf(r[k])) : fabsf(__fsqrt_rn(r[k]));
    }
    a8_encode_block<false>(m, r, word, m8, r8, mbyte, rbyte);
    if (vec) {
      __stcs(reinterpret_cast<uint2*>(s.m8 + iv), make_uint2(m8[0], m8[1]));
      __stcs(reinterpret_cast<uint2*>(s.r8 + iv), make_uint2(r8[0], r8[1]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k * 32 + lane;
        if (j >= left) continue;
        s.m8[i0 + j] = static_cast<uint8_t>(m8[k >> 2] >> (8 * (k & 3)));
        s.r8[i0 + j] = static_cast<uint8_t>(r8[k >> 2] >> (8 * (k & 3)));
      }
    }
    if (lane == 0) {
      s.s[2ll * blk] = static_cast<uint8_t>(mbyte);
      s.s[2ll * blk + 1] = static_cast<uint8_t>(rbyte);
    }
  }
}

// Codes -> plain moments: bf16 (first moment, root), both exact, or fp32
// (first moment, second moment = root squared, exact too: 12 bits).
template <int kSegs>
__global__ void __launch_bounds__(kMixThreads)
adam8_read_kernel(const __grid_constant__ A8Params<kSegs> a) {
  const int lane = threadIdx.x & 31;
  const uint32_t stride = gridDim.x * (kMixThreads / 32);
  uint32_t u = blockIdx.x * (kMixThreads / 32) + (threadIdx.x >> 5);
  if (u >= a.n_units) return;
  uint32_t cur = find_seg(a.seg, a.n_seg, u);
  for (; u < a.n_units; u += stride) {
    while (cur + 1 < a.n_seg && u >= a.seg[cur + 1].ubeg) ++cur;
    const A8Seg& s = a.seg[cur];
    const uint32_t blk = u - s.ubeg;
    const long long i0 = static_cast<long long>(blk) * kA8Block;
    const long long left = s.numel - i0;
    const bool vec = (s.flags & kMixVec) && left >= kA8Block;
    const bool b16 = s.flags & kMixGradBf16;
    const long long iv = i0 + lane * 8;
    const float mf = a8_factor(s.s[2ll * blk]), rf = a8_factor(s.s[2ll * blk + 1]);
    float m[8], r[8];
    if (vec) {
      const uint2 mw = __ldcs(reinterpret_cast<const uint2*>(s.m8 + iv));
      const uint2 rw = __ldcs(reinterpret_cast<const uint2*>(s.r8 + iv));
      a8_decode_m4(mw.x, mf, *reinterpret_cast<float(*)[4]>(m));
      a8_decode_m4(mw.y, mf, *reinterpret_cast<float(*)[4]>(m + 4));
      a8_decode_r4(rw.x, rf, *reinterpret_cast<float(*)[4]>(r));
      a8_decode_r4(rw.y, rf, *reinterpret_cast<float(*)[4]>(r + 4));
      if (b16) {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.m) + iv), pack_bf16x8(m));
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.v) + iv), pack_bf16x8(r));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] *= r[k];
        store_f32x8(static_cast<float*>(s.m) + iv, m);
        store_f32x8(static_cast<float*>(s.v) + iv, r);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k * 32 + lane;
        if (j >= left) continue;
        const long long i = i0 + j;
        float x[4], y[4];
        a8_decode_m4(s.m8[i], mf, x);
        a8_decode_r4(s.r8[i], rf, y);
        if (b16) {
          static_cast<uint16_t*>(s.m)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
          static_cast<uint16_t*>(s.v)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(y[0]));
        } else {
          static_cast<float*>(s.m)[i] = x[0];
          static_cast<float*>(s.v)[i] = y[0] * y[0];
        }
      }
    }
  }
}

}  // namespace muonb200
