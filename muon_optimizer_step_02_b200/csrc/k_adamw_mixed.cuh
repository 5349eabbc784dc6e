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
// Bytes per element: parameter 8, gradient 4 or 2, moments 16 or 4 (and 4 per
// 256), average 8, copy 2.  Measured on a 65,536 x 1024 table with bf16
// gradients and a copy: 313 us with 32-bit moments (28 bytes: 6.0 TB/s, 0.92 of
// the measured copy bandwidth), 174-190 us with 8-bit ones, rounded
// stochastically (16 bytes: 5.6-6.2 TB/s, 0.86-0.94), 195-200 us when it runs on
// end, for then the GPU's power limit lowers the clock.  The 8-bit step is
// bound by memory and by issue about equally (573 instructions per warp and
// block of 256, an issue slot in use in 77 of 100 cycles), so it is built to
// issue little: two elements to a register pair wherever the arithmetic has a
// two-value form, addresses and tensor look-up in uniform registers, the next
// block's data on their way through shared memory while one is computed.
//
// Source: PR #1893 "Record: L_ParallelResiduals_UNetSkips_DepthRecur_Muon_
// 1.0901", table "Architecture and training stack", rows "Optimizer" (AdamW
// on embeddings/scalars) and "EMA"; the page gives no setting and no state
// format.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "k_adam8.cuh"
#include "sm100_ptx.cuh"

namespace muonb200 {

constexpr int kMixThreads = 128;      // 4 warps: a unit of 4 blocks of 256 elements
constexpr int kMixResident = 6;       // thread blocks per SM (78 registers); 8-bit table above with
                                      // 5, 6, 7: 179, 174, 194 us
constexpr int kMixUnit = kMixThreads * 8;
constexpr int kMixMaxSegs = 400;      // 400 x 76 bytes of kernel parameters (limit 32,764)

// A tensor's element count, its place among the launch's tensors and its flags
// in one word.
constexpr unsigned long long kSegBf16 = 1ull << 56;   // gradient (plain moments) in bf16
constexpr unsigned long long kSegVec = 2ull << 56;    // every array aligned for wide accesses
constexpr int kSegPlace = 40;
constexpr unsigned long long kSegNumel = (1ull << kSegPlace) - 1;

struct MixSeg {
  float* p;
  const void* g;
  void* m;           // fp32, or codes
  void* v;           // fp32, or codes of the root
  uint8_t* s;        // scale bytes (m, r) per block; null: fp32 moments
  float* e;          // null: no EMA
  uint16_t* c;       // null: no bf16 copy
  unsigned long long numel;   // and place, flags
  float lr_scale, wd_scale;
};
static_assert(sizeof(MixSeg) == 72, "kMixMaxSegs counts on 72 + 4 bytes");

template <int kSegs>
struct MixParams {
  MixSeg seg[kSegs];         // those with 8-bit states first
  uint32_t ubeg[kSegs + 1];  // first unit of each tensor in the launch, and the end
  uint32_t n_seg, units8;    // units of tensors with 8-bit states
  int32_t* step_dev;         // [0] steps taken, [1] ticket; or null
  const float* lr_dev;       // or null
  const float* coef_dev;     // or null
  double pow1[31], pow2[31]; // beta^(2^j)
  int32_t step;              // t when step_dev is null
  uint32_t key;              // random key before the step number
  uint32_t first_tensor;
  int32_t advance;           // this launch advances *step_dev
  float lr, wd;
  float one;                 // 1 (see add2)
  float2 b1, omb1, minus_b2, minus_omb2, eps, d, omd;   // each twice, for two elements
};

// Values of 8 elements, two to a register pair: products and sums are issued
// for two at a time, each rounded as a single one.
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// A lane's 8 elements of a full block, 8 lane to 8 lane + 7: 32 bytes of fp32
// in one access, 16 of bf16, 8 of codes.
__device__ __forceinline__ void load8(const float* p, float2 (&x)[4]) {
  asm volatile("ld.global.cs.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0].x), "=f"(x[0].y), "=f"(x[1].x), "=f"(x[1].y), "=f"(x[2].x),
                 "=f"(x[2].y), "=f"(x[3].x), "=f"(x[3].y)
               : "l"(p));
}

__device__ __forceinline__ void store8(float* p, const float2 (&x)[4]) {
  asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
               "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y),
               "f"(x[3].x), "f"(x[3].y)
               : "memory");
}

__device__ __forceinline__ void unpack8(const uint4& raw, float2 (&x)[4]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load8_bf16(const uint16_t* p, float2 (&x)[4]) {
  unpack8(__ldcs(reinterpret_cast<const uint4*>(p)), x);
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float2 (&x)[4]) {
  __stcs(reinterpret_cast<uint4*>(p), pack8(x));
}

__device__ __forceinline__ uint2 load8_codes(const uint8_t* p) {
  return __ldcs(reinterpret_cast<const uint2*>(p));
}

__device__ __forceinline__ void store8_codes(uint8_t* p, const uint32_t (&w)[2]) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
}

__device__ __forceinline__ float bf16_at(const void* p, long long i) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

__device__ __forceinline__ float& at(float2 (&x)[4], int k) {
  return k & 1 ? x[k >> 1].y : x[k >> 1].x;
}

constexpr float kMixRootLow = 0x1p-49f;

__device__ __forceinline__ float scaled_root(float r, float g, float b2, float omb2, float up,
                                             float down) {
  const float rs = __fmul_rn(r, up), gs = __fmul_rn(g, up);
  const float v = __fadd_rn(__fmul_rn(__fmul_rn(rs, rs), b2),
                            __fmul_rn(__fmul_rn(gs, gs), omb2));
  return __fmul_rn(__fsqrt_rn(v), down);
}

// Largest of three, NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Square roots of two values, given and returned with a minus sign, rounded to
// the nearest for values in [2^-98, 2^128) (NaN or inexact elsewhere): an
// estimate s = v y from y = v^(-1/2), and one step of Newton's iteration on
// its exact residual, s + (v - s^2) y / 2.  The signs let every operation
// take its operands as they are.
__device__ __forceinline__ float2 minus_root2(float2 minus_v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(-minus_v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(-minus_v.y));
  const float2 s = mul2(minus_v, y);
  return __ffma2_rn(__ffma2_rn(s, s, minus_v), mul2(y, make_float2(0.5f, 0.5f)), s);
}

// Minus the square roots of any two values, rounded to the nearest.
__device__ __forceinline__ float2 minus_root_any(float2 v) {
  float2 x = minus_root2(make_float2(-v.x, -v.y));
  if (!(v.x >= 0x1p-98f && v.x < INFINITY)) x.x = -__fsqrt_rn(v.x);
  if (!(v.y >= 0x1p-98f && v.y < INFINITY)) x.y = -__fsqrt_rn(v.y);
  return x;
}

// 1 / x to one unit in the last place; x below the normal range counts as 0.
__device__ __forceinline__ float reciprocal(float x) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// The warp's number, in a form that the compiler knows to be the same for all
// of its lanes, so that what follows from it (blocks, addresses, branches)
// stays out of the lanes' registers.
__device__ __forceinline__ int warp_number() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// Last tensor whose first unit is at or before u.
__device__ __forceinline__ uint32_t find_seg(const uint32_t* ubeg, uint32_t n, uint32_t u) {
  uint32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if (ubeg[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What a launch's tensors share, and one tensor's share of it.
struct MixStep {
  float2 coef, minus_rbc2, keep, rate;
  uint32_t key;    // random key of the tensor
};

// New moments of a lane's 8 elements from g, m and v (a root for 8-bit states);
// nr = -r'.  Returns whether some root may be zero.
template <bool kEight, class P>
__device__ __forceinline__ bool mixed_moments(const P& a, const MixStep& w, float2 (&g)[4],
                                              float2 (&m)[4], float2 (&v)[4], float2 (&nr)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    g[k] = mul2(g[k], w.coef);
    m[k] = add2(mul2(m[k], a.b1), mul2(g[k], a.omb1), a.one);
    const float2 v0 = kEight ? mul2(v[k], v[k]) : v[k];
    const float2 nv = add2(mul2(v0, a.minus_b2), mul2(mul2(g[k], g[k]), a.minus_omb2), a.one);
    nr[k] = minus_root2(nv);
    if (!kEight) v[k] = make_float2(-nv.x, -nv.y);
  }
  // Where r' leaves [2^-49, 2^64) or is no number: the exact root of a 32-bit
  // state's v'; an 8-bit state holds roots whose squares fp32 does not, and
  // there r' comes from inputs scaled by a power of two.
  const float low = max3(max3(max3(max3(nr[0].x, nr[0].y, nr[1].x), nr[1].y, nr[2].x), nr[2].y,
                              nr[3].x), nr[3].y, nr[3].y);
  const bool odd = !(low <= -kMixRootLow);
  if (odd) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float& x = at(nr, k);
      if (x <= -kMixRootLow) continue;
      if (!kEight) {
        x = -__fsqrt_rn(at(v, k));
        continue;
      }
      const float b2 = -a.minus_b2.x, omb2 = -a.minus_omb2.x;
      x = -scaled_root(at(v, k), at(g, k), b2, omb2, 0x1p70f, 0x1p-70f);
      if (!isfinite(x)) x = -scaled_root(at(v, k), at(g, k), b2, omb2, 0x1p-70f, 0x1p70f);
    }
  }
  return odd;
}

// Full blocks with 8-bit states come through shared memory, copied there while
// the block before is computed, in two groups: what the moments need
// (gradient, codes) is replaced by the next block's as soon as it is read,
// what the weights need (parameters, averages) likewise, later.  fp32 arrays
// are copied in 16-byte pieces, lane l taking pieces l and 32 + l (so that a
// warp's access is one stretch of memory) where it reads 2 l and 2 l + 1; the
// other arrays by the lane that will read them.  Whatever the gradients' types
// from one block to the next, a warp's part of every array is its own (256
// fp32 values, or as many bf16 in its first half).  Places in a thread block's
// buffer:
constexpr int kBufG = 0, kBufCodes = 4096, kBufP = 6144, kBufE = 10240, kMixBuf = 14336;

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kBytes)
                 : "memory");
}

// A warp's 256 fp32 values, in their order.
__device__ __forceinline__ void copy_f32(uint32_t to, const float* from, int lane) {
  to += (threadIdx.x & ~31) * 32 + lane * 16;
  copy_async<16>(to, from + lane * 4);
  copy_async<16>(to + 512, from + 128 + lane * 4);
}

__device__ __forceinline__ void from_buf_f32(uint32_t at, float2 (&x)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x[0].x), "=f"(x[0].y), "=f"(x[1].x), "=f"(x[1].y)
               : "r"(at + threadIdx.x * 32) : "memory");
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x[2].x), "=f"(x[2].y), "=f"(x[3].x), "=f"(x[3].y)
               : "r"(at + threadIdx.x * 32 + 16) : "memory");
}

__device__ __forceinline__ void to_buf_f32(uint32_t at, const float2 (&x)[4]) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + threadIdx.x * 32),
               "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y)
               : "memory");
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + threadIdx.x * 32 + 16),
               "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y)
               : "memory");
}

__device__ __forceinline__ float word_of_buf(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}

__device__ __forceinline__ uint8_t byte_of_buf(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return static_cast<uint8_t>(x);
}

__device__ __forceinline__ void from_buf_bf16(uint32_t at, int lane, float2 (&x)[4]) {
  uint4 w;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "r"(at + (threadIdx.x & ~31) * 32 + lane * 16) : "memory");
  unpack8(w, x);
}

__device__ __forceinline__ uint2 from_buf_codes(uint32_t at) {
  uint2 w;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
               : "=r"(w.x), "=r"(w.y) : "r"(at + threadIdx.x * 8) : "memory");
  return w;
}

// Waits until at most kPending of the lanes' groups are under way.
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
  __syncwarp();
}

__device__ __forceinline__ void copies_group() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Where a unit's block of this warp lies.
struct MixPlace {
  uint32_t cur, end;   // tensor, and its last unit + 1
  uint32_t blk;
  long long i0, left;
  bool full;           // a full block of an aligned tensor
};

// Elements of the tensor in a place's block.
__device__ __forceinline__ int block_elements(const MixPlace& at) {
  return at.left < kA8Block ? static_cast<int>(at.left) : kA8Block;
}

template <class P>
__device__ __forceinline__ void find_place(const P& a, uint32_t u, int warp, MixPlace& at) {
  if (u >= at.end) {
    at.cur = find_seg(a.ubeg, a.n_seg, u);
    at.end = a.ubeg[at.cur + 1];
  }
  const auto& s = a.seg[at.cur];
  at.blk = (u - a.ubeg[at.cur]) * (kMixUnit / kA8Block) + warp;
  at.i0 = static_cast<long long>(at.blk) * kA8Block;
  at.left = static_cast<long long>(s.numel & kSegNumel) - at.i0;
  at.full = (s.numel & kSegVec) && at.left >= kA8Block;
}

// Starts the copies that the moments need; returns the scale bytes.
__device__ __forceinline__ uint32_t fetch_moments(const MixSeg& s, const MixPlace& at,
                                                  uint32_t buf, int lane) {
  if (s.numel & kSegBf16)
    copy_async<16>(buf + kBufG + (threadIdx.x & ~31) * 32 + lane * 16,
                   static_cast<const uint16_t*>(s.g) + at.i0 + lane * 8);
  else
    copy_f32(buf + kBufG, static_cast<const float*>(s.g) + at.i0, lane);
  const uint32_t codes = buf + kBufCodes + threadIdx.x * 8;
  copy_async<8>(codes, static_cast<uint8_t*>(s.m) + at.i0 + lane * 8);
  copy_async<8>(codes + kMixThreads * 8, static_cast<uint8_t*>(s.v) + at.i0 + lane * 8);
  // (as two bytes joined here: one 16-bit load, first used by the next block,
  // was measured 10 % slower over the whole kernel, on a 65,536 x 1024 table)
  return s.s[2ll * at.blk] | static_cast<uint32_t>(s.s[2ll * at.blk + 1]) << 8;
}

// Starts the copies that the weights need.
__device__ __forceinline__ void fetch_weights(const MixSeg& s, const MixPlace& at, uint32_t buf,
                                              int lane) {
  copy_f32(buf + kBufP, s.p + at.i0, lane);
  if (s.e) copy_f32(buf + kBufE, s.e + at.i0, lane);
}

// New weights, averages and copies of a lane's 8 elements.
template <class P>
__device__ __forceinline__ void mixed_weights(const P& a, const MixStep& w,
                                              const float2 (&m)[4], const float2 (&nr)[4],
                                              float2 (&p)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 den = __ffma2_rn(nr[k], w.minus_rbc2, a.eps);
    const float2 upd = mul2(m[k], make_float2(reciprocal(den.x), reciprocal(den.y)));
    p[k] = __ffma2_rn(upd, w.rate, mul2(p[k], w.keep));
  }
}

template <class P>
__device__ __forceinline__ void mixed_average(const P& a, const float2 (&p)[4], float2 (&e)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) e[k] = __ffma2_rn(e[k], a.d, mul2(p[k], a.omd));
}

// The same for a block that is not full or not aligned: element by element,
// zeros past the tensor's end.
__device__ __forceinline__ void fetch_ragged(const MixSeg& s, const MixPlace& at,
                                             unsigned char* buf, int lane) {
  const bool g16 = (s.numel & kSegBf16) != 0;
  const int n = block_elements(at);
  const long long i = at.i0 + lane;
  const float* sp = s.p + i;
  const float* se = s.e ? s.e + i : sp;      // (read, and not used, without an average)
  const uint8_t* sm = static_cast<uint8_t*>(s.m) + i;
  const uint8_t* sr = static_cast<uint8_t*>(s.v) + i;
  const uint16_t* g2 = static_cast<const uint16_t*>(s.g) + i;
  const float* g4 = static_cast<const float*>(s.g) + i;
  float p[8], e[8];
  uint32_t g[8], m[8], r[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {   // everything is requested before the first use
    const bool in = k * 32 + lane < n;
    g[k] = 0u;
    if (in) g[k] = g16 ? g2[k * 32] : __float_as_uint(g4[k * 32]);
    m[k] = in ? sm[k * 32] : 0u;
    r[k] = in ? sr[k * 32] : 0u;
    p[k] = in ? sp[k * 32] : 0.f;
    e[k] = in ? se[k * 32] : 0.f;
  }
  __syncwarp();   // the lanes have read the block before
  const int first = threadIdx.x & ~31;
  unsigned char* wide = buf + first * 32 + lane * 4;
  unsigned char* codes = buf + kBufCodes + first * 8 + lane;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (g16)
      *reinterpret_cast<uint16_t*>(buf + kBufG + first * 32 + lane * 2 + k * 64) =
          static_cast<uint16_t>(g[k]);
    else
      *reinterpret_cast<uint32_t*>(wide + kBufG + k * 128) = g[k];
    codes[k * 32] = static_cast<uint8_t>(m[k]);
    codes[kMixThreads * 8 + k * 32] = static_cast<uint8_t>(r[k]);
    *reinterpret_cast<float*>(wide + kBufP + k * 128) = p[k];
    *reinterpret_cast<float*>(wide + kBufE + k * 128) = e[k];
  }
  __syncwarp();
}

// A block with an 8-bit state, its copies under way; next_moments and
// next_weights start the next block's once this one's have been read.
template <bool kStochastic, bool kG16, class P, class FM, class FW>
__device__ __forceinline__ void mixed_block8(const P& a, const MixSeg& s, const MixStep& w,
                                             const MixPlace& at, uint32_t buf, uint32_t scale,
                                             int lane, const FM& next_moments,
                                             const FW& next_weights) {
  const long long i = at.i0 + lane * 8;
  float2 m[4], nr[4];
  bool odd;
  {
    float2 g[4], r[4];
    copies_wait<1>();
    if (kG16) from_buf_bf16(buf + kBufG, lane, g);
    else from_buf_f32(buf + kBufG, g);
    const float mf = a8_factor(scale & 0xffu), rf = a8_factor(scale >> 8);
    const uint2 mw = from_buf_codes(buf + kBufCodes);
    const uint2 rw = from_buf_codes(buf + kBufCodes + kMixThreads * 8);
    a8_decode_m4(mw.x, mf, m);
    a8_decode_m4(mw.y, mf, m + 2);
    a8_decode_r4(rw.x, rf, r);
    a8_decode_r4(rw.y, rf, r + 2);
    __syncwarp();   // before other lanes' pieces are replaced
    next_moments();
    odd = mixed_moments<true>(a, w, g, m, r, nr);
  }
  {
    float2 p[4], e[4];
    copies_wait<1>();
    from_buf_f32(buf + kBufP, p);
    if (s.e) from_buf_f32(buf + kBufE, e);
    mixed_weights(a, w, m, nr, p);
    if (s.e) mixed_average(a, p, e);
    __syncwarp();   // before other lanes' pieces are replaced
    if (at.full) {
      next_weights();
      store8(s.p + i, p);
      if (s.c) store8_bf16(s.c + i, p);
      if (s.e) store8(s.e + i, e);
    } else {
      // through shared memory, so that a warp's stores are one stretch (from
      // the lanes' 8 elements each, 16.8 M unaligned elements took 200 us, now
      // 104; aligned ones 45-50)
      to_buf_f32(buf + kBufP, p);
      if (s.e) to_buf_f32(buf + kBufE, e);
      __syncwarp();
      const uint32_t own = buf + (threadIdx.x & ~31) * 32 + lane * 4;
      const int n = block_elements(at);
      float* sp = s.p + at.i0 + lane;
      uint16_t* sc = s.c + at.i0 + lane;
      float* se = s.e + at.i0 + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k * 32 + lane >= n) continue;
        const float y = word_of_buf(own + kBufP + k * 128);
        sp[k * 32] = y;
        if (s.c) sc[k * 32] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        if (s.e) se[k * 32] = word_of_buf(own + kBufE + k * 128);
      }
    }
  }
  if (!at.full) {
    // past the tensor's end nothing enters the block's largest
    const int n = block_elements(at) - lane * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= n) ::muonb200::at(m, k) = ::muonb200::at(nr, k) = 0.f;
    odd = true;
  }
  uint32_t x[8], m8[2], r8[2], mbyte, rbyte;
  if (kStochastic) {
    // mix32(key of the block ^ element) but for its last step; of its first
    // step, the element's number (below 256) does not reach the upper half
    uint32_t bkey = mix32(w.key ^ at.blk);
    bkey = (bkey ^ (bkey >> 16)) ^ (lane * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = (bkey ^ k) * 0x57735285u;
      x[k] = (x[k] ^ (x[k] >> 15)) * 0x4746E6A3u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = 0u;
  }
  a8_encode_block<kStochastic>(m, nr, x, odd, m8, r8, mbyte, rbyte);
  uint8_t* cm = static_cast<uint8_t*>(s.m);
  uint8_t* cr = static_cast<uint8_t*>(s.v);
  if (at.full) {
    store8_codes(cm + i, m8);
    store8_codes(cr + i, r8);
  } else {
    __syncwarp();
    const uint32_t own = buf + kBufP + (threadIdx.x & ~31) * 32;
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(own + lane * 8), "r"(m8[0]), "r"(m8[1])
                 : "memory");
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(own + 256 + lane * 8), "r"(r8[0]),
                 "r"(r8[1])
                 : "memory");
    __syncwarp();
    const int n = block_elements(at);
    cm += at.i0 + lane;
    cr += at.i0 + lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k * 32 + lane >= n) continue;
      cm[k * 32] = byte_of_buf(own + lane + k * 32);
      cr[k * 32] = byte_of_buf(own + 256 + lane + k * 32);
    }
    __syncwarp();
    next_weights();
  }
  if (lane == 0) {
    if (at.full) {
      reinterpret_cast<uint16_t*>(s.s)[at.blk] = static_cast<uint16_t>(mbyte | rbyte << 8);
    } else {
      s.s[2ll * at.blk] = static_cast<uint8_t>(mbyte);
      s.s[2ll * at.blk + 1] = static_cast<uint8_t>(rbyte);
    }
  }
}

// A full block of an aligned tensor with a 32-bit state.
template <bool kG16, class P>
__device__ __forceinline__ void mixed_full32(const P& a, const MixSeg& s, const MixStep& w,
                                             const MixPlace& at, int lane) {
  const long long i = at.i0 + lane * 8;
  float2 p[4], g[4], m[4], v[4], nr[4], e[4];
  load8(static_cast<const float*>(s.m) + i, m);
  load8(static_cast<const float*>(s.v) + i, v);
  if (kG16) load8_bf16(static_cast<const uint16_t*>(s.g) + i, g);
  else load8(static_cast<const float*>(s.g) + i, g);
  load8(s.p + i, p);
  if (s.e) load8(s.e + i, e);
  mixed_moments<false>(a, w, g, m, v, nr);
  mixed_weights(a, w, m, nr, p);
  store8(s.p + i, p);
  if (s.c) store8_bf16(s.c + i, p);
  if (s.e) {
    mixed_average(a, p, e);
    store8(s.e + i, e);
  }
  store8(static_cast<float*>(s.m) + i, m);
  store8(static_cast<float*>(s.v) + i, v);
}

// Any block with a 32-bit state, element by element: lane l takes l, l + 32, ...
template <class P>
__device__ __forceinline__ void mixed_ragged32(const P& a, const MixSeg& s, const MixStep& w,
                                               const MixPlace& at, int lane) {
  const bool g16 = (s.numel & kSegBf16) != 0;
  float2 p[4], g[4], m[4], v[4], nr[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = k * 32 + lane;
    const long long i = at.i0 + j;
    const bool in = j < at.left;
    ::muonb200::at(p, k) = in ? s.p[i] : 0.f;
    ::muonb200::at(g, k) = !in ? 0.f : g16 ? bf16_at(s.g, i) : static_cast<const float*>(s.g)[i];
    ::muonb200::at(m, k) = in ? static_cast<const float*>(s.m)[i] : 0.f;
    ::muonb200::at(v, k) = in ? static_cast<const float*>(s.v)[i] : 0.f;
  }
  mixed_moments<false>(a, w, g, m, v, nr);
  mixed_weights(a, w, m, nr, p);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = k * 32 + lane;
    const long long i = at.i0 + j;
    if (j >= at.left) continue;
    const float x = ::muonb200::at(p, k);
    s.p[i] = x;
    if (s.e) s.e[i] = fmaf(s.e[i], a.d.x, __fmul_rn(x, a.omd.x));
    if (s.c) s.c[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    static_cast<float*>(s.m)[i] = ::muonb200::at(m, k);
    static_cast<float*>(s.v)[i] = ::muonb200::at(v, k);
  }
}

// A thread block takes a unit of 4 blocks of 256 elements at a time, one warp
// per block, so that everything about the tensor (table look-up, pointers) is
// uniform over the thread block.  Full blocks of aligned tensors move 8
// elements per lane at a time; ragged ends and unaligned tensors go element by
// element.  Tensors with 8-bit states come first, in a loop of their own (one
// loop for both forms spilled registers).
template <bool kStochastic, int kSegs>
__global__ void __launch_bounds__(kMixThreads, kMixResident)
adamw_mixed_kernel(const __grid_constant__ MixParams<kSegs> a) {
  __shared__ __align__(16) unsigned char s_buf[kMixBuf];
  __shared__ float s_bc[2];
  const int lane = threadIdx.x & 31, warp = warp_number();
  const uint32_t buf = static_cast<uint32_t>(__cvta_generic_to_shared(s_buf));
  const uint32_t n_units = a.ubeg[a.n_seg];
  MixPlace next;
  next.end = 0;
  next.full = false;
  uint32_t scale = 0;
  uint32_t u = blockIdx.x;
  if (u < a.units8) find_place(a, u, warp, next);
  grid_launch_dependents();
  grid_dependency_wait();   // nothing above touches memory
  if (next.full) scale = fetch_moments(a.seg[next.cur], next, buf, lane);
  copies_group();
  if (next.full) fetch_weights(a.seg[next.cur], next, buf, lane);
  copies_group();

  const uint32_t t = a.step_dev ? static_cast<uint32_t>(*a.step_dev) + 1u
                                : static_cast<uint32_t>(a.step);
  const float coef = a.coef_dev ? *a.coef_dev : 1.f;
  const float lr0 = a.lr_dev ? *a.lr_dev : a.lr;
  const bool skip = __any_sync(0xffffffffu, !isfinite(coef));
  if (threadIdx.x < 32) {
    const double* pw = threadIdx.x == 0 ? a.pow1 : a.pow2;
    double x = 1.0;
    for (uint32_t rest = t; rest; rest &= rest - 1) x *= pw[__ffs(rest) - 1];
    const float y = static_cast<float>(1.0 - x);
    if (threadIdx.x == 0) s_bc[0] = __frcp_rn(y);
    if (threadIdx.x == 1) s_bc[1] = __frcp_rn(__fsqrt_rn(y));
  }
  __syncthreads();   // every thread has read the step count
  // The last thread block to have read the count moves it on; the ticket's
  // answer is awaited at the end.
  const uint32_t last = gridDim.x - 1;
  uint32_t ticket = last + 1;
  if (a.advance && threadIdx.x == kMixThreads - 1)
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                 : "=r"(ticket) : "l"(a.step_dev + 1), "r"(last) : "memory");
  if (skip) {
    copies_wait<0>();
    return;
  }
  const float bc1 = s_bc[0];
  MixStep w;
  w.coef = pair(coef);
  w.minus_rbc2 = pair(-s_bc[1]);
  const uint32_t key = kStochastic ? mix32(a.key ^ t) : 0u;

  const auto set_tensor = [&](const MixSeg& s) {
    const float lr = lr0 * s.lr_scale;
    w.keep = pair(1.f - lr * (a.wd * s.wd_scale));
    w.rate = pair(-lr * bc1);
    if (kStochastic)
      w.key = mix32(key ^ (a.first_tensor +
                           (static_cast<uint32_t>(s.numel >> kSegPlace) & 0xffffu)));
  };

  uint32_t set = 0xffffffffu;
  for (; u < a.units8; u += gridDim.x) {
    const MixPlace at = next;
    const MixSeg& s = a.seg[at.cur];
    if (at.cur != set) set_tensor(s);
    set = at.cur;
    uint32_t scale_now = scale;
    next.full = false;
    if (u + gridDim.x < a.units8) find_place(a, u + gridDim.x, warp, next);
    const auto next_moments = [&]() {
      if (next.full) scale = fetch_moments(a.seg[next.cur], next, buf, lane);
      copies_group();
    };
    const auto next_weights = [&]() {
      if (next.full) fetch_weights(a.seg[next.cur], next, buf, lane);
      copies_group();
    };
    if (at.left <= 0) {
      next_moments();
      next_weights();
      continue;
    }
    if (!at.full) {
      scale_now = s.s[2ll * at.blk] | static_cast<uint32_t>(s.s[2ll * at.blk + 1]) << 8;
      fetch_ragged(s, at, s_buf, lane);
    }
    if (s.numel & kSegBf16)
      mixed_block8<kStochastic, true>(a, s, w, at, buf, scale_now, lane, next_moments,
                                      next_weights);
    else
      mixed_block8<kStochastic, false>(a, s, w, at, buf, scale_now, lane, next_moments,
                                       next_weights);
  }
  copies_wait<0>();

  for (; u < n_units; u += gridDim.x) {
    find_place(a, u, warp, next);
    const MixSeg& s = a.seg[next.cur];
    if (next.cur != set) set_tensor(s);
    set = next.cur;
    if (next.full) {
      if (s.numel & kSegBf16) mixed_full32<true>(a, s, w, next, lane);
      else mixed_full32<false>(a, s, w, next, lane);
    } else if (next.left > 0) {
      mixed_ragged32(a, s, w, next, lane);
    }
  }
  if (ticket == last) *a.step_dev = static_cast<int32_t>(t);
}

// ---- 8-bit states from and to plain arrays --------------------------------

constexpr int kA8MaxSegs = 500;   // 500 x 52 bytes of kernel parameters
// Thread blocks per SM, as many as their 37 and 32 registers leave room for
// (writing with 16: a second, partial round, 10 % slower).
constexpr int kA8WriteResident = 12, kA8ReadResident = 16;

struct A8Seg {
  uint8_t *m8, *r8, *s;
  void* m;                    // fp32 or bf16
  void* v;                    // fp32: the second moment; bf16: its root
  unsigned long long numel;   // and the flags
};
static_assert(sizeof(A8Seg) == 48, "kA8MaxSegs counts on 48 + 4 bytes");

template <int kSegs>
struct A8Params {
  A8Seg seg[kSegs];
  uint32_t ubeg[kSegs + 1];
  uint32_t n_seg;
};

// Plain moments -> codes (rounded to the nearest).  10 bytes per element from
// fp32: 67 M elements in 104-112 us (6.0-6.4 TB/s); 6 from bf16: 98 us (4.1 TB/s),
// the ALU pipe in use in 76 of 100 cycles.
template <int kSegs>
__global__ void __launch_bounds__(kMixThreads)
adam8_write_kernel(const __grid_constant__ A8Params<kSegs> a) {
  const int lane = threadIdx.x & 31, warp = warp_number();
  const uint32_t n_units = a.ubeg[a.n_seg];
  uint32_t cur = 0, end = 0;
  grid_launch_dependents();
  grid_dependency_wait();
  for (uint32_t u = blockIdx.x; u < n_units; u += gridDim.x) {
    if (u >= end) {
      cur = find_seg(a.ubeg, a.n_seg, u);
      end = a.ubeg[cur + 1];
    }
    const A8Seg& s = a.seg[cur];
    const uint32_t blk = (u - a.ubeg[cur]) * (kMixUnit / kA8Block) + warp;
    const long long i0 = static_cast<long long>(blk) * kA8Block;
    const long long left = static_cast<long long>(s.numel & kSegNumel) - i0;
    if (left <= 0) continue;
    const int n = left < kA8Block ? static_cast<int>(left) : kA8Block;
    const bool vec = (s.numel & kSegVec) && left >= kA8Block;
    const bool b16 = (s.numel & kSegBf16) != 0;
    const long long iv = i0 + lane * 8;
    float2 m[4], r[4];
    if (vec) {
      if (b16) {
        load8_bf16(static_cast<uint16_t*>(s.m) + iv, m);
        load8_bf16(static_cast<uint16_t*>(s.v) + iv, r);
      } else {
        load8(static_cast<float*>(s.m) + iv, m);
        load8(static_cast<float*>(s.v) + iv, r);
      }
    } else {
      const uint16_t *m2 = static_cast<uint16_t*>(s.m) + i0 + lane,
                     *v2 = static_cast<uint16_t*>(s.v) + i0 + lane;
      const float *m4 = static_cast<float*>(s.m) + i0 + lane,
                  *v4 = static_cast<float*>(s.v) + i0 + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool in = k * 32 + lane < n;
        at(m, k) = !in ? 0.f : b16 ? bf16_at(m2, k * 32) : m4[k * 32];
        at(r, k) = !in ? 0.f : b16 ? bf16_at(v2, k * 32) : v4[k * 32];
      }
    }
    // r: the roots with a minus sign
    if (b16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // a root below zero is not one: NaN, like a negative number's root
        float& x = at(r, k);
        x = x < 0.f ? __uint_as_float(0x7fc00000u) : -x;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = minus_root_any(r[k]);
    }
    uint32_t zero[8], m8[2], r8[2], mbyte, rbyte;
#pragma unroll
    for (int k = 0; k < 8; ++k) zero[k] = 0u;
    a8_encode_block<false>(m, r, zero, true, m8, r8, mbyte, rbyte);
    if (vec) {
      store8_codes(s.m8 + iv, m8);
      store8_codes(s.r8 + iv, r8);
    } else {
      uint8_t *cm = s.m8 + i0 + lane, *cr = s.r8 + i0 + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k * 32 + lane >= n) continue;
        cm[k * 32] = static_cast<uint8_t>(m8[k >> 2] >> (8 * (k & 3)));
        cr[k * 32] = static_cast<uint8_t>(r8[k >> 2] >> (8 * (k & 3)));
      }
    }
    if (lane == 0) {
      s.s[2ll * blk] = static_cast<uint8_t>(mbyte);
      s.s[2ll * blk + 1] = static_cast<uint8_t>(rbyte);
    }
  }
}

// A block's codes and scale bytes on their way into registers.
struct A8Codes {
  uint2 m, r;
  uint32_t scale;
};

// Codes -> plain moments: bf16 (first moment, root), both exact, or fp32
// (first moment, second moment = root squared, exact too: 12 bits).  6 bytes per
// element to bf16.  The next block's codes are requested before this one's are
// used: the 11L model's 212 tensors 8.1 -> 7.1 us, at the price of 67 -> 71 us
// (5.7 TB/s) on 67 M elements; 10 bytes per element to fp32: 118 us (5.7 TB/s).
template <int kSegs>
__global__ void __launch_bounds__(kMixThreads, kA8ReadResident)
adam8_read_kernel(const __grid_constant__ A8Params<kSegs> a) {
  const int lane = threadIdx.x & 31, warp = warp_number();
  const uint32_t n_units = a.ubeg[a.n_seg];
  MixPlace next;
  next.end = 0;
  next.full = false;
  A8Codes codes;
  const auto request = [&]() {
    const A8Seg& s = a.seg[next.cur];
    codes.m = load8_codes(s.m8 + next.i0 + lane * 8);
    codes.r = load8_codes(s.r8 + next.i0 + lane * 8);
    codes.scale = s.s[2ll * next.blk] | static_cast<uint32_t>(s.s[2ll * next.blk + 1]) << 8;
  };
  uint32_t u = blockIdx.x;
  if (u < n_units) find_place(a, u, warp, next);
  grid_launch_dependents();
  grid_dependency_wait();
  if (next.full) request();
  for (; u < n_units; u += gridDim.x) {
    const MixPlace at = next;
    const A8Codes now = codes;
    const A8Seg& s = a.seg[at.cur];
    const bool b16 = (s.numel & kSegBf16) != 0;
    next.full = false;
    if (u + gridDim.x < n_units) find_place(a, u + gridDim.x, warp, next);
    if (next.full) request();
    if (at.full) {
      const long long i = at.i0 + lane * 8;
      const float mf = a8_factor(now.scale & 0xffu), rf = a8_factor(now.scale >> 8);
      float2 m[4], r[4];
      a8_decode_m4(now.m.x, mf, m);
      a8_decode_m4(now.m.y, mf, m + 2);
      a8_decode_r4(now.r.x, rf, r);
      a8_decode_r4(now.r.y, rf, r + 2);
      if (b16) {
        store8_bf16(static_cast<uint16_t*>(s.m) + i, m);
        store8_bf16(static_cast<uint16_t*>(s.v) + i, r);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = mul2(r[k], r[k]);
        store8(static_cast<float*>(s.m) + i, m);
        store8(static_cast<float*>(s.v) + i, r);
      }
    } else if (at.left > 0) {
      const float mf = a8_factor(s.s[2ll * at.blk]), rf = a8_factor(s.s[2ll * at.blk + 1]);
      const int n = block_elements(at);
      const long long i = at.i0 + lane;
      uint32_t cm[8], cr[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool in = k * 32 + lane < n;
        cm[k] = in ? (s.m8 + i)[k * 32] : 0u;
        cr[k] = in ? (s.r8 + i)[k * 32] : 0u;
      }
      uint16_t *m2 = static_cast<uint16_t*>(s.m) + i, *v2 = static_cast<uint16_t*>(s.v) + i;
      float *m4 = static_cast<float*>(s.m) + i, *v4 = static_cast<float*>(s.v) + i;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k * 32 + lane >= n) continue;
        float2 x[2], y[2];
        a8_decode_m4(cm[k], mf, x);
        a8_decode_r4(cr[k], rf, y);
        if (b16) {
          m2[k * 32] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0].x));
          v2[k * 32] = __bfloat16_as_ushort(__float2bfloat16_rn(y[0].x));
        } else {
          m4[k * 32] = x[0].x;
          v4[k * 32] = y[0].x * y[0].x;
        }
      }
    }
  }
}

}  // namespace muonb200
