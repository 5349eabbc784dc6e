// The 8-bit form of AdamW's moments: codes, scales, rounding and random bits.
//
// A tensor's flat index space is cut into blocks of 256 elements.  The first
// moment is kept as sign, 3 exponent and 4 mantissa bits; of the second
// moment its root r = sqrt(v) is kept (the quantity the update divides by),
// as 3 exponent and 5 mantissa bits, for it needs no sign.  Each block has
// one power-of-two scale per moment, held as a byte: the exponent (biased by
// 127) of the values with the largest exponent code.  With E = byte - 127,
//   value = (1 + mantissa / 2^bits) 2^(E - 7 + exponent)   exponent 1..7
//   value = (mantissa / 2^bits) 2^(E - 6)                  exponent 0
// The byte is the least that lets the top code reach the block's largest
// magnitude; bytes lie in [20, 245], and 255 marks a block that holds a
// value that is not finite or whose magnitude passes the top code of byte
// 245 (just under 2^119): all of it reads
// as NaN.
//
// Floating codes under a power-of-two scale, rather than even steps under the
// block's exact maximum: an element whose value does not change keeps its
// code exactly when the block's scale moves (above the subnormal end), so
// the state does not drift by repeated rounding; every value is exact in
// bf16.  A rounding moves a first moment by at most 1/32 and a root by at
// most 1/64 of itself (nearest; down to E - 6).  A root above zero never
// becomes zero (its code is at least 1), so that no update is divided by eps
// alone.
//
// Encoding takes the 32-bit pattern of |x| 2^-(E + 8) 2^-112: the codes' least
// normal value then is the type's own, so that its subnormal numbers round
// where the codes' do, and the code is the top of the pattern after rounding.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace muonb200 {

constexpr int kA8Block = 256;     // elements per scale: one warp, 8 per lane
constexpr int kA8MBits = 4;       // mantissa bits of the first moment's codes
constexpr int kA8RBits = 5;       // ... of the root's
constexpr uint32_t kA8Low = 20, kA8High = 245, kA8NaN = 255;

// Two products, each rounded by itself.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// Two sums a + b, each rounded by itself.  Written as a + b or with a visible
// factor of 1, the sum of a product is joined with it into one rounding all
// the same (measured: the second moment's last bit), so the factor, which is
// 1, comes with the kernel's arguments.
__device__ __forceinline__ float2 add2(float2 a, float2 b, float one) {
  return __ffma2_rn(a, make_float2(one, one), b);
}

// Mixes 32 bits: exclusive-or with the upper bits and products with odd
// constants, chosen by measuring how often each input bit flips each output
// bit (0.500 +- 0.004 over 2^18 inputs for the worst of the 1024 pairs).
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x57735285u;
  x = (x ^ (x >> 15)) * 0x4746E6A3u;
  return x ^ (x >> 16);
}

// Scale byte of a block from the pattern of its largest magnitude.  A
// mantissa past the top code's (all `bits` ones) takes the next exponent, in
// both roundings, so that rounding up never leaves the codes.
template <int kBits>
__device__ __forceinline__ uint32_t a8_scale_byte(uint32_t largest) {
  const uint32_t e = (largest + ((1u << (23 - kBits)) - 1u)) >> 23;
  return e > kA8High ? kA8NaN : (e < kA8Low ? kA8Low : e);
}

__device__ __forceinline__ float a8_divisor(uint32_t byte) {     // 2^-(E + 8)
  return __uint_as_float((246u - byte) << 23);
}

__device__ __forceinline__ float a8_factor(uint32_t byte) {      // 2^(E + 8)
  return byte > kA8High ? __uint_as_float(0x7fc00000u) : __uint_as_float((byte + 8u) << 23);
}

// Four codes of one word -> values.  The codes' exponent and mantissa bits go
// where fp16 has its own (its subnormal numbers included), two at a time;
// `factor` is 2^(E + 8).
__device__ __forceinline__ void a8_decode_m4(uint32_t w, float factor, float2* x) {
  const float2 f2 = make_float2(factor, factor);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h = __byte_perm(w, 0, k ? 0x3424 : 0x1404);       // bytes to the halves' tops
    h = (h & 0x80008000u) | ((h >> 2) & 0x1FC01FC0u);
    x[k] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), f2);
  }
}

__device__ __forceinline__ void a8_decode_r4(uint32_t w, float factor, float2* x) {
  const float2 f2 = make_float2(factor, factor);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t h = __byte_perm(w, 0, k ? 0x4342 : 0x4140) << 5;
    x[k] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), f2);
  }
}

// Largest magnitude of three, NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Pattern of the largest magnitude of a warp's 256 values.
__device__ __forceinline__ uint32_t warp_largest(const float2 (&x)[4]) {
  float big = max_abs3(x[0].x, x[0].y, x[1].x);
  big = max_abs3(big, x[1].y, x[2].x);
  big = max_abs3(big, x[2].y, x[3].x);
  big = max_abs3(big, x[3].y, 0.f);
  return __reduce_max_sync(0xffffffffu, __float_as_uint(big) & 0x7fffffffu);
}

// Patterns of the values times 2^-(E + 8) 2^-112, before rounding; sign: the
// sign bit to give the factor.  For bytes up to 133 (magnitudes below 128) the
// two factors are one normal number.
__device__ __forceinline__ void a8_scaled(const float2 (&x)[4], uint32_t byte, uint32_t sign,
                                          float2 (&y)[4]) {
  if (byte <= 133u) {
    const float d = __uint_as_float(((134u - byte) << 23) | sign);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = mul2(x[k], make_float2(d, d));
  } else {
    const float d = __uint_as_float(__float_as_uint(a8_divisor(byte)) | sign);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = mul2(mul2(x[k], make_float2(d, d)), make_float2(0x1p-112f, 0x1p-112f));
  }
}

// Rounds a pattern to the codes' bits: from bit 23 - kBits on it then is code,
// zeros and sign.  sixteen: 16 random bits (stochastic rounding).
template <int kBits, bool kStochastic>
__device__ __forceinline__ uint32_t a8_round(uint32_t b, uint32_t sixteen) {
  constexpr int kLow = 23 - kBits;
  if (kStochastic) return b + (sixteen << (kLow - 16));
  return b + ((1u << (kLow - 1)) - 1u) + ((b >> kLow) & 1u);
}

// Upper halves of two words in one.
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  return __byte_perm(a, b, 0x7632);
}

// Encodes a lane's 8 elements of both moments; the warp holds one block.
// m: first moments, nr: roots with a minus sign (both 0 past the tensor's
// end); x: per element the 32 random bits before mix32's last step, which
// leaves their upper half (for r) as it is and joins it to the lower (for m);
// zeros: whether some of the lane's roots may be zero.
template <bool kStochastic>
__device__ __forceinline__ void a8_encode_block(const float2 (&m)[4], const float2 (&nr)[4],
                                                const uint32_t (&x)[8], bool zeros,
                                                uint32_t (&m8)[2], uint32_t (&r8)[2],
                                                uint32_t& mbyte, uint32_t& rbyte) {
  mbyte = a8_scale_byte<kA8MBits>(warp_largest(m));
  rbyte = a8_scale_byte<kA8RBits>(warp_largest(nr));
  float2 ms[4], rs[4];
  a8_scaled(m, mbyte == kA8NaN ? kA8Low : mbyte, 0u, ms);
  a8_scaled(nr, rbyte == kA8NaN ? kA8Low : rbyte, 0x80000000u, rs);
  uint32_t mh[4], rh[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t h0 = x[2 * k] >> 16, h1 = x[2 * k + 1] >> 16;
    // sign in bit 31, code in bits 25..19
    mh[k] = upper_halves(a8_round<kA8MBits, kStochastic>(__float_as_uint(ms[k].x),
                                                         (x[2 * k] ^ h0) & 0xffffu),
                         a8_round<kA8MBits, kStochastic>(__float_as_uint(ms[k].y),
                                                         (x[2 * k + 1] ^ h1) & 0xffffu));
    // a root above zero starts from code 1's pattern at least; code in bits 25..18
    constexpr float kOne = 0x1p-131f;
    static_assert(kA8RBits == 5, "kOne is code 1's pattern, 1 << 18");
    rh[k] = upper_halves(
        a8_round<kA8RBits, kStochastic>(__float_as_uint(fmaxf(rs[k].x, kOne)), h0),
        a8_round<kA8RBits, kStochastic>(__float_as_uint(fmaxf(rs[k].y, kOne)), h1));
    if (zeros) {
      if (nr[k].x == 0.f) rh[k] &= 0xffff0000u;
      if (nr[k].y == 0.f) rh[k] &= 0x0000ffffu;
    }
    // codes to the halves' upper bytes, the first moments' below their signs
    mh[k] = ((mh[k] << 5) & 0x7fff7fffu) | (mh[k] & ~0x7fff7fffu);
    rh[k] <<= 6;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    m8[k] = mbyte == kA8NaN ? 0u : __byte_perm(mh[2 * k], mh[2 * k + 1], 0x7531);
    r8[k] = rbyte == kA8NaN ? 0u : __byte_perm(rh[2 * k], rh[2 * k + 1], 0x7531);
  }
}

}  // namespace muonb200
