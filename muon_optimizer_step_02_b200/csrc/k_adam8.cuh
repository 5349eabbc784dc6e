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

// Magnitude code of |x|; sixteen: 16 random bits (stochastic rounding).
template <int kBits, bool kStochastic>
__device__ __forceinline__ uint32_t a8_encode(float ax, float divisor, uint32_t sixteen) {
  constexpr int kLow = 23 - kBits;
  uint32_t b = __float_as_uint(ax * divisor * 0x1p-112f);
  if (kStochastic) b += sixteen << (kLow - 16);
  else b += ((1u << (kLow - 1)) - 1u) + ((b >> kLow) & 1u);
  return b >> kLow;
}

// Four codes of one word -> values.  The codes' exponent and mantissa bits go
// where fp16 has its own (its subnormal numbers included), two at a time;
// `factor` is 2^(E + 8).
__device__ __forceinline__ void a8_decode_m4(uint32_t w, float factor, float (&x)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h = __byte_perm(w, 0, k ? 0x3424 : 0x1404);       // bytes to the halves' tops
    h = (h & 0x80008000u) | ((h >> 2) & 0x1FC01FC0u);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * k] = f.x * factor;
    x[2 * k + 1] = f.y * factor;
  }
}

__device__ __forceinline__ void a8_decode_r4(uint32_t w, float factor, float (&x)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t h = __byte_perm(w, 0, k ? 0x4342 : 0x4140) << 5;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * k] = f.x * factor;
    x[2 * k + 1] = f.y * factor;
  }
}

// Encodes a lane's 8 elements of both moments; the warp holds one block.
// m: first moments, r: roots (both 0 past the tensor's end); word: per
// element 32 random bits (the lower half for m, the upper for r).
template <bool kStochastic>
__device__ __forceinline__ void a8_encode_block(const float (&m)[8], const float (&r)[8],
                                                const uint32_t (&word)[8], uint32_t (&m8)[2],
                                                uint32_t (&r8)[2], uint32_t& mbyte,
                                                uint32_t& rbyte) {
  uint32_t ml = 0, rl = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ml = max(ml, __float_as_uint(m[e]) & 0x7fffffffu);
    rl = max(rl, __float_as_uint(r[e]) & 0x7fffffffu);
  }
  mbyte = a8_scale_byte<kA8MBits>(__reduce_max_sync(0xffffffffu, ml));
  rbyte = a8_scale_byte<kA8RBits>(__reduce_max_sync(0xffffffffu, rl));
  const float md = a8_divisor(mbyte), rd = a8_divisor(rbyte);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t mw = 0, rw = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * k + i;
      const uint32_t sign = (__float_as_uint(m[e]) >> 24) & 0x80u;
      const uint32_t cm =
          a8_encode<kA8MBits, kStochastic>(fabsf(m[e]), md, word[e] & 0xffffu) | sign;
      uint32_t cr = a8_encode<kA8RBits, kStochastic>(r[e], rd, word[e] >> 16);
      cr = max(cr, r[e] > 0.f ? 1u : 0u);
      mw |= cm << (8 * i);
      rw |= cr << (8 * i);
    }
    m8[k] = mbyte == kA8NaN ? 0u : mw;
    r8[k] = rbyte == kA8NaN ? 0u : rw;
  }
}

}  // namespace muonb200
