// 8-bit activation checkpoints (layout: ptb.h): groups of 32 neighbouring channels share a
// power-of-two scale 2^(E - 127), codes are int8 in -127 .. 127.
//
// E follows from the group's largest magnitude m: the smallest scale with m < 127.5 scale, so that
// no code needs clamping and every finite value is off by at most half a step.  In the bits of m
// that is an addition: the exponent field of m + 2^16 ulp, less 6 (the carry is the case of a
// mantissa of 127.5 / 64 and more).  A power of two makes both directions exact but for the one
// rounding to a code, and code times scale has at most 7 significant bits: the value that a code
// stands for is a bf16 number, so the kernels that read a checkpoint and a program that unpacks it
// to bf16 see the same values.
#pragma once

#include "ptb_device.cuh"

namespace ptb {

constexpr int kCkptGroup = 32;
constexpr unsigned kCkptBad = 255;  // the group holds a value that is not finite, or so large
                                    // (255 * 2^120 and more) that its code would stand for one

// Exponent byte of a group from the largest magnitude's bits (as integers magnitudes order like
// their values, and infinities and NaN come out above every finite one).
__device__ __forceinline__ unsigned ckpt_exponent(uint32_t max_bits) {
  if (max_bits >= 0x7f7f0000u) return kCkptBad;
  const int e = static_cast<int>((max_bits + 0x10000u) >> 23) - 6;
  return static_cast<unsigned>(e < 1 ? 1 : e);
}

// 2^(127 - E): what a value is multiplied with before it is rounded.
__device__ __forceinline__ float ckpt_inverse(unsigned e) {
  return e == kCkptBad ? 0.f : __uint_as_float((254u - e) << 23);
}

__device__ __forceinline__ float ckpt_scale(unsigned e) {
  return __uint_as_float(e == kCkptBad ? 0x7fc00000u : e << 23);
}

// Rounds to nearest even by adding 1.5 * 2^23: a sum's low byte is the code.
__device__ __forceinline__ uint32_t ckpt_pack4(float a, float b, float c, float d, float inverse) {
  const uint32_t lo = __byte_perm(__float_as_uint(fmaf(a, inverse, 12582912.f)),
                                  __float_as_uint(fmaf(b, inverse, 12582912.f)), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(fmaf(c, inverse, 12582912.f)),
                                  __float_as_uint(fmaf(d, inverse, 12582912.f)), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// The four codes of a word as fp32: a code plus 128 in the mantissa of 2^23, less 2^23 + 128.
__device__ __forceinline__ void ckpt_unpack4(uint32_t codes, float (&v)[4]) {
  const uint32_t u = codes ^ 0x80808080u;
  v[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.f;
  v[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.f;
  v[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - 8388736.f;
  v[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - 8388736.f;
}

// The same as packed pairs, times the scale.  (As one fma, (2^23 + 128 + c) s - (2^23 + 128) s, it
// would overflow for scales from 2^104 on.)
__device__ __forceinline__ void ckpt_unpack4_scaled(uint32_t codes, float scale, uint64_t (&v)[2]) {
  const uint32_t u = codes ^ 0x80808080u;
  const uint64_t s = f2(scale, scale), off = f2(-8388736.f, -8388736.f);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    v[h] = f2_mul(f2_add(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + 2 * h)),
                            __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441 + 2 * h))),
                         off),
                  s);
}

// One whole group held by a thread: its 32 values to codes and an exponent byte.
__device__ __forceinline__ void ckpt_store_group(const float (&v)[32], uint8_t* codes,
                                                 uint8_t* exponent) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  const unsigned e = ckpt_exponent(m);
  const float inv = ckpt_inverse(e);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = ckpt_pack4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], inv);
    if (e == kCkptBad) w[j] = 0;
  }
  uint4* dst = reinterpret_cast<uint4*>(codes);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  *exponent = static_cast<uint8_t>(e);
}

}  // namespace ptb
