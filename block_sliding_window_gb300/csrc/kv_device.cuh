// Device-side helpers of the serving kernels: finding a token's sequence,
// cache addresses, and the 4-bit row format (ptb.h has the layout).
#pragma once

#include "ptb_device.cuh"

namespace ptb {

// Lets a kernel use `bytes` of dynamic shared memory, once per device.  Two
// threads that set it at the same time set the same value.
constexpr int kDeviceSlots = 64;
template <typename K>
cudaError_t allow_smem(K kern, int bytes, bool (&configured)[kDeviceSlots]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDeviceSlots && configured[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < kDeviceSlots) configured[dev] = true;
  return e;
}

// 16 bytes that this SM uses once, past L1.
__device__ __forceinline__ uint4 load16_past_l1(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void store16_past_l1(void* p, const uint4& v) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Scores beyond fp32's grain.  exp2(s f - m), with m = s f of the row's largest
// score rounded to fp32, takes the exact product in its FMA: the largest weight
// comes out as 2^r, r up to half a step of m.  That cancels in O / l until r is
// tens (m of 2^31: 128, and the weight infinite or 0).  From kLargeScore on a row
// therefore goes on with f rounded up to a power of two, which makes products
// exact and r zero.  It changes no weight that counts: fp32 scores that differ
// do so by at least 2^-24 of themselves, here 32, so every weight is that of the
// largest score or below 2^-32 of it, with either factor; and as f only grows,
// maxima of parts of a row that went either way keep their order.  A row whose
// scores so far were all below -2^29 takes f itself again where one is not.
constexpr float kLargeScore = 536870912.f;  // 2^29, in the log2 domain
// The reference max of a row whose largest score is `largest`, and the factor
// that goes with it, from the row's own factor f > 0.
__device__ __forceinline__ float reference_max(float largest, float f, float& factor) {
  factor = f;
  const float m = __fmul_rn(largest, f);
  if (fabsf(m) < kLargeScore) return m;
  factor = __uint_as_float((__float_as_uint(f) + 0x007fffffu) & 0xff800000u);
  return __fmul_rn(largest, factor);
}

constexpr int kKvGroup = 32;  // channels that share one (scale, centre) pair

// The sequence of token t: the first b < batch with cu[b + 1] > t, or batch.
// A whole warp searches with 32 probes a step, so up to 32 sequences take one
// load and up to 1024 take two.  Every lane returns the same b.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t t, int lane) {
  int lo = 0, len = batch;
  while (len > 0) {
    const int step = (len + 31) >> 5;
    const int64_t at = lo + static_cast<int64_t>(lane) * step + step - 1;
    const bool past = at >= lo + len ? true : cu[at + 1] > t;
    const unsigned vote = __ballot_sync(0xffffffffu, past);
    if (vote == 0) return lo + len;
    const int f = __ffs(vote) - 1;
    if (step == 1) return min(lo + f, batch);
    const int64_t skip = static_cast<int64_t>(f) * step;
    if (skip >= len) return lo + len;
    lo += static_cast<int>(skip);
    len = min(step, len - static_cast<int>(skip));
  }
  return lo;
}

// The start of position p's page of sequence b, or null when the entry is
// outside the table or the cache.
__device__ __forceinline__ uint8_t* kv_page(const KvCache& c, int b, int64_t p) {
  const int64_t i = p >> c.page_shift;
  if (i >= c.table_pages) return nullptr;
  const int64_t page = c.table[b * c.table_stride + i];
  if (page < 0 || page >= c.pages) return nullptr;
  return c.base + page * c.page_bytes;
}

// Byte offsets inside a row of d / 2 code bytes (ng = d / 32 groups).
// Key word of channels 32 w + 8 t .. + 7:
__device__ __forceinline__ int key_word(int w, int t, int ng) { return 4 * (t * ng + w); }
// Value half-word of channels 32 w + 4 g .. + 3:
__device__ __forceinline__ int value_half(int w, int g, int ng) { return 2 * (g * ng + w); }

// The four nibbles of each 16-bit half of w as bf16 u - 8, exact: v[k] holds
// nibble k of the low and of the high half.  A nibble in mantissa bits 0 .. 3
// of 128 is 128 + u, in bits 3 .. 6 of 16 it is 16 + u: three shifts for four.
__device__ __forceinline__ uint32_t bf16x2_add(uint32_t x, float c) {
  __nv_bfloat162 v = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&x), __floats2bfloat162_rn(c, c));
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t r = w >> 8;
  v[0] = bf16x2_add((w & 0x000f000fu) | 0x43004300u, -136.f);
  v[1] = bf16x2_add(((w >> 1) & 0x00780078u) | 0x41804180u, -24.f);
  v[2] = bf16x2_add((r & 0x000f000fu) | 0x43004300u, -136.f);
  v[3] = bf16x2_add(((r >> 1) & 0x00780078u) | 0x41804180u, -24.f);
}

}  // namespace ptb
