// 8-bit activation checkpoints: packing a bf16 tensor and reading it back (format and rounding:
// checkpoint_device.cuh).
//
// Both directions are streams: 2 bytes of bf16 against 1 + 1/32 of a checkpoint per value.  A
// thread takes 16 neighbouring channels (32 bytes of bf16, 16 of codes), two lanes a group, and
// kUnits such pieces at once; the group's largest magnitude is exchanged with one shuffle.  A tensor
// without gaps between its rows is one long row.  2048 rows of 27648 packed and read back take
// 58.5 us (5.9 TB/s); with 8 channels a thread and a division for each 73.
#include "checkpoint_device.cuh"

namespace ptb {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;

// A grid of (pieces, rows): blockIdx.x, .y and the strides between a block's turns.
struct Walk {
  int64_t rows, units;  // units of 16 channels of a row: an even number
};

__global__ void __launch_bounds__(kThreads)
    pack_kernel(const __nv_bfloat16* __restrict__ x, int64_t ld_x, Walk n,
                uint8_t* __restrict__ codes, int64_t ld_codes, uint8_t* __restrict__ exps,
                int64_t ld_exps) {
  for (int64_t row = blockIdx.y; row < n.rows; row += gridDim.y) {
    const uint4* src = reinterpret_cast<const uint4*>(x + row * ld_x);
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnits); at < n.units;
         at += static_cast<int64_t>(gridDim.x) * (kThreads * kUnits)) {
      uint4 p[kUnits][2];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int64_t u = at + k * kThreads + threadIdx.x;
        p[k][0] = p[k][1] = make_uint4(0, 0, 0, 0);
        if (u < n.units) {
          p[k][0] = __ldcs(src + 2 * u);
          p[k][1] = __ldcs(src + 2 * u + 1);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int64_t u = at + k * kThreads + threadIdx.x;
        const uint32_t w[8] = {p[k][0].x, p[k][0].y, p[k][0].z, p[k][0].w,
                               p[k][1].x, p[k][1].y, p[k][1].z, p[k][1].w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const unsigned e = ckpt_exponent(m);
        const float inv = ckpt_inverse(e);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[j] = ckpt_pack4(bf16_lo(w[2 * j]), bf16_hi(w[2 * j]), bf16_lo(w[2 * j + 1]),
                            bf16_hi(w[2 * j + 1]), inv);
          if (e == kCkptBad) c[j] = 0;
        }
        if (u < n.units) {
          reinterpret_cast<uint4*>(codes + row * ld_codes)[u] = make_uint4(c[0], c[1], c[2], c[3]);
          if ((u & 1) == 0) exps[row * ld_exps + (u >> 1)] = static_cast<uint8_t>(e);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const uint8_t* __restrict__ codes, int64_t ld_codes,
                  const uint8_t* __restrict__ exps, int64_t ld_exps, Walk n,
                  __nv_bfloat16* __restrict__ x, int64_t ld_x) {
  for (int64_t row = blockIdx.y; row < n.rows; row += gridDim.y) {
    const uint4* src = reinterpret_cast<const uint4*>(codes + row * ld_codes);
    const uint8_t* scales = exps + row * ld_exps;
    uint4* dst = reinterpret_cast<uint4*>(x + row * ld_x);
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnits); at < n.units;
         at += static_cast<int64_t>(gridDim.x) * (kThreads * kUnits)) {
      uint4 c[kUnits];
      unsigned e[kUnits];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int64_t u = at + k * kThreads + threadIdx.x;
        if (u < n.units) {
          c[k] = __ldcs(src + u);
          e[k] = __ldg(scales + (u >> 1));
        }
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int64_t u = at + k * kThreads + threadIdx.x;
        if (u >= n.units) continue;
        const float s = ckpt_scale(e[k]);
        const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
        uint32_t out[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint64_t v[2];
          ckpt_unpack4_scaled(w[j], s, v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float lo, hi;
            f2_split(v[h], lo, hi);
            out[2 * j + h] = pack_bf16x2(lo, hi);
          }
        }
        dst[2 * u] = make_uint4(out[0], out[1], out[2], out[3]);
        dst[2 * u + 1] = make_uint4(out[4], out[5], out[6], out[7]);
      }
    }
  }
}

dim3 plan(const CheckpointArgs& a, Walk* n) {
  *n = {a.rows, a.cols / 16};
  if (a.rows == 1 || (a.ld_x == a.cols && a.ld_codes == a.cols && a.ld_exps == a.cols / 32))
    *n = {1, a.rows * (a.cols / 16)};
  const int64_t wide = (n->units + kThreads * kUnits - 1) / (kThreads * kUnits);
  const int64_t most = static_cast<int64_t>(a.sms) * 32;
  const int64_t x = wide < most ? wide : most;
  int64_t y = most / x;
  if (y > n->rows) y = n->rows;
  if (y > 65535) y = 65535;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < 1 ? 1 : y));
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CheckpointArgs& a, cudaStream_t stream) {
  Walk n;
  const dim3 grid = plan(a, &n);
  pack_kernel<<<grid, kThreads, 0, stream>>>(a.x, a.ld_x, n, a.codes, a.ld_codes, a.exps, a.ld_exps);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const CheckpointArgs& a, cudaStream_t stream) {
  Walk n;
  const dim3 grid = plan(a, &n);
  unpack_kernel<<<grid, kThreads, 0, stream>>>(a.codes, a.ld_codes, a.exps, a.ld_exps, n, a.x_out,
                                               a.ld_x);
  return cudaGetLastError();
}

}  // namespace ptb
