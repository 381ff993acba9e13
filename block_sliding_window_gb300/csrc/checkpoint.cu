// 8-bit activation checkpoints: packing a bf16 tensor and reading it back (format and rounding:
// checkpoint_device.cuh).
//
// Both directions are streams: 2 bytes of bf16 against 1 + 1/32 of a checkpoint per value.  A
// thread holds 8 neighbouring channels (16 bytes of bf16, 8 of codes), four lanes a group; the
// group's largest magnitude is taken over them with two shuffles.
#include "checkpoint_device.cuh"

namespace ptb {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    pack_kernel(const __nv_bfloat16* __restrict__ x, int64_t ld_x, int64_t rows, int vecs,
                uint8_t* __restrict__ codes, int64_t ld_codes, uint8_t* __restrict__ exps,
                int64_t ld_exps) {
  // vecs = cols / 8 is a multiple of 4: the four lanes of a group are in range together.
  const int64_t total = rows * vecs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
       i - (threadIdx.x & 31) < total; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const bool in = i < total;
    const int64_t row = in ? i / vecs : 0;
    const int v = in ? static_cast<int>(i - row * vecs) : 0;
    const uint4 p = in ? __ldcs(reinterpret_cast<const uint4*>(x + row * ld_x) + v)
                       : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = max(m, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const unsigned e = ckpt_exponent(m);
    const float inv = ckpt_inverse(e);
    uint2 c = make_uint2(ckpt_pack4(bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1]), inv),
                         ckpt_pack4(bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3]), inv));
    if (e == kCkptBad) c = make_uint2(0, 0);
    if (in) {
      reinterpret_cast<uint2*>(codes + row * ld_codes)[v] = c;
      if ((v & 3) == 0) exps[row * ld_exps + (v >> 2)] = static_cast<uint8_t>(e);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const uint8_t* __restrict__ codes, int64_t ld_codes,
                  const uint8_t* __restrict__ exps, int64_t ld_exps, int64_t rows, int vecs,
                  __nv_bfloat16* __restrict__ x, int64_t ld_x) {
  const int64_t total = rows * vecs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = i / vecs;
    const int v = static_cast<int>(i - row * vecs);
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(codes + row * ld_codes) + v);
    const float s = ckpt_scale(__ldg(exps + row * ld_exps + (v >> 2)));
    float a[4], b[4];
    ckpt_unpack4(c.x, a);
    ckpt_unpack4(c.y, b);
    reinterpret_cast<uint4*>(x + row * ld_x)[v] =
        make_uint4(pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(a[2] * s, a[3] * s),
                   pack_bf16x2(b[0] * s, b[1] * s), pack_bf16x2(b[2] * s, b[3] * s));
  }
}

int64_t blocks_of(int64_t rows, int64_t cols, int sms) {
  const int64_t all = (rows * (cols / 8) + kThreads - 1) / kThreads;
  const int64_t most = static_cast<int64_t>(sms) * 8;
  return all < most ? all : most;
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CheckpointArgs& a, cudaStream_t stream) {
  pack_kernel<<<static_cast<unsigned>(blocks_of(a.rows, a.cols, a.sms)), kThreads, 0, stream>>>(
      a.x, a.ld_x, a.rows, static_cast<int>(a.cols / 8), a.codes, a.ld_codes, a.exps, a.ld_exps);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const CheckpointArgs& a, cudaStream_t stream) {
  unpack_kernel<<<static_cast<unsigned>(blocks_of(a.rows, a.cols, a.sms)), kThreads, 0, stream>>>(
      a.codes, a.ld_codes, a.exps, a.ld_exps, a.rows, static_cast<int>(a.cols / 8), a.x_out, a.ld_x);
  return cudaGetLastError();
}

}  // namespace ptb
