// Causal sliding-window attention over packed sequences with grouped heads
// (definition: ptb.h).  One warp per (query row, head) walks the row's keys
// with a running maximum and sum.
#include "kv_device.cuh"

namespace ptb {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) swa_packed_kernel(const SwaPackedArgs a) {
  constexpr int E = (D + 31) / 32;  // channels a lane holds: lane, lane + 32, ...
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = row / a.heads;
  const int h = static_cast<int>(row % a.heads);
  if (row == 0)
    for (int i = lane; i < a.batch; i += 32)
      if (a.cu_q[i] < 0 || a.cu_q[i + 1] < a.cu_q[i] || a.cu_q[i + 1] > a.tokens_q)
        record_error(a.status, PTB_ERR_ARG);
  if (t >= a.tokens_q) return;
  const int b = find_sequence(a.cu_q, a.batch, t, lane);
  if (b >= a.batch) return;
  const int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  if (q0 < 0 || q0 > t || q1 > a.tokens_q || k0 < 0 || k1 < k0 || k1 > a.tokens_k) {
    if (lane == 0) record_error(a.status, PTB_ERR_ARG);
    return;
  }
  const int64_t p = (k1 - k0) - (q1 - q0) + (t - q0);
  const int kvh = h / (a.heads / a.kv_heads);
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane + 32 * e;
    q[e] = c < D ? __bfloat162float(a.q[t * a.q_st + h * a.q_sh + c]) * a.scale_log2 : 0.f;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = p - a.window + 1 > 0 ? p - a.window + 1 : 0; j <= p; ++j) {
    const __nv_bfloat16* kr = a.k + (k0 + j) * a.k_st + kvh * a.k_sh;
    const __nv_bfloat16* vr = a.v + (k0 + j) * a.v_st + kvh * a.v_sh;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane + 32 * e;
      if (c < D) s = fmaf(q[e], __bfloat162float(kr[c]), s);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mx = fmaxf(m, s);
    const float alpha = exp2f(m - mx), pr = exp2f(s - mx);
    m = mx;
    l = fmaf(l, alpha, pr);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane + 32 * e;
      if (c < D) acc[e] = fmaf(acc[e], alpha, pr * __bfloat162float(vr[c]));
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane + 32 * e;
    if (c < D)
      a.o[t * a.o_st + h * a.o_sh + c] = __float2bfloat16_rn(p >= 0 ? acc[e] / l : 0.f);
  }
}

template <int D>
cudaError_t launch_typed(const SwaPackedArgs& a, cudaStream_t stream) {
  const int64_t rows = a.tokens_q * a.heads;
  const int64_t blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  swa_packed_kernel<D><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t swa_packed_workspace(int, int64_t, int, int) { return 0; }

cudaError_t launch_swa_packed(const SwaPackedArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 16: return launch_typed<16>(a, stream);
    case 32: return launch_typed<32>(a, stream);
    case 64: return launch_typed<64>(a, stream);
    case 96: return launch_typed<96>(a, stream);
    case 128: return launch_typed<128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ptb
