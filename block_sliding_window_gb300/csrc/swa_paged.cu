// Sliding-window attention of one new token per sequence over the paged
// cache (definition and cache layout: ptb.h).  One block per (sequence,
// head); its warps take every fourth key and their running maxima, sums and
// outputs are joined in shared memory.
#include "kv_device.cuh"

namespace ptb {
namespace {

constexpr int kWarps = 4;

// Channel c of row `off` of a block of keys or values.
template <int D>
__device__ __forceinline__ float cached(const KvCache& k, const uint8_t* block, int off, int c,
                                        bool key) {
  constexpr int NG = D / kKvGroup;
  if (k.bits == 16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(block)[off * D + c]);
  if constexpr (NG > 0) {
    const int w = c / 32, x = c % 32;
    const int nibble = key ? 2 * key_word(w, x / 8, NG) + x % 8 : 2 * value_half(w, x / 4, NG) + x % 4;
    const int code = (block[off * (D / 2) + nibble / 2] >> (4 * (nibble & 1))) & 15;
    const uint32_t pair = *reinterpret_cast<const uint32_t*>(block + k.page_size * (D / 2) +
                                                             (off * NG + w) * 4);
    return fmaf(static_cast<float>(code - 8), bf16_lo(pair), bf16_hi(pair));
  }
  return 0.f;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) swa_paged_kernel(const SwaPagedArgs a) {
  constexpr int E = (D + 31) / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x, h = blockIdx.y;
  const int kvh = h / (a.heads / a.c.kv_heads);
  int64_t n = a.lens[b];
  if (n < 0 || n > a.c.table_pages * a.c.page_size) {
    if (threadIdx.x == 0) record_error(a.status, PTB_ERR_ARG);
    n = 0;
  }
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane + 32 * e;
    q[e] = c < D ? __bfloat162float(a.q[b * a.q_sb + h * a.q_sh + c]) * a.scale_log2 : 0.f;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = (n > a.window ? n - a.window : 0) + warp; j < n; j += kWarps) {
    const uint8_t* page = kv_page(a.c, b, j);
    if (!page) {
      if (lane == 0) record_error(a.status, PTB_ERR_ARG);
      continue;
    }
    const int off = static_cast<int>(j) & (a.c.page_size - 1);
    const uint8_t* kb = page + kvh * a.c.block_bytes;
    const uint8_t* vb = page + (a.c.kv_heads + kvh) * a.c.block_bytes;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane + 32 * e;
      if (c < D) s = fmaf(q[e], cached<D>(a.c, kb, off, c, true), s);
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
      if (c < D) acc[e] = fmaf(acc[e], alpha, pr * cached<D>(a.c, vb, off, c, false));
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane + 32 * e < D) so[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  float mx = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w)
    if (sl[w] != 0.f) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < kWarps; ++w)
    if (sl[w] != 0.f) total += sl[w] * exp2f(sm[w] - mx);
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (sl[w] != 0.f) o += so[w][c] * exp2f(sm[w] - mx);
    a.o[b * a.o_sb + h * a.o_sh + c] = __float2bfloat16_rn(total != 0.f ? o / total : 0.f);
  }
}

template <int D>
cudaError_t launch_typed(const SwaPagedArgs& a, cudaStream_t stream) {
  swa_paged_kernel<D><<<dim3(a.batch, a.heads), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t swa_paged_workspace(int, int, int, int, int) { return 0; }

cudaError_t launch_swa_paged(const SwaPagedArgs& a, cudaStream_t stream) {
  switch (a.c.head_dim) {
    case 16: return launch_typed<16>(a, stream);
    case 32: return launch_typed<32>(a, stream);
    case 64: return launch_typed<64>(a, stream);
    case 96: return launch_typed<96>(a, stream);
    case 128: return launch_typed<128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ptb
