// The gated feed-forward of a few tokens (a decoding step): y = [resid +] (act(x Wg^T) * (x Wu^T)) Wd^T
// for at most kThinTokens rows of x.
//
// The weights are read once and used for a handful of rows: a stream of 6 hidden ffn bytes, with
// 2 flops per byte and row.  The tcgen05 kernel (128-row tiles, one CTA per SM and weight tile) left
// a third of the SMs without a tile and reads each weight row in pieces of 128 bytes; here the rows
// of a tile are 16, so that every SM has several blocks of warps, and a warp reads long runs of each
// row straight into the registers that mma.sync takes them from:
//   - a block has 16 rows of the weights (of both gate and up) and all of K, its 8 warps a slice of K
//     each; their sums are joined in shared memory in a fixed order, then the epilogue runs;
//   - in m16n8k16 the weights are the 16-row operand and tokens the 8 columns.  A lane loads 16
//     bytes of a row, k = 8 t .. 8 t + 7 of 32: the fragment wants pairs of k in another order, but
//     the order of a contraction's index does not matter as long as x is loaded in the same one.
// Bound by memory: hidden 5120, ffn 13824, one token 67 us (6.3 TB/s; the tcgen05 kernel 86), 16 tokens
// 81, 24 tokens 91, where the reading of x by every block takes 18.  (A cluster for the
// K of 64 rows, x in shared memory: 154 us; the rounds of copies, barriers and remote sums cost more.)
#include "gated_device.cuh"

namespace ptb {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;  // rows of a weight matrix per tile

__device__ __forceinline__ uint4 load_stream(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 tokens.  MT: tiles of 16 rows of each weight matrix per block.  GATED: two weight
// matrices, act(gate) * up; else one, with the residual.
template <int NT, int MT, bool GATED>
__global__ void __launch_bounds__(kThreads, NT > 2 || MT > 1 ? 2 : 3) thin_kernel(const __grid_constant__ ThinArgs p) {
  constexpr int NW = GATED ? 2 : 1;                  // weight matrices
  constexpr int TILES = NW * MT;                     // 16-row tiles of a warp
  constexpr int U = TILES >= 4 ? 1 : 4 / TILES;      // steps of 64 k in flight
  constexpr int ROWS = TILES * kRows;
  constexpr int AHEAD = 8;                           // steps asked for before the wait
  extern __shared__ float part[];                    // [kWarps][ROWS][NT * 8 + 1]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * (MT * kRows);
  const int steps = p.K / 64;
  const int first = warp * steps / kWarps, last = (warp + 1) * steps / kWarps;

  const __nv_bfloat16* w[TILES];  // row g of each tile; row g + 8 is 8 K further on
#pragma unroll
  for (int m = 0; m < TILES; ++m)
    w[m] = (m / MT ? p.w1 : p.w0) + static_cast<int64_t>(n0 + (m % MT) * kRows + g) * p.K + 8 * t;
  const int64_t half = 8 * static_cast<int64_t>(p.K);
  const __nv_bfloat16* x[NT];
  bool live[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    live[j] = 8 * j + g < p.tokens;
    x[j] = p.x + (live[j] ? 8 * j + g : 0) * p.ld_x + 8 * t;
  }

  float acc[TILES][NT][4];
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;

  auto product = [&](int s, const uint4 (&wv)[TILES][2][2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 xv = make_uint4(0, 0, 0, 0);
        if (live[j]) xv = *reinterpret_cast<const uint4*>(x[j] + s * 64 + q * 32);
#pragma unroll
        for (int m = 0; m < TILES; ++m) {
          const uint4 &a = wv[m][0][q], &b = wv[m][1][q];
          mma_16x8x16(acc[m][j], a.x, b.x, a.y, b.y, xv.x, xv.y);
          mma_16x8x16(acc[m][j], a.z, b.z, a.w, b.w, xv.z, xv.w);
        }
      }
    }
  };
  auto load = [&](int s, uint4 (&wv)[TILES][2][2]) {
#pragma unroll
    for (int m = 0; m < TILES; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) wv[m][h][q] = load_stream(w[m] + h * half + s * 64 + q * 32);
  };

  // The down projection's first weights are on their way to L2 while the kernel in front, whose output
  // is its x, still runs (and writes no weights; what is in front of that one has ended, or this one
  // could not have started).
  if constexpr (!GATED) {
    for (int i = 0; i < AHEAD && first + i < last; ++i)
#pragma unroll
      for (int m = 0; m < TILES; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (t == 0)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(w[m] + h * half + (first + i) * 64));
  }
  wait_for_prior();
  dependents_may_start();
  int s = first;
  for (; s + U <= last; s += U) {
    uint4 wv[U][TILES][2][2];
#pragma unroll
    for (int i = 0; i < U; ++i) load(s + i, wv[i]);
#pragma unroll
    for (int i = 0; i < U; ++i) product(s + i, wv[i]);
  }
  if constexpr (U > 1) {
    for (; s < last; ++s) {
      uint4 wv[TILES][2][2];
      load(s, wv);
      product(s, wv);
    }
  }

  constexpr int PAD = NT * 8 + 1;
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[(warp * ROWS + m * kRows + g + 8 * (e >> 1)) * PAD + 8 * j + 2 * t + (e & 1)] = acc[m][j][e];
  __syncthreads();
  const GatedAct act(p.act);
  for (int i = threadIdx.x; i < MT * kRows * p.tokens; i += kThreads) {
    const int r = i % (MT * kRows), k = i / (MT * kRows);
    float v[NW];
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      v[m] = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) v[m] += part[(q * ROWS + m * MT * kRows + r) * PAD + k];
    }
    float out = GATED ? act.value(v[0]) * v[NW - 1] : v[0];
    if (!GATED && p.resid) out += __bfloat162float(p.resid[k * p.ld_resid + n0 + r]);
    p.out[k * p.ld_out + n0 + r] = __float2bfloat16_rn(out);
  }
}

template <int NT, int MT, bool GATED>
cudaError_t launch_one(const ThinArgs& a, cudaStream_t stream) {
  constexpr int bytes = kWarps * (GATED ? 2 : 1) * MT * kRows * (NT * 8 + 1) * 4;
  auto kern = thin_kernel<NT, MT, GATED>;
  if constexpr (bytes > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kern, dim3(a.N / (MT * kRows)), dim3(kThreads), bytes, stream, a);
}

// Every block reads all of x, through L1: from 9 tokens on, two 16-row tiles a block halve that where
// the blocks still cover the SMs (the down projection of 13824 by 5120, 24 tokens: the pair of kernels
// 89.5 us for 96).  With both gate and up the second pair of tiles would spill (123 us).
template <bool GATED>
cudaError_t launch(const ThinArgs& a, cudaStream_t stream) {
  const int nt = (a.tokens + 7) / 8;
  if (nt == 1) return launch_one<1, 1, GATED>(a, stream);
  if (nt > 4) return cudaErrorInvalidValue;
  if constexpr (!GATED) {
    if (a.N / (2 * kRows) >= a.sms)
      return nt == 2 ? launch_one<2, 2, GATED>(a, stream) : launch_one<4, 2, GATED>(a, stream);
  }
  return nt == 2 ? launch_one<2, 1, GATED>(a, stream) : launch_one<4, 1, GATED>(a, stream);
}

}  // namespace

cudaError_t launch_thin(const ThinArgs& a, cudaStream_t stream) {
  return a.w1 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace ptb
