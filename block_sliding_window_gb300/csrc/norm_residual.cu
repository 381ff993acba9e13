// The norms before and after a block, fused with its gate and the residual scale (ptb.h,
// ptb_norm_residual):
//   p = N(o) * post_gamma + post_beta,   y = alpha x + gate * p,   h = N(y) * pre_gamma + pre_beta,
// N the layer norm (biased variance) or the rms norm.  y is rounded to bf16 once and h is the norm
// of that rounded y, the same function of the stored stream that a separate norm would compute.
//
// Forward: one pass, 2 H bytes read for x and for o and written for y and h per row.  A row stays
// in the registers of its threads from the first load to the last store; the statistics (means,
// then centred squares) are reduced in fp32.  Rows of up to 1024 channels are a warp's, so that
// their reductions need no barrier; longer ones a block's.
#include "checkpoint_device.cuh"

namespace ptb {
namespace {

__device__ __forceinline__ void unpack8(uint4 p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the threads of a row, the same bits in all of them.  `red` holds two sets of slots for
// the warps of a block, taken in turn, so that one barrier a sum is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& turn) {
  v = warp_sum(v);
  if constexpr (!WARP) {
    float* slots = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    const int lane = threadIdx.x & 31;
    v = warp_sum(lane < warps ? slots[lane] : 0.f);
  }
  return v;
}

// VPT: 16-byte vectors of the row that a thread holds.
template <int VPT, bool WARP, bool RMS>
__global__ void __launch_bounds__(512) norm_residual_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][32];
  const int lanes = WARP ? 32 : blockDim.x;
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                           : blockIdx.x;
  if (WARP && row >= a.rows) return;
  const int nvec = a.hidden >> 3;
  const float inv_n = 1.f / static_cast<float>(a.hidden);
  int turn = 0;

  float p[VPT][8];
  uint4 xv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * lanes;
    if (v < nvec) {
      unpack8(__ldcs(reinterpret_cast<const uint4*>(a.o + row * a.ld_o) + v), p[j]);
      xv[j] = __ldcs(reinterpret_cast<const uint4*>(a.x + row * a.ld_x) + v);
    } else {
      xv[j] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) p[j][e] = 0.f;
    }
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);

  // The mean (0 for the rms norm) and 1 / sqrt(variance + eps) of p.
  auto statistics = [&](float& mean, float& rstd) {
    mean = 0.f;
    if constexpr (!RMS) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += p[j][e];
      mean = row_sum<WARP>(s, red, turn) * inv_n;
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (lane + j * lanes < nvec)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (p[j][e] - mean) * (p[j][e] - mean);
    rstd = rsqrtf(row_sum<WARP>(s, red, turn) * inv_n + a.eps);
  };

  const bool post = a.post_gamma != nullptr;
  if (post) statistics(st.x, st.y);
  const __nv_bfloat16* gate = a.gate ? a.gate + row / (a.rows / a.gates) * a.hidden : nullptr;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * lanes;
    if (v < nvec) {
      float f[8];
      if (post) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.post_gamma) + v), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[j][e] = (p[j][e] - st.x) * st.y * f[e];
        if (a.post_beta) {
          unpack8(__ldg(reinterpret_cast<const uint4*>(a.post_beta) + v), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) p[j][e] += f[e];
        }
      }
      if (gate) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(gate) + v), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[j][e] *= f[e];
      }
      unpack8(xv[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) p[j][e] = fmaf(a.alpha, f[e], p[j][e]);
      const uint4 yv = pack8(p[j]);
      reinterpret_cast<uint4*>(a.y + row * a.ld_y)[v] = yv;
      unpack8(yv, p[j]);
    }
  }
  if (a.h) {
    statistics(st.z, st.w);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * lanes;
      if (v < nvec) {
        float f[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre_gamma) + v), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[j][e] = (p[j][e] - st.z) * st.w * f[e];
        if (a.pre_beta) {
          unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre_beta) + v), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) p[j][e] += f[e];
        }
        reinterpret_cast<uint4*>(a.h + row * a.ld_h)[v] = pack8(p[j]);
      }
    }
  }
  if (a.stats && lane == 0) a.stats[row] = st;
}

// ------------------------------------------------------------ backward --
//
// With d = dy + N'(dh) (the gradient of y, from the stream and through the norm before the next
// block), oh = (o - mean) / sd and yh alike:
//   dx = alpha d,   do = N'(gate * post_gamma * d),   N'(w) = (w - mean(w) - vh mean(w vh)) / sd,
// and of the sums over rows four suffice: S0 = sum d, S1 = sum d oh, S2 = sum dh, S3 = sum dh yh.
//   dpost_beta = gate S0,  dpost_gamma = gate S1,  dgate = post_gamma S1 + post_beta S0,
//   dpre_beta = S2,  dpre_gamma = S3          (S0, S1 for each gate's rows on their own).
//
// Rows are dealt to blocks in runs, a thread has 8 channels of all its block's rows and keeps their
// sums in registers.  Each thread copies its own channels of the next rows into its own part of
// shared memory (cp.async), so the copies run ahead of the arithmetic without any barrier.  Rows of
// more channels than a block has threads for are split over a cluster, whose blocks exchange their
// two pairs of sums through shared memory of each other.  The blocks' sums are joined by a second
// kernel in a fixed order.

constexpr int kSliceMax = 6144;  // channels of one block

struct BackPlan {
  int cluster, threads, slice, groups, stages;
  size_t smem;
};

BackPlan back_plan(int64_t rows, int64_t hidden, int sms) {
  BackPlan p;
  p.cluster = 1;
  while (hidden > static_cast<int64_t>(kSliceMax) * p.cluster) p.cluster *= 2;
  const int64_t vecs = (hidden / 8 + p.cluster - 1) / p.cluster;
  p.slice = static_cast<int>(vecs) * 8;
  p.threads = static_cast<int>((vecs + 31) / 32) * 32;
  int per_sm = 768 / p.threads;
  if (per_sm < 1) per_sm = 1;
  if (per_sm > 16) per_sm = 16;
  int64_t groups = static_cast<int64_t>(sms / p.cluster) * per_sm;
  if (groups > rows) groups = rows;
  p.groups = static_cast<int>(groups < 1 ? 1 : groups);
  const size_t row = static_cast<size_t>(p.threads) * 4 * 16;
  const size_t room = (208 * 1024) / per_sm;
  int64_t st = static_cast<int64_t>(room / row);
  p.stages = static_cast<int>(st > 4 ? 4 : st < 2 ? 2 : st);
  p.smem = row * p.stages;
  return p;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sums of a pair over the threads of a row (all blocks of the cluster), the same bits everywhere.
template <bool CLUSTER>
__device__ __forceinline__ float2 pair_sum(float2 v, float2 (*red)[32], float2 (*peer)[8], int& turn,
                                           int cluster, uint32_t rank) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  float2* slots = red[turn];
  const int lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  if (lane == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  const float2 mine = lane < warps ? slots[lane] : make_float2(0.f, 0.f);
  v.x = warp_sum(mine.x);
  v.y = warp_sum(mine.y);
  if constexpr (CLUSTER) {
    // The first lanes write this block's sums into every block of the cluster.
    if (static_cast<int>(threadIdx.x) < cluster) {
      const uint32_t dst = cluster_map(&peer[turn][rank], threadIdx.x);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(v.x), "f"(v.y) : "memory");
    }
    cluster_sync();
    v = make_float2(0.f, 0.f);
    for (int r = 0; r < cluster; ++r) {
      v.x += peer[turn][r].x;
      v.y += peer[turn][r].y;
    }
  }
  turn ^= 1;
  return v;
}

template <int STAGES, bool CLUSTER, bool RMS, bool O8>
__global__ void __launch_bounds__(kSliceMax / 8, 1)
    norm_residual_backward_kernel(const __grid_constant__ NormArgs a, int cluster, int slice, int groups) {
  extern __shared__ __align__(16) uint4 ring[];  // [STAGES][4][blockDim.x]
  __shared__ float2 red[2][32];
  __shared__ float2 peer[2][8];
  const uint32_t rank = CLUSTER ? cluster_ctarank() : 0;
  const int group = blockIdx.x / cluster;
  const int64_t lo = group * a.rows / groups, hi = (group + 1) * a.rows / groups;
  const int64_t rows_per_gate = a.rows / a.gates;
  const int col = static_cast<int>(rank) * slice + threadIdx.x * 8;
  const bool in = static_cast<int>(threadIdx.x) * 8 < slice && col < a.hidden;
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr;
  const float inv_n = 1.f / static_cast<float>(a.hidden);
  int turn = 0;

  float S0[8], S1[8], S2[8], S3[8], w[8], gn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) S0[e] = S1[e] = S2[e] = S3[e] = w[e] = gn[e] = 0.f;
  if (in && pre) unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre_gamma + col)), gn);

  auto slot = [&](int stage, int t) { return ring + (stage * 4 + t) * blockDim.x + threadIdx.x; };
  auto fetch = [&](int64_t row) {
    if (in && row < hi) {
      const int stage = static_cast<int>((row - lo) % STAGES);
      if (a.dy) cp_async16(slot(stage, 0), a.dy + row * a.ld_dy + col);
      if (O8)
        cp_async8(slot(stage, 1), reinterpret_cast<const uint8_t*>(a.o) + row * a.ld_o + col);
      else
        cp_async16(slot(stage, 1), a.o + row * a.ld_o + col);
      if (pre) {
        cp_async16(slot(stage, 2), a.dh + row * a.ld_dh + col);
        cp_async16(slot(stage, 3), a.y + row * a.ld_y + col);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(lo + s);

  int64_t seg = lo / rows_per_gate;
  int64_t seg_end = 0;
  for (int64_t row = lo; row < hi; ++row) {
    if (row >= seg_end) {  // the first row, or the first of another gate
      seg = row / rows_per_gate;
      seg_end = (seg + 1) * rows_per_gate;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
      if (in) {
        float f[8];
        if (a.gate) unpack8(__ldg(reinterpret_cast<const uint4*>(a.gate + seg * a.hidden + col)), w);
        if (post) {
          unpack8(__ldg(reinterpret_cast<const uint4*>(a.post_gamma + col)), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= f[e];
        }
      }
    }
    const float4 st = __ldg(a.stats + row);
    float o_scale = 1.f;
    if (O8 && in) o_scale = ckpt_scale(__ldg(a.o_exps + row * a.ld_o_exps + col / 32));
    fetch(row + STAGES - 1);
    cp_async_wait<STAGES - 1>();
    const int stage = static_cast<int>((row - lo) % STAGES);

    float d[8], oh[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = oh[e] = 0.f;
    if (in) {
      if (a.dy) unpack8(*slot(stage, 0), d);
      if (O8) {
        const uint2 c = *reinterpret_cast<const uint2*>(slot(stage, 1));
        float f[4];
        ckpt_unpack4(c.x, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) oh[e] = f[e] * o_scale;
        ckpt_unpack4(c.y, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) oh[4 + e] = f[e] * o_scale;
      } else {
        unpack8(*slot(stage, 1), oh);
      }
    }
    if (pre) {
      float yh[8], g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) yh[e] = g[e] = 0.f;
      float2 m = make_float2(0.f, 0.f);
      if (in) {
        unpack8(*slot(stage, 2), g);
        unpack8(*slot(stage, 3), yh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          yh[e] = (yh[e] - st.z) * st.w;
          if (!RMS) S2[e] += g[e];
          S3[e] = fmaf(g[e], yh[e], S3[e]);
          g[e] *= gn[e];
          if (!RMS) m.x += g[e];
          m.y = fmaf(g[e], yh[e], m.y);
        }
      }
      m = pair_sum<CLUSTER>(m, red, peer, turn, cluster, rank);
      m.x *= inv_n;
      m.y *= inv_n;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += st.w * (g[e] - m.x - yh[e] * m.y);
    }
    if (in) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = a.alpha * d[e];
      *reinterpret_cast<uint4*>(a.dx + row * a.ld_dx + col) = pack8(f);
    }
    float2 m = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (post) oh[e] = (oh[e] - st.x) * st.y;
      if (in) {
        if (!RMS) S0[e] += d[e];
        S1[e] = fmaf(d[e], oh[e], S1[e]);
      }
      d[e] *= w[e];
      if (in) {
        m.x += d[e];
        m.y = fmaf(d[e], oh[e], m.y);
      }
    }
    if (post) {
      m = pair_sum<CLUSTER>(m, red, peer, turn, cluster, rank);
      m.x = RMS ? 0.f : m.x * inv_n;
      m.y *= inv_n;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = st.y * (d[e] - m.x - oh[e] * m.y);
    }
    if (in) *reinterpret_cast<uint4*>(a.d_o + row * a.ld_do + col) = pack8(d);

    if (in && (row + 1 == hi || row + 1 == seg_end)) {  // this gate's rows end here
      float4* dst = reinterpret_cast<float4*>(a.partials + (group + seg) * 2 * a.hidden + col);
      dst[0] = make_float4(S0[0], S0[1], S0[2], S0[3]);
      dst[1] = make_float4(S0[4], S0[5], S0[6], S0[7]);
      dst = reinterpret_cast<float4*>(a.partials + ((group + seg) * 2 + 1) * a.hidden + col);
      dst[0] = make_float4(S1[0], S1[1], S1[2], S1[3]);
      dst[1] = make_float4(S1[4], S1[5], S1[6], S1[7]);
#pragma unroll
      for (int e = 0; e < 8; ++e) S0[e] = S1[e] = 0.f;
    }
  }
  if (in && pre) {
    float* base = a.partials + (groups + a.gates) * 2 * a.hidden + group * 2 * static_cast<int64_t>(a.hidden) + col;
    float4* dst = reinterpret_cast<float4*>(base);
    dst[0] = make_float4(S2[0], S2[1], S2[2], S2[3]);
    dst[1] = make_float4(S2[4], S2[5], S2[6], S2[7]);
    dst = reinterpret_cast<float4*>(base + a.hidden);
    dst[0] = make_float4(S3[0], S3[1], S3[2], S3[3]);
    dst[1] = make_float4(S3[4], S3[5], S3[6], S3[7]);
  }
  cp_async_wait<0>();
  if constexpr (CLUSTER) cluster_sync();  // no block leaves while another may still write to it
}

// Joins the blocks' sums.  blockIdx.y = 0: dpost_gamma, dpost_beta; 1: dpre_gamma, dpre_beta;
// 2 + g: dgate of gate g.  32 channels a block; the 8 warps take the runs of rows in turn and their
// sums are added in order.
__global__ void __launch_bounds__(256)
    norm_backward_join_kernel(const __grid_constant__ NormArgs a, int groups) {
  __shared__ float part[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool in = col < a.hidden;
  const int64_t H = a.hidden;
  float s0 = 0.f, s1 = 0.f;
  if (blockIdx.y == 1) {
    const float* src = a.partials + (groups + a.gates) * 2 * H + col;
    if (in)
#pragma unroll 4
      for (int c = warp; c < groups; c += 8) {
        s0 += __ldcg(src + (c * 2) * H);
        s1 += __ldcg(src + (c * 2 + 1) * H);
      }
  } else {
    const int64_t per = a.rows / a.gates;
    const int64_t first = blockIdx.y ? blockIdx.y - 2 : 0;
    const int64_t last = blockIdx.y ? first : a.gates - 1;
    for (int64_t g = first; g <= last; ++g) {
      // The runs that hold rows of this gate: run c begins at row c * rows / groups.
      const int64_t c0 = ((g * per + 1) * groups - 1) / a.rows;
      const int64_t c1 = ((g + 1) * per * groups - 1) / a.rows;
      float t0 = 0.f, t1 = 0.f;
      if (in)
#pragma unroll 4
        for (int64_t c = c0 + ((warp - c0) & 7); c <= c1; c += 8) {
          t0 += __ldcg(a.partials + (c + g) * 2 * H + col);
          t1 += __ldcg(a.partials + ((c + g) * 2 + 1) * H + col);
        }
      const float f = in && a.gate && blockIdx.y == 0 ? __bfloat162float(a.gate[g * H + col]) : 1.f;
      s0 = fmaf(f, t0, s0);
      s1 = fmaf(f, t1, s1);
    }
  }
  part[0][warp][lane] = s0;
  part[1][warp][lane] = s1;
  __syncthreads();
  if (warp != 0 || !in) return;
  s0 = s1 = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    s0 += part[0][w][lane];
    s1 += part[1][w][lane];
  }
  if (blockIdx.y == 0) {
    if (a.dpost_gamma) a.dpost_gamma[col] = s1;
    if (a.dpost_beta) a.dpost_beta[col] = s0;
  } else if (blockIdx.y == 1) {
    if (a.dpre_gamma) a.dpre_gamma[col] = s1;
    if (a.dpre_beta) a.dpre_beta[col] = s0;
  } else {
    float v = s1;
    if (a.post_gamma) v *= __bfloat162float(a.post_gamma[col]);
    if (a.post_beta) v = fmaf(__bfloat162float(a.post_beta[col]), s0, v);
    a.dgate[(blockIdx.y - 2) * H + col] = v;
  }
}

template <bool WARP, bool RMS>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t stream) {
  const int nvec = a.hidden / 8;
  if constexpr (WARP) {
    const unsigned grid = static_cast<unsigned>((a.rows + 7) / 8);
    if (nvec <= 32)
      norm_residual_kernel<1, true, RMS><<<grid, 256, 0, stream>>>(a);
    else if (nvec <= 64)
      norm_residual_kernel<2, true, RMS><<<grid, 256, 0, stream>>>(a);
    else
      norm_residual_kernel<4, true, RMS><<<grid, 256, 0, stream>>>(a);
  } else {
    const unsigned grid = static_cast<unsigned>(a.rows);
    auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
    if (nvec <= 1024)
      norm_residual_kernel<2, false, RMS><<<grid, threads(2), 0, stream>>>(a);
    else if (nvec <= 2048)
      norm_residual_kernel<4, false, RMS><<<grid, threads(4), 0, stream>>>(a);
    else
      norm_residual_kernel<8, false, RMS><<<grid, threads(8), 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <int STAGES, bool CLUSTER, bool RMS, bool O8>
cudaError_t launch_backward(const NormArgs& a, const BackPlan& p, cudaStream_t stream) {
  auto kern = norm_residual_backward_kernel<STAGES, CLUSTER, RMS, O8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(p.smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.groups * p.cluster);
  cfg.blockDim = dim3(p.threads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  if (CLUSTER) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, a, p.cluster, p.slice, p.groups);
}

template <int STAGES>
cudaError_t launch_backward_stages(const NormArgs& a, const BackPlan& p, cudaStream_t stream) {
  const int key = (p.cluster > 1 ? 4 : 0) + (a.rms ? 2 : 0) + (a.o_exps ? 1 : 0);
  switch (key) {
    case 0: return launch_backward<STAGES, false, false, false>(a, p, stream);
    case 1: return launch_backward<STAGES, false, false, true>(a, p, stream);
    case 2: return launch_backward<STAGES, false, true, false>(a, p, stream);
    case 3: return launch_backward<STAGES, false, true, true>(a, p, stream);
    case 4: return launch_backward<STAGES, true, false, false>(a, p, stream);
    case 5: return launch_backward<STAGES, true, false, true>(a, p, stream);
    case 6: return launch_backward<STAGES, true, true, false>(a, p, stream);
    default: return launch_backward<STAGES, true, true, true>(a, p, stream);
  }
}

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, cudaStream_t stream) {
  const bool warp = a.hidden <= 1024;
  if (a.rms) return warp ? launch_forward<true, true>(a, stream) : launch_forward<false, true>(a, stream);
  return warp ? launch_forward<true, false>(a, stream) : launch_forward<false, false>(a, stream);
}

size_t norm_backward_partials(int64_t rows, int64_t hidden, int64_t gates, int sms) {
  const BackPlan p = back_plan(rows, hidden, sms);
  return static_cast<size_t>(2 * p.groups + gates) * 2 * hidden * sizeof(float);
}

cudaError_t launch_norm_residual_backward(const NormArgs& a, cudaStream_t stream) {
  const BackPlan p = back_plan(a.rows, a.hidden, a.sms);
  cudaError_t e = p.stages == 4   ? launch_backward_stages<4>(a, p, stream)
                  : p.stages == 3 ? launch_backward_stages<3>(a, p, stream)
                                  : launch_backward_stages<2>(a, p, stream);
  if (e != cudaSuccess) return e;
  const unsigned gates = a.dgate ? static_cast<unsigned>(a.gates) : 0;
  norm_backward_join_kernel<<<dim3((a.hidden + 31) / 32, 2 + gates), 256, 0, stream>>>(a, p.groups);
  return cudaGetLastError();
}

}  // namespace ptb
