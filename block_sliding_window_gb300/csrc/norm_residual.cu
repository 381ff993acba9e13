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

// Eight neighbouring channels as four register pairs: with the packed arithmetic an instruction
// serves two of them, and these kernels issue instructions rather than wait for memory (in scalar
// form 51 a value forward and 75 backward; norm_8192's 63% of the memory rate were 70% of the issue
// slots).
struct V8 {
  uint64_t p[4];
};

__device__ __forceinline__ V8 splat(float v) {
  const uint64_t q = f2(v, v);
  return {{q, q, q, q}};
}

__device__ __forceinline__ V8 unpack8(uint4 q) {
  return {{f2(bf16_lo(q.x), bf16_hi(q.x)), f2(bf16_lo(q.y), bf16_hi(q.y)),
           f2(bf16_lo(q.z), bf16_hi(q.z)), f2(bf16_lo(q.w), bf16_hi(q.w))}};
}

__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 pack8(const V8& v) {
  return make_uint4(pack2(v.p[0]), pack2(v.p[1]), pack2(v.p[2]), pack2(v.p[3]));
}

__device__ __forceinline__ V8 load8(const __nv_bfloat16* base, int v) {
  return unpack8(__ldg(reinterpret_cast<const uint4*>(base) + v));
}

__device__ __forceinline__ float both(uint64_t v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return lo + hi;
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

  V8 p[VPT];
  uint4 xv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * lanes;
    uint4 ov = make_uint4(0, 0, 0, 0);
    xv[j] = ov;
    if (v < nvec) {
      ov = __ldcs(reinterpret_cast<const uint4*>(a.o + row * a.ld_o) + v);
      xv[j] = __ldcs(reinterpret_cast<const uint4*>(a.x + row * a.ld_x) + v);
    }
    p[j] = unpack8(ov);
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);

  // The mean (0 for the rms norm) and 1 / sqrt(variance + eps) of p.
  auto statistics = [&](float& mean, float& rstd) {
    mean = 0.f;
    if constexpr (!RMS) {
      uint64_t s = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = f2_add(s, p[j].p[e]);
      mean = row_sum<WARP>(both(s), red, turn) * inv_n;
    }
    uint64_t s = 0;
    const uint64_t m = f2(-mean, -mean);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (lane + j * lanes < nvec)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t d = RMS ? p[j].p[e] : f2_add(p[j].p[e], m);
          s = f2_fma(d, d, s);
        }
    rstd = rsqrtf(row_sum<WARP>(both(s), red, turn) * inv_n + a.eps);
  };
  // v -> (v - mean) / sd * gamma + beta.  (The first part as one fma with -mean / sd would leave a
  // constant row the rounding of that quotient instead of zeros.)
  auto normalise = [&](V8& v, int at, float mean, float rstd, const __nv_bfloat16* gamma,
                       const __nv_bfloat16* beta) {
    const uint64_t r = f2(rstd, rstd), c = f2(-mean, -mean);
    const V8 g = load8(gamma, at);
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = f2_mul(RMS ? v.p[e] : f2_add(v.p[e], c), r);
    if (!RMS && beta) {
      const V8 b = load8(beta, at);
#pragma unroll
      for (int e = 0; e < 4; ++e) v.p[e] = f2_fma(v.p[e], g.p[e], b.p[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v.p[e] = f2_mul(v.p[e], g.p[e]);
    }
  };

  const bool post = a.post_gamma != nullptr;
  if (post) statistics(st.x, st.y);
  const __nv_bfloat16* gate = a.gate ? a.gate + row / (a.rows / a.gates) * a.hidden : nullptr;
  const uint64_t alpha = f2(a.alpha, a.alpha);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * lanes;
    if (v < nvec) {
      if (post) normalise(p[j], v, st.x, st.y, a.post_gamma, a.post_beta);
      if (gate) {
        const V8 g = load8(gate, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[j].p[e] = f2_mul(p[j].p[e], g.p[e]);
      }
      const V8 x = unpack8(xv[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[j].p[e] = f2_fma(alpha, x.p[e], p[j].p[e]);
      const uint4 yv = pack8(p[j]);
      reinterpret_cast<uint4*>(a.y + row * a.ld_y)[v] = yv;
      p[j] = unpack8(yv);
    }
  }
  if (a.h) {
    statistics(st.z, st.w);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * lanes;
      if (v < nvec) {
        normalise(p[j], v, st.z, st.w, a.pre_gamma, a.pre_beta);
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
  const size_t room = (216 * 1024) / per_sm - 2560;  // less the static part and the system's
  int64_t st = static_cast<int64_t>(room / row);
  p.stages = static_cast<int>(st > 6 ? 6 : st < 4 ? 4 : st);
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

// Sums of four values over the threads of a row (all blocks of the cluster), the same bits in all of
// them.  Lanes first trade pairs of values, so that four sums take six shuffles instead of twenty.
//
// Blocks of a cluster send their sums into each other's `peer` slots, each message counting its
// bytes on the receiver's barrier of the turn.  A block's sums of the turn after next cannot come in
// before this block has read these: it sends its own of the next turn only after that.
struct Exchange {
  float4 peer[2][8];
  uint64_t bar[2];
  int abort;
};

template <bool CLUSTER>
__device__ __forceinline__ float4 row_sum4(float4 v, float4 (*red)[32], Exchange* ex, unsigned& turns,
                                           int cluster, uint32_t rank, unsigned* status) {
  const int turn = turns & 1;
  const int lane = threadIdx.x & 31;
  const bool odd1 = lane & 1, odd2 = lane & 2;
  // after these, lane l holds value l & 3 summed over the lanes that differ in the low two bits
  float a = odd1 ? v.y : v.x, b = odd1 ? v.w : v.z;
  a += __shfl_xor_sync(0xffffffffu, odd1 ? v.x : v.y, 1);
  b += __shfl_xor_sync(0xffffffffu, odd1 ? v.z : v.w, 1);
  float t = odd2 ? b : a;
  t += __shfl_xor_sync(0xffffffffu, odd2 ? a : b, 2);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  float* slots = reinterpret_cast<float*>(red[turn]);
  if (lane < 4) slots[(threadIdx.x >> 5) * 4 + lane] = t;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  t = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int w = (lane >> 2) + 8 * q;
    if (w < warps) t += slots[w * 4 + (lane & 3)];
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if constexpr (CLUSTER) {
    if (static_cast<int>(threadIdx.x) < 4 * cluster) {
      if (threadIdx.x == 0) mbar_arrive_expect_tx(&ex->bar[turn], 16 * cluster);
      const uint32_t to = lane >> 2;
      const uint32_t dst = cluster_map(reinterpret_cast<float*>(&ex->peer[turn][rank]) + (lane & 3), to);
      const uint32_t bar = cluster_map(&ex->bar[turn], to);
      asm volatile(
          "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst),
          "r"(__float_as_uint(t)), "r"(bar)
          : "memory");
    }
    mbar_wait_cluster(&ex->bar[turn], (turns >> 1) & 1, &ex->abort, status);
    v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < cluster; ++r) {
      const float4 p = ex->peer[turn][r];
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
  } else {
    v.x = __shfl_sync(0xffffffffu, t, 0);
    v.y = __shfl_sync(0xffffffffu, t, 1);
    v.z = __shfl_sync(0xffffffffu, t, 2);
    v.w = __shfl_sync(0xffffffffu, t, 3);
  }
  ++turns;
  return v;
}

// Eight fp32 values in two pieces of 16 bytes.
__device__ __forceinline__ void store_v8(void* lo, void* hi, const V8& v) {
  *reinterpret_cast<ulonglong2*>(lo) = make_ulonglong2(v.p[0], v.p[1]);
  *reinterpret_cast<ulonglong2*>(hi) = make_ulonglong2(v.p[2], v.p[3]);
}
__device__ __forceinline__ V8 load_v8(const void* lo, const void* hi) {
  const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(lo);
  const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(hi);
  return {{p.x, p.y, q.x, q.y}};
}

template <int STAGES, bool CLUSTER, bool RMS, bool O8>
__global__ void __launch_bounds__(kSliceMax / 8, 1)
    norm_residual_backward_kernel(const __grid_constant__ NormArgs a, int cluster, int slice, int groups) {
  extern __shared__ __align__(16) uint4 ring[];  // [STAGES][4][blockDim.x]
  __shared__ float4 red[2][32];
  __shared__ Exchange ex;
  constexpr int AHEAD = STAGES - 2;  // rows on their way while two are worked on
  const uint32_t rank = CLUSTER ? cluster_ctarank() : 0;
  const int group = blockIdx.x / cluster;
  const int64_t lo = group * a.rows / groups, hi = (group + 1) * a.rows / groups;
  const int64_t rows_per_gate = a.rows / a.gates;
  const int col = static_cast<int>(rank) * slice + threadIdx.x * 8;
  const bool in = static_cast<int>(threadIdx.x) * 8 < slice && col < a.hidden;
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr;
  const float inv_n = 1.f / static_cast<float>(a.hidden);
  unsigned turns = 0;
  if constexpr (CLUSTER) {
    if (threadIdx.x == 0) {
      mbar_init(&ex.bar[0], 1);
      mbar_init(&ex.bar[1], 1);
      ex.abort = 0;
      mbar_fence_init();
    }
    cluster_sync();
  }

  V8 S0 = splat(0.f), S1 = S0, S2 = S0, S3 = S0, w = S0, gn = S0;
  if (in && pre) gn = load8(a.pre_gamma + col, 0);

  // This thread's slots: 16 bytes of each tensor, [stage][tensor][thread].
  char* const slots = reinterpret_cast<char*>(ring + threadIdx.x);
  const uint32_t per_tensor = blockDim.x * 16, per_stage = per_tensor * 4;
  const uint32_t ring_bytes = per_stage * STAGES;
  uint32_t fetch_at = 0;
  int64_t fetch_row = lo;
  const __nv_bfloat16* src_dy = a.dy + lo * a.ld_dy + col;
  const __nv_bfloat16* src_dh = a.dh + lo * a.ld_dh + col;
  const __nv_bfloat16* src_y = a.y + lo * a.ld_y + col;
  const char* src_o = reinterpret_cast<const char*>(a.o) + (lo * a.ld_o + col) * (O8 ? 1 : 2);
  auto fetch = [&]() {  // the next row
    if (in && fetch_row < hi) {
      char* dst = slots + fetch_at;
      if (a.dy) cp_async16(dst, src_dy);
      if (O8)
        cp_async8(dst + per_tensor, src_o);
      else
        cp_async16(dst + per_tensor, src_o);
      if (pre) {
        cp_async16(dst + 2 * per_tensor, src_dh);
        cp_async16(dst + 3 * per_tensor, src_y);
      }
      src_dy += a.ld_dy;
      src_dh += a.ld_dh;
      src_y += a.ld_y;
      src_o += a.ld_o * (O8 ? 1 : 2);
    }
    ++fetch_row;
    fetch_at += per_stage;
    if (fetch_at == ring_bytes) fetch_at = 0;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) fetch();
  auto value8 = [&](uint32_t at, int t) {
    return unpack8(*reinterpret_cast<const uint4*>(slots + at + t * per_tensor));
  };

  __nv_bfloat16* out_dx = a.dx + lo * a.ld_dx + col;
  __nv_bfloat16* out_do = a.d_o + lo * a.ld_do + col;
  const uint64_t alpha = f2(a.alpha, a.alpha);
  int64_t seg = 0, seg_end = lo;
  uint32_t stage_at = 0;
  int n;
  for (int64_t row = lo; row < hi; row += n) {
    if (row >= seg_end) {  // the first row, or the first of another gate
      seg = row / rows_per_gate;
      seg_end = (seg + 1) * rows_per_gate;
      w = splat(1.f);
      if (in) {
        if (a.gate) w = load8(a.gate + seg * a.hidden + col, 0);
        if (post) {
          const V8 f = load8(a.post_gamma + col, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) w.p[e] = f2_mul(w.p[e], f.p[e]);
        }
      }
    }
    // Two rows of one gate at a time: they share the barriers of the two rounds of sums.
    const int64_t end = seg_end < hi ? seg_end : hi;
    n = row + 1 < end ? 2 : 1;
    float4 st[2];
    float o_scale[2] = {1.f, 1.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      st[r] = __ldg(a.stats + row + (r < n ? r : 0));
      if (O8 && in && r < n)
        o_scale[r] = ckpt_scale(__ldg(a.o_exps + (row + r) * a.ld_o_exps + col / 32));
    }
    fetch();
    if (n == 2) fetch();
    cp_async_wait<AHEAD>();
    uint32_t at[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      at[r] = stage_at;
      if (r < n) stage_at += per_stage;
      if (stage_at == ring_bytes) stage_at = 0;
    }

    auto hat = [](V8 v, float mean, float r) {  // (v - mean) / sd
      const uint64_t rr = f2(r, r), c = f2(-mean, -mean);
#pragma unroll
      for (int e = 0; e < 4; ++e) v.p[e] = f2_mul(RMS ? v.p[e] : f2_add(v.p[e], c), rr);
      return v;
    };
    float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pre) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint64_t s1 = 0, s2 = 0;
        if (in && r < n) {
          const V8 g = value8(at[r], 2), yh = hat(value8(at[r], 3), st[r].z, st[r].w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!RMS) S2.p[e] = f2_add(S2.p[e], g.p[e]);
            S3.p[e] = f2_fma(g.p[e], yh.p[e], S3.p[e]);
            const uint64_t gg = f2_mul(g.p[e], gn.p[e]);
            if (!RMS) s1 = f2_add(s1, gg);
            s2 = f2_fma(gg, yh.p[e], s2);
          }
        }
        if (r) m.z = both(s1), m.w = both(s2);
        else m.x = both(s1), m.y = both(s2);
      }
      m = row_sum4<CLUSTER>(m, red, &ex, turns, cluster, rank, a.status);
    }
    auto load_o = [&](int r) {
      V8 v;
      if (O8) {
        const uint2 c = *reinterpret_cast<const uint2*>(slots + at[r] + per_tensor);
        uint64_t f[2];
        ckpt_unpack4_scaled(c.x, o_scale[r], f);
        v.p[0] = f[0], v.p[1] = f[1];
        ckpt_unpack4_scaled(c.y, o_scale[r], f);
        v.p[2] = f[0], v.p[3] = f[1];
      } else {
        v = value8(at[r], 1);
      }
      return post ? hat(v, st[r].x, st[r].y) : v;
    };
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint64_t s1 = 0, s2 = 0;
      if (in && r < n) {
        V8 d = a.dy ? value8(at[r], 0) : splat(0.f);
        if (pre) {
          const V8 g = value8(at[r], 2), yh = hat(value8(at[r], 3), st[r].z, st[r].w);
          // d += (g gn - m1 - yh m2) / sd
          const float m1 = (r ? m.z : m.x) * -inv_n, m2 = (r ? m.w : m.y) * -inv_n;
          const uint64_t c1 = f2(m1, m1), c2 = f2(m2, m2), sd = f2(st[r].w, st[r].w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t t = RMS ? f2_mul(yh.p[e], c2) : f2_fma(yh.p[e], c2, c1);
            d.p[e] = f2_fma(sd, f2_fma(g.p[e], gn.p[e], t), d.p[e]);
          }
        }
        V8 f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f.p[e] = f2_mul(alpha, d.p[e]);
        *reinterpret_cast<uint4*>(out_dx + r * a.ld_dx) = pack8(f);
        const V8 oh = load_o(r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!RMS) S0.p[e] = f2_add(S0.p[e], d.p[e]);
          S1.p[e] = f2_fma(d.p[e], oh.p[e], S1.p[e]);
          d.p[e] = f2_mul(d.p[e], w.p[e]);
          if (!RMS) s1 = f2_add(s1, d.p[e]);
          s2 = f2_fma(d.p[e], oh.p[e], s2);
        }
        if (post) {
          // kept for the second round in this thread's own slots, whose values are used up
          char* mine = slots + at[r];
          store_v8(mine, mine + 2 * per_tensor, d);
          store_v8(mine + per_tensor, mine + 3 * per_tensor, oh);
        } else {
          *reinterpret_cast<uint4*>(out_do + r * a.ld_do) = pack8(d);
        }
      }
      if (r) k.z = both(s1), k.w = both(s2);
      else k.x = both(s1), k.y = both(s2);
    }
    if (post) {
      k = row_sum4<CLUSTER>(k, red, &ex, turns, cluster, rank, a.status);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (in && r < n) {
          const float k1 = (r ? k.z : k.x) * -inv_n, k2 = (r ? k.w : k.y) * -inv_n;
          const uint64_t c1 = f2(k1, k1), c2 = f2(k2, k2), sd = f2(st[r].y, st[r].y);
          const char* mine = slots + at[r];
          V8 d = load_v8(mine, mine + 2 * per_tensor);
          const V8 oh = load_v8(mine + per_tensor, mine + 3 * per_tensor);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t t = RMS ? f2_fma(oh.p[e], c2, d.p[e]) : f2_add(f2_fma(oh.p[e], c2, c1), d.p[e]);
            d.p[e] = f2_mul(sd, t);
          }
          *reinterpret_cast<uint4*>(out_do + r * a.ld_do) = pack8(d);
        }
      }
    }
    out_dx += n * a.ld_dx;
    out_do += n * a.ld_do;

    if (in && row + n == end) {  // this gate's rows of this run end here
      float* dst = a.partials + (group + seg) * 2 * a.hidden + col;
      store_v8(dst, dst + 4, S0);
      store_v8(dst + a.hidden, dst + a.hidden + 4, S1);
      S0 = S1 = splat(0.f);
    }
  }
  if (in && pre) {
    float* dst = a.partials + (groups + a.gates) * 2 * a.hidden + group * 2 * static_cast<int64_t>(a.hidden) + col;
    store_v8(dst, dst + 4, S2);
    store_v8(dst + a.hidden, dst + a.hidden + 4, S3);
  }
  cp_async_wait<0>();
  if constexpr (CLUSTER) cluster_sync();  // no block leaves while another may still write to it
}

// Joins the blocks' sums.  blockIdx.y = 0: dpost_gamma, dpost_beta and a single gate's dgate; 1:
// dpre_gamma, dpre_beta; 2 + g: dgate of gate g of several.  32 channels a block; its warps take the
// runs of rows in turn and their sums are added in order.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(kJoinWarps * 32)
    norm_backward_join_kernel(const __grid_constant__ NormArgs a, int groups) {
  __shared__ float part[2][kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool in = col < a.hidden;
  const int64_t H = a.hidden;
  const bool pre = blockIdx.y == 1, each = blockIdx.y > 1;
  float s0 = 0.f, s1 = 0.f;
  const int64_t per = a.rows / a.gates;
  const int64_t first = each ? blockIdx.y - 2 : 0;
  const int64_t last = each || pre ? first : a.gates - 1;
  for (int64_t g = first; g <= last; ++g) {
    // The runs that hold rows of this gate: run c begins at row c * rows / groups.
    int c0 = 0, c1 = groups - 1;
    const float* src = a.partials + (groups + a.gates) * 2 * H;
    if (!pre) {
      c0 = static_cast<int>(((g * per + 1) * groups - 1) / a.rows);
      c1 = static_cast<int>(((g + 1) * per * groups - 1) / a.rows);
      src = a.partials + g * 2 * H;
    }
    src += col;
    float t0 = 0.f, t1 = 0.f;
    if (in) {
#pragma unroll 10
      for (int c = c0 + ((warp - c0) & (kJoinWarps - 1)); c <= c1; c += kJoinWarps) {
        t0 += __ldcg(src + (c * 2) * H);
        t1 += __ldcg(src + (c * 2 + 1) * H);
      }
      const bool weigh = blockIdx.y == 0 && a.gate && a.gates > 1;
      const float f = weigh ? __bfloat162float(a.gate[g * H + col]) : 1.f;
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
  for (int w = 0; w < kJoinWarps; ++w) {
    s0 += part[0][w][lane];
    s1 += part[1][w][lane];
  }
  if (pre) {
    if (a.dpre_gamma) a.dpre_gamma[col] = s1;
    if (a.dpre_beta) a.dpre_beta[col] = s0;
    return;
  }
  if (each || (a.gates == 1 && a.dgate)) {
    float v = s1;
    if (a.post_gamma) v *= __bfloat162float(a.post_gamma[col]);
    if (a.post_beta) v = fmaf(__bfloat162float(a.post_beta[col]), s0, v);
    a.dgate[first * H + col] = v;
  }
  if (!each) {
    const float f = a.gates == 1 && a.gate ? __bfloat162float(a.gate[col]) : 1.f;
    if (a.dpost_gamma) a.dpost_gamma[col] = f * s1;
    if (a.dpost_beta) a.dpost_beta[col] = f * s0;
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
    if (nvec <= 2048)
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
  cudaError_t e = p.stages == 6   ? launch_backward_stages<6>(a, p, stream)
                  : p.stages == 5 ? launch_backward_stages<5>(a, p, stream)
                                  : launch_backward_stages<4>(a, p, stream);
  if (e != cudaSuccess) return e;
  const unsigned each = a.dgate && a.gates > 1 ? static_cast<unsigned>(a.gates) : 0;
  norm_backward_join_kernel<<<dim3((a.hidden + 31) / 32, 2 + each), kJoinWarps * 32, 0, stream>>>(
      a, p.groups);
  return cudaGetLastError();
}

}  // namespace ptb
