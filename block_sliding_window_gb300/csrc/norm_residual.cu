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
#include <atomic>
#include <type_traits>

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
template <int VPT, bool WARP, bool RMS, int REGS>
__global__ void __maxnreg__(REGS) norm_residual_kernel(const __grid_constant__ NormArgs a) {
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
// With gg = dh * pre_gamma, w = gate * post_gamma and vh = (v - mean) / sd of y (yh) and of o (oh):
//   d  = dy + (gg - m1 - yh m2) / sd_y,          m1 = mean(gg), m2 = mean(gg yh)
//   dx = alpha d,   do = (w d - k1 - oh k2) / sd_o,   k1 = mean(w d), k2 = mean(w oh d)
// (rms norms: m1 = k1 = 0).  k1 and k2 are sums over d, which needs m1 and m2 first; but with d
// written out,
//   k1 = mean(w dy) + (mean(w gg) - m1 mean(w) - m2 mean(w yh)) / sd_y,   k2 alike with w oh for w,
// all ten sums (four for rms norms) come out of one look at the row and one round between the
// threads, where d first and k after took two and kept d in shared memory in between (norm_bwd_8bit
// 123 us, 36 of them in the two rounds).  Of the sums over rows four suffice:
//   S0 = sum d, S1 = sum d oh, S2 = sum dh, S3 = sum dh yh   (S0, S1 for each gate's rows apart)
//   dpost_beta = gate S0,  dpost_gamma = gate S1,  dgate = post_gamma S1 + post_beta S0,
//   dpre_beta = S2,  dpre_gamma = S3.
//
// Rows are dealt to blocks in runs, a thread has VEC * 8 channels of all its block's rows and keeps
// their sums in registers.  Each thread copies its own channels of the next rows into its own part of
// shared memory (cp.async), so the copies run ahead of the arithmetic without any barrier; two rows
// at a time share the round between the threads.  Rows of more channels than a block has threads for
// are split over a cluster, whose blocks exchange their sums through each other's shared memory.
// The blocks' sums are joined by a second kernel in a fixed order.

// Channels of one block and of a thread.  A thread keeps the sums of its channels in registers, two
// for a channel of an rms norm and four for one of a layer norm, and a quarter of the SM has
// registers for whole warps only:
//   rms norms    up to 5120 channels 640 threads of 8 (96 registers), else 384 of 16 (168) a slice;
//   layer norms  256 threads of 16 (248; with 168 the sums spill, 4096 channels 162 us), from 4097 to
//                6144 channels of 24 and one row at a time (5120 channels 111 us; two rows 126, in two
//                slices 145)
// Rows of two to four slices are cut into twice as many, so that two blocks share an SM: one works
// while the other waits for its cluster (layer norms of 12288 channels 148 us in three slices, 134 in
// six, either way on 138 SMs; rms norms 104 in two and 101 in four).
template <int VEC, bool RMS>
__host__ __device__ constexpr int back_threads() {
  return RMS ? (VEC == 1 ? 640 : 384) : 256;
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// All but the latest `ahead` (2 to 4) groups.
template <int AHEAD>
__device__ __forceinline__ void wait_ahead(int ahead) {
  if constexpr (AHEAD < 4) {
    if (ahead != AHEAD) return wait_ahead<AHEAD + 1>(ahead);
  }
  cp_async_wait<AHEAD>();
}

constexpr int kMostSums = 20;

// A warp's part of shared memory, behind the ring.
struct alignas(16) WarpArea {
  float4 stats[6];            // of the rows in the ring
  float mine[2][kMostSums];   // its sums, for the block; two turns
  float sum[kMostSums];       // everyone's, for its lanes
};

// What the blocks of a cluster tell each other: they send their sums into each other's `peer` slots,
// each message counting its bytes on the receiver's barrier of the turn.  A block's sums of the turn
// after next cannot come in before this block has read these: it sends its own of the next turn only
// after that.
struct Exchange {
  float peer[2][8][kMostSums];
  uint64_t bar[2];
  int abort;
};

constexpr size_t kShared = 226 * 1024;  // shared memory of an SM, as far as the blocks may fill it
// What one block may take of it beside its Exchange: back_plan's smem is at most this.
constexpr int kMostDynamic = static_cast<int>(kShared - sizeof(Exchange) - 1024);

struct BackPlan {
  int vec, cluster, threads, slice, groups, stages;
  size_t smem;
};

BackPlan back_plan(int64_t rows, int64_t hidden, bool rms, int sms) {
  BackPlan p;
  const int most = !rms                                ? back_threads<2, false>()
                   : hidden <= back_threads<1, true>() * 8 ? back_threads<1, true>()
                                                           : back_threads<2, true>();
  if (rms)
    p.vec = most == back_threads<1, true>() ? 1 : 2;
  else
    p.vec = hidden > most * 16 && hidden <= most * 24 ? 3 : 2;
  const int slice = most * p.vec * 8;
  p.cluster = static_cast<int>((hidden + slice - 1) / slice);
  if (p.cluster > 1 && p.cluster <= 4) p.cluster *= 2;  // two half blocks on an SM
  const int64_t vecs = (hidden / 8 + p.cluster - 1) / p.cluster;
  p.slice = static_cast<int>(vecs) * 8;
  p.threads = static_cast<int>(((vecs + p.vec - 1) / p.vec + 31) / 32) * 32;
  const size_t row = static_cast<size_t>(p.threads) * p.vec * 4 * 16;
  const size_t rest = p.threads / 32 * sizeof(WarpArea);
  // Blocks on an SM: what the registers allow and four rows a block leave room for.
  int per_sm = most / p.threads;
  const size_t fixed = rest + sizeof(Exchange) + 1024;
  while (per_sm > 1 && per_sm * (4 * row + fixed) > kShared) --per_sm;
  int64_t groups = static_cast<int64_t>(sms) * per_sm / p.cluster;
  if (groups > rows) groups = rows;
  p.groups = static_cast<int>(groups < 1 ? 1 : groups);
  const int64_t st = static_cast<int64_t>((kShared / per_sm - fixed) / row);
  p.stages = static_cast<int>(st > 6 ? 6 : st);
  p.smem = row * p.stages + rest;
  return p;
}

// Sums of V values over the threads of a row (all blocks of the cluster), the same bits in all of
// them.  Lanes first trade pairs of values, so that four sums take six shuffles instead of twenty.
template <int V, bool CLUSTER>
__device__ __forceinline__ void row_sums(float (&v)[V], WarpArea* areas, Exchange& ex,
                                         unsigned& turns, int cluster, uint32_t rank,
                                         unsigned* status) {
  static_assert(V % 4 == 0 && V <= kMostSums, "");
  const int turn = turns & 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool odd1 = lane & 1, odd2 = lane & 2;
#pragma unroll
  for (int q = 0; q < V; q += 4) {
    float a = odd1 ? v[q + 1] : v[q], b = odd1 ? v[q + 3] : v[q + 2];
    a += __shfl_xor_sync(0xffffffffu, odd1 ? v[q] : v[q + 1], 1);
    b += __shfl_xor_sync(0xffffffffu, odd1 ? v[q + 2] : v[q + 3], 1);
    float t = odd2 ? b : a;
    t += __shfl_xor_sync(0xffffffffu, odd2 ? a : b, 2);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane < 4) areas[warp].mine[turn][q + lane] = t;  // lane l has value l & 3
  }
  __syncthreads();
  float t = 0.f;
  if (lane < V) {
#pragma unroll 4
    for (int w = 0; w < warps; ++w) t += areas[w].mine[turn][lane];
  }
  if constexpr (CLUSTER) {
    if (warp == 0) {
      if (lane == 0) mbar_arrive_expect_tx(&ex.bar[turn], 4 * V * cluster);
      __syncwarp();
      if (lane < V)
        for (int to = 0; to < cluster; ++to)
          asm volatile(
              "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                  cluster_map(&ex.peer[turn][rank][lane], to)),
              "r"(__float_as_uint(t)), "r"(cluster_map(&ex.bar[turn], to))
              : "memory");
      __syncwarp();
    }
    mbar_wait_cluster_warp(&ex.bar[turn], (turns >> 1) & 1, &ex.abort, status);
    t = 0.f;
    if (lane < V)
      for (int r = 0; r < cluster; ++r) t += ex.peer[turn][r][lane];
  }
  // to every lane: this warp's own slots, read before the next round's barrier
  if (lane < V) areas[warp].sum[lane] = t;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < V; q += 4) {
    const float4 p = *reinterpret_cast<const float4*>(&areas[warp].sum[q]);
    v[q] = p.x, v[q + 1] = p.y, v[q + 2] = p.z, v[q + 3] = p.w;
  }
  __syncwarp();
  ++turns;
}

__device__ __forceinline__ void store_v8(float* dst, const V8& v) {
  ulonglong2* d = reinterpret_cast<ulonglong2*>(dst);
  d[0] = make_ulonglong2(v.p[0], v.p[1]);
  d[1] = make_ulonglong2(v.p[2], v.p[3]);
}

// A load that stays where it is written: the compiler would move a plain one down to its use.
__device__ __forceinline__ unsigned load_now(const uint8_t* p) {
  unsigned v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w) : "memory");
}

// pre_gamma of eight channels: as fp32 pairs, or as it is stored where registers are short (a layer
// norm has twice the sums to keep).
template <bool WIDE>
struct Gamma {
  V8 v;
  __device__ __forceinline__ void set(uint4 q) { v = unpack8(q); }
  __device__ __forceinline__ const V8& get() const { return v; }
};
template <>
struct Gamma<false> {
  uint4 q;
  __device__ __forceinline__ void set(uint4 p) { q = p; }
  __device__ __forceinline__ V8 get() const { return unpack8(q); }
};

// FULL: both norms and both gradients are there (the usual call); else a.dy, post_gamma or pre_gamma
// may be absent.
template <int VEC, bool CLUSTER, bool RMS, bool O8, bool FULL>
__device__ __forceinline__ void backward_rows(const NormArgs& a, int cluster, int slice, int groups,
                                              int stages) {
  extern __shared__ __align__(16) uint4 ring[];  // [stages][4][VEC][blockDim.x], then the warps' areas
  __shared__ __align__(16) Exchange ex;          // (clusters only)
  const int ahead = stages - 2;  // rows on their way while two are worked on
  const uint32_t rank = CLUSTER ? cluster_ctarank() : 0;
  const int group = blockIdx.x / cluster;
  const int64_t lo = group * a.rows / groups, hi = (group + 1) * a.rows / groups;
  const int64_t rows_per_gate = a.rows / a.gates;
  // This thread's channels.  Vectors behind the row's end hold zeros, with weights of zero, and are
  // not stored.
  const int col = static_cast<int>(rank) * slice + threadIdx.x * 8;
  const int step = blockDim.x * 8;
  bool in[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    in[j] = static_cast<int>(threadIdx.x) * 8 + j * step < slice && col + j * step < a.hidden;
  const bool post = FULL || a.post_gamma != nullptr, pre = FULL || a.pre_gamma != nullptr;
  const bool has_dy = FULL || a.dy != nullptr;
  const float inv_n = -1.f / static_cast<float>(a.hidden);  // the means are subtracted
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

  V8 S0[VEC], S1[VEC], S2[VEC], S3[VEC], w[VEC];
  Gamma<RMS> gn[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    S0[j] = S1[j] = S2[j] = S3[j] = splat(0.f);
    gn[j].set(in[j] && pre ? __ldg(reinterpret_cast<const uint4*>(a.pre_gamma + col + j * step))
                           : make_uint4(0, 0, 0, 0));
  }

  // This thread's slots: 16 bytes of each tensor and vector.
  const uint32_t per_vec = blockDim.x * 16, per_tensor = per_vec * VEC, per_stage = per_tensor * 4;
  const uint32_t mine = smem_addr(ring + threadIdx.x), ring_end = mine + per_stage * stages;
  for (int t = 0; t < 4; ++t)  // what no copy will fill
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (!in[j] || !(t == 0 ? has_dy : t == 1 ? true : pre))
        for (uint32_t at = mine + t * per_tensor + j * per_vec; at < ring_end; at += per_stage)
          sts16(at, make_uint4(0, 0, 0, 0));
  uint32_t fetch_at = mine;
  int64_t left = hi - lo;  // rows still to be fetched
  const float4* src_stats = a.stats + lo;
  const int warp = threadIdx.x >> 5;
  WarpArea* const areas = reinterpret_cast<WarpArea*>(ring + stages * 4 * VEC * blockDim.x);
  const uint32_t stats_mine = smem_addr(areas[warp].stats);
  uint32_t stats_fetch = stats_mine, stats_at = stats_mine;
  const __nv_bfloat16* src_dy = a.dy + lo * a.ld_dy + col;
  const __nv_bfloat16* src_dh = a.dh + lo * a.ld_dh + col;
  const __nv_bfloat16* src_y = a.y + lo * a.ld_y + col;
  const char* src_o = reinterpret_cast<const char*>(a.o) + (lo * a.ld_o + col) * (O8 ? 1 : 2);
  auto fetch = [&]() {  // the next row
    if (left > 0) {
      if ((threadIdx.x & 31) == 0) cp_async16(stats_fetch, src_stats);
      ++src_stats;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (!in[j]) break;
        const uint32_t at = fetch_at + j * per_vec;
        if (has_dy) cp_async16(at, src_dy + j * step);
        if (O8)
          cp_async8(at + per_tensor, src_o + j * step);
        else
          cp_async16(at + per_tensor, src_o + j * step * 2);
        if (pre) {
          cp_async16(at + 2 * per_tensor, src_dh + j * step);
          cp_async16(at + 3 * per_tensor, src_y + j * step);
        }
      }
      src_dy += a.ld_dy;
      src_dh += a.ld_dh;
      src_y += a.ld_y;
      src_o += a.ld_o * (O8 ? 1 : 2);
      --left;
    }
    fetch_at += per_stage;
    stats_fetch += 16;
    if (fetch_at == ring_end) {
      fetch_at = mine;
      stats_fetch = stats_mine;
    }
    cp_async_commit();
  };
  for (int s = 0; s < ahead; ++s) fetch();

  // Exponents are read one step ahead of their rows.
  const uint8_t* exps[VEC];
  int64_t exps_left = hi - lo;
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    exps[j] = O8 ? a.o_exps + lo * a.ld_o_exps + (in[j] ? (col + j * step) / 32 : 0) : nullptr;
  unsigned next_e[2][VEC];
  auto read_ahead = [&](int n) {  // the rows n and n + 1 behind the current ones
    if (!O8) return;
    exps_left -= n;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      exps[j] += n * a.ld_o_exps;
      if (exps_left > 0) next_e[0][j] = load_now(exps[j]);
      if (exps_left > 1) next_e[1][j] = load_now(exps[j] + a.ld_o_exps);
    }
  };
  read_ahead(0);

  __nv_bfloat16* out_dx = a.dx + lo * a.ld_dx + col;
  __nv_bfloat16* out_do = a.d_o + lo * a.ld_do + col;
  uint32_t stage_at = mine;

  auto hat = [](V8 v, float mean, float r) {  // (v - mean) / sd
    const uint64_t rr = f2(r, r), c = f2(-mean, -mean);
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = f2_mul(RMS ? v.p[e] : f2_add(v.p[e], c), rr);
    return v;
  };
  auto load_oh = [&](uint32_t at, unsigned exponent, const float4& st) {
    V8 v;
    if (O8) {
      const float scale = ckpt_scale(exponent);
      const uint2 c = lds8(at + per_tensor);
      uint64_t q[2];
      ckpt_unpack4_scaled(c.x, scale, q);
      v.p[0] = q[0], v.p[1] = q[1];
      ckpt_unpack4_scaled(c.y, scale, q);
      v.p[2] = q[0], v.p[3] = q[1];
    } else {
      v = unpack8(lds16(at + per_tensor));
    }
    return post ? hat(v, st.x, st.y) : v;
  };

  // Sums of a row: m2, B1, B2, B4, and of a layer norm m1, A1, A2, A3, A4, B3 as well.
  constexpr int SUMS = RMS ? 4 : 10;
  float w_sum = 0.f;  // of this thread's weights
  // N rows of one gate.
  auto rows = [&](auto count) {
    constexpr int N = decltype(count)::value;
    float4 st[N];
    unsigned ex8[N][VEC];
#pragma unroll
    for (int r = 0; r < N; ++r) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) ex8[r][j] = O8 ? next_e[r][j] : 0;
    }
    read_ahead(N);
#pragma unroll
    for (int r = 0; r < N; ++r) fetch();
    wait_ahead<2>(ahead);
    __syncwarp();  // lane 0's copies of the statistics are the whole warp's
    uint32_t at[N];
#pragma unroll
    for (int r = 0; r < N; ++r) {
      at[r] = stage_at;
      const uint4 q = lds16(stats_at);
      st[r] = make_float4(__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z),
                          __uint_as_float(q.w));
      if (!pre) st[r].z = st[r].w = 0.f;  // whatever is kept for a norm that is not there
      stage_at += per_stage;
      stats_at += 16;
      if (stage_at == ring_end) {
        stage_at = mine;
        stats_at = stats_mine;
      }
    }
    float v[(SUMS * N + 3) / 4 * 4];
    if (pre || post) {
#pragma unroll
      for (int r = 0; r < N; ++r) {
        uint64_t t[SUMS];
#pragma unroll
        for (int e = 0; e < SUMS; ++e) t[e] = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const uint32_t p = at[r] + j * per_vec;
          const V8 d = unpack8(lds16(p)), oh = load_oh(p, ex8[r][j], st[r]);
          const V8 g = unpack8(lds16(p + 2 * per_tensor));
          const V8 yh = hat(unpack8(lds16(p + 3 * per_tensor)), st[r].z, st[r].w), gamma = gn[j].get();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (RMS) S3[j].p[e] = f2_fma(g.p[e], yh.p[e], S3[j].p[e]);
            const uint64_t gg = f2_mul(g.p[e], gamma.p[e]), wo = f2_mul(w[j].p[e], oh.p[e]);
            t[0] = f2_fma(gg, yh.p[e], t[0]);
            t[1] = f2_fma(wo, d.p[e], t[1]);
            t[2] = f2_fma(wo, gg, t[2]);
            t[3] = f2_fma(wo, yh.p[e], t[3]);
            if constexpr (!RMS) {
              t[4] = f2_add(t[4], gg);
              t[5] = f2_fma(w[j].p[e], d.p[e], t[5]);
              t[6] = f2_fma(w[j].p[e], gg, t[6]);
              t[8] = f2_fma(w[j].p[e], yh.p[e], t[8]);
              t[9] = f2_add(t[9], wo);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < SUMS; ++e) v[r * SUMS + e] = e == 7 ? w_sum : both(t[e]);
      }
#pragma unroll
      for (int e = SUMS * N; e < (SUMS * N + 3) / 4 * 4; ++e) v[e] = 0.f;
      row_sums<(SUMS * N + 3) / 4 * 4, CLUSTER>(v, areas, ex, turns, cluster, rank, a.status);
    }
    float m1[N], m2[N], k1[N], k2[N];  // less the means
#pragma unroll
    for (int r = 0; r < N; ++r) {
      m1[r] = m2[r] = k1[r] = k2[r] = 0.f;
      const float* q = v + r * SUMS;
      if (pre) {
        m2[r] = q[0] * inv_n;
        if constexpr (!RMS) m1[r] = q[4] * inv_n;
      }
      if (post) {
        float b = fmaf(m2[r], q[3], q[2]);
        if constexpr (!RMS) {
          b = fmaf(m1[r], q[9], b);
          k1[r] = fmaf(st[r].w, fmaf(m1[r], q[7], fmaf(m2[r], q[8], q[6])), q[5]) * inv_n;
        }
        k2[r] = fmaf(st[r].w, b, q[1]) * inv_n;
      }
    }
#pragma unroll
    for (int r = 0; r < N; ++r) {
      // d = dy + gg / sd + c1 + c2 yh (c2 y for rms norms)
      const float y2 = st[r].w * m2[r] * (RMS ? st[r].w : 1.f), y1 = st[r].w * m1[r];
      const uint64_t c1 = f2(y1, y1), c2 = f2(y2, y2), sd = f2(st[r].w, st[r].w);
      const uint64_t my = f2(-st[r].z, -st[r].z);
      const uint64_t e1 = f2(k1[r], k1[r]), e2 = f2(k2[r], k2[r]), so = f2(st[r].y, st[r].y);
      const uint64_t alpha = f2(a.alpha, a.alpha);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const uint32_t p = at[r] + j * per_vec;
        V8 d = unpack8(lds16(p)), f;
        if (pre) {
          const V8 g = unpack8(lds16(p + 2 * per_tensor)), y = unpack8(lds16(p + 3 * per_tensor));
          const V8 gamma = gn[j].get();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint64_t t = d.p[e];
            if constexpr (RMS) {
              t = f2_fma(y.p[e], c2, t);
            } else {
              // here and not in the first look, where the sums take the registers
              const uint64_t yh = f2_mul(f2_add(y.p[e], my), sd);
              S2[j].p[e] = f2_add(S2[j].p[e], g.p[e]);
              S3[j].p[e] = f2_fma(g.p[e], yh, S3[j].p[e]);
              t = f2_fma(yh, c2, f2_add(t, c1));
            }
            d.p[e] = f2_fma(sd, f2_mul(g.p[e], gamma.p[e]), t);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) f.p[e] = f2_mul(alpha, d.p[e]);
        if (in[j]) *reinterpret_cast<uint4*>(out_dx + j * step) = pack8(f);
        const V8 oh = load_oh(p, ex8[r][j], st[r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!RMS) S0[j].p[e] = f2_add(S0[j].p[e], d.p[e]);
          S1[j].p[e] = f2_fma(d.p[e], oh.p[e], S1[j].p[e]);
          d.p[e] = f2_mul(d.p[e], w[j].p[e]);
          if (post) {
            d.p[e] = f2_fma(oh.p[e], e2, d.p[e]);
            d.p[e] = f2_mul(so, RMS ? d.p[e] : f2_add(d.p[e], e1));
          }
        }
        if (in[j]) *reinterpret_cast<uint4*>(out_do + j * step) = pack8(d);
      }
      out_dx += a.ld_dx;
      out_do += a.ld_do;
    }
  };

  for (int64_t row = lo; row < hi;) {  // the rows of one gate after those of another
    const int64_t seg = row / rows_per_gate;
    const int64_t seg_end = (seg + 1) * rows_per_gate;
    const int64_t end = seg_end < hi ? seg_end : hi;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[j] = splat(in[j] ? 1.f : 0.f);
      if (in[j]) {
        if (a.gate) w[j] = load8(a.gate + seg * a.hidden + col + j * step, 0);
        if (post) {
          const V8 f = load8(a.post_gamma + col + j * step, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[j].p[e] = f2_mul(w[j].p[e], f.p[e]);
        }
      }
    }
    if (!RMS) {
      uint64_t t = 0;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) t = f2_add(t, w[j].p[e]);
      w_sum = both(t);
    }
    if constexpr (VEC == 3) {  // two rows' sums would not fit beside the channels'
      for (int n = static_cast<int>(end - row); n > 0; --n) rows(std::integral_constant<int, 1>());
    } else {
      for (int n = static_cast<int>((end - row) >> 1); n > 0; --n) rows(std::integral_constant<int, 2>());
      if ((end - row) & 1) rows(std::integral_constant<int, 1>());
    }
    row = end;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (in[j]) {
        float* dst = a.partials + (group + seg) * 2 * a.hidden + col + j * step;
        store_v8(dst, S0[j]);
        store_v8(dst + a.hidden, S1[j]);
      }
      S0[j] = S1[j] = splat(0.f);
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (in[j] && pre) {
      float* dst = a.partials + (groups + a.gates) * 2 * a.hidden +
                   group * 2 * static_cast<int64_t>(a.hidden) + col + j * step;
      store_v8(dst, S2[j]);
      store_v8(dst + a.hidden, S3[j]);
    }
  dependents_may_start();
  cp_async_wait<0>();
  if constexpr (CLUSTER) cluster_sync();  // no block leaves while another may still write to it
}

template <int VEC, bool CLUSTER, bool O8, bool FULL>
__global__ void __launch_bounds__(back_threads<VEC, true>(), 1)
    norm_backward_rms_kernel(const __grid_constant__ NormArgs a, int cluster, int slice, int groups,
                             int stages) {
  backward_rows<VEC, CLUSTER, true, O8, FULL>(a, cluster, slice, groups, stages);
}

template <int VEC, bool CLUSTER, bool O8, bool FULL>
__global__ void __maxnreg__(248)
    norm_backward_layer_kernel(const __grid_constant__ NormArgs a, int cluster, int slice, int groups,
                               int stages) {
  backward_rows<VEC, CLUSTER, false, O8, FULL>(a, cluster, slice, groups, stages);
}

// Joins the blocks' sums.  blockIdx.y = 0: dpost_gamma, dpost_beta and a single gate's dgate; 1:
// dpre_gamma, dpre_beta; 2 + g: dgate of gate g of several.  A block has 32 channels, 8 threads of 4
// beside one another, and deals the runs of rows to its 32 groups of 8 threads: each has a handful of
// loads, all in flight at once.  The groups' sums are added in order.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads)
    norm_backward_join_kernel(const __grid_constant__ NormArgs a, int groups) {
  __shared__ float4 part[2][32][8];
  wait_for_prior();
  const int quad = threadIdx.x & 7, lot = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + quad * 4;
  const bool in = col < a.hidden;
  const int64_t H = a.hidden;
  const bool pre = blockIdx.y == 1, each = blockIdx.y > 1;
  const int64_t per = a.rows / a.gates;
  float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
  auto add = [](float4& s, float4 v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
  auto load = [&](int64_t row) { return __ldcg(reinterpret_cast<const float4*>(a.partials + row * H + col)); };
  if (in) {
    if (pre || a.gates == 1) {
      const int64_t base = pre ? (groups + a.gates) * 2 : 0;
#pragma unroll 5
      for (int c = lot; c < groups; c += 32) {
        add(s0, load(base + 2 * c));
        add(s1, load(base + 2 * c + 1));
      }
    } else if (each) {
      // The runs that hold rows of this gate: run c begins at row c * rows / groups.
      const int64_t g = blockIdx.y - 2;
      const int c0 = static_cast<int>(((g * per + 1) * groups - 1) / a.rows);
      const int c1 = static_cast<int>(((g + 1) * per * groups - 1) / a.rows);
#pragma unroll 2
      for (int c = c0 + lot; c <= c1; c += 32) {
        add(s0, load(2 * (c + g)));
        add(s1, load(2 * (c + g) + 1));
      }
    } else {
      for (int c = lot; c < groups; c += 32) {  // a run's gates
        const int64_t lo = static_cast<int64_t>(c) * a.rows / groups;
        const int64_t hi = static_cast<int64_t>(c + 1) * a.rows / groups;
        for (int64_t g = lo / per; g * per < hi; ++g) {
          const float4 u = load(2 * (c + g)), v = load(2 * (c + g) + 1);
          const uint2 q = __ldg(reinterpret_cast<const uint2*>(a.gate + g * H + col));
          const float4 f = make_float4(bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y));
          add(s0, make_float4(f.x * u.x, f.y * u.y, f.z * u.z, f.w * u.w));
          add(s1, make_float4(f.x * v.x, f.y * v.y, f.z * v.z, f.w * v.w));
        }
      }
    }
  }
  part[0][lot][quad] = s0;
  part[1][lot][quad] = s1;
  __syncthreads();
  // One thread a channel from here.
  const int c = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || c >= a.hidden) return;
  float t0 = 0.f, t1 = 0.f;
#pragma unroll
  for (int l = 0; l < 32; ++l) {
    t0 += reinterpret_cast<const float*>(part[0][l])[threadIdx.x];
    t1 += reinterpret_cast<const float*>(part[1][l])[threadIdx.x];
  }
  if (pre) {
    if (a.dpre_gamma) a.dpre_gamma[c] = t1;
    if (a.dpre_beta) a.dpre_beta[c] = t0;
    return;
  }
  if (each || (a.gates == 1 && a.dgate)) {
    float v = t1;
    if (a.post_gamma) v *= __bfloat162float(a.post_gamma[c]);
    if (a.post_beta) v = fmaf(__bfloat162float(a.post_beta[c]), t0, v);
    a.dgate[(each ? blockIdx.y - 2 : 0) * H + c] = v;
  }
  if (!each) {
    const float f = a.gates == 1 && a.gate ? __bfloat162float(a.gate[c]) : 1.f;
    if (a.dpost_gamma) a.dpost_gamma[c] = f * t1;
    if (a.dpost_beta) a.dpost_beta[c] = f * t0;
  }
}

// Vectors and registers a thread: what keeps most rows under way on an SM without spilling much, since a
// row is a chain of loads, sums and barriers.  Layer norms have four rounds of sums, which cost less with
// more vectors (84 MB of each tensor: 5120 channels 77 us with two, 73 with three of 60 registers, 68 with
// four of 64; 8192 86 and 70, 16384 in 512 threads 118 with five of 128, 80; 20480 114 and 90 with five of
// 64; 32768 121 with eight, 97).  rms norms: 56 us up to 8192, 16384 82 and 68, 32768 94 and 78.  Of a
// warp's rows: layer norms of 256 channels 69 us with 32 registers and 76 with 46, 512 62 with 48 and 65
// with 64, 1024 65 with 64 and 76 with 88.
template <bool RMS>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t stream) {
  const int nvec = a.hidden / 8;
  const unsigned rows = static_cast<unsigned>(a.rows), warps = (rows + 7) / 8;
  auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
  if (nvec <= 32)
    norm_residual_kernel<1, true, RMS, 32><<<warps, 256, 0, stream>>>(a);
  else if (nvec <= 64)
    norm_residual_kernel<2, true, RMS, 48><<<warps, 256, 0, stream>>>(a);
  else if (nvec <= 128)
    norm_residual_kernel<4, true, RMS, RMS ? 72 : 64><<<warps, 256, 0, stream>>>(a);
  else if (nvec <= (RMS ? 1024 : 256))
    norm_residual_kernel<2, false, RMS, 40><<<rows, threads(2), 0, stream>>>(a);
  else if (nvec > 1024 && nvec <= 1536)
    norm_residual_kernel<3, false, RMS, 64><<<rows, threads(3), 0, stream>>>(a);
  else if (nvec > (RMS ? 1536 : 2048) && nvec <= 2560)
    norm_residual_kernel<5, false, RMS, 64><<<rows, threads(5), 0, stream>>>(a);
  else
    norm_residual_kernel<4, false, RMS, 64><<<rows, threads(4), 0, stream>>>(a);
  return cudaGetLastError();
}

template <int VEC, bool CLUSTER, bool RMS, bool O8, bool FULL>
cudaError_t launch_backward(const NormArgs& a, BackPlan& p, cudaStream_t stream) {
  void (*kern)(NormArgs, int, int, int, int);
  if constexpr (RMS)
    kern = norm_backward_rms_kernel<VEC, CLUSTER, O8, FULL>;
  else
    kern = norm_backward_layer_kernel<VEC, CLUSTER, O8, FULL>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  // The limit belongs to the kernel, which serves many sizes, and not to a launch: the largest, once for
  // each device.  (The size of each call would be another thread's limit between its set-up and its launch.)
  static std::atomic<uint64_t> raised{0};
  static_assert(kMaxDevices <= 64, "");
  if (!(raised.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
    if (e != cudaSuccess) return e;
    raised.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
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
  if (CLUSTER && p.cluster > 1) {
    // Clusters leave places over in each GPC: as many groups as run at once, or the last would be a
    // wave of their own.  The count follows from the cluster's and the block's size and from how the
    // device's SMs lie in its GPCs, which need not be alike on two devices.
    static std::atomic<uint16_t> known[kMaxDevices][9][back_threads<VEC, RMS>() / 32 + 1];
    std::atomic<uint16_t>& kept = known[dev][p.cluster][p.threads / 32];
    int most = kept.load(std::memory_order_relaxed);
    if (most == 0) {
      e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (most < 1) most = 1;
      kept.store(static_cast<uint16_t>(most), std::memory_order_relaxed);
    }
    if (p.groups > most) p.groups = most;
    cfg.gridDim = dim3(p.groups * p.cluster);
  }
  return cudaLaunchKernelEx(&cfg, kern, a, p.cluster, p.slice, p.groups, p.stages);
}

template <int VEC, bool CLUSTER, bool RMS>
cudaError_t launch_backward(const NormArgs& a, BackPlan& p, cudaStream_t stream) {
  const bool full = a.dy && a.dh && a.post_gamma;
  if (a.o_exps)
    return full ? launch_backward<VEC, CLUSTER, RMS, true, true>(a, p, stream)
                : launch_backward<VEC, CLUSTER, RMS, true, false>(a, p, stream);
  return full ? launch_backward<VEC, CLUSTER, RMS, false, true>(a, p, stream)
              : launch_backward<VEC, CLUSTER, RMS, false, false>(a, p, stream);
}

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, cudaStream_t stream) {
  return a.rms ? launch_forward<true>(a, stream) : launch_forward<false>(a, stream);
}

size_t norm_backward_partials(int64_t rows, int64_t hidden, int64_t gates, int sms) {
  const int a = back_plan(rows, hidden, true, sms).groups, b = back_plan(rows, hidden, false, sms).groups;
  return static_cast<size_t>(2 * (a > b ? a : b) + gates) * 2 * hidden * sizeof(float);
}

cudaError_t launch_norm_residual_backward(const NormArgs& a, cudaStream_t stream) {
  BackPlan p = back_plan(a.rows, a.hidden, a.rms != 0, a.sms);
  cudaError_t e;
  if (a.rms)  // (a slice of 16 channels a thread may be a cluster of one block)
    e = p.vec == 1 ? launch_backward<1, false, true>(a, p, stream)
                   : launch_backward<2, true, true>(a, p, stream);
  else if (p.vec == 3)
    e = launch_backward<3, false, false>(a, p, stream);
  else
    e = p.cluster > 1 ? launch_backward<2, true, false>(a, p, stream)
                      : launch_backward<2, false, false>(a, p, stream);
  if (e != cudaSuccess) return e;
  const unsigned each = a.dgate && a.gates > 1 ? static_cast<unsigned>(a.gates) : 0;
  return launch_dependent(norm_backward_join_kernel, dim3((a.hidden + 31) / 32, 2 + each),
                          dim3(kJoinThreads), 0, stream, a, p.groups);
}

}  // namespace ptb
