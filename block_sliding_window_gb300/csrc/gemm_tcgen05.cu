// The two GEMMs of the parallel transformer block on tcgen05 tensor cores.
//
//   [QKV | up]  : U = [xn W_qkv^T | gelu_tanh(xn W_up^T)]      (one GEMM, N = 3H + F)
//   [out | down]: y = x + [ctx | G] [W_o | W_down]^T            (one GEMM, K = H + F)
//
// The PTB computes the attention and MLP branches from the same LN(x) and
// sums both with the residual (MegaScale study notes, ch.2 §2.2, PTB row),
// so the two input projections share one GEMM and the two output
// projections share one GEMM whose epilogue adds x.  GeLU is fused into the
// first GEMM's epilogue (§2.5, Table 3, efficient-operators row).
//
// Kernel structure (one persistent CTA per SM, 192 threads; 320 with eight epilogue warps):
//   warp 0      TMA producer: 128 x 64 A tile and BN x 64 B tile per stage
//               into a ring of shared-memory stages (128-byte swizzle).
//   warp 1      owns the TMEM allocation; one thread issues tcgen05.mma
//               (M = 128, N = BN, K = 16) into a double-buffered fp32
//               accumulator in TMEM and commits stage / tile completion to
//               mbarriers.  (Measured on GB300: with 128 x 256 tiles a
//               64-wide k-block takes ~790 cycles for 512 cycles of MMA work,
//               matching the shared-memory traffic per k-block -- 48 KB of
//               operand reads plus 48 KB of TMA writes at ~128 B/clk.)
//   warps 2..5  (2..9 for the GEMMs of a gated feed-forward with bf16
//               outputs: epi_warps) epilogue: tcgen05.ld of the accumulator
//               (warp w reads TMEM lanes 32*(w%4) .. +31, i.e. one output row
//               per thread), GELU or residual add in fp32, bf16 stores.  The epilogue of
//               one work unit overlaps the main loop of the next.
//
// Work units.  The tiles that fill whole waves (a multiple of the grid) are
// processed whole, M-fastest, so the M tiles of one weight block run at the
// same time and share it through L2; odd waves walk K backwards, so each wave
// starts on the k-slabs the previous one left in L2.  The remaining R < grid tiles of the
// last, partial wave are each split along K into S pieces (R*S <= grid), one
// piece per otherwise idle CTA.  A piece writes its fp32 partial tile to the
// workspace, and each epilogue warp bumps an arrival counter of its 32-row
// quarter of the tile (two warps of a quarter have one each, for their chunks
// of columns); the warp that arrives last sums the S partials of what it
// counts in piece order (so the bits do not depend on who finished) and runs
// the epilogue for it.  Nothing ever waits on another CTA or another warp.
//
// Every mbarrier wait is bounded (see mbar_wait); on a timeout all roles
// unwind, wait for their own copies and MMAs, free TMEM and return.
#include "checkpoint_device.cuh"
#include "gated_device.cuh"
#include "ptb_device.cuh"

namespace ptb {
namespace {

constexpr int BM = 128;
// One k-block is one 128-byte swizzle row: 64 bf16 or 128 e4m3 elements,
// consumed by four MMAs (K = 16 bf16 or K = 32 e4m3 each, 32 bytes apart).
template <bool FP8>
struct Elem {
  static constexpr int kBK = FP8 ? 128 : 64;
};
constexpr int kMmasPerBlock = 4;

// Warps of the epilogue.  The gated epilogues do ten times the others' work for a value (two or three
// outputs, an exponential, groups of 8-bit codes) and a weight gradient of a few hundred tokens has a
// short main loop: both outlast it on four warps.  On eight, two share the rows of a TMEM quarter and
// take its 32-column chunks in turn.  A training step of 777 tokens, hidden 2048, ffn 5440: 252 us with
// four warps everywhere, 240 with eight in the gated epilogues, 235 with eight in all three; from 1500
// tokens and hidden 5120 on, where main loops are longer, no difference.
template <int EPI>
__host__ __device__ constexpr int epi_warps() {
  return EPI == kEpiGated || EPI == kEpiDgated || EPI == kEpiBf16 ? 8 : 4;
}
template <int EPI>
__host__ __device__ constexpr int gemm_threads() {
  return 64 + 32 * epi_warps<EPI>();
}

// The GEMMs of a gated feed-forward follow one another with nothing between them: each is set up
// (barriers, tensor memory) on the SMs that the one in front has left.  A training step of 777 tokens,
// hidden 2048, ffn 5440 takes 220 us that way and 227 without; 256 tokens of 256 by 256 12 and 14.8.
template <int EPI>
__host__ __device__ constexpr bool dependent() {
  return EPI == kEpiGated || EPI == kEpiDgated || EPI == kEpiBf16;
}

// The weight-gradient GEMMs (fp32 output, both operands MN-major) write
// their large outputs through shared memory: each epilogue warp stages its
// 32 rows x 32 columns (rows padded to 36 floats) and then writes whole
// 128-byte row segments, 4 rows per store instruction, instead of one
// 16-byte piece of 32 different rows.  Measured on GB300 (13B-class
// training step): the two weight-gradient GEMMs 7% and 9% faster; the same
// staging (and its 18 KB of shared memory) on every variant made the other
// GEMMs 3-15% slower, so only these variants use it.
constexpr int kF32Pad = 36;
constexpr int kF32StageBytes = 4 * 32 * kF32Pad * 4;

template <int EPI, int LAYOUT>
__host__ __device__ constexpr bool staged_f32() {
  return EPI == kEpiF32 && LAYOUT == kLayoutNN;
}

template <int BN, bool STAGE = false>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr int kABytes = BM * 128;  // 128-byte rows: 64 bf16 or 128 e4m3
  static constexpr int kBBytes = BN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes =
      kStages * kStageBytes + kBarBytes + (STAGE ? kF32StageBytes : 0) + 1024;
};

__device__ __forceinline__ float gelu_tanh(float z) {
  const float k0 = 0.7978845608028654f;  // sqrt(2 / pi)
  const float k1 = 0.044715f;
  return 0.5f * z * (1.0f + tanhf(k0 * (z + k1 * z * z * z)));
}

// One unit of work: k-blocks [kb0, kb1) of one output tile.  slot >= 0 marks
// a K piece of a remainder tile (its index in the partial-tile buffer).
struct Unit {
  int tile, kb0, kb1, slot;
};

// The i-th unit of worker `self` of `count` (a CTA, or a CTA pair); false
// when the worker has no more work.
__device__ __forceinline__ bool unit_at(const GemmArgs& p, int num_tiles, int num_kb, int i,
                                        Unit& u, int self, int count) {
  if (p.split_s < 2) {
    const int tile = self + i * count;
    if (tile >= num_tiles) return false;
    u = {tile, 0, num_kb, -1};
    return true;
  }
  const int whole = num_tiles - p.split_r;  // a multiple of count
  const int n_whole = whole / count;
  if (i < n_whole) {
    u = {self + i * count, 0, num_kb, -1};
    return true;
  }
  if (i == n_whole && self < p.split_r * p.split_s) {
    const int r = self / p.split_s;
    const int s = self % p.split_s;
    u = {whole + r, s * num_kb / p.split_s, (s + 1) * num_kb / p.split_s, self};
    return true;
  }
  return false;
}

// The t-th k-block a unit processes.  Whole-tile units of odd waves (odd
// unit index i) walk K backwards: a wave's tiles read the shared operand
// k-slab by k-slab in step, and the operand of the long-K GEMMs is larger
// than L2, so a wave that starts where the previous one ended finds its
// first k-slabs still in L2 instead of re-reading them from DRAM.  K pieces
// of split tiles keep the forward order.
__device__ __forceinline__ int unit_kb(const Unit& u, int i, int t) {
  return ((i & 1) && u.slot < 0) ? u.kb1 - 1 - t : u.kb0 + t;
}

// e4m3 operands carry one scale per A row and one per B row (= output
// column): C[m, n] = a_scale[m] * b_scale[n] * sum_k A8[m, k] B8[n, k].
__device__ __forceinline__ void dequantize(const GemmArgs& p, int row, int col, float (&acc)[32]) {
  const float sa = row < p.M ? __ldg(p.a_scale + row) : 0.f;
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    const float4 sb = __ldg(reinterpret_cast<const float4*>(p.b_scale + col) + v);
    acc[4 * v] *= sa * sb.x;
    acc[4 * v + 1] *= sa * sb.y;
    acc[4 * v + 2] *= sa * sb.z;
    acc[4 * v + 3] *= sa * sb.w;
  }
}

// d/dz gelu_tanh(z) = 0.5 (1 + t) + 0.5 z (1 - t^2) c (1 + 3 a z^2),
// t = tanh(c (z + a z^3)), c = sqrt(2 / pi), a = 0.044715.
__device__ __forceinline__ float gelu_tanh_grad(float z) {
  const float k0 = 0.7978845608028654f;
  const float k1 = 0.044715f;
  const float t = tanhf(k0 * (z + k1 * z * z * z));
  return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * k0 * (1.0f + 3.0f * k1 * z * z);
}

__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* dst_row, const uint32_t (&packed)[16]) {
  uint4* dst = reinterpret_cast<uint4*>(dst_row);
#pragma unroll
  for (int v = 0; v < 4; ++v)
    dst[v] = make_uint4(packed[4 * v], packed[4 * v + 1], packed[4 * v + 2], packed[4 * v + 3]);
}

// Epilogue of one 32-column chunk of one output row: acc (fp32) -> out.
template <int EPI>
__device__ __forceinline__ void store_chunk(const GemmArgs& p, int row, int col,
                                            const float (&acc)[32]) {
  // Destination region (a 32-column chunk never straddles a split point).
  void* base = p.out;
  int64_t ld = p.ld_out;
  int64_t r = row, c = col;
  if (col >= p.out_split_col) {
    base = p.out1;
    ld = p.ld_out1;
    c -= p.out_split_col;
  } else if (row >= p.out_split_row) {
    base = p.out1;
    ld = p.ld_out1;
    r -= p.out_split_row;
  }
  if constexpr (EPI == kEpiF32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + r * ld + c);
#pragma unroll
    for (int v = 0; v < 8; ++v)
      dst[v] = make_float4(acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]);
    return;
  }
  uint32_t packed[16];
  if constexpr (EPI == kEpiQkvGelu) {
    if (col >= p.gelu_col) {
      if (p.aux) {  // keep the pre-activation for the backward pass
#pragma unroll
        for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(acc[2 * j], acc[2 * j + 1]);
        store_bf16x32(p.aux + row * p.ld_aux + (col - p.gelu_col), packed);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
        packed[j] = pack_bf16x2(gelu_tanh(acc[2 * j]), gelu_tanh(acc[2 * j + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(acc[2 * j], acc[2 * j + 1]);
    }
  } else if constexpr (EPI == kEpiDgelu) {
    if (col >= p.gelu_col) {
      const uint4* src = reinterpret_cast<const uint4*>(p.aux + row * p.ld_aux + (col - p.gelu_col));
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint4 z = __ldg(src + v);
        const uint32_t zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = v * 8 + j * 2;
          packed[v * 4 + j] = pack_bf16x2(acc[e] * gelu_tanh_grad(bf16_lo(zs[j])),
                                          acc[e + 1] * gelu_tanh_grad(bf16_hi(zs[j])));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(acc[2 * j], acc[2 * j + 1]);
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(p.resid + row * p.ld_resid + col);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint4 x = __ldg(src + v);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = v * 8 + j * 2;
        packed[v * 4 + j] = pack_bf16x2(acc[e] + bf16_lo(xs[j]), acc[e + 1] + bf16_hi(xs[j]));
      }
    }
  }
  store_bf16x32(static_cast<__nv_bfloat16*>(base) + r * ld + c, packed);
}

// 16 columns in one 32-byte store, a whole sector, for rows that begin on 32 bytes.
__device__ __forceinline__ void store_bf16x16(__nv_bfloat16* dst, const uint32_t (&packed)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
               "r"(packed[0]), "r"(packed[1]), "r"(packed[2]), "r"(packed[3]), "r"(packed[4]),
               "r"(packed[5]), "r"(packed[6]), "r"(packed[7])
               : "memory");
}

__device__ __forceinline__ void load16(const __nv_bfloat16* src, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
          "=r"(w[7])
        : "l"(src));
  } else {
    const uint4 p = __ldg(reinterpret_cast<const uint4*>(src));
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w, w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
  }
}

// bf16 [resid +] acc of 32 columns of a row, rows beyond out_split_row to out1.  p.wide: every row of
// both outputs begins on 32 bytes.
__device__ __forceinline__ void store_bf16(const GemmArgs& p, int row, int col,
                                           const float (&acc)[32]) {
  const bool second = row >= p.out_split_row;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(second ? p.out1 : p.out) +
                       (second ? (row - p.out_split_row) * p.ld_out1 : row * p.ld_out) + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
    if (p.resid) {
      const uint4* src = reinterpret_cast<const uint4*>(p.resid + row * p.ld_resid + col + 16 * h);
      const uint4 x = src[0], y = src[1];  // the output may be the residual itself
      const uint32_t r[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = pack_bf16x2(acc[16 * h + 2 * j] + bf16_lo(r[j]), acc[16 * h + 2 * j + 1] + bf16_hi(r[j]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(acc[16 * h + 2 * j], acc[16 * h + 2 * j + 1]);
    }
    if (p.wide) {
      store_bf16x16(dst + 16 * h, w);
    } else {
      uint4* d = reinterpret_cast<uint4*>(dst + 16 * h);
      d[0] = make_uint4(w[0], w[1], w[2], w[3]);
      d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

__device__ __forceinline__ void pack_row(const float (&v)[32], uint32_t (&packed)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
}

// Forward of a gated feed-forward, 32 columns of one row: gate g and up u (fp32 accumulators) ->
// act(g) * u, rounded once; what the backward pass keeps is rounded from the accumulators, too.
__device__ __forceinline__ void store_gated(const GemmArgs& p, int row, int col,
                                            const float (&g)[32], const float (&u)[32]) {
  const GatedAct act(p.act);
  uint32_t packed[16];
  if (p.kept) {
    const int64_t at = static_cast<int64_t>(row) * 2 * p.ffn + col;
    if (p.kept_exps) {
      uint8_t* codes = static_cast<uint8_t*>(p.kept);
      ckpt_store_group(g, codes + at, p.kept_exps + at / kCkptGroup);
      ckpt_store_group(u, codes + at + p.ffn, p.kept_exps + (at + p.ffn) / kCkptGroup);
    } else {
      __nv_bfloat16* kept = static_cast<__nv_bfloat16*>(p.kept);
      pack_row(g, packed);
      store_bf16x32(kept + at, packed);
      pack_row(u, packed);
      store_bf16x32(kept + at + p.ffn, packed);
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t half[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = 16 * h + 2 * j;
      half[j] = pack_bf16x2(act.value(g[e]) * u[e], act.value(g[e + 1]) * u[e + 1]);
    }
    store_bf16x16(out + 16 * h, half);
  }
}

// What the forward pass kept of 32 columns of a row: gate and up, bf16 pairs or codes.
struct Kept {
  uint32_t g[16], u[16];
  float sg, su;
};

__device__ __forceinline__ void load_kept(const GemmArgs& p, int row, int col, Kept& k) {
  if (row >= p.M || col >= p.N) return;
  const int64_t at = static_cast<int64_t>(row) * 2 * p.ffn + col;
  const bool wide = (reinterpret_cast<uintptr_t>(p.kept) & 31) == 0;
  if (p.kept_exps) {
    const uint8_t* codes = static_cast<const uint8_t*>(p.kept) + at;
    load16(reinterpret_cast<const __nv_bfloat16*>(codes), wide, reinterpret_cast<uint32_t(&)[8]>(k.g));
    load16(reinterpret_cast<const __nv_bfloat16*>(codes + p.ffn), wide,
           reinterpret_cast<uint32_t(&)[8]>(k.u));
    k.sg = ckpt_scale(__ldg(p.kept_exps + at / kCkptGroup));
    k.su = ckpt_scale(__ldg(p.kept_exps + (at + p.ffn) / kCkptGroup));
  } else {
    const __nv_bfloat16* kept = static_cast<const __nv_bfloat16*>(p.kept) + at;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load16(kept + 16 * h, wide, reinterpret_cast<uint32_t(&)[8]>(k.g[8 * h]));
      load16(kept + p.ffn + 16 * h, wide, reinterpret_cast<uint32_t(&)[8]>(k.u[8 * h]));
    }
  }
}

// Four neighbouring values, columns 4 q .. 4 q + 3 of the 32.
__device__ __forceinline__ void kept4(const uint32_t (&w)[16], float scale, bool codes, int q,
                                      float (&v)[4]) {
  if (codes) {
    ckpt_unpack4(w[q], v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= scale;
  } else {
    v[0] = bf16_lo(w[2 * q]), v[1] = bf16_hi(w[2 * q]);
    v[2] = bf16_lo(w[2 * q + 1]), v[3] = bf16_hi(w[2 * q + 1]);
  }
}

// Backward of act(g) * u for its gradient d, 32 columns of one row, g and u as they were kept:
// act(g) * u once more for the weight gradient of the down projection, d u act'(g) and d act(g).
__device__ __forceinline__ void store_dgated(const GemmArgs& p, int row, int col,
                                             const float (&d)[32], const Kept& kept) {
  const GatedAct act(p.act);
  const bool codes = p.kept_exps != nullptr;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + col;
  __nv_bfloat16* out1 = static_cast<__nv_bfloat16*>(p.out1) + row * p.ld_out1 + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pa[8], pg[8], pu[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float g[4], u[4];
      kept4(kept.g, kept.sg, codes, 4 * h + q, g);
      kept4(kept.u, kept.su, codes, 4 * h + q, u);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float d0 = d[16 * h + 4 * q + e], d1 = d[16 * h + 4 * q + e + 1];
        float a0, s0, a1, s1;
        act.value_and_slope(g[e], a0, s0);
        act.value_and_slope(g[e + 1], a1, s1);
        const int j = 2 * q + e / 2;
        pa[j] = pack_bf16x2(a0 * u[e], a1 * u[e + 1]);
        pg[j] = pack_bf16x2(d0 * u[e] * s0, d1 * u[e + 1] * s1);
        pu[j] = pack_bf16x2(d0 * a0, d1 * a1);
      }
    }
    store_bf16x16(out + 16 * h, pa);
    store_bf16x16(out1 + 16 * h, pg);
    store_bf16x16(out1 + p.ffn + 16 * h, pu);
  }
}

// Output tile origin of tile index t (M index fastest, or N index fastest).
__device__ __forceinline__ void tile_origin(const GemmArgs& p, int t, int num_m, int num_n, int bm,
                                            int bn, int& m0, int& n0) {
  if (p.n_fastest) {
    m0 = (t / num_n) * bm;
    n0 = (t % num_n) * bn;
  } else {
    m0 = (t % num_m) * bm;
    n0 = (t / num_m) * bn;
  }
}

// fp32 epilogue of one 32-column chunk for the 32 consecutive rows of a warp
// (lane i holds row row0 + i): staged in `st` (32 x kF32Pad floats) and
// stored row segment by row segment.  Warp-collective.
__device__ __forceinline__ void store_chunk_f32_warp(const GemmArgs& p, int row, int col,
                                                     const float (&acc)[32], int lane,
                                                     float* st) {
  float* mine = st + lane * kF32Pad;
#pragma unroll
  for (int v = 0; v < 8; ++v)
    *reinterpret_cast<float4*>(mine + 4 * v) =
        make_float4(acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]);
  __syncwarp();
  const int row0 = row - lane;
  const int c4 = lane & 7;
  const bool second_col = col >= p.out_split_col;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + (lane >> 3);
    const float4 v = *reinterpret_cast<const float4*>(st + r * kF32Pad + 4 * c4);
    const int grow = row0 + r;
    if (grow < p.M) {
      float* base = static_cast<float*>(p.out);
      int64_t ld = p.ld_out, rr = grow, cc = col + 4 * c4;
      if (second_col) {
        base = static_cast<float*>(p.out1);
        ld = p.ld_out1;
        cc -= p.out_split_col;
      } else if (grow >= p.out_split_row) {
        base = static_cast<float*>(p.out1);
        ld = p.ld_out1;
        rr -= p.out_split_row;
      }
      *reinterpret_cast<float4*>(base + rr * ld + cc) = v;
    }
  }
  __syncwarp();
}

// Partial tiles: the 32 x 32 chunk of rows prow .. and columns c .. of piece `slot` is 4 KB in the
// order in which a warp writes and reads it, 16 bytes of each lane side by side (whole lines; rows
// of a partial would give each instruction 32 of them).
template <int BN, int ROWS>
__device__ __forceinline__ float4* partial_chunk(const GemmArgs& p, int slot, int prow, int c) {
  const int64_t chunk = (static_cast<int64_t>(slot) * (ROWS / 32) + (prow >> 5)) * (BN / 32) + (c >> 5);
  return reinterpret_cast<float4*>(p.partials) + chunk * 256 + (prow & 31);
}

// Sums of the K pieces' partials, 32 columns of this thread's row at a time, in piece order.  Each
// thread copies what it will add through its own part of the operands' ring, which no load or MMA uses
// behind a worker's last unit: the copies of kSlots pieces are on their way at a time.
// (Loaded into registers, a piece at a time, the join took 0.8 us more for each piece: 200 tokens by
// 2048 by 10880 in nine pieces 36 us, 30 this way.)
template <int BN, int EPI, int ROWS>
struct PieceSums {
  static constexpr int kSlots = epi_warps<EPI>() == 8 ? 5 : 8;  // of 4 KB a warp
  static constexpr int kRingBytes = epi_warps<EPI>() * kSlots * 4096;  // 160 KB, or 128 on four warps
  static constexpr int kStride = 32 * (epi_warps<EPI>() / 4);
  static constexpr int64_t kPiece = static_cast<int64_t>(ROWS / 32) * (BN / 32) * 256;
  const float4* src;  // piece 0
  uint32_t slots, at = 0;
  int first, chunks, pieces, chunk = 0, piece = 0;

  // Columns first, first + kStride .. below `end` of tile columns; of the gated epilogue each of them
  // and then the one BN / 2 behind it.
  __device__ __forceinline__ PieceSums(const GemmArgs& p, int slot, int prow, int first_, int end,
                                       uint8_t* ring, int warp)
      : slots(smem_addr(ring) + warp * kSlots * 4096 + (prow & 31) * 16), first(first_),
        pieces(p.split_s) {
    src = partial_chunk<BN, ROWS>(p, slot / pieces * pieces, prow, 0);
    chunks = end > first ? (end - first + kStride - 1) / kStride : 0;
    if (EPI == kEpiGated) chunks *= 2;
#pragma unroll 1
    for (int k = 0; k < kSlots; ++k) fetch();
  }
  __device__ __forceinline__ void fetch() {
    if (chunk < chunks) {
      const int c = EPI == kEpiGated ? first + (chunk >> 1) * kStride + (chunk & 1) * (BN / 2)
                                     : first + chunk * kStride;
      const float4* from = src + piece * kPiece + (c >> 5) * 256;
#pragma unroll
      for (int v = 0; v < 8; ++v) cp_async16(slots + at + v * 512, from + 32 * v);
      if (++piece == pieces) {
        piece = 0;
        ++chunk;
      }
    }
    cp_async_commit();
    at = at == (kSlots - 1) * 4096 ? 0 : at + 4096;
  }
  // The next chunk.
  __device__ __forceinline__ void sum(float (&acc)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = 0.f;
#pragma unroll 1
    for (int s = 0; s < pieces; ++s) {
      cp_async_wait<kSlots - 1>();
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const uint4 q = lds16(slots + at + v * 512);
        acc[4 * v] += __uint_as_float(q.x);
        acc[4 * v + 1] += __uint_as_float(q.y);
        acc[4 * v + 2] += __uint_as_float(q.z);
        acc[4 * v + 3] += __uint_as_float(q.w);
      }
      fetch();
    }
  }
};

// The epilogue of one unit for one thread's output row `row`: a whole tile
// goes straight from TMEM through store_chunk; a K piece of a split tile
// publishes its fp32 partial (row `prow` of the ROWS-row partial tile) and
// counts its warp's arrival on p.counters[counter], and the warp that
// arrives last for those 32 rows sums all pieces in piece order and stores.
template <int BN, int EPI, bool FP8, int ROWS, bool STAGE>
__device__ __forceinline__ void epilogue_unit(const GemmArgs& p, const Unit& u, int row, int prow,
                                              int counter, uint32_t t_row, int n0, int lane,
                                              float* f32_stage, int half, uint8_t* ring) {
  // This warp's chunks of 32 columns, from `first` on below `width`.  (Where a quarter has one warp only,
  // `first` is a constant, and the bound is found once: a loop that tested n0 + c < p.N from a `first` of
  // its warp cost the fp32 weight gradients 4%, 512 tokens, hidden 12288, ffn 49152: 1032 and 1674 us for
  // 989 and 1593.)
  constexpr int stride = 32 * (epi_warps<EPI>() / 4);
  const int first = epi_warps<EPI>() == 4 ? 0 : 32 * half;
  const int width = min(BN, p.N - n0);
  bool finish = true;
  const int warp = prow / 32 % 4 + 4 * half;  // of the epilogue
  if (u.slot >= 0) {
    if (row - lane >= p.M) return;  // none of the warp's rows are there
    // A K piece: publish the fp32 partial, then count the arrival.
#pragma unroll 1
    for (int c = first; c < BN; c += stride) {
      if (EPI != kEpiGated && n0 + c >= p.N) break;
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_row + c, r);
      tmem_ld_wait();
      float4* dst = partial_chunk<BN, ROWS>(p, u.slot, prow, c);
#pragma unroll
      for (int v = 0; v < 8; ++v)
        __stcg(dst + 32 * v,
               make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                           __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3])));
    }
    // Each warp owns its 32 rows (or its half of their chunks): it counts
    // its own arrival for them, and the last warp to arrive finishes them.  No warp waits for another.
    __threadfence();
    __syncwarp();
    unsigned prev = 0;
    if (lane == 0) prev = atomicAdd(p.counters + counter, 1u);
    prev = __shfl_sync(0xffffffffu, prev, 0);
    finish = prev == static_cast<unsigned>(p.split_s - 1);
    if (finish) __threadfence();
  }
  if constexpr (EPI == kEpiGated) {
    // Columns c and BN / 2 + c of the tile are gate and up of output column n0 / 2 + c.
    const int end = min(BN / 2, p.ffn - n0 / 2);
    if (u.slot < 0) {
#pragma unroll 1
      for (int c = first; c < end; c += stride) {
        float v[2][32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(t_row + h * (BN / 2) + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[h][j] = __uint_as_float(r[j]);
        }
        if (row < p.M) store_gated(p, row, n0 / 2 + c, v[0], v[1]);
      }
    } else if (finish) {
      PieceSums<BN, EPI, ROWS> pieces(p, u.slot, prow, first, end, ring, warp);
#pragma unroll 1
      for (int c = first; c < end; c += stride) {
        float v[2][32];
        pieces.sum(v[0]);
        pieces.sum(v[1]);
        if (row < p.M) store_gated(p, row, n0 / 2 + c, v[0], v[1]);
      }
    }
    return;
  }
  // (kEpiDgated) each chunk's kept values are asked for before the chunk in front of it is worked on
  Kept kept, next;
  if (EPI == kEpiDgated && finish) load_kept(p, row, n0 + first, next);
  if constexpr (EPI == kEpiBf16) {
    if (u.slot < 0) {  // two chunks on their way at a time
#pragma unroll 1
      for (int c = first; c < width; c += 2 * stride) {
        const bool two = c + stride < width;
        uint32_t r[2][32];
        tmem_ld_32x32b_x32(t_row + c, r[0]);
        if (two) tmem_ld_32x32b_x32(t_row + c + stride, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float acc[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] = __uint_as_float(r[h][j]);
          if (row < p.M && (h == 0 || two)) store_bf16(p, row, n0 + c + h * stride, acc);
        }
      }
      return;
    }
  }
  if (finish && u.slot < 0) {
#pragma unroll 1
    for (int c = first; c < width; c += stride) {
      if constexpr (EPI == kEpiDgated) {
        kept = next;
        if (c + stride < BN) load_kept(p, row, n0 + c + stride, next);
      }
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_row + c, r);
      tmem_ld_wait();
      float acc[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] = __uint_as_float(r[j]);
      if constexpr (FP8) dequantize(p, row, n0 + c, acc);
      if constexpr (STAGE)
        store_chunk_f32_warp(p, row, n0 + c, acc, lane, f32_stage);
      else if (row < p.M) {
        if constexpr (EPI == kEpiDgated)
          store_dgated(p, row, n0 + c, acc, kept);
        else if constexpr (EPI == kEpiBf16)
          store_bf16(p, row, n0 + c, acc);
        else
          store_chunk<EPI>(p, row, n0 + c, acc);
      }
    }
  } else if (finish) {
    // Sum every piece's partial (this warp's own included) in piece order,
    // so the result does not depend on which warp happened to finish.
    PieceSums<BN, EPI, ROWS> pieces(p, u.slot, prow, first, width, ring, warp);
#pragma unroll 1
    for (int c = first; c < width; c += stride) {
      if constexpr (EPI == kEpiDgated) {
        kept = next;
        if (c + stride < BN) load_kept(p, row, n0 + c + stride, next);
      }
      float acc[32];
      pieces.sum(acc);
      if constexpr (FP8) dequantize(p, row, n0 + c, acc);
      if constexpr (STAGE)
        store_chunk_f32_warp(p, row, n0 + c, acc, lane, f32_stage);
      else if (row < p.M) {
        if constexpr (EPI == kEpiDgated)
          store_dgated(p, row, n0 + c, acc, kept);
        else if constexpr (EPI == kEpiBf16)
          store_bf16(p, row, n0 + c, acc);
        else
          store_chunk<EPI>(p, row, n0 + c, acc);
      }
    }
  }
}

template <int BN, int EPI, bool FP8, int LAYOUT>
__global__ void __launch_bounds__(gemm_threads<EPI>(), 1) gemm_kernel(const __grid_constant__ GemmArgs p) {
  constexpr bool kStage = staged_f32<EPI, LAYOUT>();
  using C = Cfg<BN, kStage>;
  constexpr int BK = Elem<FP8>::kBK;
  // MN-major operands arrive as 64-wide MN blocks of 64 K rows (8 KB each).
  constexpr bool kAmn = (LAYOUT & 1) != 0;
  constexpr bool kBmn = (LAYOUT & 2) != 0;
  constexpr uint32_t kMnBlock = 64 * 128;
  static_assert(!(FP8 && LAYOUT != kLayoutKK), "e4m3 operands are K-major only");
  static_assert(PieceSums<BN, EPI, BM>::kRingBytes <= C::kStages * C::kStageBytes,
                "the join of K pieces would reach past the ring into the barriers");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty_bar = full_bar + C::kStages;
  uint64_t* tfull_bar = empty_bar + C::kStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* done_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_m = (p.M + BM - 1) / BM;
  const int num_n = (p.N + BN - 1) / BN;  // columns behind N: zeros by TMA, not stored
  const int num_tiles = num_m * num_n;
  const int num_kb = (p.K + BK - 1) / BK;  // a K tail is zero-filled by TMA

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], epi_warps<EPI>());
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.a0);
    tma_prefetch_desc(&p.a1);
    tma_prefetch_desc(&p.b0);
    tma_prefetch_desc(&p.b1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if constexpr (dependent<EPI>()) {
    wait_for_prior();
    dependents_may_start();
  }

  auto stage_a = [&](int s) { return smem + s * C::kStageBytes; };
  auto stage_b = [&](int s) { return smem + s * C::kStageBytes + C::kABytes; };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      // L2 priority of each operand's loads as the launcher chose it (the
      // layer's GEMMs keep both, evict_last).  Measured on this kernel with
      // the weights at normal priority instead of evict_first, the 175B
      // layer ran 11% slower; an L2 prefetch of the tiles 8 k-blocks ahead,
      // 48% slower.
      const uint64_t pol = p.a_keep ? l2_policy_evict_last() : l2_policy_evict_first();
      const uint64_t pol_b = p.b_keep ? l2_policy_evict_last() : l2_policy_evict_first();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0;  // bit s: stage s has had a load issued
      uint32_t armed_parity = 0;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && unit_at(p, num_tiles, num_kb, i, u, blockIdx.x, gridDim.x); ++i) {
        int m0, n0;
        tile_origin(p, u.tile, num_m, num_n, BM, BN, m0, n0);
        const bool nlo = n0 < p.n_split;
        const int by = nlo ? n0 : n0 - p.n_split;
        for (int t = 0; t < u.kb1 - u.kb0; ++t) {
          const int kb = unit_kb(u, i, t);
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const int k = kb * BK;
          const bool klo = k < p.k_split;
          const int kx = klo ? k : k - p.k_split;
          mbar_arrive_expect_tx(&full_bar[stage], C::kStageBytes);
          const CUtensorMap* amap = klo ? &p.a0 : &p.a1;
          const CUtensorMap* bmap = (nlo && klo) ? &p.b0 : &p.b1;
          if constexpr (kAmn) {
#pragma unroll
            for (int h = 0; h < BM / 64; ++h)
              tma_load_2d(stage_a(stage) + h * kMnBlock, amap, &full_bar[stage], m0 + 64 * h, kx,
                          pol);
          } else {
            tma_load_2d(stage_a(stage), amap, &full_bar[stage], kx, m0, pol);
          }
          if constexpr (kBmn) {
#pragma unroll
            for (int h = 0; h < BN / 64; ++h)
              tma_load_2d(stage_b(stage) + h * kMnBlock, bmap, &full_bar[stage], by + 64 * h, kx,
                          pol_b);
          } else if constexpr (EPI == kEpiGated) {
            // Rows n0 / 2 .. of the gate's weights, then the same rows of up's.
            tma_load_2d(stage_b(stage), &p.b0, &full_bar[stage], kx, n0 / 2, pol_b);
            tma_load_2d(stage_b(stage) + BN / 2 * 128, &p.b1, &full_bar[stage], kx, n0 / 2, pol_b);
          } else {
            tma_load_2d(stage_b(stage), bmap, &full_bar[stage], kx, by, pol_b);
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // Unwinding: let every copy this thread issued land before the CTA
        // (and its shared memory) goes away.
        volatile int no_abort = 0;
        for (int s = 0; s < C::kStages; ++s)
          if (armed & (1u << s))
            mbar_wait(&full_bar[s], (armed_parity >> s) & 1u, &no_abort, p.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    if (lane == 0) {
      constexpr uint32_t idesc = (FP8 ? umma_idesc_e4m3(BM, BN) : umma_idesc_bf16(BM, BN)) |
                                 (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && unit_at(p, num_tiles, num_kb, i, u, blockIdx.x, gridDim.x); ++i) {
        const int acc = i & 1;
        const uint32_t acc_phase = (i >> 1) & 1;
        if (!mbar_wait(&tempty_bar[acc], acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int t = 0; t < u.kb1 - u.kb0; ++t) {
          if (!mbar_wait(&full_bar[stage], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = kAmn ? sw128_mnmajor_desc(smem_addr(stage_a(stage)), kMnBlock)
                                      : sw128_kmajor_desc(smem_addr(stage_a(stage)));
          const uint64_t bdesc = kBmn ? sw128_mnmajor_desc(smem_addr(stage_b(stage)), kMnBlock)
                                      : sw128_kmajor_desc(smem_addr(stage_b(stage)));
          // One MMA step along K: +32 bytes inside a K-major swizzled row
          // (+2 in the descriptor's 16-byte units), or 16 rows of 128 bytes
          // of an MN-major block (+128).
          constexpr uint64_t kStepA = kAmn ? 128 : 2;
          constexpr uint64_t kStepB = kBmn ? 128 : 2;
#pragma unroll
          for (int kk = 0; kk < kMmasPerBlock; ++kk) {
            const uint32_t accum = (t != 0 || kk != 0) ? 1u : 0u;
            if constexpr (FP8)
              umma_e4m3_ss(d_tmem, adesc + kStepA * kk, bdesc + kStepB * kk, idesc, accum);
            else
              umma_bf16_ss(d_tmem, adesc + kStepA * kk, bdesc + kStepB * kk, idesc, accum);
          }
          umma_commit(&empty_bar[stage]);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit(&tfull_bar[acc]);
      }
      // Wait for every MMA this thread issued before TMEM is released.
      umma_commit(done_bar);
      volatile int no_abort = 0;
      mbar_wait(done_bar, 0, &no_abort, p.status);
    }
  } else {
    // --------------------------------------------------------- epilogue --
    const int quarter = warp & 3;
    const int row_local = quarter * 32 + lane;
    float* f32_stage = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes + C::kBarBytes) +
                       quarter * 32 * kF32Pad;
    Unit u;
    for (int i = 0; unit_at(p, num_tiles, num_kb, i, u, blockIdx.x, gridDim.x); ++i) {
      const int acc_buf = i & 1;
      const uint32_t acc_phase = (i >> 1) & 1;
      if (!mbar_wait_warp(&tfull_bar[acc_buf], acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      int m0, n0;
      tile_origin(p, u.tile, num_m, num_n, BM, BN, m0, n0);
      const int row = m0 + row_local;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc_buf * BN);
      epilogue_unit<BN, EPI, FP8, BM, kStage>(p, u, row, row_local,
                                              (u.slot / p.split_s) * epi_warps<EPI>() + warp - 2,
                                              t_row, n0, lane, f32_stage, (warp - 2) >> 2, smem);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[acc_buf]);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ------------------------------------------------------------ CTA pairs --
// 256 x 256 output tiles on a CTA pair (a cluster of two CTAs on the two SMs
// of a TPC, tcgen05 cta_group::2).  Rank r loads rows m0 + 128 r of A and
// columns by + 128 r of B into its own shared memory; rank 0 issues M = 256,
// N = 256 MMAs that read both CTAs' tiles at the same offsets, and each CTA's
// TMEM receives its 128 rows of the accumulator.  Per SM and 64-wide k-block
// the stage is 32 KB instead of 48 KB, so the shared-memory traffic of TMA
// writes plus operand reads drops by a third.
//   warp 0      both ranks: TMA producer into their own ring of 5
//               stages (pair_stages).  The
//               copies of both ranks complete on rank 0's `full` barrier of
//               the stage (cta_group::2 TMA), which rank 0 arms with the
//               bytes of both.  (A first version relayed rank 1's stages with
//               a cluster-scope release arrive per stage and ran at 31%
//               tensor activity.)
//   warp 1      both ranks allocate TMEM together (cta_group::2).  Rank 0
//               issues the MMAs and commits stage and tile completion to the
//               barriers at the same offset in both CTAs.
//   warps 2..5  (2..9) both ranks: epilogue of their 128 rows; each warp then
//               arrives on rank 0's `tempty` barrier (8 or 16 arrivals per
//               tile).
// The remainder wave is split along K per pair as in the single-CTA kernel
// (256-row partial tiles, 8 or 16 arrival counters per tile).
constexpr int kPairBN = 256;
// Stages of the ring.  Fewer stages leave more of the SM's unified L1 /
// shared memory to L1.  With both operands loaded evict_last, 5 stages for
// every GEMM against 6 for [QKV | up] (5 for the others): 175B-class layer
// 4.41-4.47 vs 4.45-4.50 ms, 13B-class, e4m3 and training within noise; 6
// for all and 7 for [QKV | up] were slower everywhere (175B-class 4.54-4.57
// ms, training 14.3-14.7 vs 14.2-14.4 ms).  (Under the earlier evict_first
// weights, 6 had been 1.7% better for [QKV | up] at 13B.)
template <int EPI>
__host__ __device__ constexpr int pair_stages() { return 5; }
template <bool STAGE = false, int NSTAGES = 6>
struct PairCfg {
  static constexpr int kABytes = BM * 128;
  static constexpr int kBBytes = (kPairBN / 2) * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTmemCols = 2 * kPairBN;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes =
      NSTAGES * kStageBytes + kBarBytes + (STAGE ? kF32StageBytes : 0) + 1024;
};

template <int EPI, int LAYOUT, bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(gemm_threads<EPI>(), 1)
    gemm_pair_kernel(const __grid_constant__ GemmArgs p) {
  constexpr bool kStage = staged_f32<EPI, LAYOUT>();
  using C = PairCfg<kStage, pair_stages<EPI>()>;
  constexpr int BN = kPairBN;
  constexpr int BK = Elem<FP8>::kBK;
  static_assert(!(FP8 && LAYOUT != kLayoutKK), "e4m3 operands are K-major only");
  constexpr int NS = pair_stages<EPI>();
  // MN-major operands arrive as 64-wide MN blocks of 64 K rows (8 KB each).
  constexpr bool kAmn = (LAYOUT & 1) != 0;
  constexpr bool kBmn = (LAYOUT & 2) != 0;
  constexpr uint32_t kMnBlock = 64 * 128;
  static_assert(PieceSums<BN, EPI, 2 * BM>::kRingBytes <= NS * C::kStageBytes,
                "the join of K pieces would reach past the ring into the barriers");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + NS * C::kStageBytes);
  uint64_t* empty_bar = full_bar + NS;
  uint64_t* tfull_bar = empty_bar + NS;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* done_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int npairs = static_cast<int>(gridDim.x >> 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_m = (p.M + 2 * BM - 1) / (2 * BM);
  const int num_n = (p.N + BN - 1) / BN;  // columns behind N: zeros by TMA, not stored
  const int num_tiles = num_m * num_n;
  const int num_kb = (p.K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full_bar[s], 1);  // used in rank 0 only
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 2 * epi_warps<EPI>());
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.a0);
    tma_prefetch_desc(&p.a1);
    tma_prefetch_desc(&p.b0);
    tma_prefetch_desc(&p.b1);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before anything crosses the pair
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if constexpr (dependent<EPI>()) {
    wait_for_prior();
    dependents_may_start();
  }

  auto stage_a = [&](int s) { return smem + s * C::kStageBytes; };
  auto stage_b = [&](int s) { return smem + s * C::kStageBytes + C::kABytes; };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      const uint64_t pol = p.a_keep ? l2_policy_evict_last() : l2_policy_evict_first();
      const uint64_t pol_b = p.b_keep ? l2_policy_evict_last() : l2_policy_evict_first();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_parity = 0;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && unit_at(p, num_tiles, num_kb, i, u, pair, npairs); ++i) {
        int m0, n0;
        tile_origin(p, u.tile, num_m, num_n, 2 * BM, BN, m0, n0);
        const bool nlo = n0 < p.n_split;
        const int by = (nlo ? n0 : n0 - p.n_split) + static_cast<int>(rank) * (BN / 2);
        const int my_m = m0 + static_cast<int>(rank) * BM;
        for (int t = 0; t < u.kb1 - u.kb0; ++t) {
          const int kb = unit_kb(u, i, t);
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const int k = kb * BK;
          const bool klo = k < p.k_split;
          const int kx = klo ? k : k - p.k_split;
          const uint32_t leader_full = cluster_map(&full_bar[stage], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * C::kStageBytes);
          const CUtensorMap* amap = klo ? &p.a0 : &p.a1;
          const CUtensorMap* bmap = (nlo && klo) ? &p.b0 : &p.b1;
          if constexpr (kAmn) {
#pragma unroll
            for (int h = 0; h < BM / 64; ++h)
              tma_load_2d_pair(stage_a(stage) + h * kMnBlock, amap, leader_full, my_m + 64 * h,
                               kx, pol);
          } else {
            tma_load_2d_pair(stage_a(stage), amap, leader_full, kx, my_m, pol);
          }
          if constexpr (kBmn) {
#pragma unroll
            for (int h = 0; h < BN / 128; ++h)
              tma_load_2d_pair(stage_b(stage) + h * kMnBlock, bmap, leader_full, by + 64 * h, kx,
                               pol_b);
          } else if constexpr (EPI == kEpiGated) {
            // Rank 0 brings the gate's rows, rank 1 the same rows of up.
            tma_load_2d_pair(stage_b(stage), rank == 0 ? &p.b0 : &p.b1, leader_full, kx, n0 / 2,
                             pol_b);
          } else {
            tma_load_2d_pair(stage_b(stage), bmap, leader_full, kx, by, pol_b);
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // Unwinding: let every copy this thread issued land before the CTA
        // (and its shared memory) goes away.  Rank 0 waits for its stages;
        // rank 1's completions go to rank 0, so it gives them 100 us.
        volatile int no_abort = 0;
        if (rank == 0) {
          for (int s = 0; s < NS; ++s)
            if (armed & (1u << s))
              mbar_wait(&full_bar[s], (armed_parity >> s) & 1u, &no_abort, p.status);
        } else {
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 100000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ----------------------------------------------------- MMA issuer --
      constexpr uint32_t idesc =
          (FP8 ? umma_idesc_e4m3(2 * BM, BN) : umma_idesc_bf16(2 * BM, BN)) |
          (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
      constexpr uint64_t kStepA = kAmn ? 128 : 2;
      constexpr uint64_t kStepB = kBmn ? 128 : 2;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && unit_at(p, num_tiles, num_kb, i, u, pair, npairs); ++i) {
        const int acc = i & 1;
        const uint32_t acc_phase = (i >> 1) & 1;
        if (!mbar_wait_cluster(&tempty_bar[acc], acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int t = 0; t < u.kb1 - u.kb0; ++t) {
          if (!mbar_wait_cluster(&full_bar[stage], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = kAmn ? sw128_mnmajor_desc(smem_addr(stage_a(stage)), kMnBlock)
                                      : sw128_kmajor_desc(smem_addr(stage_a(stage)));
          const uint64_t bdesc = kBmn ? sw128_mnmajor_desc(smem_addr(stage_b(stage)), kMnBlock)
                                      : sw128_kmajor_desc(smem_addr(stage_b(stage)));
#pragma unroll
          for (int kk = 0; kk < kMmasPerBlock; ++kk) {
            const uint32_t accum = (t != 0 || kk != 0) ? 1u : 0u;
            if constexpr (FP8)
              umma_e4m3_pair(d_tmem, adesc + kStepA * kk, bdesc + kStepB * kk, idesc, accum);
            else
              umma_bf16_pair(d_tmem, adesc + kStepA * kk, bdesc + kStepB * kk, idesc, accum);
          }
          umma_commit_pair(&empty_bar[stage], 0x3);
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit_pair(&tfull_bar[acc], 0x3);
      }
      // Every MMA this thread issued completes before TMEM is released in
      // either CTA.
      umma_commit_pair(done_bar, 0x3);
      volatile int no_abort = 0;
      mbar_wait(done_bar, 0, &no_abort, p.status);
    } else if (lane == 0) {
      // The pair's MMAs read this CTA's shared memory and write its TMEM:
      // wait for the last of them (rank 0 always commits this barrier).
      volatile int no_abort = 0;
      mbar_wait(done_bar, 0, &no_abort, p.status);
    }
  } else {
    // --------------------------------------------------------- epilogue --
    const int quarter = warp & 3;
    const int row_local = quarter * 32 + lane;
    float* f32_stage = reinterpret_cast<float*>(smem + NS * C::kStageBytes + C::kBarBytes) +
                       quarter * 32 * kF32Pad;
    Unit u;
    for (int i = 0; unit_at(p, num_tiles, num_kb, i, u, pair, npairs); ++i) {
      const int acc_buf = i & 1;
      const uint32_t acc_phase = (i >> 1) & 1;
      if (!mbar_wait_cluster_warp(&tfull_bar[acc_buf], acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      int m0, n0;
      tile_origin(p, u.tile, num_m, num_n, 2 * BM, BN, m0, n0);
      const int prow = static_cast<int>(rank) * BM + row_local;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc_buf * BN);
      epilogue_unit<BN, EPI, FP8, 2 * BM, kStage>(
          p, u, m0 + prow, prow,
          ((u.slot / p.split_s) * 2 + static_cast<int>(rank)) * epi_warps<EPI>() + warp - 2, t_row, n0,
          lane, f32_stage, (warp - 2) >> 2, smem);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map(&tempty_bar[acc_buf], 0));
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of either CTA still signals the other
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::kTmemCols);
  }
}

template <int EPI, int LAYOUT, bool FP8 = false>
cudaError_t launch_pair(const GemmArgs& a, cudaStream_t stream) {
  using C = PairCfg<staged_f32<EPI, LAYOUT>(), pair_stages<EPI>()>;
  auto kern = gemm_pair_kernel<EPI, LAYOUT, FP8>;
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  if (a.grid % 2) return cudaErrorInvalidValue;
  if constexpr (dependent<EPI>())
    return launch_dependent(kern, dim3(a.grid), dim3(gemm_threads<EPI>()), C::kSmemBytes, stream, a);
  kern<<<a.grid, gemm_threads<EPI>(), C::kSmemBytes, stream>>>(a);
  return cudaGetLastError();
}

template <int BN, int EPI, bool FP8, int LAYOUT>
cudaError_t launch_typed(const GemmArgs& a, cudaStream_t stream) {
  using C = Cfg<BN, staged_f32<EPI, LAYOUT>()>;
  auto kern = gemm_kernel<BN, EPI, FP8, LAYOUT>;
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  if constexpr (dependent<EPI>())
    return launch_dependent(kern, dim3(a.grid), dim3(gemm_threads<EPI>()), C::kSmemBytes, stream, a);
  kern<<<a.grid, gemm_threads<EPI>(), C::kSmemBytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Arrival counters for 32 rows of a split tile.
int gemm_counters(int epilogue) {
  return (epilogue == kEpiGated    ? epi_warps<kEpiGated>()
          : epilogue == kEpiDgated ? epi_warps<kEpiDgated>()
          : epilogue == kEpiBf16   ? epi_warps<kEpiBf16>()
                                   : 4) / 4;
}

GemmPlan plan_gemm(int64_t tiles, int64_t num_kb, int sms, int block_n, int rows, int counters,
                   int most_s) {
  GemmPlan g;
  g.grid = static_cast<int>(tiles < sms ? tiles : sms);
  g.split_r = 0;
  g.split_s = 1;
  // Remainder tiles of the last, partial wave (all tiles if fewer than SMs).
  const int64_t r = tiles - (tiles / sms) * sms;
  if (r > 0) {
    int64_t s = sms / r;
    const int64_t s_k = num_kb / kMinSplitKBlocks;  // each piece keeps >= kMinSplitKBlocks
    if (s_k < s) s = s_k;
    if (most_s < s) s = most_s;
    if (s >= 2) {
      g.split_r = static_cast<int>(r);
      g.split_s = static_cast<int>(s);
      if (tiles < sms) g.grid = static_cast<int>(r * s);
    }
  }
  g.partial_bytes = static_cast<size_t>(g.split_r) * g.split_s * rows * block_n * sizeof(float);
  g.counter_bytes = static_cast<size_t>(g.split_r) * (rows / 32) * counters * sizeof(unsigned);
  return g;
}

namespace {

template <int EPI, bool FP8, int LAYOUT>
cudaError_t launch_bn(const GemmArgs& a, cudaStream_t stream) {
  switch (a.block_n) {
    case 256: return launch_typed<256, EPI, FP8, LAYOUT>(a, stream);
    case 128: return launch_typed<128, EPI, FP8, LAYOUT>(a, stream);
    case 64: return launch_typed<64, EPI, FP8, LAYOUT>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gemm(const GemmArgs& a, cudaStream_t stream) {
  if (a.split_s >= 2 && a.split_r > 0 && !a.counters_zero) {
    cudaError_t e =
        cudaMemsetAsync(a.counters, 0, a.split_r * (a.pair ? 8 : 4) * gemm_counters(a.epilogue) *
                                           sizeof(unsigned), stream);
    if (e != cudaSuccess) return e;
  }
  if (a.pair) {  // 256-wide N tiles on CTA pairs
    if (a.block_n != kPairBN) return cudaErrorInvalidValue;
    if (a.fp8) {
      if (a.layout != kLayoutKK) return cudaErrorInvalidValue;
      if (a.epilogue == kEpiQkvGelu) return launch_pair<kEpiQkvGelu, kLayoutKK, true>(a, stream);
      if (a.epilogue == kEpiResidual) return launch_pair<kEpiResidual, kLayoutKK, true>(a, stream);
      return cudaErrorInvalidValue;
    }
    if (a.layout == kLayoutKK && a.epilogue == kEpiQkvGelu)
      return launch_pair<kEpiQkvGelu, kLayoutKK>(a, stream);
    if (a.layout == kLayoutKK && a.epilogue == kEpiResidual)
      return launch_pair<kEpiResidual, kLayoutKK>(a, stream);
    if (a.layout == kLayoutKK && a.epilogue == kEpiBf16)
      return launch_pair<kEpiBf16, kLayoutKK>(a, stream);
    if (a.layout == kLayoutKK && a.epilogue == kEpiGated)
      return launch_pair<kEpiGated, kLayoutKK>(a, stream);
    if (a.layout == kLayoutKN && a.epilogue == kEpiDgelu)
      return launch_pair<kEpiDgelu, kLayoutKN>(a, stream);
    if (a.layout == kLayoutKN && a.epilogue == kEpiDgated)
      return launch_pair<kEpiDgated, kLayoutKN>(a, stream);
    if (a.layout == kLayoutKN && a.epilogue == kEpiBf16)
      return launch_pair<kEpiBf16, kLayoutKN>(a, stream);
    if (a.layout == kLayoutNN && a.epilogue == kEpiBf16)
      return launch_pair<kEpiBf16, kLayoutNN>(a, stream);
    if (a.layout == kLayoutKN && a.epilogue == kEpiF32)
      return launch_pair<kEpiF32, kLayoutKN>(a, stream);
    if (a.layout == kLayoutNN && a.epilogue == kEpiF32)
      return launch_pair<kEpiF32, kLayoutNN>(a, stream);
    return cudaErrorInvalidValue;
  }
  // The instantiated (epilogue, operand type, layout) combinations: the
  // forward GEMMs (bf16 and e4m3, K-major) and the backward GEMMs (bf16).
  if (a.layout == kLayoutKK) {
    if (a.epilogue == kEpiQkvGelu)
      return a.fp8 ? launch_bn<kEpiQkvGelu, true, kLayoutKK>(a, stream)
                   : launch_bn<kEpiQkvGelu, false, kLayoutKK>(a, stream);
    if (a.epilogue == kEpiResidual)
      return a.fp8 ? launch_bn<kEpiResidual, true, kLayoutKK>(a, stream)
                   : launch_bn<kEpiResidual, false, kLayoutKK>(a, stream);
    if (a.epilogue == kEpiBf16 && !a.fp8) return launch_bn<kEpiBf16, false, kLayoutKK>(a, stream);
    if (a.epilogue == kEpiGated && !a.fp8) {
      // Half of a tile's columns are the gate's: tiles of 64 would leave 32 rows of weights a box.
      if (a.block_n == 256) return launch_typed<256, kEpiGated, false, kLayoutKK>(a, stream);
      if (a.block_n == 128) return launch_typed<128, kEpiGated, false, kLayoutKK>(a, stream);
    }
    return cudaErrorInvalidValue;
  }
  if (a.fp8) return cudaErrorInvalidValue;
  if (a.layout == kLayoutKN) {
    if (a.epilogue == kEpiDgelu) return launch_bn<kEpiDgelu, false, kLayoutKN>(a, stream);
    if (a.epilogue == kEpiDgated) return launch_bn<kEpiDgated, false, kLayoutKN>(a, stream);
    if (a.epilogue == kEpiBf16) return launch_bn<kEpiBf16, false, kLayoutKN>(a, stream);
    if (a.epilogue == kEpiF32) return launch_bn<kEpiF32, false, kLayoutKN>(a, stream);
    return cudaErrorInvalidValue;
  }
  if (a.layout == kLayoutNN && a.epilogue == kEpiF32)
    return launch_bn<kEpiF32, false, kLayoutNN>(a, stream);
  if (a.layout == kLayoutNN && a.epilogue == kEpiBf16)
    return launch_bn<kEpiBf16, false, kLayoutNN>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ptb
