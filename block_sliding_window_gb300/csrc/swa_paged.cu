// Sliding-window attention of one new token per sequence over the paged
// cache (definition and cache layout: ptb.h).
//
// The cache is read once and bounds the kernel: 2 d bytes per key and value
// row in bf16, d / 2 + d / 8 in 4 bits, against 4 d operations per query head.
// The G query heads of a kv head share its rows, so the products run on the
// tensor cores (mma.sync m16n8k16; a step has far too few rows for tcgen05's
// 128), transposed to fill them: S^T = K Q^T with 16 keys as rows and 8 heads
// as columns, O^T += V^T P^T with 16 channels as rows.
//
// Work split.  The unit is a block of 32 keys of one (sequence, kv head, up to
// 16 query heads).  All units of the call, in order, are dealt to the blocks,
// one per SM, and a block's to its warps, in equal contiguous shares, whatever
// the sequences' lengths: one long sequence spreads over the whole GPU and a
// ragged batch stays even.  A warp works alone: it streams its units through
// its own ring in shared memory, keeps maximum, sum and output of the current
// segment in registers, and writes the output itself where it holds all of a
// segment.  Partial results of cut segments are joined in shared memory at
// the block's end, and those cut between blocks by a second kernel, launched
// to overlap this one's end.  The order is fixed: the same bits every time.
// (Joining all warps' parts in the second kernel cost 10 us on one long
// sequence, of 22.)
//
// 4-bit rows:
//   q.k = sum_w scale_w (q.u)_w + (centre_w - 8 scale_w) Q_w,  Q_w = sum of q over group w,
//   sum_j p_j v_j = sum_j (p_j scale_jw)(u_j - 8) + sum_j p_j centre_jw.
// Nibbles become numbers by a mask alone, as subnormals: a shift serves four.
// Keys: fp16 u 2^-24 and u 2^-20 are operands as they are; q enters as fp16,
// scaled by a power of two (exact down to 2^-28 of the row's largest), the
// channels of the second kind by 2^-4 of it.  The scale is applied to each
// group's product, and the rest is one more product with the pairs as they lie
// (Q_w in two bf16 terms).
// Values: bf16 u 2^-133 and u 2^-129 become multiples of u - 8 by an FMA; the
// scale goes into P, and the centres are one more product.  p and p * scale are
// rounded to bf16 once, as P is in the other attention kernels.
// The integer pipe (0.5 instructions a clock and SM quarter, measured) bounds
// the 4-bit kernel: with nibbles in the mantissas of 64 and 128, two shifts more
// for four and an addition, 64 long sequences took 200 us, now 159.  (e4m3
// products, for which a masked word is an operand as it lies, were slower: the
// compiler builds them from fp16 ones.)
// Measured on 64 sequences, 64 heads of 128 over 8: bf16 6.0 TB/s (140 us; the
// cache alone at the rate of a copy 124); 4 bits 5.4 TB/s (159 us; 127; the
// copies alone take 130).  One sequence of 16000 keys: 12 us, half of it the two
// launches' ends.
// Rows that the mask leaves out (before the window, past the length, pages out
// of range) may hold anything: their scores are replaced and their values or
// pairs zeroed before use.
#include <cuda_fp16.h>

#include <type_traits>

#include "kv_device.cuh"

namespace ptb {
namespace {

constexpr int kBlockKeys = 32;   // keys of a unit
constexpr int kMinUnits = 4;     // a block's share is at least this many units
constexpr int kJoinThreads = 256;

template <int D, int BITS, int NT>
struct Cfg {
  static constexpr int kAtoms = (D + 63) / 64;
  static constexpr int NG = D / kKvGroup;
  // Keys or values of a unit in shared memory.  Bits 16: 64-channel column
  // blocks of 32 rows of 128 swizzled bytes.  Bits 4: 32 rows of codes, then
  // their pairs.
  static constexpr int kSideBytes =
      BITS == 16 ? kAtoms * kBlockKeys * 128 : kBlockKeys * (D / 2 + D / 8);
  static constexpr int kStageBytes = 2 * kSideBytes;
  // Bits 4: two stages a warp do as well as three and leave room for the
  // partial result.
  static constexpr int kStages = BITS == 4 ? 2 : 3;
  // Warps of a block, one block per SM: as many as registers (4 bits: 168 or
  // 255 a thread) or shared memory (16 bits) allow.  4 bits, 64 sequences:
  // 14 warps of 128 registers take 174 us, 12 of 164 159.
  static constexpr int kWarps =
      BITS == 4 ? (NT == 1 ? 12 : 8) : (D > 64 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 8 : 7));
  // A partial result: maxima and sums of 8 NT heads, then their outputs.
  static constexpr int kSlotBytes = 8 * NT * (2 + D) * 4;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static_assert(kRingBytes >= kSlotBytes, "a warp's last partial result lies over its ring");
  static constexpr int kWarpBytes = (kRingBytes + kSlotBytes + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = 1024 + kWarps * (kWarpBytes + 128);
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct PagedParams {
  CUtensorMap map;  // bits 16: {d, rows of a page, pages}
  SwaPagedArgs a;
  int group, head_blocks;  // G; blocks of 8 NT query heads of a kv head
  float* parts;            // [2 x blocks]: partial results as in shared memory
  int4* cuts;              // [blocks]: the segment that goes on into the block
};

// The keys that sequence b's query attends to, in units.
struct Span {
  int n, lo;       // positions lo .. n - 1
  int unit0, units;
};

__device__ __forceinline__ Span span_of(const SwaPagedArgs& a, int b) {
  Span s;
  const int64_t cap = a.c.table_pages << a.c.page_shift;
  int n = a.lens[b];
  if (n < 0 || n > cap) n = 0;
  s.n = n;
  s.lo = n > a.window ? n - a.window : 0;
  s.unit0 = s.lo / kBlockKeys;
  s.units = n > 0 ? (n - 1) / kBlockKeys - s.unit0 + 1 : 0;
  return s;
}

// Units of all sequences together, per head block (one warp).
__device__ __forceinline__ int64_t total_units(const SwaPagedArgs& a, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < a.batch; b += 32) sum += span_of(a, b).units;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Units of a block's share.
__device__ __forceinline__ int64_t share_of(int64_t units, int blocks) {
  const int64_t s = (units + blocks - 1) / blocks;
  return s > kMinUnits ? s : kMinUnits;
}

// A place among the units: unit i of head block hh (0 .. kv_heads *
// head_blocks - 1) of sequence b.
struct Place {
  int b, hh, i;
  Span s;
};

// The place of unit u < total (one warp).
__device__ __forceinline__ Place place_of(const SwaPagedArgs& a, int heads, int64_t u, int lane) {
  Place p;
  int64_t before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    const int64_t mine = b < a.batch ? static_cast<int64_t>(span_of(a, b).units) * heads : 0;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned vote = __ballot_sync(0xffffffffu, u < before + sum);
    if (vote || b0 + 32 >= a.batch) {
      const int f = vote ? __ffs(vote) - 1 : 31;
      p.b = min(b0 + f, a.batch - 1);
      u -= before + __shfl_sync(0xffffffffu, sum - mine, f);
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  p.s = span_of(a, p.b);
  const int units = p.s.units > 0 ? p.s.units : 1;
  p.hh = static_cast<int>(u / units);
  p.i = static_cast<int>(u % units);
  return p;
}

// The next unit after p; false behind the last.
__device__ __forceinline__ void next_place(const SwaPagedArgs& a, int heads, Place& p) {
  if (++p.i < p.s.units) return;
  p.i = 0;
  if (++p.hh < heads) return;
  p.hh = 0;
  do {
    if (++p.b >= a.batch) return;
    p.s = span_of(a, p.b);
  } while (p.s.units == 0);
}

// ------------------------------------------------------------- primitives --

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from a zero accumulator.
__device__ __forceinline__ void mma_bf16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The same with fp16 operands.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit values held by a warp (lane 4 r + c:
// row r, columns 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes global -> shared, past L1; completion by groups.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                         int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Nibbles 0 .. 3 of both 16-bit halves of w as fp16 numbers: in mantissa bits
// 0 .. 3 of a subnormal, u is u 2^-24, in bits 4 .. 7 u 2^-20.  One shift for four.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t r = w >> 8;
  v[0] = w & 0x000f000fu;
  v[1] = w & 0x00f000f0u;
  v[2] = r & 0x000f000fu;
  v[3] = r & 0x00f000f0u;
}
// The same as bf16 numbers around zero: in the lowest bits of a bf16 a nibble is
// u 2^-133, four bits up u 2^-129 (subnormals and the first binade are evenly
// spaced), and an FMA makes them (u - 8) 2^-6 and (u - 8) 2^-2, both exact.
constexpr float kLowNibble = 64.f, kHighNibble = 4.f;  // what undoes the factors
__device__ __forceinline__ void codes_bf16_scaled(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t r = w >> 8;
  const uint32_t x[4] = {w & 0x000f000fu, w & 0x00f000f0u, r & 0x000f000fu, r & 0x00f000f0u};
  const __nv_bfloat162 up = __floats2bfloat162_rn(0x1p127f, 0x1p127f);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float c = -8.f / (k & 1 ? kHighNibble : kLowNibble);
    __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[k]), up,
                               __floats2bfloat162_rn(c, c));
    v[k] = *reinterpret_cast<uint32_t*>(&y);
  }
}
// N consecutive words (N 1 .. 4) at 4 N-byte alignment (4-byte for N = 3).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&r)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x, r[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}
__device__ __forceinline__ uint32_t lds16(const uint8_t* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}

// Row `r` (0 .. 15) of a 16-key tile of 4-bit rows stands for this key: the
// order in which a lane's four value rows fall into different banks.
__device__ __forceinline__ int key_of_row(int r) {
  return ((r & 7) >> 1) + 4 * (r & 1) + (r & 8);
}

// What a warp leaves of segments that it holds in part.
struct WarpParts {
  int has0, end0, b0, hh0;  // a segment that began earlier; end0: it ends here
  int has1, b1, hh1, pad;   // a segment that goes on in the next warp
};
static_assert(128 % sizeof(WarpParts) == 0, "stepped through in 128-byte blocks");

// ------------------------------------------------------------------ kernel --

template <int D, int BITS, int NT>
__global__ void __launch_bounds__(Cfg<D, BITS, NT>::kWarps * 32, 1)
    swa_paged_kernel(const __grid_constant__ PagedParams P) {
  using C = Cfg<D, BITS, NT>;
  constexpr int NG = C::NG;
  constexpr int MS = D / 16;  // 16-channel steps
  constexpr int kWarps = C::kWarps;
  const SwaPagedArgs& a = P.a;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = base + warp * C::kWarpBytes;
  const uint8_t* ring_rows = smem_raw + (ring - smem_addr(smem_raw));
  uint8_t* tail = smem_raw + (base - smem_addr(smem_raw)) + kWarps * C::kWarpBytes + warp * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);                     // [kStages]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + C::kStages);
  volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);  // [kStages]

  WarpParts* parts = reinterpret_cast<WarpParts*>(tail + 64);
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&full[s], 1);
    *abort_flag = 0;
    parts->has0 = parts->end0 = parts->has1 = 0;
    mbar_fence_init();
  }
  __syncwarp();

  const int heads = a.c.kv_heads * P.head_blocks;
  // Sequences without keys: zeros; lengths out of range: recorded as well.
  for (int b = blockIdx.x * kWarps + warp; b < a.batch; b += gridDim.x * kWarps) {
    const int n = a.lens[b];
    if (n < 0 || n > (a.c.table_pages << a.c.page_shift))
      if (lane == 0) record_error(a.status, PTB_ERR_ARG);
    if (span_of(a, b).units == 0)
      for (int x = lane; x < a.heads * (D / 8); x += 32)
        *reinterpret_cast<uint4*>(a.o + b * a.o_sb + (x / (D / 8)) * a.o_sh + x % (D / 8) * 8) =
            make_uint4(0, 0, 0, 0);
  }
  // This block's share, and this warp's part of it.
  const int64_t total = total_units(a, lane) * heads;
  const int64_t share = share_of(total, gridDim.x);
  const int64_t c0 = blockIdx.x * share, c1 = c0 + share < total ? c0 + share : total;
  if (c0 >= c1) {  // the whole block
    if (threadIdx.x == 0) P.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  const int64_t part = (c1 - c0 + kWarps - 1) / kWarps;
  const int64_t u0 = c0 + warp * part < c1 ? c0 + warp * part : c1;
  const int64_t u1 = u0 + part < c1 ? u0 + part : c1;

  const int page = a.c.page_size;
  const int sub_shift = page < kBlockKeys ? a.c.page_shift : 5;
  const int sub_keys = 1 << sub_shift;          // keys of a unit that lie in one page
  const int subs = kBlockKeys >> sub_shift;     // 1 or 2
  const uint32_t page_bytes = static_cast<uint32_t>(a.c.page_bytes);  // < 2^31

  // ------------------------------------------------------------ producer --
  // Bits 16: tensor-map copies, issued by one lane each (sub-block `lane /
  // copies`; the 64-channel column blocks of keys, then of values), counted
  // on the stage's mbarrier.  Bits 4: 16-byte copies by all lanes, one commit
  // group a unit.  (Bulk copies of 2 KB and 0.5 KB cost 60 more instructions
  // a unit: each is issued by a loop over the lanes that carry one.)
  constexpr int kCopies = 2 * C::kAtoms;
  const int copy_sub = lane / kCopies, copy_part = lane % kCopies;
  const int copy_side = copy_part / C::kAtoms, copy_atom = copy_part % C::kAtoms;
  const uint32_t value_side = static_cast<uint32_t>(a.c.kv_heads * a.c.block_bytes);
  const uint8_t* lane_base = a.c.base + lane * 16;

  Place ld = place_of(a, heads, u0 < u1 ? u0 : c0, lane);
  Place at = ld;
  volatile int* begin = reinterpret_cast<volatile int*>(tail + 96);  // the share's first place
  if (threadIdx.x == 0) {
    begin[0] = ld.b;
    begin[1] = ld.hh;
    begin[2] = ld.i;
    begin[3] = ld.s.units;
  }
  int64_t to_load = u1 - u0;  // units whose copies are still to be issued
  // Pages of the coming sub-blocks, one a lane; -1: not needed, or out of range.
  int page_reg = -1, page_next = 32;
  int64_t head_src = 0;  // this kv head's keys in a page: bytes (bits 4) or row (bits 16)
  auto issue = [&](int stage) {
    const int key0 = (ld.s.unit0 + ld.i) * kBlockKeys;
    if (page_next >= 32) {
      const int64_t pos = static_cast<int64_t>(key0) + (lane << sub_shift);
      page_reg = -1;
      if (pos < ld.s.n && pos + sub_keys > ld.s.lo) {
        page_reg = a.c.table[ld.b * a.c.table_stride + (pos >> a.c.page_shift)];
        if (page_reg < 0 || page_reg >= a.c.pages) {
          page_reg = -1;
          record_error(a.status, PTB_ERR_ARG);
        }
      }
      page_next = 0;
      head_src = (ld.hh / P.head_blocks) * (BITS == 16 ? page : a.c.block_bytes);
    }
    const int pg0 = __shfl_sync(0xffffffffu, page_reg, page_next);
    const int pg1 = subs == 1 ? pg0 : __shfl_sync(0xffffffffu, page_reg, page_next + 1);
    page_next += subs;
    uint32_t mask = 0xffffffffu;
    if (key0 < ld.s.lo || key0 + kBlockKeys > ld.s.n || (pg0 | pg1) < 0) {
      const int from = max(ld.s.lo - key0, 0), to = min(ld.s.n - key0, kBlockKeys);
      mask = (to == 32 ? 0xffffffffu : (1u << to) - 1u) & ~((1u << from) - 1u);
      if (pg0 < 0) mask &= subs == 1 ? 0u : 0xffff0000u;
      if (pg1 < 0) mask &= subs == 1 ? 0u : 0xffffu;
    }
    if constexpr (BITS == 16) {
      const int n = pg0 < 0 ? 0 : 1, valid = n + (subs == 1 || pg1 < 0 ? 0 : 1);
      if (lane == 0) {
        masks[stage] = mask;
        if (valid)
          mbar_arrive_expect_tx(&full[stage], valid * (C::kStageBytes >> (subs - 1)));
        else
          mbar_arrive(&full[stage]);
      }
      __syncwarp();  // armed, and the stage has been read by every lane
      const int pg = copy_sub == 0 ? pg0 : pg1;
      if (copy_sub < subs && pg >= 0) {
        const int off = (key0 + (copy_sub << sub_shift)) & (page - 1);
        tma_rows(ring + stage * C::kStageBytes + copy_side * C::kSideBytes +
                     copy_atom * kBlockKeys * 128 + copy_sub * sub_keys * 128,
                 &P.map, &full[stage], copy_atom * 64,
                 static_cast<int>(head_src) + copy_side * a.c.kv_heads * page + off, pg);
      }
    } else {
      if (lane == 0) masks[stage] = mask;
      __syncwarp();  // the stage has been read by every lane
      constexpr int kCodes = kBlockKeys * (D / 2) / 16, kPairs = kBlockKeys * (D / 8) / 16;
      const uint32_t dst = ring + stage * C::kStageBytes + lane * 16;
      const uint32_t head_at = static_cast<uint32_t>(head_src);
      if (subs == 1) {
        // All rows in one page: every address is a lane's base plus constants.
        if (pg0 >= 0) {
          const uint8_t* block = lane_base + static_cast<uint64_t>(static_cast<uint32_t>(pg0)) * page_bytes;
          const int off = key0 & (page - 1);
          const uint8_t* k_codes = block + (head_at + off * (D / 2));
          const uint8_t* k_pairs = block + (head_at + page * (D / 2) + off * (D / 8));
          const uint8_t *v_codes = k_codes + value_side, *v_pairs = k_pairs + value_side;
#pragma unroll
          for (int i = 0; i < (kCodes + 31) / 32; ++i)
            if (kCodes >= i * 32 + 32 || i * 32 + lane < kCodes) {
              copy16(dst + i * 512, k_codes + i * 512);
              copy16(dst + i * 512 + C::kSideBytes, v_codes + i * 512);
            }
          if (kPairs >= 32 || lane < kPairs) {
            copy16(dst + kBlockKeys * (D / 2), k_pairs);
            copy16(dst + kBlockKeys * (D / 2) + C::kSideBytes, v_pairs);
          }
        }
      } else {
        // Pages of 16 rows: the unit is two whole blocks.
        const uint8_t* block0 = lane_base + static_cast<uint64_t>(static_cast<uint32_t>(pg0)) * page_bytes + head_at;
        const uint8_t* block1 = lane_base + static_cast<uint64_t>(static_cast<uint32_t>(pg1)) * page_bytes + head_at;
        auto rows = [&](auto n, uint32_t from, uint32_t to) {
          constexpr int chunks = decltype(n)::value, half = chunks / 2;
#pragma unroll
          for (int i = 0; i < (chunks + 31) / 32; ++i) {
            const bool second = i * 32 + lane >= half;
            if (i * 32 + lane < chunks && (second ? pg1 : pg0) >= 0) {
              const uint8_t* p = (second ? block1 - half * 16 : block0) + (from + i * 512);
              copy16(to + i * 512, p);
              copy16(to + i * 512 + C::kSideBytes, p + value_side);
            }
          }
        };
        rows(std::integral_constant<int, kCodes>(), 0, dst);
        rows(std::integral_constant<int, kPairs>(), 16 * (D / 2), dst + kBlockKeys * (D / 2));
      }
    }
    --to_load;
    if (++ld.i >= ld.s.units) {
      --ld.i;
      next_place(a, heads, ld);
      page_next = 32;
    }
  };

#pragma unroll
  for (int s = 0; s < C::kStages; ++s) {
    if (to_load > 0) issue(s);
    if constexpr (BITS == 4) copy_commit();  // a group a stage, empty behind the last unit
  }

  // ------------------------------------------------------------ consumer --
  int64_t u = u0;
  int stage = 0;
  uint32_t parity = 0;
  bool ok = true;
  while (u < u1 && ok) {
    // ---- one segment: units at.i .. of (sequence, kv head, head block)
    const int first = at.i;
    const int kvh = at.hh / P.head_blocks;
    const int head0 = kvh * P.group + (at.hh % P.head_blocks) * 8 * NT;  // first query head
    const int nheads = min(8 * NT, (kvh + 1) * P.group - head0);
    const int64_t left = u1 - u;
    const int count = static_cast<int>(left < at.s.units - first ? left : at.s.units - first);

    // Queries as B fragments (column = head g): for 16 bits channels 16 s + 2 t,
    // + 1 and + 8, + 9; for 4 bits in the order of the codes, scaled by a
    // power of two into fp16.
    uint32_t qf[NT][MS][2];
    uint32_t qs[NT][2];  // Q_t: (-8 Q, Q) 2^-24 in two bf16 terms
    float to_log2[NT][2];  // scores of heads 2 t, 2 t + 1 to the log2 domain, now
    [[maybe_unused]] float own_log2[NT][2];  // and as their queries have it (4 bits)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool live = nt * 8 + g < nheads;
      const __nv_bfloat16* q = a.q + at.b * a.q_sb + (head0 + (live ? nt * 8 + g : 0)) * a.q_sh;
      to_log2[nt][0] = to_log2[nt][1] = a.scale_log2;
      if constexpr (BITS == 16) {
#pragma unroll
        for (int s = 0; s < MS; ++s) {
          qf[nt][s][0] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t) : 0u;
          qf[nt][s][1] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 + 2 * t) : 0u;
        }
      } else {
        uint4 v[NG];
        uint32_t mx = 0;  // largest |q|, as bits: NaN above infinity above all numbers
#pragma unroll
        for (int wq = 0; wq < NG; ++wq) {
          v[wq] = make_uint4(0, 0, 0, 0);
          if (live) v[wq] = *reinterpret_cast<const uint4*>(q + 32 * wq + 8 * t);
          const uint32_t x[4] = {v[wq].x, v[wq].y, v[wq].z, v[wq].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, max((x[e] << 16) & 0x7fffffffu, x[e] & 0x7fff0000u));
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // The power of two that brings the largest |q| into [2^14, 2^15), the
        // scores' unit being 2^-24 of it; a query that is not finite, or of
        // 2^119 or more (no such power is left), gives NaN.
        const int expo = static_cast<int>(mx >> 23);
        const int shift = max(min(127 + 14 - expo, 127), 24 - 127);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
        const float down =
            __uint_as_float(expo >= 127 + 119 ? 0x7fffffffu
                                              : static_cast<uint32_t>(127 + 24 - shift) << 23);
        qs[nt][0] = qs[nt][1] = 0;
#pragma unroll
        for (int wq = 0; wq < NG; ++wq) {
          const uint32_t x[4] = {v[wq].x, v[wq].y, v[wq].z, v[wq].w};
          float y[8], sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] = bf16_lo(x[e]) * up;
            y[2 * e + 1] = bf16_hi(x[e]) * up;
            sum += y[2 * e] + y[2 * e + 1];
          }
          qf[nt][2 * wq][0] = pack_f16x2(y[0], y[4]);
          qf[nt][2 * wq][1] = pack_f16x2(y[1] * 0.0625f, y[5] * 0.0625f);
          qf[nt][2 * wq + 1][0] = pack_f16x2(y[2], y[6]);
          qf[nt][2 * wq + 1][1] = pack_f16x2(y[3] * 0.0625f, y[7] * 0.0625f);
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          sum *= 0x1p-24f;
          const uint32_t top = pack_bf16x2(-8.f * sum, sum);
          if (t == wq) {
            qs[nt][0] = top;
            qs[nt][1] = pack_bf16x2(-8.f * sum - bf16_lo(top), sum - bf16_hi(top));
          }
        }
        // Never 0 or infinite: a masked score times 0 would not stay minus infinity, and
        // times infinity a finite score below zero would become a masked one.  Beyond
        // the last power of two the row is NaN (scale |q| of 2^116.4 and more).
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          to_log2[nt][e] *= __shfl_sync(0xffffffffu, down, 8 * t + 4 * e);
          if (to_log2[nt][e] == 0.f) to_log2[nt][e] = 0x1p-126f;
          if (to_log2[nt][e] > 0x1p127f) to_log2[nt][e] = __uint_as_float(0x7fffffffu);
          own_log2[nt][e] = to_log2[nt][e];
        }
      }
    }

    float o[NT][MS][4];
    float oc[NT][4];  // sum_j p_j centre_j of group g (4 bits)
    float m_ref[NT][2], l[NT][2];
    bool large = false;  // some score was large (kLargeScore); the same in all lanes
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int s = 0; s < MS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) oc[nt][e] = 0.f;
      m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    for (int blk = 0; blk < count; ++blk) {
      if constexpr (BITS == 16) {
        if (!mbar_wait_warp(&full[stage], parity, abort_flag, a.status)) {
          ok = false;
          break;
        }
      } else {
        copy_wait<C::kStages - 1>();
        __syncwarp();
      }
      const uint32_t keys = ring + stage * C::kStageBytes;
      const uint32_t vals = keys + C::kSideBytes;
      const uint8_t* key_rows = ring_rows + stage * C::kStageBytes;
      const uint8_t* val_rows = key_rows + C::kSideBytes;
      // 4 bits: codes and pairs of the two 16-key tiles within a side.
      constexpr uint32_t code1 = 16 * (D / 2), pair0 = kBlockKeys * (D / 2);
      constexpr uint32_t pair1 = pair0 + 16 * (D / 8);
      const uint32_t mask = masks[stage];

      // ---- scores of the unit's two 16-key tiles: s[tile][nt]: keys g (0, 1)
      // and g + 8 (2, 3), heads 2 t (0, 2) and 2 t + 1 (1, 3)
      float s[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (BITS == 16) {
          const int row = 16 * h + (lane & 15);
#pragma unroll
          for (int m = 0; m < MS; ++m) {
            const int chunk = (m % 4) * 2 + (lane >> 4);
            uint32_t f[4];
            ldmatrix4(f, keys + (m / 4) * kBlockKeys * 128 + row * 128 + ((chunk ^ (row & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (m == 0)
                mma_bf16_zero(s[h][nt], f[0], f[1], f[2], f[3], qf[nt][m][0], qf[nt][m][1]);
              else
                mma_bf16(s[h][nt], f[0], f[1], f[2], f[3], qf[nt][m][0], qf[nt][m][1]);
            }
          }
        } else {
          const int ka = key_of_row(g), kb = ka + 8;
          const uint8_t* codes = key_rows + (h ? code1 : 0);
          const uint8_t* pairs = key_rows + (h ? pair1 : pair0);
          uint32_t ca[NG], cb[NG], pa[NG], pb[NG];
          lds_words<NG>(ca, codes + ka * (D / 2) + t * 4 * NG);
          lds_words<NG>(cb, codes + kb * (D / 2) + t * 4 * NG);
          lds_words<NG>(pa, pairs + ka * (D / 8));
          lds_words<NG>(pb, pairs + kb * (D / 8));
          // All lanes load (beyond the last group: group 0), so that none is away
          // when the products begin; the queries' terms of such lanes are zero.
          const int group = t < NG ? t : 0;
          uint32_t wa = lds32(pairs + ka * (D / 8) + 4 * group);
          uint32_t wb = lds32(pairs + kb * (D / 8) + 4 * group);
          if constexpr (NG < 4) {
            wa = t < NG ? wa : 0u;
            wb = t < NG ? wb : 0u;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16_zero(s[h][nt], wa, wb, wa, wb, qs[nt][0], qs[nt][1]);
#pragma unroll
          for (int wq = 0; wq < NG; ++wq) {
            const float sa = bf16_lo(pa[wq]), sb = bf16_lo(pb[wq]);
            uint32_t na[4], nb[4];
            codes_f16(ca[wq], na);
            codes_f16(cb[wq], nb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float acc[4];
              mma_f16_zero(acc, na[0], nb[0], na[1], nb[1], qf[nt][2 * wq][0], qf[nt][2 * wq][1]);
              mma_f16(acc, na[2], nb[2], na[3], nb[3], qf[nt][2 * wq + 1][0], qf[nt][2 * wq + 1][1]);
              s[h][nt][0] = fmaf(sa, acc[0], s[h][nt][0]);
              s[h][nt][1] = fmaf(sa, acc[1], s[h][nt][1]);
              s[h][nt][2] = fmaf(sb, acc[2], s[h][nt][2]);
              s[h][nt][3] = fmaf(sb, acc[3], s[h][nt][3]);
            }
          }
        }
      }
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ra = BITS == 16 ? g : key_of_row(g);
          const bool va = (mask >> (16 * h + ra)) & 1u, vb = (mask >> (16 * h + ra + 8)) & 1u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s[h][nt][0] = va ? s[h][nt][0] : -INFINITY;
            s[h][nt][1] = va ? s[h][nt][1] : -INFINITY;
            s[h][nt][2] = vb ? s[h][nt][2] : -INFINITY;
            s[h][nt][3] = vb ? s[h][nt][3] : -INFINITY;
          }
        }
      }

      // ---- weights.  The reference max of a head is the same in all lanes and
      // is the largest score so far, so that the weight of a key that dominates
      // its row is 1, and 1 and its value's scale survive the rounding to bf16.
      // (Raised only past 2^8, rows of a heavy key were off by that rounding: 14
      // sequences of two heads by 1.3 and up to 1.9 times the output's own
      // rounding, now 1.09 and 1.16.  It costs 0.5% in bf16, 3% on groups above
      // 16; in 4 bits 3% on windows of 1024 and nothing on long sequences.)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float raw[2], mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          raw[e] = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
          mx[e] = __fmul_rn(raw[e], to_log2[nt][e]);
        }
        if (__any_sync(0xffffffffu, mx[0] > m_ref[nt][0] || mx[1] > m_ref[nt][1])) {
          float alpha[2], m[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
              raw[e] = fmaxf(raw[e], __shfl_xor_sync(0xffffffffu, raw[e], x));
            m[e] = fmaxf(m_ref[nt][e], __fmul_rn(raw[e], to_log2[nt][e]));
          }
          if (large || __any_sync(0xffffffffu, fmaxf(fabsf(m[0]), fabsf(m[1])) >= kLargeScore)) {
            large = true;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (m[e] > m_ref[nt][e])
                m[e] = reference_max(raw[e], BITS == 16 ? a.scale_log2 : own_log2[nt][e], to_log2[nt][e]);
            __syncwarp();
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            alpha[e] = m[e] == -INFINITY ? 1.f : fast_exp2(m_ref[nt][e] - m[e]);
            m_ref[nt][e] = m[e];
            l[nt][e] *= alpha[e];
          }
#pragma unroll
          for (int m = 0; m < MS; ++m) {
            o[nt][m][0] *= alpha[0];
            o[nt][m][1] *= alpha[1];
            o[nt][m][2] *= alpha[0];
            o[nt][m][3] *= alpha[1];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) oc[nt][e] *= alpha[e & 1];
        }
      }

      // ---- tile by tile: P, then O^T += V^T P^T
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float p[NT][4];        // keys g, g + 8, heads 2 t, 2 t + 1, as the scores
        uint32_t pf[NT][2];    // P^T fragments: column = head g, rows keys 2 t, 2 t + 1 / + 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m0 = m_ref[nt][0] == -INFINITY ? 0.f : m_ref[nt][0];
          const float m1 = m_ref[nt][1] == -INFINITY ? 0.f : m_ref[nt][1];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[nt][e] = fast_exp2(fmaf(s[h][nt][e], to_log2[nt][e & 1], (e & 1) ? -m1 : -m0));
          l[nt][0] += p[nt][0] + p[nt][2];
          l[nt][1] += p[nt][1] + p[nt][3];
          pf[nt][0] = transpose8x8(pack_bf16x2(p[nt][0], p[nt][1]));
          pf[nt][1] = transpose8x8(pack_bf16x2(p[nt][2], p[nt][3]));
        }
        if constexpr (BITS == 16) {
          const int row = 16 * h + (lane & 7) + ((lane >> 4) << 3);
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (mask != 0xffffffffu) {
            const uint32_t bits = mask >> (16 * h + 2 * t);
            keep0 = ((bits & 1u) ? 0xffffu : 0u) | ((bits & 2u) ? 0xffff0000u : 0u);
            keep1 = ((bits & 256u) ? 0xffffu : 0u) | ((bits & 512u) ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int m = 0; m < MS; ++m) {
            const int chunk = (m % 4) * 2 + ((lane >> 3) & 1);
            uint32_t f[4];
            ldmatrix4_trans(f, vals + (m / 4) * kBlockKeys * 128 + row * 128 +
                                   ((chunk ^ (row & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16(o[nt][m], f[0] & keep0, f[1] & keep0, f[2] & keep1, f[3] & keep1,
                       pf[nt][0], pf[nt][1]);
          }
        } else {
          // Rows of this lane: keys t, t + 4 (first half), t + 8, t + 12.
          const uint8_t* codes = val_rows + (h ? code1 : 0);
          const uint8_t* pairs = val_rows + (h ? pair1 : pair0);
          const int ka = key_of_row(g);  // this lane's rows of p: keys ka, ka + 8
          uint32_t pa[NG], pb[NG];
          lds_words<NG>(pa, pairs + ka * (D / 8));
          lds_words<NG>(pb, pairs + (ka + 8) * (D / 8));
          uint32_t cw[4];  // pair of group g (rows from NG on repeat group 0)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            cw[x] = lds32(pairs + (t + 4 * x) * (D / 8) + 4 * (g < NG ? g : 0));
          if (mask != 0xffffffffu) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              cw[x] = ((mask >> (16 * h + t + 4 * x)) & 1u) ? cw[x] : 0u;
            const bool va = (mask >> (16 * h + ka)) & 1u, vb = (mask >> (16 * h + ka + 8)) & 1u;
#pragma unroll
            for (int wv = 0; wv < NG; ++wv) {
              pa[wv] = va ? pa[wv] : 0u;
              pb[wv] = vb ? pb[wv] : 0u;
            }
          }
          // Centres: row g of the product is group g.
          const uint32_t c0 = __byte_perm(cw[0], cw[1], 0x7632);
          const uint32_t c1 = __byte_perm(cw[2], cw[3], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16(oc[nt], c0, 0u, c1, 0u, pf[nt][0], pf[nt][1]);
          // Codes: half-word w of this lane's NG holds channels 32 w + 4 g .. + 3.
          uint32_t cv[4][(NG + 1) / 2];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint8_t* row = codes + (t + 4 * x) * (D / 2) + g * 2 * NG;
            if constexpr (NG % 2 == 0) {
              lds_words<NG / 2>(cv[x], row);
            } else {
#pragma unroll
              for (int wv = 0; wv < NG; ++wv) {
                const uint32_t hw = lds16(row + 2 * wv);
                if (wv & 1)
                  cv[x][wv / 2] |= hw << 16;
                else
                  cv[x][wv / 2] = hw;
              }
            }
          }
#pragma unroll
          for (int wv = 0; wv < NG; ++wv) {
            const uint32_t sel = (wv & 1) ? 0x7632u : 0x5410u;
            const uint32_t v0 = __byte_perm(cv[0][wv / 2], cv[1][wv / 2], sel);
            const uint32_t v1 = __byte_perm(cv[2][wv / 2], cv[3][wv / 2], sel);
            uint32_t e[4], f[4];
            codes_bf16_scaled(v0, e);
            codes_bf16_scaled(v1, f);
            const float sa = bf16_lo(pa[wv]), sb = bf16_lo(pb[wv]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t w0 = transpose8x8(pack_bf16x2(p[nt][0] * sa, p[nt][1] * sa));
              const uint32_t w1 = transpose8x8(pack_bf16x2(p[nt][2] * sb, p[nt][3] * sb));
              mma_bf16(o[nt][2 * wv], e[0], e[1], f[0], f[1], w0, w1);
              mma_bf16(o[nt][2 * wv + 1], e[2], e[3], f[2], f[3], w0, w1);
            }
          }
        }
      }

      // ---- refill the stage
      if (to_load > 0) issue(stage);
      if constexpr (BITS == 4) copy_commit();
      if (++stage == C::kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }
    if (!ok) break;

    // ---- end of the segment
    const bool whole = first == 0 && count == at.s.units;
    // A segment that began in an earlier warp leaves its partial result in the
    // warp's slot; one that goes on in a later warp is the warp's last, and
    // lies over the ring, which is done.
    float* slot = reinterpret_cast<float*>(
        smem_raw + (ring - smem_addr(smem_raw)) + (first > 0 ? C::kRingBytes : 0));
    if (!whole && lane == 0) {
      if (first > 0) {
        parts->has0 = 1;
        parts->end0 = first + count == at.s.units;
        parts->b0 = at.b;
        parts->hh0 = at.hh;
      } else {
        parts->has1 = 1;
        parts->b1 = at.b;
        parts->hh1 = at.hh;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
      if constexpr (BITS == 4) {
        // The centres' sums of group w lie in lanes 4 w + t.
#pragma unroll
        for (int wv = 0; wv < NG; ++wv) {
          const float z0 = __shfl_sync(0xffffffffu, oc[nt][0], 4 * wv + t);
          const float z1 = __shfl_sync(0xffffffffu, oc[nt][1], 4 * wv + t);
#pragma unroll
          for (int m = 2 * wv; m < 2 * wv + 2; ++m) {
            o[nt][m][0] = fmaf(o[nt][m][0], kLowNibble, z0);
            o[nt][m][1] = fmaf(o[nt][m][1], kLowNibble, z1);
            o[nt][m][2] = fmaf(o[nt][m][2], kHighNibble, z0);
            o[nt][m][3] = fmaf(o[nt][m][3], kHighNibble, z1);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = nt * 8 + 2 * t + e;
        if (head >= nheads) continue;
        if (whole) {
          const float inv = l[nt][e] != 0.f ? 1.f / l[nt][e] : 0.f;
          __nv_bfloat16* out = a.o + at.b * a.o_sb + (head0 + head) * a.o_sh;
          if constexpr (BITS == 16) {
#pragma unroll
            for (int m = 0; m < MS; ++m) {
              out[16 * m + g] = __float2bfloat16_rn(o[nt][m][e] * inv);
              out[16 * m + 8 + g] = __float2bfloat16_rn(o[nt][m][e + 2] * inv);
            }
          } else {
#pragma unroll
            for (int wv = 0; wv < NG; ++wv)
              *reinterpret_cast<uint2*>(out + 32 * wv + 4 * g) = make_uint2(
                  pack_bf16x2(o[nt][2 * wv][e] * inv, o[nt][2 * wv][e + 2] * inv),
                  pack_bf16x2(o[nt][2 * wv + 1][e] * inv, o[nt][2 * wv + 1][e + 2] * inv));
          }
        } else {
          if (g == 0) {
            slot[head] = m_ref[nt][e];
            slot[8 * NT + head] = l[nt][e];
          }
          float* out = slot + 16 * NT + head * D;
          if constexpr (BITS == 16) {
#pragma unroll
            for (int m = 0; m < MS; ++m) {
              out[16 * m + g] = o[nt][m][e];
              out[16 * m + 8 + g] = o[nt][m][e + 2];
            }
          } else {
#pragma unroll
            for (int wv = 0; wv < NG; ++wv)
              *reinterpret_cast<float4*>(out + 32 * wv + 4 * g) =
                  make_float4(o[nt][2 * wv][e], o[nt][2 * wv][e + 2], o[nt][2 * wv + 1][e],
                              o[nt][2 * wv + 1][e + 2]);
          }
        }
      }
    }
    u += count;
    at.i += count - 1;
    if (u < u1) next_place(a, heads, at);
  }
  if (BITS == 16 && !ok) {
    // Let this warp's copies land before the block goes away.
    volatile int no_abort = 0;
    const int64_t flight = u1 - u - to_load;
    for (int64_t n = 0; n < flight && n < C::kStages; ++n) {
      mbar_wait_warp(&full[stage], parity, &no_abort, a.status);
      if (++stage == C::kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    // For the join kernel: sequence, head block, first share and number of
    // shares of the segment that the block's share begins inside of.
    const int64_t f0 = c0 - begin[2];
    const int first = static_cast<int>(f0 / share);
    P.cuts[blockIdx.x] =
        begin[2] > 0 ? make_int4(begin[0], begin[1], first,
                                 static_cast<int>((f0 + begin[3] - 1) / share) - first + 1)
                     : make_int4(0, 0, 0, 0);
  }

  // -------------------------------------------------- join within the block --
  // A chain is a cut segment's partial results in this block: the slot of the
  // warp where it begins (slot 0 of warp 0: it began in an earlier block) and
  // slots 0 of the warps that follow, up to its end.  Warps take the chains'
  // heads in turn, a lane a part (statistics) or 4 channels (outputs); 96
  // windows of 1024 took 60 us with look-ups part by part, 55 so.  A segment
  // with its beginning and end here is finished; of the others the block
  // leaves one partial result each (slot 0: begun earlier; slot 1: goes on)
  // for the join kernel.
  auto parts_of = [&](int w) {
    return parts + (w - warp) * (128 / static_cast<int>(sizeof(WarpParts)));
  };
  auto slot_of = [&](int w, bool begins) {
    return reinterpret_cast<const float*>(smem_raw + (base - smem_addr(smem_raw)) +
                                          w * C::kWarpBytes + (begins ? 0 : C::kRingBytes));
  };
  const WarpParts* its = parts_of(lane < kWarps ? lane : 0);
  const unsigned has0 = __ballot_sync(0xffffffffu, lane < kWarps && its->has0);
  const unsigned ends = __ballot_sync(0xffffffffu, lane < kWarps && its->end0);
  const unsigned has1 = __ballot_sync(0xffffffffu, lane < kWarps && its->has1);
  int turn = warp;  // heads that other warps take before this one's next
  for (unsigned left = has1 << 1 | (has0 & 1u); left; left &= left - 1) {
    const int c = __ffs(left) - 1;
    const bool begins = c > 0;  // in warp c - 1 of this block
    const int w0 = begins ? c - 1 : 0, from = begins ? c : 0;
    const int run = __ffs(~(has0 >> from)) - 1, end = __ffs(ends >> from);
    const bool ended = end > 0 && end <= run;
    const int n = (ended ? end : run) + (begins ? 1 : 0);  // parts, in warps w0 ..
    const int b = begins ? parts_of(w0)->b1 : parts_of(0)->b0;
    const int hh = begins ? parts_of(w0)->hh1 : parts_of(0)->hh0;
    const int kvh = hh / P.head_blocks;
    const int head0 = kvh * P.group + (hh % P.head_blocks) * 8 * NT;
    const int nheads = min(8 * NT, (kvh + 1) * P.group - head0);
    for (; turn < nheads; turn += kWarps) {
      const int head = turn;
      const bool part = lane < n;
      const float* p = slot_of(w0 + (part ? lane : 0), begins && (lane == 0 || !part));
      const float m = part ? p[head] : -INFINITY;
      float mx = m, sum = part ? p[8 * NT + head] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float f = fast_exp2(m - (mx == -INFINITY ? 0.f : mx));
      sum *= f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const bool live = lane * 4 < D;
#pragma unroll 2
      for (int i = 0; i < n; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        const float4 v = *reinterpret_cast<const float4*>(slot_of(w0 + i, begins && i == 0) +
                                                          16 * NT + head * D + (live ? lane * 4 : 0));
        acc.x = fmaf(fi, v.x, acc.x);
        acc.y = fmaf(fi, v.y, acc.y);
        acc.z = fmaf(fi, v.z, acc.z);
        acc.w = fmaf(fi, v.w, acc.w);
      }
      if (begins && ended) {
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        if (live)
          *reinterpret_cast<uint2*>(a.o + b * a.o_sb + (head0 + head) * a.o_sh + lane * 4) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      } else {
        float* out = P.parts + (2 * blockIdx.x + (begins ? 1 : 0)) * (C::kSlotBytes / 4);
        if (lane == 0) {
          out[head] = mx;
          out[8 * NT + head] = sum;
        }
        if (live) *reinterpret_cast<float4*>(out + 16 * NT + head * D + lane * 4) = acc;
      }
    }
    turn -= nheads;
  }
}

// Joins the blocks' shares of the segments that were cut between them.  Block
// w looks at the boundary between shares w and w + 1: where it falls inside a
// segment of n shares, the n - 1 blocks of its boundaries split the segment's
// heads among them.
template <int NT>
__global__ void __launch_bounds__(kJoinThreads) swa_paged_join_kernel(const PagedParams P, int d) {
  const SwaPagedArgs& a = P.a;
  __shared__ float4 so[kJoinThreads / 32][32];
  __shared__ float sl[kJoinThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Every block waits, so that this kernel ends after the one before it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = P.cuts[blockIdx.x + 1];
  const int n = cut.w;                        // shares of the segment
  if (n == 0) return;                         // no segment goes on here
  const int w0 = cut.z;
  const int me = blockIdx.x - w0;             // this boundary among n - 1
  const int kvh = cut.y / P.head_blocks;
  const int head0 = kvh * P.group + (cut.y % P.head_blocks) * 8 * NT;
  const int nheads = min(8 * NT, (kvh + 1) * P.group - head0);
  auto slot_of = [&](int x) {
    return P.parts + static_cast<int64_t>(2 * (w0 + x) + (x == 0 ? 1 : 0)) * (8 * NT * (2 + d));
  };
  // A head at a time, 4 channels a lane.  Few shares: a warp takes a head
  // alone; many: all warps share one.
  const bool alone = n <= kJoinThreads / 32;
  const bool live = lane * 4 < d;
  for (int head = me + (alone ? warp * (n - 1) : 0); head < nheads;
       head += (n - 1) * (alone ? kJoinThreads / 32 : 1)) {
    float mx = -INFINITY;
    for (int x = lane; x < n; x += 32) mx = fmaxf(mx, slot_of(x)[head]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int x = alone ? 0 : warp; x < n; x += alone ? 1 : kJoinThreads / 32) {
      const float* p = slot_of(x);
      const float f = fast_exp2(p[head] - ref);
      l = fmaf(f, p[8 * NT + head], l);
      if (live) {
        const float4 v = *reinterpret_cast<const float4*>(p + 16 * NT + head * d + lane * 4);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
    }
    if (!alone) {
      so[warp][lane] = acc;
      if (lane == 0) sl[warp] = l;
      __syncthreads();
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
#pragma unroll
      for (int x = 0; x < kJoinThreads / 32; ++x) {
        const float4 v = so[x][lane];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        l += sl[x];
      }
      __syncthreads();
    }
    if ((alone || warp == 0) && live) {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      *reinterpret_cast<uint2*>(a.o + cut.x * a.o_sb + (head0 + head) * a.o_sh + lane * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
  }
}

int head_tiles(int group) { return group > 8 ? 2 : 1; }

template <int D, int BITS, int NT>
cudaError_t launch_typed(PagedParams& prm, cudaStream_t stream) {
  using C = Cfg<D, BITS, NT>;
  auto kern = swa_paged_kernel<D, BITS, NT>;
  static bool configured[kDeviceSlots] = {};
  cudaError_t e = allow_smem(kern, C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  const int grid = prm.a.sms;
  kern<<<grid, C::kWarps * 32, C::kSmemBytes, stream>>>(prm);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid - 1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  // Launched to overlap the first kernel's end where that one is long: with 64
  // heads over 8, calls of 100 to 400 MB take 2 us less so (4 bits, 100 MB: 30.9
  // us a call for 32.9).  Shorter ones are bound by the host, 20 us either way,
  // and replayed from a graph they lose by it in 4 bits (8 to 100 MB: 0.6 to 0.9
  // us; bf16 no difference).  The lengths are not known here, so the bound goes
  // by the table: a short call under a wide one loses that much.
  const KvCache& c = prm.a.c;
  const int64_t most = c.table_pages << c.page_shift;
  const double bytes = 2.0 * prm.a.batch * c.kv_heads *
                       static_cast<double>(most < prm.a.window ? most : prm.a.window) *
                       (static_cast<double>(c.block_bytes) / c.page_size);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = bytes > 100e6 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, swa_paged_join_kernel<NT>, static_cast<const PagedParams&>(prm), D);
}

template <int D, int BITS>
cudaError_t launch_nt(PagedParams& prm, cudaStream_t stream) {
  return head_tiles(prm.group) == 1 ? launch_typed<D, BITS, 1>(prm, stream)
                                    : launch_typed<D, BITS, 2>(prm, stream);
}

template <int BITS>
cudaError_t launch_d(PagedParams& prm, cudaStream_t stream) {
  switch (prm.a.c.head_dim) {
    case 32: return launch_nt<32, BITS>(prm, stream);
    case 64: return launch_nt<64, BITS>(prm, stream);
    case 96: return launch_nt<96, BITS>(prm, stream);
    case 128: return launch_nt<128, BITS>(prm, stream);
    default: break;
  }
  if constexpr (BITS == 16)
    if (prm.a.c.head_dim == 16) return launch_nt<16, BITS>(prm, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

// A block's cut, and two partial results: maxima, sums and outputs of up to
// 8 NT heads.
size_t swa_paged_workspace(int, int heads, int kv_heads, int head_dim, int sms) {
  return sms * (2ull * 8 * head_tiles(heads / kv_heads) * (2 + head_dim) * sizeof(float) +
                sizeof(int4));
}

cudaError_t launch_swa_paged(const SwaPagedArgs& a, cudaStream_t stream) {
  PagedParams prm;
  prm.a = a;
  prm.group = a.heads / a.c.kv_heads;
  const int tile = 8 * head_tiles(prm.group);
  prm.head_blocks = (prm.group + tile - 1) / tile;
  prm.cuts = static_cast<int4*>(a.workspace);
  prm.parts = reinterpret_cast<float*>(prm.cuts + a.sms);
  if (a.c.bits == 4) return launch_d<4>(prm, stream);
  const int sub = a.c.page_size < kBlockKeys ? a.c.page_size : kBlockKeys;
  const uint64_t row = 2ull * a.c.head_dim;
  const uint64_t dims[3] = {static_cast<uint64_t>(a.c.head_dim), a.c.page_bytes / row,
                            static_cast<uint64_t>(a.c.pages)};
  const uint64_t strides[2] = {row, static_cast<uint64_t>(a.c.page_bytes)};
  const uint32_t box[3] = {64, static_cast<uint32_t>(sub), 1};
  if (!make_tensor_map(&prm.map, reinterpret_cast<const __nv_bfloat16*>(a.c.base), 3, dims, strides,
                       box))
    return cudaErrorInvalidValue;
  return launch_d<16>(prm, stream);
}

}  // namespace ptb
