// The paged cache of keys and values: appending new tokens, with the
// position rotation and (bits = 4) the quantization on the way, and reading
// rows back (layout and arithmetic: ptb.h).
//
// Both are single passes over memory.  Into bf16 an append runs at memory's rate
// (5490 tokens, 64 + 8 heads of 128, rotated keys kept: 37.7 us, 6.3 TB/s); into
// 4 bits instructions bound it (80% of the issue slots; 17785 tokens of 32 heads
// of 64: 90 us).  Reading those back takes 42 us (28 at the rate of a copy: a
// token's rows lie in 64 blocks of a page, 40 bytes each); heads of 128, 13 for 13.
//
// Append: a warp takes a token and a batch of its head rows; a lane holds 8
// neighbouring channels (16 bytes) of a row and a row lies in one warp (d / 8
// lanes), so the rotation's other half and a 32-channel group's minimum and
// maximum come from shuffles.  The batch's rows are loaded before the token's
// sequence, position and page are looked up, which hides those dependent
// loads.  In-place rotation is safe: a row is read in full by its warp before
// any of it is written.
//
// Gather: a lane holds what lies together in a 4-bit row, 8 channels of every
// group of a key (4 lanes a row) or 4 of every group of a value (8 lanes).
#include "kv_device.cuh"

namespace ptb {
namespace {

// Blocks of two warps: 64 threads fill an SM up again as soon as two warps end
// (17785 tokens of 32 heads of 64, 4 bits: append and gather 129 us; 134 with 128
// threads, 133 with 32).  Rows go past L1 (139 us with 128 threads without).
constexpr int kKvThreads = 64;
constexpr int kBatch = 4;  // loads of rows that a lane has in flight (142 us; 161 with 2 or 8)

// Token and batch of a warp's number.  A 64-bit division costs as much as a
// third of the rest of a warp's look-ups, so it is left to calls that need it.
__device__ __forceinline__ void split_item(int64_t item, int batches, int64_t& t, int& batch) {
  if (item <= 0xffffffffll)
    t = static_cast<uint32_t>(item) / static_cast<uint32_t>(batches);
  else
    t = item / batches;
  batch = static_cast<int>(item - t * batches);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) {
  return *reinterpret_cast<__nv_bfloat162*>(&v);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}

// One (scale, centre) pair and the 8 codes of this lane, from 8 bf16 values
// of a group that 4 neighbouring lanes share.
//
// u = round(y / s) + 8 with y = x - centre.  The quotient has to be that of an
// IEEE division, or ties (frequent: bf16 values over a bf16 scale) would fall
// either way; one exact remainder and one correction give it (P. Markstein,
// IBM J. Res. Dev. 34 (1990), Theorem 7: with r the rounded reciprocal of s
// and q within an ulp, q + r (y - q s) by two FMAs is y / s rounded).
__device__ __forceinline__ uint32_t quantize_group(const uint4& w, uint32_t& pair) {
  const __nv_bfloat162 v0 = as_bf162(w.x), v1 = as_bf162(w.y), v2 = as_bf162(w.z),
                       v3 = as_bf162(w.w);
  // NaN stays in both, an infinity makes the range infinite.
  __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(v0, v1), __hmin2_nan(v2, v3));
  __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(v0, v1), __hmax2_nan(v2, v3));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo2 = __hmin2_nan(lo2, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(lo2), o)));
    hi2 = __hmax2_nan(hi2, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(hi2), o)));
  }
  const float lo = __bfloat162float(__hmin_nan(__low2bfloat16(lo2), __high2bfloat16(lo2)));
  const float hi = __bfloat162float(__hmax_nan(__low2bfloat16(hi2), __high2bfloat16(hi2)));
  const float range = __fsub_rn(hi, lo);
  if (!(range < INFINITY)) {
    pair = 0x7fc07fc0u;  // NaN, NaN: the whole group reads as NaN
    return 0;
  }
  constexpr float k15 = 1.f / 15;
  float fifteenth = __fmul_rn(range, k15);
  fifteenth = range > 1e-28f ? fmaf(fmaf(-fifteenth, 15.f, range), k15, fifteenth)
                             : __fdiv_rn(range, 15.f);
  const __nv_bfloat16 scale = __float2bfloat16_rn(fifteenth);
  const float s = __bfloat162float(scale);
  const __nv_bfloat16 centre = __float2bfloat16_rn(__fadd_rn(lo, 8.f * s));
  const float z = __bfloat162float(centre);
  pair = static_cast<uint32_t>(__bfloat16_as_ushort(scale)) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(centre)) << 16);
  const uint32_t raw[4] = {w.x, w.y, w.z, w.w};
  const float inv = __frcp_rn(s);
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  uint32_t codes = 0;
  if (s > 1e-30f) {  // no remainder underflows
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      const float y = __fsub_rn((e & 1) ? bf16_hi(raw[e >> 1]) : bf16_lo(raw[e >> 1]), z);
      float q = __fmul_rn(y, inv);
      q = fmaf(fmaf(-q, s, y), inv, q);
      codes = codes * 16u + __float_as_uint(__fadd_rn(fminf(fmaxf(q, -8.f), 7.f), kMagic));
    }
    codes -= (0x4b400000u - 8u) * 0x11111111u;  // kMagic's bits less 8, in each of the eight
  } else {
#pragma unroll 1
    for (int e = 7; e >= 0; --e) {
      const uint32_t word = e < 2 ? raw[0] : (e < 4 ? raw[1] : (e < 6 ? raw[2] : raw[3]));
      const float y = __fsub_rn((e & 1) ? bf16_hi(word) : bf16_lo(word), z);
      const float q = rintf(__fdiv_rn(y, s > 0.f ? s : 1.f));
      codes = codes * 16u + static_cast<uint32_t>(fminf(fmaxf(q, -8.f), 7.f) + 8.f);
    }
  }
  return codes;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_lo(v[e]);
    x[2 * e + 1] = bf16_hi(v[e]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// A warp's number is token * batches + batch; a batch is kBatch steps of RPW
// rows of one kind: q, then k, then v.
template <int D>
__global__ void __launch_bounds__(kKvThreads)
    kv_append_kernel(const KvAppendArgs a, int q_batches, int kv_batches) {
  constexpr int L = D / 8;     // lanes a row
  constexpr int RPW = 32 / L;  // rows a warp holds at once
  constexpr int NG = D / kKvGroup;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5);
  const int batches = q_batches + 2 * kv_batches;
  int64_t t;
  int batch;
  split_item(item, batches, t, batch);
  if (t >= a.tokens) return;
  const bool is_q = batch < q_batches;
  batch -= is_q ? 0 : q_batches;
  const bool is_v = !is_q && batch >= kv_batches;
  batch -= is_v ? kv_batches : 0;
  const int rows = is_q ? a.heads : a.c.kv_heads;
  const int sub = lane / L;  // row of this lane among the RPW
  const int c = lane - sub * L;
  const int h0 = batch * (kBatch * RPW) + sub;
  const int64_t sh = is_q ? a.q_sh : (is_v ? a.v_sh : a.k_sh);
  const __nv_bfloat16* src =
      (is_q ? a.q + t * a.q_st : (is_v ? a.v + t * a.v_st : a.k + t * a.k_st)) + h0 * sh + 8 * c;

  uint4 w[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    w[i] = sub < RPW && h0 + i * RPW < rows
               ? load16_past_l1(src + i * RPW * sh)
               : make_uint4(0, 0, 0, 0);

  const int b = find_sequence(a.cu, a.batch, t, lane);
  if (b >= a.batch) return;  // a row behind the last sequence
  const int64_t first = a.cu[b], past = a.past[b];
  const int64_t pos = past + (t - first);
  if (first < 0 || first > t || a.cu[b + 1] > a.tokens || past < 0 || pos >= a.positions) {
    if (lane == 0) record_error(a.status, PTB_ERR_ARG);
    return;
  }
  if (!is_v && a.rot_dim) {
    const bool rotated = sub < RPW && 8 * c < a.rot_dim;
    const int half = a.rot_dim / 2;
    const bool lower = 8 * c < half;
    // (cos, sin) of this lane's channels, the same for every head; the sign of
    // the sine is its sign in the lane's outputs: x cos + other sin.
    float co[8], si[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) co[e] = si[e] = 0.f;
    if (rotated) {
      const float* cr = a.cos + pos * half;
      const float* sr = a.sin + pos * half;
      if (a.interleaved) {
        const float4 x = *reinterpret_cast<const float4*>(cr + 4 * c);
        const float4 y = *reinterpret_cast<const float4*>(sr + 4 * c);
        co[0] = co[1] = x.x, co[2] = co[3] = x.y, co[4] = co[5] = x.z, co[6] = co[7] = x.w;
        si[1] = y.x, si[3] = y.y, si[5] = y.z, si[7] = y.w;
        si[0] = -y.x, si[2] = -y.y, si[4] = -y.z, si[6] = -y.w;
      } else {
        const int at = lower ? 8 * c : 8 * c - half;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(cr + at + e);
          const float4 y = *reinterpret_cast<const float4*>(sr + at + e);
          co[e] = x.x, co[e + 1] = x.y, co[e + 2] = x.z, co[e + 3] = x.w;
          si[e] = lower ? -y.x : y.x, si[e + 1] = lower ? -y.y : y.y;
          si[e + 2] = lower ? -y.z : y.z, si[e + 3] = lower ? -y.w : y.w;
        }
      }
    }
    // The lane whose vector this one turns against: half a rotation away.
    const int other = (!a.interleaved && rotated) ? sub * L + (lower ? c + half / 8 : c - half / 8)
                                                  : lane;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      uint4 p = w[i];
      if (!a.interleaved) {
        p.x = __shfl_sync(0xffffffffu, w[i].x, other);
        p.y = __shfl_sync(0xffffffffu, w[i].y, other);
        p.z = __shfl_sync(0xffffffffu, w[i].z, other);
        p.w = __shfl_sync(0xffffffffu, w[i].w, other);
      }
      if (rotated) {
        float x[8], y[8], out[8];
        unpack8(w[i], x);
        unpack8(p, y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          out[e] = __fadd_rn(__fmul_rn(x[e], co[e]),
                             __fmul_rn(a.interleaved ? x[e ^ 1] : y[e], si[e]));
        w[i] = pack8(out);
      }
    }
  }
  __syncwarp();  // in place: every row has been read
  __nv_bfloat16* out = is_q ? a.q_out : (is_v ? nullptr : a.k_out);
  if (out) {
    const int64_t oh = is_q ? a.qo_sh : a.ko_sh;
    out += t * (is_q ? a.qo_st : a.ko_st) + h0 * oh + 8 * c;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (sub < RPW && h0 + i * RPW < rows)
        store16_past_l1(out + i * RPW * oh, w[i]);
  }
  if (is_q) return;

  uint8_t* page = kv_page(a.c, b, pos);
  if (!page) {
    if (lane == 0) record_error(a.status, PTB_ERR_ARG);
    return;
  }
  const int off = static_cast<int>(pos) & (a.c.page_size - 1);
  uint8_t* block = page + ((is_v ? a.c.kv_heads : 0) + h0) * a.c.block_bytes;
  const int64_t step = RPW * a.c.block_bytes;
  if (a.c.bits == 16) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (sub < RPW && h0 + i * RPW < rows)
        store16_past_l1(block + i * step + off * (2 * D) + 16 * c, w[i]);
  } else if constexpr (NG > 0) {
    const int g = c >> 2;  // group, and the vector's place in it
    uint8_t* row = block + off * (D / 2);
    uint8_t* pairs = block + a.c.page_size * (D / 2) + (off * NG + g) * 4;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (batch * (kBatch * RPW) + i * RPW >= rows) break;
      uint32_t pair;
      const uint32_t codes = quantize_group(w[i], pair);
      if (sub < RPW && h0 + i * RPW < rows) {
        uint8_t* r = row + i * step;
        if (!is_v) {
          *reinterpret_cast<uint32_t*>(r + key_word(g, c & 3, NG)) = codes;
        } else {
          *reinterpret_cast<uint16_t*>(r + value_half(g, 2 * (c & 3), NG)) =
              static_cast<uint16_t>(codes);
          *reinterpret_cast<uint16_t*>(r + value_half(g, 2 * (c & 3) + 1, NG)) =
              static_cast<uint16_t>(codes >> 16);
        }
        if ((c & 3) == 0) *reinterpret_cast<uint32_t*>(pairs + i * step) = pair;
      }
    }
  }
}

// N (1 .. 4) consecutive words at 4-byte alignment, 16- or 8-byte where N is 4 or 2.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&r)[N], const uint8_t* p) {
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

// The values of eight codes, v[k] = (nibble k of the low half, of the high
// half) as bf16 pairs: centre + scale * (u - 8), rounded once.
__device__ __forceinline__ void code_values(uint32_t codes, uint32_t scale2, uint32_t centre2,
                                            uint32_t (&v)[4]) {
  codes_bf16(codes, v);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = as_u32(__hfma2(as_bf162(v[k]), as_bf162(scale2), as_bf162(centre2)));
}

// A warp's number is token * batches + batch of rows (k heads, then v heads).
template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads) kv_gather_kernel(const KvGatherArgs a, int batches,
                                                               int batch_rows) {
  constexpr int NG = D / kKvGroup;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5);
  int64_t t;
  int batch;
  split_item(item, batches, t, batch);
  if (t >= a.tokens) return;
  const int b = find_sequence(a.cu, a.batch, t, lane);
  if (b >= a.batch) return;
  const int64_t first = a.cu[b], start = a.start[b];
  const int64_t pos = start + (t - first);
  const uint8_t* page = first < 0 || first > t || a.cu[b + 1] > a.tokens || start < 0
                            ? nullptr
                            : kv_page(a.c, b, pos);
  if (!page) {
    if (lane == 0) record_error(a.status, PTB_ERR_ARG);
    return;
  }
  const int off = static_cast<int>(pos) & (a.c.page_size - 1);
  const int kv = a.c.kv_heads;
  const int row_base = batch * batch_rows;
  const int row_end = min(row_base + batch_rows, 2 * kv);
  auto row_out = [&](int r) {
    return r < kv ? a.k + t * a.k_st + r * a.k_sh : a.v + t * a.v_st + (r - kv) * a.v_sh;
  };
  if constexpr (BITS == 16) {
    constexpr int L = D / 8, RPW = 32 / L;
    const int sub = lane / L, c = lane - sub * L;
#pragma unroll 4
    for (int r = row_base + sub; r < row_end; r += RPW)
      if (sub < RPW)
        store16_past_l1(row_out(r) + 8 * c,
                        load16_past_l1(page + r * a.c.block_bytes + off * (2 * D) + 16 * c));
  } else {
    // Keys: 4 lanes a row.
    const int t4 = lane & 3, g = lane & 7;
#pragma unroll 2
    for (int r = row_base + (lane >> 2); r < min(row_end, kv); r += 8) {
      const uint8_t* block = page + r * a.c.block_bytes;
      uint32_t codes[NG], pair[NG];
      load_words<NG>(codes, block + off * (D / 2) + key_word(0, t4, NG));
      load_words<NG>(pair, block + a.c.page_size * (D / 2) + off * (D / 8));
      __nv_bfloat16* out = row_out(r) + 8 * t4;
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        uint32_t v[4];
        code_values(codes[w], __byte_perm(pair[w], pair[w], 0x1010),
                    __byte_perm(pair[w], pair[w], 0x3232), v);
        store16_past_l1(
            out + 32 * w,
            make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                       __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)));
      }
    }
    // Values: 8 lanes a row.
#pragma unroll 2
    for (int r = max(row_base, kv) + (lane >> 3); r < row_end; r += 4) {
      const uint8_t* block = page + r * a.c.block_bytes;
      const uint16_t* src =
          reinterpret_cast<const uint16_t*>(block + off * (D / 2) + value_half(0, g, NG));
      // Two groups a word: half-words w and w + 1.
      constexpr int NW = (NG + 1) / 2;
      uint32_t codes[NW], pair[2 * NW];
      if constexpr (NG % 2 == 0) {
        load_words<NW>(codes, reinterpret_cast<const uint8_t*>(src));
      } else {
#pragma unroll
        for (int w = 0; w < NW; ++w)
          codes[w] = src[2 * w] |
                     (2 * w + 1 < NG ? static_cast<uint32_t>(src[2 * w + 1]) << 16 : 0u);
        pair[2 * NW - 1] = 0;
      }
      load_words<NG>(*reinterpret_cast<uint32_t(*)[NG]>(&pair[0]),
                     block + a.c.page_size * (D / 2) + off * (D / 8));
      __nv_bfloat16* out = row_out(r) + 4 * g;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        uint32_t v[4];
        code_values(codes[w], __byte_perm(pair[2 * w], pair[2 * w + 1], 0x5410),
                    __byte_perm(pair[2 * w], pair[2 * w + 1], 0x7632), v);
        *reinterpret_cast<uint2*>(out + 64 * w) =
            make_uint2(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410));
        if (2 * w + 1 < NG)
          *reinterpret_cast<uint2*>(out + 64 * w + 32) =
              make_uint2(__byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
      }
    }
  }
}

template <int D>
cudaError_t append_typed(const KvAppendArgs& a, cudaStream_t stream) {
  constexpr int kRows = kBatch * (32 / (D / 8));
  const int q_batches = (a.heads + kRows - 1) / kRows;
  const int kv_batches = (a.c.kv_heads + kRows - 1) / kRows;
  const int batches = q_batches + 2 * kv_batches;
  const int64_t blocks = (a.tokens * batches + kKvThreads / 32 - 1) / (kKvThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  kv_append_kernel<D><<<static_cast<unsigned>(blocks), kKvThreads, 0, stream>>>(a, q_batches,
                                                                                  kv_batches);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t gather_bits(const KvGatherArgs& a, cudaStream_t stream) {
  // Rows of a warp: 64 where that leaves enough warps to fill the GPU (16k
  // tokens of 32 heads: 42 us, 46 with 16), else 16, two 8-row steps of keys.
  const int rows = 2 * a.c.kv_heads;
  const int batch_rows = a.tokens * ((rows + 63) / 64) >= 64ll * a.sms ? 64 : 16;
  const int batches = (rows + batch_rows - 1) / batch_rows;
  const int64_t blocks = (a.tokens * batches + kKvThreads / 32 - 1) / (kKvThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  kv_gather_kernel<D, BITS>
      <<<static_cast<unsigned>(blocks), kKvThreads, 0, stream>>>(a, batches, batch_rows);
  return cudaGetLastError();
}

template <int D>
cudaError_t gather_typed(const KvGatherArgs& a, cudaStream_t stream) {
  if (a.c.bits == 16) return gather_bits<D, 16>(a, stream);
  if constexpr (D % kKvGroup == 0) return gather_bits<D, 4>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  switch (a.c.head_dim) {
    case 16: return append_typed<16>(a, stream);
    case 32: return append_typed<32>(a, stream);
    case 64: return append_typed<64>(a, stream);
    case 96: return append_typed<96>(a, stream);
    case 128: return append_typed<128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_gather(const KvGatherArgs& a, cudaStream_t stream) {
  switch (a.c.head_dim) {
    case 16: return gather_typed<16>(a, stream);
    case 32: return gather_typed<32>(a, stream);
    case 64: return gather_typed<64>(a, stream);
    case 96: return gather_typed<96>(a, stream);
    case 128: return gather_typed<128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ptb
