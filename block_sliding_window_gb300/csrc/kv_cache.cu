// The paged cache of keys and values: appending new tokens, with the
// position rotation and (bits = 4) the quantization on the way, and reading
// rows back (layout and arithmetic: ptb.h).
//
// Both are single passes over memory.  A lane holds 8 neighbouring channels
// (16 bytes) of one head row and a row lies in one warp (d / 8 lanes), so the
// rotation's other half and a 32-channel group's minimum and maximum come
// from shuffles, and in-place rotation is safe: a row is read in full by its
// warp before any of it is written.
#include "kv_device.cuh"

namespace ptb {
namespace {

constexpr int kKvThreads = 128;

// One (scale, centre) pair and the 8 codes of this lane, from 8 bf16 values
// of a group that 4 neighbouring lanes share.
__device__ __forceinline__ uint32_t quantize_group(const float (&x)[8], uint32_t& pair) {
  float lo = x[0], hi = x[0];
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    finite = finite && fabsf(x[e]) < INFINITY;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    finite = __shfl_xor_sync(0xffffffffu, finite ? 1 : 0, o) && finite;
  }
  const float range = __fsub_rn(hi, lo);
  if (!finite || !(range < INFINITY)) {
    pair = 0x7fc07fc0u;  // NaN, NaN: the whole group reads as NaN
    return 0;
  }
  const __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
  const float s = __bfloat162float(scale);
  const __nv_bfloat16 centre = __float2bfloat16_rn(__fadd_rn(lo, 8.f * s));
  const float z = __bfloat162float(centre);
  pair = static_cast<uint32_t>(__bfloat16_as_ushort(scale)) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(centre)) << 16);
  const float div = s > 0.f ? s : 1.f;
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float u = rintf(__fdiv_rn(__fsub_rn(x[e], z), div)) + 8.f;
    codes |= static_cast<uint32_t>(fminf(fmaxf(u, 0.f), 15.f)) << (4 * e);
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

// Grid: x = token, y = chunk of head rows (all q heads, then k, then v).
template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvAppendArgs a, int chunk) {
  constexpr int L = D / 8;        // lanes a row
  constexpr int RPW = 32 / L;     // rows a warp holds at once
  constexpr int NG = D / kKvGroup;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int b = find_sequence(a.cu, a.batch, t, lane);
  if (b >= a.batch) return;  // a row behind the last sequence
  const int64_t first = a.cu[b], past = a.past[b];
  const int64_t pos = past + (t - first);
  if (first < 0 || first > t || past < 0 || pos >= a.positions) {
    if (threadIdx.x == 0) record_error(a.status, PTB_ERR_ARG);
    return;
  }
  uint8_t* page = kv_page(a.c, b, pos);
  if (!page && threadIdx.x == 0) record_error(a.status, PTB_ERR_ARG);
  const int off = static_cast<int>(pos) & (a.c.page_size - 1);

  const int sub = lane / L;       // row of this lane among the warp's RPW
  const int c = lane - sub * L;   // its 8-channel vector
  const bool rotated = sub < RPW && 8 * c < a.rot_dim;
  const int half = a.rot_dim / 2;
  // 8 (cos, sin) of this lane's channels: the same for every head.
  float co[8], si[8];
  if (rotated) {
    const float* cr = a.cos + pos * half;
    const float* sr = a.sin + pos * half;
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        co[2 * e] = co[2 * e + 1] = cr[4 * c + e];
        si[2 * e] = si[2 * e + 1] = sr[4 * c + e];
      }
    } else {
      const int at = 8 * c < half ? 8 * c : 8 * c - half;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = cr[at + e];
        si[e] = sr[at + e];
      }
    }
  }
  const int rows = a.heads + 2 * a.c.kv_heads;
  const int row_end = min(rows, static_cast<int>(blockIdx.y + 1) * chunk);
  for (int r0 = blockIdx.y * chunk + warp * RPW; r0 < row_end; r0 += (kKvThreads / 32) * RPW) {
    const int r = r0 + sub;
    const bool live = sub < RPW && r < row_end;
    const bool is_q = r < a.heads, is_k = !is_q && r < a.heads + a.c.kv_heads;
    const int h = is_q ? r : (is_k ? r - a.heads : r - a.heads - a.c.kv_heads);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) {
      const __nv_bfloat16* src = is_q ? a.q + t * a.q_st + h * a.q_sh
                                      : (is_k ? a.k + t * a.k_st + h * a.k_sh
                                              : a.v + t * a.v_st + h * a.v_sh);
      w = *reinterpret_cast<const uint4*>(src + 8 * c);
    }
    if (a.rot_dim) {
      // The vector that this one turns against: half a rotation away.
      const int other = sub * L + (8 * c < half ? c + half / 8 : c - half / 8);
      const int from = (!a.interleaved && rotated) ? other : lane;
      uint4 p;
      p.x = __shfl_sync(0xffffffffu, w.x, from);
      p.y = __shfl_sync(0xffffffffu, w.y, from);
      p.z = __shfl_sync(0xffffffffu, w.z, from);
      p.w = __shfl_sync(0xffffffffu, w.w, from);
      if (rotated && live && (is_q || is_k)) {
        float x[8], y[8], out[8];
        unpack8(w, x);
        unpack8(p, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other_x = a.interleaved ? x[e ^ 1] : y[e];
          const bool lower = a.interleaved ? (e & 1) == 0 : 8 * c < half;
          const float u = __fmul_rn(x[e], co[e]), v = __fmul_rn(other_x, si[e]);
          out[e] = lower ? __fsub_rn(u, v) : __fadd_rn(u, v);
        }
        w = pack8(out);
      }
    }
    __syncwarp();  // in place: the whole row has been read
    if (live && is_q)
      *reinterpret_cast<uint4*>(a.q_out + t * a.qo_st + h * a.qo_sh + 8 * c) = w;
    if (live && is_k && a.k_out)
      *reinterpret_cast<uint4*>(a.k_out + t * a.ko_st + h * a.ko_sh + 8 * c) = w;
    uint8_t* block = page ? page + (is_k ? h : a.c.kv_heads + h) * a.c.block_bytes : nullptr;
    if (a.c.bits == 16) {
      if (live && !is_q && page)
        *reinterpret_cast<uint4*>(block + off * (2 * D) + 16 * c) = w;
    } else if constexpr (NG > 0) {
      float x[8];
      unpack8(w, x);
      uint32_t pair;
      const uint32_t codes = quantize_group(x, pair);
      if (live && !is_q && page) {
        uint8_t* row = block + off * (D / 2);
        const int g = c >> 2;  // group, and the vector's place in it
        if (is_k) {
          *reinterpret_cast<uint32_t*>(row + key_word(g, c & 3, NG)) = codes;
        } else {
          *reinterpret_cast<uint16_t*>(row + value_half(g, 2 * (c & 3), NG)) =
              static_cast<uint16_t>(codes);
          *reinterpret_cast<uint16_t*>(row + value_half(g, 2 * (c & 3) + 1, NG)) =
              static_cast<uint16_t>(codes >> 16);
        }
        if ((c & 3) == 0)
          *reinterpret_cast<uint32_t*>(block + a.c.page_size * (D / 2) + (off * NG + g) * 4) =
              pair;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_gather_kernel(const KvGatherArgs a, int chunk) {
  constexpr int L = D / 8;
  constexpr int RPW = 32 / L;
  constexpr int NG = D / kKvGroup;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int b = find_sequence(a.cu, a.batch, t, lane);
  if (b >= a.batch) return;
  const int64_t first = a.cu[b], start = a.start[b];
  const int64_t pos = start + (t - first);
  const uint8_t* page = first < 0 || first > t || start < 0 ? nullptr : kv_page(a.c, b, pos);
  if (!page) {
    if (threadIdx.x == 0) record_error(a.status, PTB_ERR_ARG);
    return;
  }
  const int off = static_cast<int>(pos) & (a.c.page_size - 1);
  const int sub = lane / L, c = lane - sub * L;
  const int rows = 2 * a.c.kv_heads;
  const int row_end = min(rows, static_cast<int>(blockIdx.y + 1) * chunk);
  for (int r0 = blockIdx.y * chunk + warp * RPW; r0 < row_end; r0 += (kKvThreads / 32) * RPW) {
    const int r = r0 + sub;
    if (sub >= RPW || r >= row_end) continue;
    const bool is_k = r < a.c.kv_heads;
    const int h = is_k ? r : r - a.c.kv_heads;
    const uint8_t* block = page + r * a.c.block_bytes;
    uint4 w;
    if (a.c.bits == 16) {
      w = *reinterpret_cast<const uint4*>(block + off * (2 * D) + 16 * c);
    } else {
      const uint8_t* row = block + off * (D / 2);
      const int g = c >> 2;
      const uint32_t codes =
          is_k ? *reinterpret_cast<const uint32_t*>(row + key_word(g, c & 3, NG))
               : *reinterpret_cast<const uint16_t*>(row + value_half(g, 2 * (c & 3), NG)) |
                     (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(
                          row + value_half(g, 2 * (c & 3) + 1, NG)))
                      << 16);
      const uint32_t pair = *reinterpret_cast<const uint32_t*>(
          block + a.c.page_size * (D / 2) + (off * NG + g) * 4);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = fmaf(static_cast<float>(static_cast<int>((codes >> (4 * e)) & 15u) - 8),
                    bf16_lo(pair), bf16_hi(pair));
      w = pack8(x);
    }
    __nv_bfloat16* dst = is_k ? a.k + t * a.k_st + h * a.k_sh : a.v + t * a.v_st + h * a.v_sh;
    *reinterpret_cast<uint4*>(dst + 8 * c) = w;
  }
}

// Head rows a block takes: all of a token's, or fewer when the tokens alone
// would leave SMs without blocks.
int rows_per_block(int64_t tokens, int rows, int rpw, int sms) {
  const int least = (kKvThreads / 32) * rpw;
  int chunk = rows;
  while (chunk > least && tokens * ((rows + chunk - 1) / chunk) < 8ll * sms)
    chunk = (chunk + 1) / 2;
  return chunk < least ? least : (chunk + rpw - 1) / rpw * rpw;
}

template <int D>
cudaError_t append_typed(const KvAppendArgs& a, cudaStream_t stream) {
  const int rows = a.heads + 2 * a.c.kv_heads;
  const int chunk = rows_per_block(a.tokens, rows, 32 / (D / 8), a.sms);
  const dim3 grid(static_cast<unsigned>(a.tokens), (rows + chunk - 1) / chunk);
  kv_append_kernel<D><<<grid, kKvThreads, 0, stream>>>(a, chunk);
  return cudaGetLastError();
}

template <int D>
cudaError_t gather_typed(const KvGatherArgs& a, cudaStream_t stream) {
  const int rows = 2 * a.c.kv_heads;
  const int chunk = rows_per_block(a.tokens, rows, 32 / (D / 8), a.sms);
  const dim3 grid(static_cast<unsigned>(a.tokens), (rows + chunk - 1) / chunk);
  kv_gather_kernel<D><<<grid, kKvThreads, 0, stream>>>(a, chunk);
  return cudaGetLastError();
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
