// Internal declarations shared by the translation units of libptb.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "ptb.h"

namespace ptb {

constexpr int kMaxDevices = 64;  // device ordinals that the library takes: 0 .. 63

// Launches `kern` so that it may start before the kernel in front of it in the stream has ended (see
// wait_for_prior, which it has to call).
template <typename... Args>
cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Epilogue of the tcgen05 GEMM.
enum GemmEpilogue : int {
  kEpiQkvGelu = 0,   // store bf16(acc); columns >= gelu_col store bf16(gelu_tanh(acc)) (and,
                     // with aux set, the pre-activation bf16(acc) at aux[row, col - gelu_col])
  kEpiResidual = 1,  // store bf16(acc + resid)
  kEpiDgelu = 2,     // columns >= gelu_col store bf16(acc * gelu_tanh'(aux[row, col - gelu_col])),
                     // the others bf16(acc)
  kEpiF32 = 3,       // store fp32 acc
  kEpiBf16 = 4,      // store bf16(acc), with resid set bf16(acc + resid)
  kEpiGated = 5,     // a tile holds block_n / 2 columns of the gate and the same of up: store
                     // bf16(act(gate) * up); with kept set, also gate and up themselves
  kEpiDgated = 6,    // acc is the gradient of act(gate) * up: store bf16(act(gate) * up) (out) and
                     // the gradients of gate and up (out1, two halves), gate and up from kept
};

// Activation of a gated feed-forward (ptb.h).
enum GatedActivation : int { kActSilu = 0, kActGelu = 1 };

// Operand layouts in shared memory (bit 0: A, bit 1: B).  K-major: the
// stored matrix is [M or N rows][K]; MN-major: it is [K rows][M or N], so the
// GEMM reads its transpose without a copy.
enum GemmLayout : int {
  kLayoutKK = 0,  // A K-major, B K-major
  kLayoutKN = 2,  // A K-major, B MN-major
  kLayoutNN = 3,  // A MN-major, B MN-major
};

// One GEMM launch: C[M, N] = A[M, K] * B[N, K]^T with A and B split into two
// tensor maps each.  Columns n < n_split read B from map b0 (index n), the
// rest from b1 (index n - n_split); inner indices k < k_split read A and B
// from a0/b0 (index k), the rest from a1/b1 (index k - k_split).  At most
// one of the two splits is active.  Maps of K-major operands are over
// [rows, K] (box 64 x 128 or 64 x block_n), maps of MN-major operands over
// [K, M or N] (box 64 x 64).
struct GemmArgs {
  CUtensorMap a0, a1, b0, b1;
  int M, N, K;
  int n_split, k_split;
  int block_n;  // 64, 128 or 256
  int layout;   // GemmLayout
  int n_fastest;  // tile order: 0 = M index fastest, 1 = N index fastest
  int a_keep, b_keep;  // L2 priority of the operand's loads: 1 evict_last, 0 evict_first
  int pair;  // 1: 256 x 256 tiles on CTA pairs (grid = 2 x pairs); bf16, K-major, block_n 256
  // Output: element (row, col) goes to out[row, col] (row stride ld_out),
  // except that columns >= out_split_col go to out1[row, col - out_split_col]
  // and rows >= out_split_row to out1[row - out_split_row, col] (row stride
  // ld_out1).  bf16 elements, fp32 for kEpiF32.
  void* out;
  int64_t ld_out;
  void* out1;
  int64_t ld_out1;
  int out_split_col, out_split_row;
  const __nv_bfloat16* resid;
  int64_t ld_resid;
  __nv_bfloat16* aux;  // kEpiQkvGelu: optional pre-activation out; kEpiDgelu: pre-activation in
  int64_t ld_aux;
  int gelu_col;
  int epilogue;
  int grid;  // persistent CTAs (<= number of SMs)
  unsigned* status;
  // K split of the last, partial wave (split_s < 2: no split).
  int split_r;          // remainder tiles that are split
  int split_s;          // pieces per remainder tile
  float* partials;      // [split_r * split_s] tiles of fp32
  unsigned* counters;   // [split_r][4 (8 for pairs) x gemm_counters] arrival counters
  int counters_zero;    // 0: the launch clears them first; 1: the caller has
  // e4m3 operands (fp8 != 0): K counted in e4m3 elements, 128 per k-block;
  // a_scale [M] and b_scale [N] dequantize the fp32 accumulator.
  int fp8;
  const float* a_scale;
  const float* b_scale;
  // Gated epilogues: gate and up of each row, [M, 2 ffn], gate first: bf16, or, with kept_exps
  // set, a checkpoint's codes and exponents.
  int act;
  int ffn;
  int wide;  // kEpiBf16: every output row begins on 32 bytes
  void* kept;
  uint8_t* kept_exps;
};

// Each K piece of a split tile keeps at least this many 64-wide k-blocks.
constexpr int kMinSplitKBlocks = 8;

struct GemmPlan {
  int grid, split_r, split_s;
  size_t partial_bytes, counter_bytes;
};

// Grid and K split for `tiles` output tiles of `num_kb` k-blocks on `sms`
// SMs: whole waves of tiles, then the remainder tiles split along K over the
// SMs the last wave would leave idle.
// `workers` is the number of CTAs (or CTA pairs), `rows` the tile height
// (128, or 256 for pairs).
// `counters`: arrival counters for 32 rows (gemm_counters of the epilogue).
// `most_s` caps the pieces of a tile.
GemmPlan plan_gemm(int64_t tiles, int64_t num_kb, int workers, int block_n, int rows = 128,
                   int counters = 1, int most_s = 1 << 30);
int gemm_counters(int epilogue);

struct SwaArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  int64_t q_sb, q_sh, q_ss, k_sb, k_sh, k_ss, v_sb, v_sh, v_ss, o_sb, o_sh, o_ss;
  int batch, heads, seq, head_dim, window;
  float scale_log2;  // softmax scale * log2(e)
  int* counts;       // optional per-row attended-key counts
  float* lse;        // optional [batch][heads][seq]: log2 of row i's softmax denominator in
                     // base-2 units, log2(sum_j 2^(q_i.k_j * scale * log2 e))
  unsigned* status;  // device status word (bounded waits record timeouts here)
  int sms;           // SMs of the device (persistent grid size)
};

// Backward of causal SWA over strided [batch][heads][seq][head_dim] bf16 views
// (element (b, h, i, c) at base + b*sb + h*sh + i*ss + c).
struct SwaBwdArgs {
  const __nv_bfloat16 *q, *k, *v, *o, *dout;
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t q_sb, q_sh, q_ss, k_sb, k_sh, k_ss, v_sb, v_sh, v_ss, o_sb, o_sh, o_ss;
  int64_t do_sb, do_sh, do_ss, dq_sb, dq_sh, dq_ss, dk_sb, dk_sh, dk_ss, dv_sb, dv_sh, dv_ss;
  const float* lse;  // [batch][heads][seq], as SwaArgs::lse of the forward pass
  float* delta;      // [batch][heads][seq] scratch: sum_c dO * o per row
  int batch, heads, seq, head_dim, window;
  float scale, scale_log2;  // softmax scale, and scale * log2(e)
  unsigned* status;
  int sms;
};

// Encodes a bf16 tiled tensor map with 128-byte swizzle (rank <= 5; dims and
// strides innermost first, strides in bytes for dims 1..rank-1).  Needs the
// driver entry point, which the per-device set-up of the C ABI loads.
bool make_tensor_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                     const uint64_t* strides_bytes, const uint32_t* box);

// ------------------------------------------------------------- serving --

// The paged cache of keys and values (layout: ptb.h).
struct KvCache {
  uint8_t* base;
  int64_t pages, page_bytes;  // page_bytes = 2 * kv_heads * block_bytes
  int64_t block_bytes;        // one kv head's keys or values of one page
  const int32_t* table;       // [batch][table_stride], table_pages entries used
  int64_t table_stride, table_pages;
  int page_size, page_shift, kv_heads, head_dim, bits;
};

struct KvAppendArgs {
  KvCache c;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_out;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh, ko_st, ko_sh;
  const float *cos, *sin;
  int64_t positions;
  int rot_dim, interleaved;
  const int32_t *cu, *past;
  int batch, heads;
  int64_t tokens;
  unsigned* status;
  int sms;
};

struct KvGatherArgs {
  KvCache c;
  __nv_bfloat16 *k, *v;
  int64_t k_st, k_sh, v_st, v_sh;
  const int32_t *cu, *start;
  int batch;
  int64_t tokens;
  unsigned* status;
  int sms;
};

struct SwaPackedArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;
  const int32_t *cu_q, *cu_k;
  int batch, heads, kv_heads, head_dim, window;
  int64_t tokens_q, tokens_k;
  float scale_log2;
  void* workspace;
  unsigned* status;
  int sms;
};

struct SwaPagedArgs {
  KvCache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  int64_t q_sb, q_sh, o_sb, o_sh;
  const int32_t* lens;
  int batch, heads, window;
  float scale_log2;
  void* workspace;
  unsigned* status;
  int sms;
};

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv_gather(const KvGatherArgs& a, cudaStream_t stream);
size_t swa_packed_workspace(int batch, int64_t tokens_q, int heads, int kv_heads, int sms);
cudaError_t launch_swa_packed(const SwaPackedArgs& a, cudaStream_t stream);
size_t swa_paged_workspace(int batch, int heads, int kv_heads, int head_dim, int sms);
cudaError_t launch_swa_paged(const SwaPagedArgs& a, cudaStream_t stream);

// -------------------------------------------- blocks with gates and norms --

// out[t, n] = act(x w0^T) * (x w1^T), or without w1 [resid +] x w0^T, for at most kThinTokens rows of
// x; weights [N, K], K a multiple of 64, N of 16.
constexpr int kThinTokens = 32;
struct ThinArgs {
  const __nv_bfloat16 *x, *w0, *w1, *resid;
  __nv_bfloat16* out;
  int64_t ld_x, ld_resid, ld_out;
  int tokens, N, K, act, sms;
};

struct CheckpointArgs {
  const __nv_bfloat16* x;   // pack
  __nv_bfloat16* x_out;     // unpack
  uint8_t *codes, *exps;
  int64_t ld_x, ld_codes, ld_exps;
  int64_t rows, cols;
  int sms;
};

// y = alpha x + gate * N(o), h = N(y) (ptb_norm_residual), and its backward.
struct NormArgs {
  const __nv_bfloat16 *x, *o;
  int64_t ld_x, ld_o;
  const uint8_t* o_exps;  // backward: not null when o is a checkpoint's codes
  int64_t ld_o_exps;
  const __nv_bfloat16 *post_gamma, *post_beta, *pre_gamma, *pre_beta;
  const __nv_bfloat16* gate;
  int64_t gates;
  float alpha, eps;
  int rms;
  int64_t rows;
  int hidden;
  __nv_bfloat16 *y, *h;  // forward
  int64_t ld_y, ld_h;
  float4* stats;         // (mean, 1/sd) of o and of y, per row
  // backward
  const __nv_bfloat16 *dy, *dh;
  int64_t ld_dy, ld_dh;
  __nv_bfloat16 *dx, *d_o;
  int64_t ld_dx, ld_do;
  float *dpost_gamma, *dpost_beta, *dgate, *dpre_gamma, *dpre_beta;
  float* partials;
  unsigned* status;
  int sms;
};

cudaError_t launch_checkpoint_pack(const CheckpointArgs& a, cudaStream_t stream);
cudaError_t launch_checkpoint_unpack(const CheckpointArgs& a, cudaStream_t stream);
cudaError_t launch_thin(const ThinArgs& a, cudaStream_t stream);
cudaError_t launch_norm_residual(const NormArgs& a, cudaStream_t stream);
// Bytes of NormArgs::partials.
size_t norm_backward_partials(int64_t rows, int64_t hidden, int64_t gates, int sms);
cudaError_t launch_norm_residual_backward(const NormArgs& a, cudaStream_t stream);

cudaError_t launch_gemm(const GemmArgs& a, cudaStream_t stream);
cudaError_t launch_layernorm(const __nv_bfloat16* x, const __nv_bfloat16* gamma,
                             const __nv_bfloat16* beta, int64_t rows, int hidden, float eps,
                             __nv_bfloat16* out, cudaStream_t stream, float2* stats = nullptr);
// Backward of the LayerNorm plus the residual path of the block:
//   dx = dy + r * (g - mean(g) - xh * mean(g * xh)),  g = dxn * gamma,
//   xh = (x - mean) * r, with (mean, r) from the forward pass's stats;
//   dgamma = sum over rows of dxn * xh,  dbeta = sum over rows of dxn.
// `partials` holds 2 * hidden * ln_backward_chunks(rows) floats.
int64_t ln_backward_chunks(int64_t rows);
cudaError_t launch_layernorm_backward(const __nv_bfloat16* x, const __nv_bfloat16* gamma,
                                      const float2* stats, const float* dxn,
                                      const __nv_bfloat16* dy, int64_t rows, int hidden,
                                      __nv_bfloat16* dx, float* dgamma, float* dbeta,
                                      float* partials, cudaStream_t stream);
cudaError_t launch_swa_backward(const SwaBwdArgs& a, cudaStream_t stream);
cudaError_t launch_swa(const SwaArgs& a, cudaStream_t stream);
cudaError_t launch_layernorm_fp8(const __nv_bfloat16* x, const __nv_bfloat16* gamma,
                                 const __nv_bfloat16* beta, int64_t rows, int hidden, float eps,
                                 uint8_t* out, float* scale, cudaStream_t stream);
cudaError_t launch_quantize_rows(const __nv_bfloat16* src0, int64_t ld0, int n0,
                                 const __nv_bfloat16* src1, int64_t ld1, int n1, int64_t rows,
                                 int64_t row0, uint8_t* out, float* scale, cudaStream_t stream);
cudaError_t launch_wait_probe(uint64_t limit_ns, unsigned* status, cudaStream_t stream);

}  // namespace ptb
