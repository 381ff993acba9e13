// C ABI of libptb, the parts of blocks with a gated feed-forward: the feed-forward with its
// backward pass, the norms before and after a block with its gate and residual scale, and the
// 8-bit activation checkpoints (declared in include/ptb.h).
#include <cmath>
#include <cstring>

#include "api_internal.h"

using namespace ptb;
using namespace ptb::api;

namespace {

constexpr int64_t kMaxRows = 1ll << 30;

#define PTB_TRY(expr)                   \
  do {                                  \
    const ptb_status st_ = (expr);      \
    if (st_ != PTB_OK) return st_;      \
  } while (0)

// A matrix of `rows` rows of `cols` elements; `unit` elements are 16 bytes.  A single row has no stride.
ptb_status check_rows(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t unit) {
  if (rows == 0) return PTB_OK;
  if (!p) return PTB_ERR_ARG;
  if (rows > 1 && ld < cols) return PTB_ERR_ARG;
  if (!aligned(p, 16) || (rows > 1 && ld % unit)) return PTB_ERR_ALIGN;
  return PTB_OK;
}

// A vector of parameters that may be absent.
ptb_status check_vector(const void* p) { return aligned(p, 16) ? PTB_OK : PTB_ERR_ALIGN; }

ptb_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!need) return PTB_OK;
  if (!workspace) return PTB_ERR_ARG;
  if (bytes < need) return PTB_ERR_WORKSPACE;
  return aligned(workspace, kAlign) ? PTB_OK : PTB_ERR_ALIGN;
}

ptb_status check_checkpoint(const void* codes, int64_t ld_codes, const uint8_t* exps,
                            int64_t ld_exps, int64_t rows, int64_t cols) {
  if (rows == 0) return PTB_OK;
  if (!exps || (rows > 1 && ld_exps < cols / 32)) return PTB_ERR_ARG;
  return check_rows(codes, ld_codes, rows, cols, 16);
}

// ---------------------------------------------------------- gated GEMMs --

GemmCall call_up(int64_t t, int64_t h, int64_t f) {  // [gate | up] = x [W_gate ; W_up]^T
  GemmCall c;
  c.layout = kLayoutKK;
  c.epilogue = kEpiGated, c.ragged = true;
  c.M = t, c.N = 2 * f, c.K = h;
  c.lda0 = h, c.ldb0 = h;
  c.ld_out = f, c.ffn = f;
  return c;
}
GemmCall call_da(int64_t t, int64_t h, int64_t f) {  // da = dy W_down
  GemmCall c;
  c.layout = kLayoutKN;
  c.epilogue = kEpiDgated, c.ragged = true;
  c.M = t, c.N = f, c.K = h;
  c.lda0 = h, c.ldb0 = f;
  c.ld_out = f, c.ld_out1 = 2 * f, c.ffn = f;
  return c;
}
GemmCall call_dw_down(int64_t t, int64_t h, int64_t f, int bits) {  // dy^T a
  GemmCall c;
  c.layout = kLayoutNN;
  c.epilogue = bits == 32 ? kEpiF32 : kEpiBf16, c.ragged = true;
  c.M = h, c.N = f, c.K = t;
  c.lda0 = h, c.ldb0 = f, c.ld_out = f;
  return c;
}
GemmCall call_dw_up(int64_t t, int64_t h, int64_t f, int bits) {  // [dg | du]^T x
  GemmCall c;
  c.layout = kLayoutNN;
  c.epilogue = bits == 32 ? kEpiF32 : kEpiBf16, c.ragged = true;
  c.M = 2 * f, c.N = h, c.K = t;
  c.lda0 = 2 * f, c.ldb0 = h, c.ld_out = h, c.ld_out1 = h;
  c.out_split_row = f;
  return c;
}
GemmCall call_dx(int64_t t, int64_t h, int64_t f) {  // dg W_gate + du W_up
  GemmCall c;
  c.layout = kLayoutKN;
  c.epilogue = kEpiBf16, c.ragged = true;
  c.M = t, c.N = h, c.K = 2 * f, c.k_split = f;
  c.lda0 = 2 * f, c.lda1 = 2 * f, c.ldb0 = h, c.ldb1 = h, c.ld_out = h;
  return c;
}

GemmCall call_down(int64_t t, int64_t h, int64_t f) {  // a W_down^T
  GemmCall c;
  c.layout = kLayoutKK;
  c.epilogue = kEpiBf16, c.ragged = true;
  c.M = t, c.N = h, c.K = f;
  c.lda0 = f, c.ldb0 = f, c.ld_out = h;
  return c;
}

struct Regions {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t at = off;
    off += round_up(bytes, kAlign);
    return at;
  }
};

// Few tokens go through the kernel that streams the weights.  Every block of it reads all of x, which
// from 17 tokens on costs more than the tiles of the other kernel, unless there is little to stream: 24
// tokens, hidden 2048, ffn 5440 26 us and 34, 4096 and 11008 63 both, 5120 and 13824 91 and 86.
bool thin(int64_t tokens, int64_t hidden, int64_t ffn) {
  return tokens <= kThinTokens / 2 || (tokens <= kThinTokens && hidden * ffn < 40'000'000);
}

// The GEMMs of a call have arrival counters of their own, which one memset clears: a memset in front of
// each was a fifth of the nodes of a small call's graph.
struct ForwardLayout {
  size_t a, gemm, gemm_bytes, counters[2], total;
};

ForwardLayout forward_layout(int64_t t, int64_t h, int64_t f, int sms) {
  ForwardLayout l;
  Regions r;
  const CallSizes up = call_sizes(call_up(t, h, f), sms), down = call_sizes(call_down(t, h, f), sms);
  l.a = r.take(static_cast<size_t>(t) * f * 2);
  l.gemm_bytes = up.scratch > down.scratch ? up.scratch : down.scratch;
  l.gemm = r.take(l.gemm_bytes);
  l.counters[0] = r.take(up.counters);
  l.counters[1] = r.take(down.counters);
  l.total = r.off;
  return l;
}

struct BackwardLayout {
  size_t a, dgu, x, gemm, gemm_bytes, counters[4], total;
};

BackwardLayout backward_layout(int64_t t, int64_t h, int64_t f, bool x8, int bits, int sms) {
  BackwardLayout l;
  Regions r;
  l.a = r.take(static_cast<size_t>(t) * f * 2);
  l.dgu = r.take(static_cast<size_t>(t) * f * 4);
  l.x = r.take(x8 ? static_cast<size_t>(t) * h * 2 : 0);
  l.gemm_bytes = 0;
  const CallSizes sizes[] = {call_sizes(call_da(t, h, f), sms), call_sizes(call_dw_down(t, h, f, bits), sms),
                             call_sizes(call_dw_up(t, h, f, bits), sms), call_sizes(call_dx(t, h, f), sms)};
  for (const CallSizes& s : sizes) l.gemm_bytes = s.scratch > l.gemm_bytes ? s.scratch : l.gemm_bytes;
  l.gemm = r.take(l.gemm_bytes);
  for (int k = 0; k < 4; ++k) l.counters[k] = r.take(sizes[k].counters);
  l.total = r.off;
  return l;
}

// Clears the counters of a layout from `first` to its end; their place in it, for GEMM k.
ptb_status clear_counters(char* ws, size_t first, size_t total, cudaStream_t stream) {
  if (total == first) return PTB_OK;
  return launch_status(cudaMemsetAsync(ws + first, 0, total - first, stream));
}
unsigned* counters_at(char* ws, size_t at) { return reinterpret_cast<unsigned*>(ws + at); }

bool gated_shape_ok(int64_t tokens, int64_t hidden, int64_t ffn) {
  return tokens > 0 && check_gemm_shape(tokens, hidden, ffn) == PTB_OK && 2 * ffn <= kMaxRows;
}

ptb_status check_gated(int64_t tokens, int64_t hidden, int64_t ffn, int32_t activation) {
  if (tokens < 0 || (activation != kActSilu && activation != kActGelu)) return PTB_ERR_ARG;
  PTB_TRY(check_gemm_shape(tokens ? tokens : 1, hidden, ffn));
  return 2 * ffn <= kMaxRows ? PTB_OK : PTB_ERR_SHAPE;
}

}  // namespace

extern "C" {

size_t ptb_gated_ffn_workspace_size(int64_t tokens, int64_t hidden, int64_t ffn) {
  if (!gated_shape_ok(tokens, hidden, ffn)) return 0;
  return forward_layout(tokens, hidden, ffn, current_sms()).total;
}

ptb_status ptb_gated_ffn(const ptb_bf16* x, int64_t ld_x, const ptb_bf16* w_gate,
                         const ptb_bf16* w_up, const ptb_bf16* w_down, const ptb_bf16* residual,
                         int64_t ld_residual, int64_t tokens, int64_t hidden, int64_t ffn,
                         int32_t activation, ptb_bf16* y, int64_t ld_y, void* kept,
                         uint8_t* kept_exps, void* workspace, size_t workspace_bytes,
                         ptb_stream stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (!w_gate || !w_up || !w_down || (kept_exps && !kept)) return PTB_ERR_ARG;
  PTB_TRY(check_gated(tokens, hidden, ffn, activation));
  if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || !aligned(kept, 16))
    return PTB_ERR_ALIGN;
  PTB_TRY(check_rows(x, ld_x, tokens, hidden, 8));
  PTB_TRY(check_rows(y, ld_y, tokens, hidden, 8));
  if (residual) PTB_TRY(check_rows(residual, ld_residual, tokens, hidden, 8));
  if (tokens == 1) ld_x = ld_y = ld_residual = hidden;  // not used, but tensor maps want one
  if (y && y == residual && ld_y != ld_residual) return PTB_ERR_ARG;
  const size_t need = ptb_gated_ffn_workspace_size(tokens, hidden, ffn);
  PTB_TRY(check_workspace(workspace, workspace_bytes, need));
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (tokens == 0) return PTB_OK;
  const ForwardLayout l = forward_layout(tokens, hidden, ffn, ds->sms);
  char* ws = static_cast<char*>(workspace);
  ptb_bf16* a = reinterpret_cast<ptb_bf16*>(ws + l.a);
  if (thin(tokens, hidden, ffn) && !kept) {
    ThinArgs n;
    std::memset(&n, 0, sizeof(n));
    n.x = bf(x), n.ld_x = ld_x;
    n.w0 = bf(w_gate), n.w1 = bf(w_up);
    n.out = bf(a), n.ld_out = ffn;
    n.tokens = static_cast<int>(tokens), n.N = static_cast<int>(ffn), n.K = static_cast<int>(hidden);
    n.act = activation, n.sms = ds->sms;
    PTB_TRY(launch_status(launch_thin(n, stream)));
    n.x = bf(a), n.ld_x = ffn;
    n.w0 = bf(w_down), n.w1 = nullptr;
    n.resid = bf(residual), n.ld_resid = ld_residual;
    n.out = bf(y), n.ld_out = ld_y;
    n.N = static_cast<int>(hidden), n.K = static_cast<int>(ffn);
    return launch_status(launch_thin(n, stream));
  }
  // 1. a = act(x W_gate^T) * (x W_up^T)
  PTB_TRY(clear_counters(ws, l.counters[0], l.total, stream));
  GemmCall c = call_up(tokens, hidden, ffn);
  c.counters = counters_at(ws, l.counters[0]);
  c.a0 = x, c.lda0 = ld_x, c.b0 = w_gate, c.b1 = w_up;
  c.out = a;
  c.act = activation;
  c.kept = kept, c.kept_exps = kept_exps;
  PTB_TRY(gemm_call(ds, c, ws + l.gemm, l.gemm_bytes, stream));
  // 2. y = [residual +] a W_down^T
  c = call_down(tokens, hidden, ffn);
  c.counters = counters_at(ws, l.counters[1]);
  c.a0 = a, c.b0 = w_down;
  c.out = y, c.ld_out = ld_y;
  c.resid = residual, c.ld_resid = ld_residual;
  return gemm_call(ds, c, ws + l.gemm, l.gemm_bytes, stream);
}

size_t ptb_gated_ffn_backward_workspace_size(int64_t tokens, int64_t hidden, int64_t ffn,
                                             int32_t x_bits) {
  if (!gated_shape_ok(tokens, hidden, ffn) || (x_bits != 16 && x_bits != 8)) return 0;
  const int sms = current_sms();
  const size_t a = backward_layout(tokens, hidden, ffn, x_bits == 8, 16, sms).total;
  const size_t b = backward_layout(tokens, hidden, ffn, x_bits == 8, 32, sms).total;
  return a > b ? a : b;
}

ptb_status ptb_gated_ffn_backward(const ptb_bf16* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                  const uint8_t* x_exps, int64_t ld_x_exps,
                                  const ptb_bf16* w_gate, const ptb_bf16* w_up,
                                  const ptb_bf16* w_down, const void* kept,
                                  const uint8_t* kept_exps, int64_t tokens, int64_t hidden,
                                  int64_t ffn, int32_t activation, ptb_bf16* dx, int64_t ld_dx,
                                  void* dw_gate, void* dw_up, void* dw_down, int32_t grad_bits,
                                  void* workspace, size_t workspace_bytes, ptb_stream stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (!w_gate || !w_up || !w_down || !dw_gate || !dw_up || !dw_down) return PTB_ERR_ARG;
  if ((tokens > 0 && !kept) || (grad_bits != 16 && grad_bits != 32)) return PTB_ERR_ARG;
  PTB_TRY(check_gated(tokens, hidden, ffn, activation));
  const void* ptrs[] = {w_gate, w_up, w_down, dw_gate, dw_up, dw_down, kept};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return PTB_ERR_ALIGN;
  PTB_TRY(check_rows(dy, ld_dy, tokens, hidden, 8));
  PTB_TRY(check_rows(dx, ld_dx, tokens, hidden, 8));
  if (x_exps)
    PTB_TRY(check_checkpoint(x, ld_x, x_exps, ld_x_exps, tokens, hidden));
  else
    PTB_TRY(check_rows(x, ld_x, tokens, hidden, 8));
  const size_t need = ptb_gated_ffn_backward_workspace_size(tokens, hidden, ffn, x_exps ? 8 : 16);
  PTB_TRY(check_workspace(workspace, workspace_bytes, need));
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (tokens == 0) {  // sums over no token
    const size_t bytes = static_cast<size_t>(hidden) * ffn * (grad_bits / 8);
    for (void* p : {dw_gate, dw_up, dw_down})
      PTB_TRY(launch_status(cudaMemsetAsync(p, 0, bytes, stream)));
    return PTB_OK;
  }
  if (tokens == 1) {  // not used, but tensor maps want one
    ld_dy = ld_dx = hidden;
    if (!x_exps) ld_x = hidden;
  }
  const BackwardLayout l =
      backward_layout(tokens, hidden, ffn, x_exps != nullptr, grad_bits, ds->sms);
  char* ws = static_cast<char*>(workspace);
  ptb_bf16* a = reinterpret_cast<ptb_bf16*>(ws + l.a);
  ptb_bf16* dgu = reinterpret_cast<ptb_bf16*>(ws + l.dgu);
  void* scratch = ws + l.gemm;
  const ptb_bf16* xb = static_cast<const ptb_bf16*>(x);
  if (x_exps) {  // the weight gradients' GEMM reads bf16, which is what the codes stand for
    CheckpointArgs u;
    std::memset(&u, 0, sizeof(u));
    u.codes = static_cast<uint8_t*>(const_cast<void*>(x));
    u.exps = const_cast<uint8_t*>(x_exps);
    u.ld_codes = ld_x, u.ld_exps = ld_x_exps;
    u.x_out = reinterpret_cast<__nv_bfloat16*>(ws + l.x);
    u.ld_x = hidden;
    u.rows = tokens, u.cols = hidden;
    u.sms = ds->sms;
    PTB_TRY(launch_status(launch_checkpoint_unpack(u, stream)));
    xb = reinterpret_cast<const ptb_bf16*>(ws + l.x);
    ld_x = hidden;
  }
  // 1. da = dy W_down; a, [dg | du] from it and the kept gate and up
  PTB_TRY(clear_counters(ws, l.counters[0], l.total, stream));
  GemmCall c = call_da(tokens, hidden, ffn);
  c.counters = counters_at(ws, l.counters[0]);
  c.a0 = dy, c.lda0 = ld_dy, c.b0 = w_down;
  c.out = a, c.out1 = dgu;
  c.act = activation;
  c.kept = const_cast<void*>(kept), c.kept_exps = const_cast<uint8_t*>(kept_exps);
  PTB_TRY(gemm_call(ds, c, scratch, l.gemm_bytes, stream));
  // 2. dW_down = dy^T a
  c = call_dw_down(tokens, hidden, ffn, grad_bits);
  c.counters = counters_at(ws, l.counters[1]);
  c.a0 = dy, c.lda0 = ld_dy, c.b0 = a;
  c.out = dw_down;
  PTB_TRY(gemm_call(ds, c, scratch, l.gemm_bytes, stream));
  // 3. [dW_gate ; dW_up] = [dg | du]^T x
  c = call_dw_up(tokens, hidden, ffn, grad_bits);
  c.counters = counters_at(ws, l.counters[2]);
  c.a0 = dgu, c.b0 = xb, c.ldb0 = ld_x;
  c.out = dw_gate, c.out1 = dw_up;
  PTB_TRY(gemm_call(ds, c, scratch, l.gemm_bytes, stream));
  // 4. dx = dg W_gate + du W_up: the last, so that dx may be dy or x
  c = call_dx(tokens, hidden, ffn);
  c.counters = counters_at(ws, l.counters[3]);
  c.a0 = dgu, c.a1 = dgu + ffn, c.b0 = w_gate, c.b1 = w_up;
  c.out = dx, c.ld_out = ld_dx;
  return gemm_call(ds, c, scratch, l.gemm_bytes, stream);
}

// ------------------------------------------------------------ the norms --

ptb_status ptb_norm_residual(const ptb_bf16* x, int64_t ld_x, const ptb_bf16* o, int64_t ld_o,
                             const ptb_bf16* post_gamma, const ptb_bf16* post_beta,
                             const ptb_bf16* gate, int64_t gates, float alpha,
                             const ptb_bf16* pre_gamma, const ptb_bf16* pre_beta, int32_t rms,
                             float eps, int64_t rows, int64_t hidden, ptb_bf16* y, int64_t ld_y,
                             ptb_bf16* h, int64_t ld_h, float* stats, ptb_stream stream) {
  if (rows < 0 || hidden < 1 || gates < 1 || (rms != 0 && rms != 1)) return PTB_ERR_ARG;
  if ((post_beta && !post_gamma) || (pre_beta && !pre_gamma) || (rms && (post_beta || pre_beta)))
    return PTB_ERR_ARG;
  if (rows > 0 && (h != nullptr) != (pre_gamma != nullptr)) return PTB_ERR_ARG;
  if (!std::isfinite(alpha) || !std::isfinite(eps) || eps <= 0.f) return PTB_ERR_ARG;
  if (hidden % 8 || hidden > 32768 || rows > kMaxRows || gates > 65533 || rows % gates)
    return PTB_ERR_SHAPE;
  PTB_TRY(check_rows(x, ld_x, rows, hidden, 8));
  PTB_TRY(check_rows(o, ld_o, rows, hidden, 8));
  PTB_TRY(check_rows(y, ld_y, rows, hidden, 8));
  if (h) PTB_TRY(check_rows(h, ld_h, rows, hidden, 8));
  for (const void* p : {post_gamma, post_beta, pre_gamma, pre_beta, gate}) PTB_TRY(check_vector(p));
  PTB_TRY(check_vector(stats));
  if (rows == 1) ld_x = ld_o = ld_y = ld_h = hidden;  // not used
  if (rows > 0 && (h == y || (y == x && ld_y != ld_x) || (y == o && ld_y != ld_o) ||
                   (h && h == x && ld_h != ld_x) || (h && h == o && ld_h != ld_o)))
    return PTB_ERR_ARG;
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (rows == 0) return PTB_OK;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = bf(x), a.ld_x = ld_x, a.o = bf(o), a.ld_o = ld_o;
  a.post_gamma = bf(post_gamma), a.post_beta = bf(post_beta);
  a.pre_gamma = bf(pre_gamma), a.pre_beta = bf(pre_beta);
  a.gate = bf(gate), a.gates = gates;
  a.alpha = alpha, a.eps = eps, a.rms = rms;
  a.rows = rows, a.hidden = static_cast<int>(hidden);
  a.y = bf(y), a.ld_y = ld_y, a.h = bf(h), a.ld_h = ld_h;
  a.stats = reinterpret_cast<float4*>(stats);
  a.sms = ds->sms;
  return launch_status(launch_norm_residual(a, static_cast<cudaStream_t>(stream)));
}

size_t ptb_norm_residual_backward_workspace_size(int64_t rows, int64_t hidden, int64_t gates) {
  if (rows < 1 || rows > kMaxRows || hidden < 1 || hidden % 8 || hidden > 32768 || gates < 1 ||
      gates > 65533 || rows % gates)
    return 0;
  return round_up(norm_backward_partials(rows, hidden, gates, current_sms()), kAlign);
}

ptb_status ptb_norm_residual_backward(
    const ptb_bf16* dy, int64_t ld_dy, const ptb_bf16* dh, int64_t ld_dh, const ptb_bf16* y,
    int64_t ld_y, const void* o, int64_t ld_o, const uint8_t* o_exps, int64_t ld_o_exps,
    const float* stats, const ptb_bf16* post_gamma, const ptb_bf16* post_beta,
    const ptb_bf16* gate, int64_t gates, float alpha, const ptb_bf16* pre_gamma, int32_t rms,
    int64_t rows, int64_t hidden, ptb_bf16* dx, int64_t ld_dx, ptb_bf16* d_o, int64_t ld_do,
    float* dpost_gamma, float* dpost_beta, float* dgate, float* dpre_gamma, float* dpre_beta,
    void* workspace, size_t workspace_bytes, ptb_stream stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (rows < 0 || hidden < 1 || gates < 1 || (rms != 0 && rms != 1)) return PTB_ERR_ARG;
  if ((post_beta && !post_gamma) || (rms && (post_beta || dpost_beta || dpre_beta)))
    return PTB_ERR_ARG;
  if ((dpost_gamma && !post_gamma) || (dpost_beta && !post_gamma) || (dgate && !gate) ||
      ((dpre_gamma || dpre_beta) && !pre_gamma))
    return PTB_ERR_ARG;
  if (rows > 0 && ((dh != nullptr) != (pre_gamma != nullptr) || (!dy && !dh) || !stats))
    return PTB_ERR_ARG;
  if (!std::isfinite(alpha)) return PTB_ERR_ARG;
  if (hidden % 8 || hidden > 32768 || rows > kMaxRows || gates > 65533 || rows % gates ||
      (o_exps && hidden % 32))
    return PTB_ERR_SHAPE;
  if (dy) PTB_TRY(check_rows(dy, ld_dy, rows, hidden, 8));
  if (dh) PTB_TRY(check_rows(dh, ld_dh, rows, hidden, 8));
  if (dh) PTB_TRY(check_rows(y, ld_y, rows, hidden, 8));
  if (o_exps)
    PTB_TRY(check_checkpoint(o, ld_o, o_exps, ld_o_exps, rows, hidden));
  else
    PTB_TRY(check_rows(o, ld_o, rows, hidden, 8));
  PTB_TRY(check_rows(dx, ld_dx, rows, hidden, 8));
  PTB_TRY(check_rows(d_o, ld_do, rows, hidden, 8));
  for (const void* p : {post_gamma, post_beta, gate, pre_gamma}) PTB_TRY(check_vector(p));
  PTB_TRY(check_vector(stats));
  for (const float* p : {dpost_gamma, dpost_beta, dgate, dpre_gamma, dpre_beta})
    if (!aligned(p, 4)) return PTB_ERR_ALIGN;
  if (rows > 0 && dx == d_o) return PTB_ERR_ARG;
  if (rows == 1) {  // not used
    ld_dy = ld_dh = ld_y = ld_o = ld_dx = ld_do = hidden;
    ld_o_exps = hidden / 32;
  }
  // In place: a row's gradients may replace what they were computed from, at the same strides.
  const struct {
    const void* p;
    int64_t ld;
  } ins[] = {{dy, ld_dy}, {dh, ld_dh}, {y, ld_y}, {o, o_exps ? -1 : ld_o}};
  for (const auto& i : ins)
    if (rows > 0 && i.p && ((i.p == dx && i.ld != ld_dx) || (i.p == d_o && i.ld != ld_do)))
      return PTB_ERR_ARG;
  const size_t need = ptb_norm_residual_backward_workspace_size(rows, hidden, gates);
  PTB_TRY(check_workspace(workspace, workspace_bytes, need));
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (rows == 0) {  // sums over no row
    for (float* p : {dpost_gamma, dpost_beta, dpre_gamma, dpre_beta})
      if (p) PTB_TRY(launch_status(cudaMemsetAsync(p, 0, hidden * 4, stream)));
    if (dgate) PTB_TRY(launch_status(cudaMemsetAsync(dgate, 0, gates * hidden * 4, stream)));
    return PTB_OK;
  }
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dy = bf(dy), a.ld_dy = ld_dy, a.dh = bf(dh), a.ld_dh = ld_dh;
  a.y = const_cast<__nv_bfloat16*>(bf(y)), a.ld_y = ld_y;
  a.o = static_cast<const __nv_bfloat16*>(o), a.ld_o = ld_o;
  a.o_exps = o_exps, a.ld_o_exps = ld_o_exps;
  a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
  a.post_gamma = bf(post_gamma), a.post_beta = bf(post_beta), a.pre_gamma = bf(pre_gamma);
  a.gate = bf(gate), a.gates = gate ? gates : 1;  // without a gate there is nothing to sum by gates
  a.alpha = alpha, a.rms = rms;
  a.rows = rows, a.hidden = static_cast<int>(hidden);
  a.dx = bf(dx), a.ld_dx = ld_dx, a.d_o = bf(d_o), a.ld_do = ld_do;
  a.dpost_gamma = dpost_gamma, a.dpost_beta = dpost_beta, a.dgate = dgate;
  a.dpre_gamma = dpre_gamma, a.dpre_beta = dpre_beta;
  a.partials = static_cast<float*>(workspace);
  a.status = ds->status;
  a.sms = ds->sms;
  return launch_status(launch_norm_residual_backward(a, stream));
}

// ------------------------------------------------------ 8-bit checkpoints --

ptb_status ptb_checkpoint_pack(const ptb_bf16* x, int64_t ld_x, int64_t rows, int64_t cols,
                               void* codes, int64_t ld_codes, uint8_t* exps, int64_t ld_exps,
                               ptb_stream stream) {
  if (rows < 0 || cols < 1) return PTB_ERR_ARG;
  if (cols % 32 || cols > kMaxRows || rows > kMaxRows) return PTB_ERR_SHAPE;
  PTB_TRY(check_rows(x, ld_x, rows, cols, 8));
  PTB_TRY(check_checkpoint(codes, ld_codes, exps, ld_exps, rows, cols));
  if (rows > 0 && static_cast<const void*>(x) == codes) return PTB_ERR_ARG;
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (rows == 0) return PTB_OK;
  CheckpointArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = bf(x), a.ld_x = ld_x;
  a.codes = static_cast<uint8_t*>(codes), a.ld_codes = ld_codes;
  a.exps = exps, a.ld_exps = ld_exps;
  a.rows = rows, a.cols = cols, a.sms = ds->sms;
  return launch_status(launch_checkpoint_pack(a, static_cast<cudaStream_t>(stream)));
}

ptb_status ptb_checkpoint_unpack(const void* codes, int64_t ld_codes, const uint8_t* exps,
                                 int64_t ld_exps, int64_t rows, int64_t cols, ptb_bf16* x,
                                 int64_t ld_x, ptb_stream stream) {
  if (rows < 0 || cols < 1) return PTB_ERR_ARG;
  if (cols % 32 || cols > kMaxRows || rows > kMaxRows) return PTB_ERR_SHAPE;
  PTB_TRY(check_rows(x, ld_x, rows, cols, 8));
  PTB_TRY(check_checkpoint(codes, ld_codes, exps, ld_exps, rows, cols));
  if (rows > 0 && static_cast<const void*>(x) == codes) return PTB_ERR_ARG;
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (rows == 0) return PTB_OK;
  CheckpointArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x_out = bf(x), a.ld_x = ld_x;
  a.codes = static_cast<uint8_t*>(const_cast<void*>(codes)), a.ld_codes = ld_codes;
  a.exps = const_cast<uint8_t*>(exps), a.ld_exps = ld_exps;
  a.rows = rows, a.cols = cols, a.sms = ds->sms;
  return launch_status(launch_checkpoint_unpack(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
