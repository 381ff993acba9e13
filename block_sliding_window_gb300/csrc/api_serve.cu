// C ABI of libptb, serving: the paged cache of keys and values (appends with
// the position rotation, reads) and sliding-window attention over packed
// prompts and over the cache (MegaScale study notes, ch.2 §2.2, SWA row, on
// batches of sequences of different lengths).  This file checks arguments;
// the kernels are in kv_cache.cu, swa_packed.cu and swa_paged.cu.
#include <cmath>
#include <cstring>

#include "api_internal.h"

using namespace ptb;
using namespace ptb::api;

namespace {

constexpr int64_t kMaxTokens = 1ll << 30;  // token rows and positions stay in int
constexpr int32_t kMaxHeads = 65535;
constexpr int32_t kMaxPackedGroup = 128;  // a query tile holds at least one token of all its heads

bool page_size_ok(int32_t p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }

int64_t kv_block_bytes(int32_t page_size, int32_t head_dim, int32_t bits) {
  const int64_t row = bits == 16 ? 2 * head_dim : head_dim / 2 + head_dim / 8;
  return page_size * row;
}

bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0 && s < (1ll << 39); }

// 0 stands for the default.  Times log2(e) the scale has to stay below 2^127: an
// infinite factor makes NaN of a score of zero, and the kernels round it up to a
// power of two for large scores.
bool scale_ok(float s) { return s >= 0.f && s <= 0x1p126f; }

// Shape, alignment and table of a cache; the device is not touched.
ptb_status fill_cache(KvCache* c, const void* base, int64_t pages, const int32_t* table,
                      int64_t table_stride, int64_t table_pages, int32_t kv_heads,
                      int32_t head_dim, int32_t page_size, int32_t bits) {
  if (!base || !table || pages < 1 || table_pages < 1 || table_stride < table_pages)
    return PTB_ERR_ARG;
  if (kv_heads < 1 || head_dim < 1) return PTB_ERR_ARG;
  if (ptb_kv_page_size(kv_heads, page_size, head_dim, bits) == 0) return PTB_ERR_SHAPE;
  if (pages > (1ll << 31) - 1 || table_pages > kMaxTokens / page_size) return PTB_ERR_SHAPE;
  if (!aligned(base, 16) || !aligned(table, 4)) return PTB_ERR_ALIGN;
  c->base = static_cast<uint8_t*>(const_cast<void*>(base));
  c->pages = pages;
  c->block_bytes = kv_block_bytes(page_size, head_dim, bits);
  c->page_bytes = 2 * kv_heads * c->block_bytes;
  c->table = table;
  c->table_stride = table_stride;
  c->table_pages = table_pages;
  c->page_size = page_size;
  c->page_shift = 0;
  while ((1 << c->page_shift) < page_size) ++c->page_shift;
  c->kv_heads = kv_heads;
  c->head_dim = head_dim;
  c->bits = bits;
  return PTB_OK;
}

// A strided tensor of `rows` rows; one without rows may have no pointer.
ptb_status check_view(const void* p, int64_t st, int64_t sh, int64_t rows) {
  if (!p && rows > 0) return PTB_ERR_ARG;
  if (!aligned(p, 16) || !stride_ok(st) || !stride_ok(sh)) return PTB_ERR_ALIGN;
  return PTB_OK;
}

}  // namespace

#define PTB_TRY(expr)                   \
  do {                                  \
    const ptb_status st_ = (expr);      \
    if (st_ != PTB_OK) return st_;      \
  } while (0)

extern "C" {

size_t ptb_kv_page_size(int32_t kv_heads, int32_t page_size, int32_t head_dim, int32_t bits) {
  if (kv_heads < 1 || kv_heads > kMaxHeads || !page_size_ok(page_size) || !head_dim_ok(head_dim))
    return 0;
  if (bits != 16 && !(bits == 4 && head_dim % 32 == 0)) return 0;
  const int64_t bytes = 2 * kv_heads * kv_block_bytes(page_size, head_dim, bits);
  return bytes < (1ll << 31) ? static_cast<size_t>(bytes) : 0;  // offsets in a page stay in 32 bits
}

ptb_status ptb_kv_append(const ptb_bf16* q, int64_t q_st, int64_t q_sh, const ptb_bf16* k,
                         int64_t k_st, int64_t k_sh, const ptb_bf16* v, int64_t v_st, int64_t v_sh,
                         const float* cos, const float* sin, int64_t positions, int32_t rot_dim,
                         int32_t interleaved, const int32_t* cu_seqlens, const int32_t* past,
                         int32_t batch, int64_t tokens, int32_t heads, int32_t kv_heads,
                         int32_t head_dim, ptb_bf16* q_out, int64_t qo_st, int64_t qo_sh,
                         ptb_bf16* k_out, int64_t ko_st, int64_t ko_sh, void* cache, int64_t pages,
                         const int32_t* page_table, int64_t table_stride, int64_t table_pages,
                         int32_t page_size, int32_t bits, ptb_stream stream) {
  KvAppendArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!cu_seqlens || !past || batch < 1 || tokens < 0 || kv_heads < 1 || head_dim < 1)
    return PTB_ERR_ARG;
  if ((q != nullptr) != (q_out != nullptr) || (q && heads < 1) || rot_dim < 0) return PTB_ERR_ARG;
  if (rot_dim > 0 && (!cos || !sin || positions < 1)) return PTB_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return PTB_ERR_ARG;
  if (tokens > kMaxTokens || heads > kMaxHeads || rot_dim % 16 || rot_dim > head_dim)
    return PTB_ERR_SHAPE;
  PTB_TRY(fill_cache(&a.c, cache, pages, page_table, table_stride, table_pages, kv_heads, head_dim,
                     page_size, bits));
  PTB_TRY(check_view(k, k_st, k_sh, tokens));
  PTB_TRY(check_view(v, v_st, v_sh, tokens));
  if (q) {
    PTB_TRY(check_view(q, q_st, q_sh, tokens));
    PTB_TRY(check_view(q_out, qo_st, qo_sh, tokens));
    if (q_out == q && (qo_st != q_st || qo_sh != q_sh)) return PTB_ERR_ARG;
  }
  if (k_out) {
    PTB_TRY(check_view(k_out, ko_st, ko_sh, tokens));
    if (k_out == k && (ko_st != k_st || ko_sh != k_sh)) return PTB_ERR_ARG;
  }
  if (q_out && (q_out == k || q_out == v || q_out == k_out)) return PTB_ERR_ARG;
  if (k_out && (k_out == v || k_out == q)) return PTB_ERR_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(past, 4)) return PTB_ERR_ALIGN;
  if (rot_dim > 0 && (!aligned(cos, 16) || !aligned(sin, 16))) return PTB_ERR_ALIGN;
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (tokens == 0) return PTB_OK;
  a.q = bf(q), a.k = bf(k), a.v = bf(v), a.q_out = bf(q_out), a.k_out = bf(k_out);
  a.q_st = q_st, a.q_sh = q_sh, a.k_st = k_st, a.k_sh = k_sh, a.v_st = v_st, a.v_sh = v_sh;
  a.qo_st = qo_st, a.qo_sh = qo_sh, a.ko_st = ko_st, a.ko_sh = ko_sh;
  a.cos = cos, a.sin = sin;
  a.positions = rot_dim ? positions : kMaxTokens;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.cu = cu_seqlens, a.past = past;
  a.batch = batch;
  a.heads = q ? heads : 0;
  a.tokens = tokens;
  a.status = ds->status;
  a.sms = ds->sms;
  return launch_status(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

ptb_status ptb_kv_gather(const void* cache, int64_t pages, const int32_t* page_table,
                         int64_t table_stride, int64_t table_pages, const int32_t* cu_seqlens,
                         const int32_t* start, int32_t batch, int64_t tokens, int32_t kv_heads,
                         int32_t head_dim, int32_t page_size, int32_t bits, ptb_bf16* k,
                         int64_t k_st, int64_t k_sh, ptb_bf16* v, int64_t v_st, int64_t v_sh,
                         ptb_stream stream) {
  KvGatherArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!cu_seqlens || !start || batch < 1 || tokens < 0) return PTB_ERR_ARG;
  if (tokens > kMaxTokens) return PTB_ERR_SHAPE;
  PTB_TRY(fill_cache(&a.c, cache, pages, page_table, table_stride, table_pages, kv_heads, head_dim,
                     page_size, bits));
  PTB_TRY(check_view(k, k_st, k_sh, tokens));
  PTB_TRY(check_view(v, v_st, v_sh, tokens));
  if (k && k == v) return PTB_ERR_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(start, 4)) return PTB_ERR_ALIGN;
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (tokens == 0) return PTB_OK;
  a.k = bf(k), a.v = bf(v);
  a.k_st = k_st, a.k_sh = k_sh, a.v_st = v_st, a.v_sh = v_sh;
  a.cu = cu_seqlens, a.start = start;
  a.batch = batch;
  a.tokens = tokens;
  a.status = ds->status;
  a.sms = ds->sms;
  return launch_status(launch_kv_gather(a, static_cast<cudaStream_t>(stream)));
}

size_t swa_attention_packed_workspace_size(int32_t batch, int64_t tokens_q, int32_t heads,
                                           int32_t kv_heads) {
  if (batch < 1 || tokens_q < 0 || tokens_q > kMaxTokens || kv_heads < 1 || heads < kv_heads ||
      heads % kv_heads || heads / kv_heads > kMaxPackedGroup || heads > kMaxHeads)
    return 0;
  return round_up(swa_packed_workspace(batch, tokens_q, heads, kv_heads, current_sms()), kAlign);
}

ptb_status swa_attention_packed(const ptb_bf16* q, int64_t q_st, int64_t q_sh, const ptb_bf16* k,
                                int64_t k_st, int64_t k_sh, const ptb_bf16* v, int64_t v_st,
                                int64_t v_sh, const int32_t* cu_seqlens_q,
                                const int32_t* cu_seqlens_k, int32_t batch, int64_t tokens_q,
                                int64_t tokens_k, int32_t heads, int32_t kv_heads,
                                int32_t head_dim, int32_t window, float scale, ptb_bf16* o,
                                int64_t o_st, int64_t o_sh, void* workspace,
                                size_t workspace_bytes, ptb_stream stream) {
  if (!cu_seqlens_q || batch < 1 || tokens_q < 0 || tokens_k < 0 || heads < 1 || kv_heads < 1 ||
      window < 1)
    return PTB_ERR_ARG;
  if (!scale_ok(scale)) return PTB_ERR_ARG;
  if (!head_dim_ok(head_dim) || heads % kv_heads || heads / kv_heads > kMaxPackedGroup ||
      heads > kMaxHeads || batch > 65535 || tokens_q > kMaxTokens || tokens_k > kMaxTokens)
    return PTB_ERR_SHAPE;
  PTB_TRY(check_view(q, q_st, q_sh, tokens_q));
  PTB_TRY(check_view(k, k_st, k_sh, tokens_k));
  PTB_TRY(check_view(v, v_st, v_sh, tokens_k));
  PTB_TRY(check_view(o, o_st, o_sh, tokens_q));
  if (o && (o == k || o == v)) return PTB_ERR_ARG;
  if (o && (o == q && (o_st != q_st || o_sh != q_sh))) return PTB_ERR_ARG;
  if (!aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4)) return PTB_ERR_ALIGN;
  const size_t need = swa_attention_packed_workspace_size(batch, tokens_q, heads, kv_heads);
  if (need) {
    if (!workspace) return PTB_ERR_ARG;
    if (workspace_bytes < need) return PTB_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return PTB_ERR_ALIGN;
  }
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  if (tokens_q == 0) return PTB_OK;
  SwaPackedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = bf(q), a.k = bf(k), a.v = bf(v), a.o = bf(o);
  a.q_st = q_st, a.q_sh = q_sh, a.k_st = k_st, a.k_sh = k_sh;
  a.v_st = v_st, a.v_sh = v_sh, a.o_st = o_st, a.o_sh = o_sh;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k ? cu_seqlens_k : cu_seqlens_q;
  a.batch = batch;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  // A window of the longest possible sequence or more is plain causal
  // attention; clamping it keeps the kernels' index expressions inside int.
  a.window = window > tokens_k ? static_cast<int>(tokens_k > 0 ? tokens_k : 1) : window;
  a.tokens_q = tokens_q;
  a.tokens_k = tokens_k;
  const float sc = scale == 0.f ? 1.0f / std::sqrt(static_cast<float>(head_dim)) : scale;
  a.scale_log2 = sc * 1.4426950408889634f;
  a.workspace = workspace;
  a.status = ds->status;
  a.sms = ds->sms;
  return launch_status(launch_swa_packed(a, static_cast<cudaStream_t>(stream)));
}

size_t swa_attention_paged_workspace_size(int32_t batch, int32_t heads, int32_t kv_heads,
                                          int32_t head_dim) {
  if (batch < 1 || batch > 65535 || kv_heads < 1 || heads < kv_heads || heads % kv_heads ||
      heads > kMaxHeads || !head_dim_ok(head_dim))
    return 0;
  return round_up(swa_paged_workspace(batch, heads, kv_heads, head_dim, current_sms()), kAlign);
}

ptb_status swa_attention_paged(const ptb_bf16* q, int64_t q_sb, int64_t q_sh, const void* cache,
                               int64_t pages, const int32_t* page_table, int64_t table_stride,
                               int64_t table_pages, const int32_t* seq_lens, int32_t batch,
                               int32_t heads, int32_t kv_heads, int32_t head_dim,
                               int32_t page_size, int32_t bits, int32_t window, float scale,
                               ptb_bf16* o, int64_t o_sb, int64_t o_sh, void* workspace,
                               size_t workspace_bytes, ptb_stream stream) {
  SwaPagedArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!seq_lens || batch < 1 || heads < 1 || kv_heads < 1 || window < 1) return PTB_ERR_ARG;
  if (!scale_ok(scale)) return PTB_ERR_ARG;
  if (batch > 65535 || heads > kMaxHeads || heads % kv_heads) return PTB_ERR_SHAPE;
  PTB_TRY(fill_cache(&a.c, cache, pages, page_table, table_stride, table_pages, kv_heads, head_dim,
                     page_size, bits));
  PTB_TRY(check_view(q, q_sb, q_sh, batch));
  PTB_TRY(check_view(o, o_sb, o_sh, batch));
  if (o == q && (o_sb != q_sb || o_sh != q_sh)) return PTB_ERR_ARG;
  if (!aligned(seq_lens, 4)) return PTB_ERR_ALIGN;
  const size_t need = swa_attention_paged_workspace_size(batch, heads, kv_heads, head_dim);
  if (need) {
    if (!workspace) return PTB_ERR_ARG;
    if (workspace_bytes < need) return PTB_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return PTB_ERR_ALIGN;
  }
  DeviceState* ds = nullptr;
  PTB_TRY(device_state(&ds));
  a.q = bf(q), a.o = bf(o);
  a.q_sb = q_sb, a.q_sh = q_sh, a.o_sb = o_sb, a.o_sh = o_sh;
  a.lens = seq_lens;
  a.batch = batch;
  a.heads = heads;
  a.window = window;
  const float sc = scale == 0.f ? 1.0f / std::sqrt(static_cast<float>(head_dim)) : scale;
  a.scale_log2 = sc * 1.4426950408889634f;
  a.workspace = workspace;
  a.status = ds->status;
  a.sms = ds->sms;
  return launch_status(launch_swa_paged(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
