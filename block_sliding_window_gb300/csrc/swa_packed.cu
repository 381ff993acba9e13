// Causal sliding-window attention over packed sequences with grouped heads
// (definition: ptb.h), on tcgen05 tensor cores.
//
// A query tile is the 128 rows of an MMA: TQ = 128 / G consecutive tokens
// times the G query heads of one key/value head, so a K/V tile is loaded once
// for all of them and a short sequence still fills its tile.  A work item is
// two such tiles (2 TQ tokens of one sequence, one kv head) that share every
// 64-key tile of their band.  Items differ in length, so a one-block kernel
// first lists the query blocks of all sequences, longest first (counting
// sort), and the persistent attention kernel's CTAs take them in snake
// order.  A call that cannot have more items than there are SMs skips the
// list: each CTA finds its own item.
//
// 448 threads, one CTA per SM (the roles and the score / P V pipeline are
// those of the equal-length kernel in swa_tcgen05.cu):
//   warp 0       TMA: Q tiles as boxes {64 channels, G heads, TQ tokens}, K
//                and V tiles as {64 channels, 1 head, 64 tokens}
//   warps 1..4   four MMA-issuing threads: S = Q K^T and O += P V of the two
//                query tiles (P in tensor memory)
//   warps 5..12  softmax, one query row per thread: online maximum and sum in
//                the log2 domain, then O / l as a row
//   warp 13      clears what the mask leaves out: a tile that some row masks
//                also holds rows of later positions, of the next sequence or
//                of no sequence; their weight is 0, but 0 times a NaN or an
//                infinity in V would reach every row of the tile.  This warp
//                scans the masked rows of V and, where one holds such a value,
//                zeroes what is not finite in the tile before the P V product
//                may read it; rows that do attend to such a value get it added
//                at the end of the item (rare path).  The scan costs 3 to 5%.
// Every mbarrier wait is bounded; on a timeout all roles unwind.
//
// What bounds it.  In long prompts the tensor pipe: a 64-key tile is 2 x 384
// cycles of scores (their operands come from shared memory, 48 cycles a K = 16
// step where the products take 32) and 2 x 256 of P V, of 1600 measured; the
// rest is the round trip score -> softmax -> P V -> score over two buffers
// (waits 155, TMEM load 370, weights and their store 850 cycles).  In short
// ones an item's end (last P V, output: 1.5 us) and, on grouped heads, memory.
// Measured: one prompt of 16001 tokens, 16 heads of 128: 727 us, 1.44 PFLOP/s;
// 4 prompts, 128 heads of 96, window 1024: 163 us; 64 ragged prompts, 64 heads
// over 8, window 512: 151 us, 3.5 TB/s.  (A row's own factor for large scores is
// 1% of that: 149 and 161 us with one factor for all.)
#include "kv_device.cuh"

namespace ptb {
namespace {

constexpr int BQ = 128;       // rows per query tile (= MMA M)
constexpr int QT = 2;         // query tiles per work item
constexpr int BKV = 64;       // keys per K/V tile (= MMA N of S, K of PV)
constexpr int kThreads = 448;
constexpr int kCleanWarp = 13;
constexpr int kHeldItems = 64;  // a CTA's first items, held in shared memory
constexpr int kBadSlots = 8;  // more than the items that the K/V ring can hold at once
constexpr float kRescaleLog2 = 8.0f;  // raise the reference max only past 2^8

template <int D>
struct Cfg {
  static constexpr int kAtoms = (D + 63) / 64;
  static constexpr int kQTileBytes = kAtoms * BQ * 128;
  static constexpr int kKVBytes = kAtoms * BKV * 128;
  static constexpr int kFixed = QT * kQTileBytes + kHeldItems * 16 + 512 + 1024;
  static constexpr int kNSFit = (227 * 1024 - kFixed) / (2 * kKVBytes);
  static constexpr int kNS = kNSFit < 6 ? kNSFit : 6;
  static constexpr int kSmemBytes = kFixed + kNS * 2 * kKVBytes;
  static constexpr int kTmemCols = 512;
  __host__ __device__ static constexpr int s_col(int x, int buf) { return x * 256 + buf * BKV; }
  __host__ __device__ static constexpr int o_col(int x) { return x * 256 + 2 * BKV; }
};
static_assert(Cfg<128>::kNS + 1 < kBadSlots && Cfg<16>::kNS + 1 < kBadSlots, "bad-value slots");

struct PackedParams {
  CUtensorMap tq, tk, tv;  // {d, heads, tokens}
  int wide_stores;         // every output row starts on a 32-byte boundary
  SwaPackedArgs a;
  int group, tq_tokens;    // G, TQ
  unsigned inv_group;      // r / G = r * inv_group >> 16 for r < 128
  const int* count;        // null: the CTA finds its own item
  const int4* blocks;      // as sequence_block() makes them
};

struct Item {
  int q_row, ntok, p0, k_row, kvh, kt_hi, n_tiles;
};

__device__ __forceinline__ Item make_item(const int4& b, int kvh, int window) {
  Item it;
  it.q_row = b.x;
  it.ntok = b.y;
  it.p0 = b.z;
  it.k_row = b.w;
  it.kvh = kvh;
  const int last = it.p0 + it.ntok - 1;
  const int first = max(0, it.p0 - window + 1);
  it.kt_hi = last >= 0 ? last / BKV : 0;
  it.n_tiles = last >= 0 ? it.kt_hi - first / BKV + 1 : 0;
  return it;
}

// Does key tile [key0, key0 + 63] meet the band of query tile x of the item?
__device__ __forceinline__ bool tile_relevant(const Item& it, int x, int key0, int tq, int window) {
  if (x * tq >= it.ntok) return false;
  const int r0 = it.p0 + x * tq;
  const int r1 = it.p0 + min((x + 1) * tq, it.ntok) - 1;
  return key0 <= r1 && key0 + BKV - 1 >= r0 - window + 1;
}

// Does some row of the item mask some key of the tile?
__device__ __forceinline__ bool tile_masked(const Item& it, int key0, int window) {
  return key0 + BKV - 1 > it.p0 || key0 < it.p0 + it.ntok - window;
}

// The query blocks of sequence b, or 0 when its offsets are out of range.
__device__ __forceinline__ int sequence_blocks(const SwaPackedArgs& a, int b, int block_tokens,
                                               bool* bad) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.tokens_q || k0 < 0 || k1 < k0 || k1 > a.tokens_k) {
    *bad = true;
    return 0;
  }
  return (q1 - q0 + block_tokens - 1) / block_tokens;
}

// Query block i of sequence b: first row of q and o, tokens (1 .. 2 TQ),
// position of the first one (negative: before the first key), and the row of
// the sequence's position 0 in k and v.
__device__ __forceinline__ int4 sequence_block(const SwaPackedArgs& a, int b, int i,
                                               int block_tokens) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  const int t = i * block_tokens;
  return make_int4(q0 + t, min(block_tokens, q1 - q0 - t), (k1 - k0) - (q1 - q0) + t, k0);
}

// ------------------------------------------------------------------ list --

// Lists the query blocks of all sequences, most key tiles first: a counting
// sort over kBuckets classes of tile counts.  One block; a warp takes a
// sequence at a time and its lanes the sequence's blocks.  The offsets are
// read once, together: with a dependent read per sequence the kernel took
// 6 us for 64 prompts.
constexpr int kBuckets = 1024;
constexpr int kListHeld = 1024;  // sequences whose offsets are held in shared memory

__global__ void __launch_bounds__(1024) packed_list_kernel(const SwaPackedArgs a, int block_tokens,
                                                           int max_tiles, int* count,
                                                           int4* blocks, int capacity) {
  __shared__ int cursor[kBuckets];
  __shared__ int warp_sum[32];
  __shared__ int4 held[kListHeld];  // q0, q1, k0, k1; q1 = q0 where they are out of range
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cursor[threadIdx.x] = 0;
  bool bad = false;
  auto offsets = [&](int b) -> int4 {
    int4 s = make_int4(a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1]);
    if (s.x < 0 || s.y < s.x || s.y > a.tokens_q || s.z < 0 || s.w < s.z || s.w > a.tokens_k) {
      bad = true;
      s.y = s.x;
    }
    return s;
  };
  if (threadIdx.x < a.batch) held[threadIdx.x] = offsets(threadIdx.x);
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int b = warp; b < a.batch; b += 32) {
      const int4 s = b < kListHeld ? held[b] : offsets(b);
      for (int t = lane * block_tokens; t < s.y - s.x; t += 32 * block_tokens) {
        const int4 e = make_int4(s.x + t, min(block_tokens, s.y - s.x - t),
                                 (s.w - s.z) - (s.y - s.x) + t, s.z);
        const Item it = make_item(e, 0, a.window);
        // Tile counts below kBuckets are their own class.
        const int cls = kBuckets - 1 -
                        min(kBuckets - 1, max_tiles < kBuckets
                                              ? it.n_tiles
                                              : static_cast<int>(static_cast<float>(it.n_tiles) *
                                                                 (kBuckets - 1) / max_tiles));
        const int at = atomicAdd(&cursor[cls], 1);
        if (pass == 1 && at < capacity) blocks[at] = e;
      }
    }
    __syncthreads();
    if (pass == 0) {
      // Exclusive prefix sum of the class sizes.
      const int mine = cursor[threadIdx.x];
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      if (lane == 31) warp_sum[warp] = sum;
      __syncthreads();
      int before = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      cursor[threadIdx.x] = before + sum - mine;
      if (threadIdx.x == kBuckets - 1) {
        // Offsets that go back and forth can name more blocks than the tokens
        // have: the list ends at its capacity.
        *count = min(before + sum, capacity);
        if (before + sum > capacity) record_error(a.status, PTB_ERR_ARG);
      }
      __syncthreads();
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(a.status, PTB_ERR_ARG);
}

// Block number `n` of all sequences in their order, by one warp; false when
// there are not so many.
__device__ __forceinline__ bool find_block(const SwaPackedArgs& a, int block_tokens, int n,
                                           int lane, int4* out) {
  bool bad = false;
  int seen = 0, my_b = -1, my_i = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + lane;
    const int mine = b < a.batch ? sequence_blocks(a, b, block_tokens, &bad) : 0;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    if (n >= seen + sum - mine && n < seen + sum) {
      my_b = b;
      my_i = n - (seen + sum - mine);
    }
    seen += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (bad && n == 0) record_error(a.status, PTB_ERR_ARG);
  const unsigned vote = __ballot_sync(0xffffffffu, my_b >= 0);
  if (!vote) return false;
  const int from = __ffs(vote) - 1;
  my_b = __shfl_sync(0xffffffffu, my_b, from);
  my_i = __shfl_sync(0xffffffffu, my_i, from);
  *out = sequence_block(a, my_b, my_i, block_tokens);
  return true;
}

// ------------------------------------------------------------- attention --

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int32_t c0, int32_t c1,
                                                int32_t c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Bits 15 and 31: the low / high bf16 of w is not finite.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    swa_packed_kernel(const __grid_constant__ PackedParams P) {
  using C = Cfg<D>;
  constexpr int NS = C::kNS;
  const SwaPackedArgs& a = P.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                               // [QT][kQTileBytes]
  uint8_t* sK = sQ + QT * C::kQTileBytes;           // [NS][kKVBytes]
  uint8_t* sV = sK + NS * C::kKVBytes;              // [NS][kKVBytes]
  int4* held = reinterpret_cast<int4*>(sV + NS * C::kKVBytes);  // [kHeldItems]
  uint64_t* bars = reinterpret_cast<uint64_t*>(held + kHeldItems);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + 1;
  uint64_t* kv_full = q_empty + 1;      // [NS]
  uint64_t* kv_empty = kv_full + NS;    // [NS]
  uint64_t* v_clean = kv_empty + NS;    // [NS]: V holds finite values where rows mask it
  uint64_t* s_full = v_clean + NS;      // [QT][2]
  uint64_t* p_full = s_full + 2 * QT;   // [QT][2]: P in score buffer 0 / 1
  uint64_t* pv_done = p_full + 2 * QT;  // [QT][2]: P V of score buffer 0 / 1
  uint64_t* done_bar = pv_done + 2 * QT;  // [2 * QT]: one per issuing thread
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 2 * QT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* own_count = abort_flag + 1;
  volatile int* bad_item = own_count + 1;  // [kBadSlots]: item k cleared values: k + 1 in k % slots
  static_assert((2 + 3 * C::kNS + 4 * 2 * QT) * 8 + 4 * (3 + kBadSlots) <= 512, "barriers");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int TQ = P.tq_tokens, G = P.group;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, QT);  // both score threads release Q
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2 * QT + 1);  // every issuing thread and the cleaning warp
      mbar_init(&v_clean[s], 1);
    }
    for (int x = 0; x < 2 * QT; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&done_bar[x], 1);
    }
    *abort_flag = 0;
    for (int s = 0; s < kBadSlots; ++s) bad_item[s] = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&P.tq);
    tma_prefetch_desc(&P.tk);
    tma_prefetch_desc(&P.tv);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (P.count) {
    // The list comes from the kernel before this one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else if (warp == 2) {
    int4 e = make_int4(0, 0, 0, 0);
    const bool found = find_block(a, QT * TQ, blockIdx.x / a.kv_heads, lane, &e);
    if (lane == 0) {
      held[0] = e;
      *own_count = found ? 1 : 0;
    }
  }
  // The list of this CTA's items, so that no role waits for global memory
  // between two of them.
  const int listed = P.count ? *P.count * a.kv_heads : 0;
  if (P.count && threadIdx.x < kHeldItems) {
    const int item = snake_item(threadIdx.x);
    if (item < listed) held[threadIdx.x] = P.blocks[item / a.kv_heads];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int num_items = P.count ? listed : (*own_count ? gridDim.x : 0);
  auto item_at = [&](int k, int item) -> Item {
    const int4 e = k < kHeldItems ? held[k] : P.blocks[item / a.kv_heads];
    return make_item(e, item % a.kv_heads, a.window);
  };

  if (warp == 0) {
    // ------------------------------------------------------------- TMA --
    if (lane == 0) {
      bool ok = true;
      uint32_t kv_count = 0, q_count = 0;
      uint32_t armed = 0, armed_parity = 0;
      for (int k = 0, item = snake_item(0); ok && item < num_items; item = snake_item(++k)) {
        const Item it = item_at(k, item);
        if (it.n_tiles == 0) continue;
        if (!mbar_wait(q_empty, (q_count & 1) ^ 1u, abort_flag, a.status)) {
          ok = false;
          break;
        }
        const int tiles = it.ntok > TQ ? 2 : 1;
        mbar_arrive_expect_tx(q_full, tiles * C::kAtoms * G * TQ * 128);
        for (int x = 0; x < tiles; ++x)
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_3d(sQ + x * C::kQTileBytes + at * BQ * 128, &P.tq, q_full, at * 64,
                        it.kvh * G, it.q_row + x * TQ);
        ++q_count;
        for (int j = 0; j < it.n_tiles; ++j, ++kv_count) {
          const int st = kv_count % NS;
          const uint32_t ph = (kv_count / NS) & 1;
          if (!mbar_wait(&kv_empty[st], ph ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          const int row = it.k_row + (it.kt_hi - j) * BKV;
          mbar_arrive_expect_tx(&kv_full[st], 2 * C::kKVBytes);
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at) {
            tma_load_3d(sK + st * C::kKVBytes + at * BKV * 128, &P.tk, &kv_full[st], at * 64,
                        it.kvh, row);
            tma_load_3d(sV + st * C::kKVBytes + at * BKV * 128, &P.tv, &kv_full[st], at * 64,
                        it.kvh, row);
          }
          armed |= 1u << st;
          armed_parity = (armed_parity & ~(1u << st)) | (ph << st);
        }
        // Behind this item's tiles, the next one's queries start on their way
        // to L2 (64 ragged prompts: 149 us, 151 without; before the tiles they
        // hold those up).
        const int next = snake_item(k + 1);
        if (next < num_items) {
          const Item nx = item_at(k + 1, next);
          for (int x = 0; x < (nx.ntok > TQ ? 2 : 1); ++x)
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              tma_prefetch_3d(&P.tq, at * 64, nx.kvh * G, nx.q_row + x * TQ);
        }
      }
      // Let every copy this thread issued land before the CTA goes away.
      volatile int no_abort = 0;
      for (int s = 0; s < NS; ++s)
        if (armed & (1u << s))
          mbar_wait(&kv_full[s], (armed_parity >> s) & 1u, &no_abort, a.status);
      if (q_count > 0) mbar_wait(q_full, (q_count - 1) & 1, &no_abort, a.status);
    }
  } else if (warp <= 2 * QT) {
    // ------------------------------------------------------------- MMA --
    const bool pv_role = warp > QT;
    const int x = pv_role ? warp - 1 - QT : warp - 1;
    if (lane == 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(BQ, BKV);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(BQ, D) | (1u << 16);  // B (V) MN-major
      bool ok = true;
      uint32_t kv_count = 0, q_count = 0, issued = 0;
      const uint64_t qd = sw128_kmajor_desc(smem_addr(sQ + x * C::kQTileBytes));
      for (int k = 0, item = snake_item(0); ok && item < num_items; item = snake_item(++k)) {
        const Item it = item_at(k, item);
        if (it.n_tiles == 0) continue;
        if (!pv_role) {
          if (!mbar_wait(q_full, q_count & 1, abort_flag, a.status)) break;
          ++q_count;
        }
        bool first_pv = true;
        // What lies between a wait and the first product adds to every tile's
        // round trip, so a role waits last for what comes last (scores: the
        // P V of two tiles before; P V: P) and has its descriptors by then.
        // Parity waits are exact only within one phase: both threads of a
        // query tile observe and release every stage in order, also the tiles
        // outside their band.
        for (int j = 0; j < it.n_tiles; ++j, ++kv_count) {
          const int st = kv_count % NS;
          const uint32_t ph = (kv_count / NS) & 1;
          const bool relevant = tile_relevant(it, x, (it.kt_hi - j) * BKV, TQ, a.window);
          const uint32_t n = issued, buf = n & 1;
          if (!mbar_wait(&kv_full[st], ph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          if (!pv_role) {
            if (relevant) {
              const uint64_t kd = sw128_kmajor_desc(smem_addr(sK + st * C::kKVBytes));
              const uint32_t d_tmem = tmem + C::s_col(x, buf);
              // Score buffer n % 2 still holds P number n - 2 until its P V ends.
              if (n >= 2 && !mbar_wait(&pv_done[2 * x + buf], ((n - 2) >> 1) & 1, abort_flag,
                                       a.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t at = kk / 4, off = (kk % 4) * 32;
                umma_bf16_ss(d_tmem, qd + ((at * BQ * 128 + off) >> 4),
                             kd + ((at * BKV * 128 + off) >> 4), idesc_s, kk > 0);
              }
              umma_commit(&s_full[2 * x + buf]);
              ++issued;
            }
            // The P V thread releases the stage after this product has ended.
            mbar_arrive(&kv_empty[st]);
            if (j == it.n_tiles - 1) umma_commit(q_empty);  // Q_X is free once these finish
          } else {
            if (!mbar_wait(&v_clean[st], ph, abort_flag, a.status)) {
              ok = false;
              break;
            }
            if (!relevant) {
              mbar_arrive(&kv_empty[st]);
              continue;
            }
            const uint64_t vd = sw128_mnmajor_desc(smem_addr(sV + st * C::kKVBytes), BKV * 128);
            const uint32_t p_tmem = tmem + C::s_col(x, buf);
            const uint32_t d_tmem = tmem + C::o_col(x);
            if (!mbar_wait(&p_full[2 * x + buf], (n >> 1) & 1, abort_flag, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BKV / 16; ++kk)  // 16 keys = 8 packed P columns
              umma_bf16_ts(d_tmem, p_tmem + kk * 8, vd + ((kk * 16 * 128) >> 4), idesc_pv,
                           (!first_pv || kk > 0) ? 1u : 0u);
            umma_commit(&pv_done[2 * x + buf]);
            umma_commit(&kv_empty[st]);  // this query tile is done with the stage
            ++issued;
            first_pv = false;
          }
        }
      }
      const int me = pv_role ? QT + x : x;
      umma_commit(&done_bar[me]);
      volatile int no_abort = 0;
      mbar_wait(&done_bar[me], 0, &no_abort, a.status);
    }
  } else if (warp == kCleanWarp) {
    // ----------------------------------------------------------- clean --
    bool ok = true;
    uint32_t kv_count = 0;
    for (int k = 0, item = snake_item(0); ok && item < num_items; item = snake_item(++k)) {
      const Item it = item_at(k, item);
      for (int j = 0; j < it.n_tiles; ++j, ++kv_count) {
        const int st = kv_count % NS;
        if (!mbar_wait_warp(&kv_full[st], (kv_count / NS) & 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        const int key0 = (it.kt_hi - j) * BKV;
        if (tile_masked(it, key0, a.window)) {
          // Rows that some query of the item masks: before `lower` and from
          // `upper` on (groups of four, a warp's 512 bytes of one column block).
          const int lower = (min(max(it.p0 + it.ntok - a.window - key0, 0), BKV) + 3) / 4;
          const int upper = max(min(max(it.p0 + 1 - key0, 0), BKV) / 4, lower);
          uint4* v = reinterpret_cast<uint4*>(sV + st * C::kKVBytes) + lane;
          // 0 times a value that is not finite is NaN and stays: one bf16x2
          // FMA for two values.
          __nv_bfloat162 nan[4];
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) nan[e] = zero;
          auto scan = [&](int i0, int i1) {
#pragma unroll 4
            for (int i = i0; i < i1; ++i)
#pragma unroll
              for (int at = 0; at < C::kAtoms; ++at) {
                const uint4 w = v[(at * (BKV / 4) + i) * 32];
                nan[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.x), zero, nan[0]);
                nan[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.y), zero, nan[1]);
                nan[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.z), zero, nan[2]);
                nan[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.w), zero, nan[3]);
              }
          };
          scan(0, lower);
          scan(upper, BKV / 4);
          nan[0] = __hadd2(__hadd2(nan[0], nan[1]), __hadd2(nan[2], nan[3]));
          if (__any_sync(0xffffffffu, (*reinterpret_cast<uint32_t*>(&nan[0]) & 0x7fff7fffu) != 0)) {
            for (int i = 0; i < C::kKVBytes / 512; ++i) {
              uint4 w = v[i * 32];
              w.x &= ~(not_finite2(w.x) / 0x8000u * 0xffffu);
              w.y &= ~(not_finite2(w.y) / 0x8000u * 0xffffu);
              w.z &= ~(not_finite2(w.z) / 0x8000u * 0xffffu);
              w.w &= ~(not_finite2(w.w) / 0x8000u * 0xffffu);
              v[i * 32] = w;
            }
            fence_proxy_async_smem();
            if (lane == 0) bad_item[k % kBadSlots] = k + 1;
          }
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(&v_clean[st]);
          mbar_arrive(&kv_empty[st]);
        }
      }
    }
  } else {
    // --------------------------------------------------------- softmax --
    const int x = (warp - 1 - 2 * QT) >> 2;  // query tile of this warpgroup
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row in the query tile = TMEM lane
    const int tok = static_cast<int>((r * P.inv_group) >> 16);  // r / G: token of the tile
    const bool row_used = r < G * TQ;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lane_base + C::o_col(x);
    uint32_t seen = 0;  // relevant tiles of this query tile so far (all items)
    bool ok = true;

    // P V number n of this query tile completes phase n / 2 of
    // pv_done[x][n % 2]; one barrier per score buffer keeps every parity wait
    // within one phase.
    auto wait_pv = [&](uint32_t n) -> bool {
      if (!mbar_wait_warp(&pv_done[2 * x + (n & 1)], (n >> 1) & 1, abort_flag, a.status))
        return false;
      tc_fence_after();
      return true;
    };

    for (int k = 0, item = snake_item(0); ok && item < num_items; item = snake_item(++k)) {
      const Item it = item_at(k, item);
      if (x * TQ >= it.ntok) continue;
      const int i = it.p0 + x * TQ + tok;  // position of this thread's query
      float m_ref = -INFINITY, l_run = 0.f;
      float scale = a.scale_log2;  // of this row (kLargeScore)
      bool any_pv = false;
      for (int j = 0; j < it.n_tiles; ++j) {
        const int key0 = (it.kt_hi - j) * BKV;
        if (!tile_relevant(it, x, key0, TQ, a.window)) continue;
        const int buf = seen & 1;
        if (!mbar_wait_warp(&s_full[2 * x + buf], (seen >> 1) & 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        static_assert(BKV == 64, "two 32-column TMEM loads per score row");
        uint32_t raw0[32], raw1[32];
        tmem_ld_32x32b_x32(tmem + lane_base + C::s_col(x, buf), raw0);
        tmem_ld_32x32b_x32(tmem + lane_base + C::s_col(x, buf) + 32, raw1);
        tmem_ld_wait();
        float v[BKV];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          v[e] = __uint_as_float(raw0[e]);
          v[32 + e] = __uint_as_float(raw1[e]);
        }
        const bool interior = (key0 + BKV - 1 <= i) && (key0 >= i - a.window + 1);
        if (!interior) {
          const int hi = min(i - key0, BKV - 1), lo = max(i - a.window + 1 - key0, 0);
          uint64_t keep = hi < lo ? 0 : (~0ull >> (BKV - 1 - hi)) & (~0ull << lo);
          uint32_t keep0 = static_cast<uint32_t>(keep), keep1 = static_cast<uint32_t>(keep >> 32);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v[e] = (keep0 & (1u << e)) ? v[e] : -INFINITY;
            v[32 + e] = (keep1 & (1u << e)) ? v[32 + e] : -INFINITY;
          }
        }
        // Row max as a tree of three-input maxima, then one f32x2 FMA (scale
        // and shift) and one f32x2 add (row sum) per two scores.
        float m1[22], m2[8];
#pragma unroll
        for (int t = 0; t < 21; ++t) m1[t] = fmax3(v[3 * t], v[3 * t + 1], v[3 * t + 2]);
        m1[21] = v[63];
#pragma unroll
        for (int t = 0; t < 7; ++t) m2[t] = fmax3(m1[3 * t], m1[3 * t + 1], m1[3 * t + 2]);
        m2[7] = m1[21];
        float mx = fmax3(fmax3(m2[0], m2[1], m2[2]), fmax3(m2[3], m2[4], m2[5]), fmaxf(m2[6], m2[7]));
        const float raw_max = mx;
        mx = __fmul_rn(mx, scale);  // row max in the log2 domain, rounded for every use
        // Raise the reference max only when the row max passes it by 2^8.
        float alpha = 1.f;
        const bool raise = mx > m_ref + kRescaleLog2;
        if (raise) {
          const float m = reference_max(raw_max, a.scale_log2, scale);
          alpha = fast_exp2(m_ref - m);  // 0 while m_ref is -inf
          l_run *= alpha;
          m_ref = m;
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t scale2 = f2(scale, scale), shift2 = f2(-m_use, -m_use);
        uint64_t sum2[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
        uint32_t pk[BKV / 2];
#pragma unroll
        for (int e = 0; e < BKV; e += 2) {
          float t0, t1;
          f2_split(f2_fma(f2(v[e], v[e + 1]), scale2, shift2), t0, t1);
          const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
          sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2(p0, p1));  // four chains
          pk[e / 2] = pack_bf16x2(p0, p1);
        }
        float s0, s1;
        f2_split(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), s0, s1);
        l_run += s0 + s1;
        // P (bf16 pairs) over the first 32 columns of the scores just read; lanes
        // that raised their maximum are back with the others.
        __syncwarp();
        tmem_st_32x32b_x32(tmem + lane_base + C::s_col(x, buf), pk);
        if (any_pv && __any_sync(0xffffffffu, raise)) {
          // O must hold every earlier P V of this item before it is rescaled.
          if (!wait_pv(seen - 1)) {
            tmem_st_wait();
            ok = false;
            break;
          }
          if constexpr (D % 32 == 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_tmem + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_32x32b_x32(o_tmem + c, o);
            }
          } else {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_tmem, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x16(o_tmem, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + buf]);
        any_pv = true;
        ++seen;
      }
      if (!ok) break;
      // The last P V of the item, then O / l (rows without keys: zeros).
      if (any_pv && !wait_pv(seen - 1)) {
        ok = false;
        break;
      }
      const float inv = l_run != 0.f ? 1.f / l_run : 0.f;
      // A later item's mark says nothing about this one: look for such values.
      const bool bad = any_pv && bad_item[k % kBadSlots] > k;
      // Rows go out of registers, 32 bytes a store where rows start on 32-byte
      // boundaries (else 16), past L1: a store fills whole sectors, and 64
      // ragged prompts took 163 us with lines allocated in L1, 151 without.
      // Staging rows in shared memory to store whole lines was slower (186),
      // and so were tensor-map stores.
      __nv_bfloat16* out = a.o + static_cast<int64_t>(it.q_row + x * TQ + tok) * a.o_st +
                           static_cast<int64_t>(it.kvh * G + r - tok * G) * a.o_sh;
      const bool live = row_used && x * TQ + tok < it.ntok;
      // The loops over columns here and in the rescaling stay loops: the code of
      // all roles shares the instruction cache (unrolled: 177 us for 168).
      constexpr int kCols = D < 32 ? D : 32;  // columns per TMEM wait
#pragma unroll 1
      for (int c = 0; c < D; c += kCols) {
        uint32_t o[kCols];
        if (any_pv) {
          if constexpr (kCols == 32) {
            tmem_ld_32x32b_x32(o_tmem + c, o);
          } else {
            tmem_ld_32x32b_x16(o_tmem + c, o);
          }
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < kCols; ++e) o[e] = 0;
        }
        if (live) {
          float f[kCols];
#pragma unroll
          for (int e = 0; e < kCols; ++e) f[e] = __uint_as_float(o[e]) * inv;
          if (bad) {
            // Values that are not finite and that this row attends to, out of
            // the tiles that were cleared.
            for (int key = max(0, i - a.window + 1); key <= i; ++key) {
              if (!tile_masked(it, key & ~(BKV - 1), a.window)) {
                key |= BKV - 1;  // on to the next tile
                continue;
              }
              const __nv_bfloat16* row =
                  a.v + static_cast<int64_t>(it.k_row + key) * a.v_st + it.kvh * a.v_sh + c;
#pragma unroll
              for (int e = 0; e < kCols; ++e) {
                const float z = __bfloat162float(row[e]);
                if (!(fabsf(z) < INFINITY)) f[e] += z;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < kCols; e += 16) {
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = pack_bf16x2(f[e + 2 * q], f[e + 2 * q + 1]);
            if (P.wide_stores) {
              asm volatile(
                  "st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                      out + c + e),
                  "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                  "r"(w[7])
                  : "memory");
            } else {
              store16_past_l1(out + c + e, make_uint4(w[0], w[1], w[2], w[3]));
              store16_past_l1(out + c + e + 8, make_uint4(w[4], w[5], w[6], w[7]));
            }
          }
        }
        __syncwarp();  // the next columns' load is the whole warp's
      }
      tc_fence_before();
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch_typed(const PackedParams& prm, int grid, bool after_list, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = swa_packed_kernel<D>;
  static bool configured[kDeviceSlots] = {};
  cudaError_t e = allow_smem(kern, C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  // Set up while the list is written; the kernel waits for it before reading.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_list ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, prm);
}

// {d, heads, tokens}: boxes of 64 channels x `heads_box` heads x `tokens_box` tokens.
bool packed_map(CUtensorMap* map, const __nv_bfloat16* base, int d, int heads, int64_t tokens,
                int64_t st, int64_t sh, int heads_box, int tokens_box) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(tokens)};
  const uint64_t strides[2] = {static_cast<uint64_t>(sh) * 2, static_cast<uint64_t>(st) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(heads_box), static_cast<uint32_t>(tokens_box)};
  return make_tensor_map(map, base, 3, dims, strides, box);
}

// Tokens of a work item.
int block_tokens(int heads, int kv_heads) { return QT * (BQ / (heads / kv_heads)); }

// The most query blocks that `batch` sequences of `tokens` in all can have.
int64_t most_blocks(int batch, int64_t tokens, int block) { return tokens / block + batch; }

}  // namespace

// The list: its length (16 bytes), then the blocks; none where every SM takes
// at most one item.
size_t swa_packed_workspace(int batch, int64_t tokens_q, int heads, int kv_heads, int sms) {
  const int64_t n = most_blocks(batch, tokens_q, block_tokens(heads, kv_heads));
  if (n * kv_heads <= sms) return 0;
  return static_cast<size_t>(16 + n * sizeof(int4));
}

cudaError_t launch_swa_packed(const SwaPackedArgs& a, cudaStream_t stream) {
  PackedParams prm;
  prm.a = a;
  prm.group = a.heads / a.kv_heads;
  prm.tq_tokens = BQ / prm.group;
  prm.inv_group = (65536u + prm.group - 1) / prm.group;
  if (!packed_map(&prm.tq, a.q, a.head_dim, a.heads, a.tokens_q, a.q_st, a.q_sh, prm.group,
                  prm.tq_tokens))
    return cudaErrorInvalidValue;
  prm.wide_stores = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && a.o_st % 16 == 0 && a.o_sh % 16 == 0;
  // Without keys the maps are never used; they still need a valid address.
  const bool keys = a.tokens_k > 0;
  if (!packed_map(&prm.tk, keys ? a.k : a.q, a.head_dim, a.kv_heads, keys ? a.tokens_k : 1, a.k_st,
                  a.k_sh, 1, BKV) ||
      !packed_map(&prm.tv, keys ? a.v : a.q, a.head_dim, a.kv_heads, keys ? a.tokens_k : 1, a.v_st,
                  a.v_sh, 1, BKV))
    return cudaErrorInvalidValue;
  const int block = QT * prm.tq_tokens;
  const int64_t blocks = most_blocks(a.batch, a.tokens_q, block);
  const int64_t items = blocks * a.kv_heads;
  if (items > 0x3fffffff) return cudaErrorInvalidValue;  // item numbers stay in int
  const bool list = items > a.sms;
  prm.count = nullptr;
  prm.blocks = nullptr;
  if (list) {
    int* count = static_cast<int*>(a.workspace);
    int4* out = reinterpret_cast<int4*>(count + 4);
    const int64_t span = a.window < a.tokens_k ? a.window : a.tokens_k;
    const int max_tiles = static_cast<int>((span + block) / BKV + 2);
    packed_list_kernel<<<1, 1024, 0, stream>>>(a, block, max_tiles, count, out,
                                               static_cast<int>(blocks));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    prm.count = count;
    prm.blocks = out;
  }
  const int grid = static_cast<int>(items < a.sms ? items : a.sms);
  switch (a.head_dim) {
    case 16: return launch_typed<16>(prm, grid, list, stream);
    case 32: return launch_typed<32>(prm, grid, list, stream);
    case 64: return launch_typed<64>(prm, grid, list, stream);
    case 96: return launch_typed<96>(prm, grid, list, stream);
    case 128: return launch_typed<128>(prm, grid, list, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ptb
