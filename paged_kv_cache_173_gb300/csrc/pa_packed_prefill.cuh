// pa_packed_prefill.cuh -- causal attention over whole prompts in packed rows, on the
// tcgen05 tensor cores, with the cache write of the prompts' keys and values.
//
//  packed_prefill_tc_kernel  one CTA per SM; an item of work is a pair of query tiles of
//                            a (KV head, sequence), a tile up to 128 rows (128 / G tokens
//                            x G heads, G any group up to 16).  Q K^T and P V in tensor
//                            memory, one softmax thread per row.
//
// Warps: two warpgroups of softmax (a tile each); one that writes the item's own keys and
// values into the pools and the outputs; and one with an MMA warp per tile, a warp that finds
// the work items and makes masked values safe, and one for the loads of K and V (TMA, 128 keys
// at a time).
//
// The bound is the tensor cores: 4 x 128 x 128 x d multiply-adds per pair and 128 keys, 2062
// cycles at d = 128; at d = 64 the softmax, whose 256 x 128 scores take the four schedulers
// 1530 cycles (1024 of them the exponentials).  Long prompts take 2700 and 2490 cycles.  What
// stands against the rest:
//  - A tile's chain (scores, weights, P V, next scores) is longer than its MMAs.  Two tiles
//    alternate; the weights leave in halves; the offset of the exponent is taken from the block
//    before, and the weights' own sum says whether it holds, so that no maximum is looked for
//    first (half a block 300 cycles earlier).  At d = 64 there is room in tensor memory for P
//    beside S, and Q K^T runs ahead of P V.
//  - The end of an item: outputs and the cache write have warps of their own, Q of the next
//    item comes from L2, and its first MMAs wait for nothing else.  (By the softmax threads:
//    8 prompts of 1024 tokens without groups 204 us against 115.)
//  - Values that are not finite in keys that a row does not see: a warp looks the few blocks
//    concerned through as they land, one instruction per pair of elements (five: 8.2 against
//    7.0 us for one short prompt).
//  - Items are taken longest first, by CTAs that come to the end of their last one.
// Tried and dropped: two softmax threads per row (both share one MUFU, and their 80 registers
// spill: 233 us for the 200 below); Q K^T in halves of 64 keys (an MMA of N = 64 from shared
// memory takes 48 cycles, one of N = 128 64); items in groups whose keys fit L2 (ragged
// prompts 175 -> 187 us).
// Measured, cache write included, call behind call through the binding on changing inputs (what
// a server sees: inputs from DRAM, the clock lowered by the power limit) and, second, replays of a
// graph on one set of inputs (2.07 GHz, tensor pipe active 64%):
//   fp16, 32/8 heads of 128, 8 prompts of 2048 tokens   231 us (1.19 PFLOP/s), 200 us (1.37)
//   the same, one prompt of 61                          6.4 us, 6.4 us
//   bf16, 16 prompts of 1 to 2048                       173 us, 165 us
//   fp16, 64/8 heads, 6000 + 8192 tokens                1.06 ms (1.49 PFLOP/s), 1.02 ms (1.55)
//   bf16, 28/4 heads of 64, 12 of 200 to 1500           72 us, 71 us
//   fp16, 32/8 heads of 64, 8 of 2048                   164 us in replays
// Registers: 168 / 96 / 80 by role, no spills (a spilled register makes every arrival wait for
// local memory: 208 -> 228 us) but 20 bytes of the items' warp at d = 64 in ragged batches, beside
// the search (batches that hardly search, 64 sequences: 29.5 us with them, 29.7 without).
//
// The method: causal multi-query attention ("in-depth reading", section 5.1, item 5;
// "vAttention", contiguous prefill), online softmax of "vLLM PagedAttention source
// walk-through", section 3.4.
#pragma once

#include "pa_block.cuh"
#include "pa_prefill.cuh"
#include "pa_tc.cuh"

namespace pa {

namespace {

struct PackedParams {
  CUtensorMap tmap_q;  // q as rows x heads x dims: box of 64 dims x G heads x 128 / G rows, 128-byte swizzle
  CUtensorMap tmap_k;  // key likewise: 64 dims x 1 head x 128 rows
  CUtensorMap tmap_v;
  void* out;
  const void* key;
  const void* value;
  int64_t k_stride;  // elements
  int64_t v_stride;
  void* k_cache;  // null: no cache write
  void* v_cache;
  const int64_t* slot_mapping;
  int64_t num_slots;
  const int32_t* query_start_loc;
  uint64_t pair_magic;  // ceil(2^64 / tokens of a pair): the high half of a product with it divides
  int num_seqs;
  int num_rows;
  int max_query_len;
  int num_heads;
  int num_kv_heads;
  int group;
  int inv_g;  // 65536 / group + 1: r / group = r * inv_g >> 16 for the rows r < 128 of a tile
  int tile_tokens;
  int pairs;
  // grid order: (KV head, sequence, pair) or, longest_first = 0, (pair, KV head, sequence).  Ragged
  // kernels: one dimension, KV head and place in the list of all sequences' pairs, longest first.
  int longest_first;
  float scale_log2;
};

template <typename T, int HEAD_DIM>
struct PpCfg {
  static constexpr bool BF16 = !std::is_same<T, __half>::value;
  static constexpr int SOFT = TC_TILES * TC_ROWS;  // softmax threads
  static constexpr int SIDE_WARP = SOFT / 32;      // cache write, masked values
  static constexpr int SIDE = 128;
  static constexpr int MMA_WARP = SIDE_WARP + SIDE / 32;
  static constexpr int ITEM_WARP = MMA_WARP + TC_TILES;
  static constexpr int LOAD_WARP = ITEM_WARP + 1;
  static constexpr int THREADS = SOFT + SIDE + 128;
  static constexpr int SOFT_REGS = 168;
  static constexpr int SIDE_REGS = 96;
  static constexpr int MMA_REGS = 80;
  // what the warpgroups hold is what the block was launched with
  static_assert(SOFT * SOFT_REGS + SIDE * SIDE_REGS + 128 * MMA_REGS <= THREADS * 128, "registers");
  static constexpr int DBOX = HEAD_DIM / BOX_DIMS;
  static constexpr int QATOM = TC_ROWS * 128;
  static constexpr int QBYTES = DBOX * QATOM;
  static constexpr int KATOM = TC_KEYS * 128;
  static constexpr int KBYTES = DBOX * KATOM;
  static constexpr int SMEM_MAX = 227 * 1024;
  static constexpr int RESERVE = 3 * 1024;  // items, sums, barriers
  static constexpr int STAGES_FIT = (SMEM_MAX - RESERVE - TC_TILES * QBYTES) / KBYTES;
  static constexpr int KSTAGES = STAGES_FIT / 2 < 4 ? STAGES_FIT / 2 : 4;
  static constexpr int VSTAGES = STAGES_FIT - KSTAGES < 4 ? STAGES_FIT - KSTAGES : 4;
  static_assert(KSTAGES >= 2 && VSTAGES >= 2 && KSTAGES <= VSTAGES, "the rings");
  static constexpr int K_OFF = TC_TILES * QBYTES;
  static constexpr int V_OFF = K_OFF + KSTAGES * KBYTES;
  static constexpr int INFO_OFF = V_OFF + VSTAGES * KBYTES;
  // Published items.  The MMAs are at most one item ahead of the outputs that are still being written, the loads
  // VSTAGES blocks, so as many items, ahead of them, and one more is published.
  static constexpr int ITEMS = 8;
  static_assert(VSTAGES + 3 <= ITEMS, "the ring of items");
  static constexpr int INFO = 8;  // words of an item
  // An item of more blocks asks for its successor near its end: an item that is taken waits for the CTA that took it,
  // while others are free (one prompt of 2048 tokens, two items a CTA: 43 us asked for at once).
  static constexpr int ASK_AT_ONCE = 4;
  static constexpr int SUM_OFF = INFO_OFF + ITEMS * INFO * 4;  // [tile][row] sum of the weights
  static constexpr int RESP_OFF = SUM_OFF + TC_TILES * TC_ROWS * 4;
  static constexpr int BAR_OFF = RESP_OFF + 16;
  static constexpr int DONE = VSTAGES;  // ring of completed steps
  static constexpr int NBARS = KSTAGES + 2 * VSTAGES + DONE + 11 * TC_TILES + ITEMS + 2;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int LAYOUT_BYTES = SLOT_OFF + 16;
  static constexpr int SMEM_BYTES = LAYOUT_BYTES;
  static_assert(SMEM_BYTES <= SMEM_MAX, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  // A tile's 256 columns: S 128, then O.  With 64 channels there is room for P beside S, and Q K^T of a block runs
  // ahead of P V of the one before, once the softmax is done with the scores of that (EARLY); else P goes over S, and
  // it runs behind P V.
  static constexpr bool EARLY = HEAD_DIM == 64;
  static constexpr int P_COL = EARLY ? 128 : 0;
  static constexpr int O_COL = EARLY ? 192 : 128;
  static constexpr uint32_t ID_S = umma_idesc_f16(TC_ROWS, TC_KEYS, BF16, false);
  static constexpr uint32_t ID_PV = umma_idesc_f16(TC_ROWS, HEAD_DIM, BF16, true);
  // log2 of the largest weight when the running maximum has just moved; it may grow by 2^8 from there.
  // float16: up to 2^15, so that small weights keep their bits.  bfloat16 has float32's range, and weights
  // of 2^-8 at most keep a sum of 2^8 of its largest values within it.
  static constexpr float MID = BF16 ? -16.f : 7.f;
  // The largest sum of 64 weights that leaves the maximum where it is (64 equal ones at the maximum: 2^(MID + 6)).
  static constexpr float LIMIT = BF16 ? 0.25f : 32768.f;
  // A weight's exponent is x a + (MID - m) for the score x, one FMA, with m = rounded_up(t a) of the score t that the
  // row is measured from: m lies |m| 2^-22 above t a, and MID - m is rounded by 2^-24 of it at most.  While it is
  // below this bound, that makes the weights smaller by 2^-6 of a power of two; from 2^27 on they would all be 0 in
  // fp16.  Past the bound t is taken off first, (x - t) a + MID, which holds for scores of any size: a warp with such
  // a row weighs its scores once more, from tensor memory, at twice the time.
  static constexpr float WIDE = 65536.f;
};

// ---------------------------------------------------------------- work items
struct PackedItem {
  int s, kvh;
  int ta;    // first token of tile 0
  int q0;    // row of the sequence's first token
  int qlen;  // its tokens

  __device__ __forceinline__ int tiles(int tt) const { return ta + tt < qlen ? 2 : 1; }
  // one past tile u's last token, which is as many keys as its last row sees, and the key blocks that it meets
  __device__ __forceinline__ int tile_end(int u, int tt) const { return min(qlen, ta + (u + 1) * tt); }
  __device__ __forceinline__ int tile_blocks(int u, int tt) const {
    return u < tiles(tt) ? (tile_end(u, tt) + TC_KEYS - 1) / TC_KEYS : 0;
  }
  __device__ __forceinline__ int kend(int tt) const { return tile_end(1, tt); }
  __device__ __forceinline__ int blocks(int tt) const { return (kend(tt) + TC_KEYS - 1) / TC_KEYS; }
  // The first block with a key that some row of the item does not see.  The item's last block is always one:
  // ta is even, so ta + 1 tokens fill no block.
  __device__ __forceinline__ int first_masked() const { return ta / TC_KEYS; }
};

// The rows of sequence i: the first one, and how many are computed (at most 0: none).
__device__ __forceinline__ int rows_of(const PackedParams& p, int i, int& q0) {
  q0 = min(max(__ldg(p.query_start_loc + i), 0), p.num_rows);
  return min(min(max(__ldg(p.query_start_loc + i + 1), 0), p.num_rows) - q0, p.max_query_len);
}

// The pairs of query tiles of sequence i (0 past the last).
__device__ __forceinline__ int pairs_of(const PackedParams& p, int i) {
  if (i >= p.num_seqs) return 0;
  int q0;
  const int n = rows_of(p, i, q0);
  return n <= 0 ? 0 : static_cast<int>(__umul64hi(static_cast<uint64_t>(n - 1), p.pair_magic)) + 1;
}

// What a warp's last search of the list found: the pair, C of it, and the length of the list (-1: no search yet).
struct ListPlace {
  int pair = 0, c = 0, total = -1;
};

// Place `at` of the list of all sequences' pairs, the pairs of highest number first and those of
// one number in the sequences' order: (pair, sequence), or false past the last.  The whole warp
// searches; C(x), the pairs numbered above x, is the sum over the sequences of max(0, pairs - 1 - x),
// and the pair the least x with C(x) <= at (-1: past the last).  The place found before narrows the search:
// among prompts of one pair nothing is left of it.  A pass over the sequences takes four values of x, and a lane
// has four of the sequences on their way.  (One value and one sequence at a time, from scratch: a prompt of 1024
// beside 1000 of one token 659 us, now 155; one of 8192 beside 255 of one 238, now 179.)
__device__ __forceinline__ bool listed_pair(const PackedParams& p, int at, int& pair, int& s, ListPlace& known) {
  constexpr int X = 4, SEQS = 4;
  const int lane = threadIdx.x & 31;
  int lo = -1, hi = p.pairs - 1;  // the least x is in [lo, hi]
  int c_hi = 0;                   // C(hi)
  if (known.total >= 0) {
    if (at >= known.total) return false;
    lo = 0;
    if (at >= known.c) hi = known.pair, c_hi = known.c;
    else lo = known.pair + 1;
  }
#pragma unroll 1
  while (lo < hi) {
    int n[X];
#pragma unroll
    for (int k = 0; k < X; ++k) n[k] = 0;
    const int wide = hi - lo;
#pragma unroll 1
    for (int i = lane; i < p.num_seqs; i += 32 * SEQS) {
      int m[SEQS];
#pragma unroll
      for (int y = 0; y < SEQS; ++y) m[y] = pairs_of(p, i + 32 * y) - 1 - lo;
#pragma unroll
      for (int k = 0; k < X; ++k)
#pragma unroll
        for (int y = 0; y < SEQS; ++y) n[k] += max(0, m[y] - wide * k / X);
    }
    int from = lo, to = hi;
    bool found = false;
#pragma unroll
    for (int k = 0; k < X; ++k) {
      const int x = lo + wide * k / X;
      const int c = __reduce_add_sync(kFullMask, n[k]);
      if (k == 0 && lo < 0) known.total = c;
      if (!found) {
        if (c <= at) {
          found = true;
          to = x;
          c_hi = c;
        } else {
          from = x + 1;
        }
      }
    }
    lo = from;
    hi = to;
  }
  if (hi < 0) return false;
  known.pair = pair = hi;
  known.c = c_hi;
  s = -1;
  int rank = at - c_hi;
#pragma unroll 1
  for (int i = 0; i < p.num_seqs; i += 32 * SEQS) {
    unsigned has[SEQS];
#pragma unroll
    for (int y = 0; y < SEQS; ++y) has[y] = __ballot_sync(kFullMask, pairs_of(p, i + 32 * y + lane) > hi);
#pragma unroll
    for (int y = 0; y < SEQS; ++y) {
      const int n = __popc(has[y]);
      if (rank >= 0 && rank < n) s = i + 32 * y + static_cast<int>(__fns(has[y], 0, rank + 1));
      rank -= n;
    }
    if (rank < 0) break;
  }
  return s >= 0;
}

// The item of a grid index, by whole warps; false: nothing to do.
template <bool IS_RAGGED>
__device__ __forceinline__ bool find_packed_item(const PackedParams& p, uint3 id, PackedItem& it, ListPlace& known) {
  int pair;
  if constexpr (IS_RAGGED) {
    it.kvh = id.x % p.num_kv_heads;
    if (!listed_pair(p, id.x / p.num_kv_heads, pair, it.s, known)) return false;
  } else {
    const bool lf = p.longest_first;
    pair = p.pairs - 1 - static_cast<int>(lf ? id.z : id.x);  // the longest pairs start first
    it.kvh = lf ? id.x : id.y;
    it.s = lf ? id.y : id.z;
  }
  it.qlen = rows_of(p, it.s, it.q0);
  it.ta = 2 * pair * p.tile_tokens;
  return it.ta < it.qlen;
}

// NaN in the rows of an item, by `n` threads.
template <typename T, int HEAD_DIM>
__device__ __forceinline__ void write_nan_rows(const PackedParams& p, const PackedItem& it, int i, int n) {
  constexpr int U = HEAD_DIM / 8;
  const uint32_t v = pack2<T>(NAN, NAN);
  const int rows = (it.kend(p.tile_tokens) - it.ta) * p.group;
#pragma unroll 1
  for (; i < rows * U; i += n) {
    const int r = i / U;
    const int t = r / p.group;
    T* row = static_cast<T*>(p.out) + (static_cast<size_t>(it.q0 + it.ta + t) * p.num_heads + it.kvh * p.group + r -
                                       t * p.group) * HEAD_DIM;
    reinterpret_cast<uint4*>(row)[i % U] = make_uint4(v, v, v, v);
  }
}

// The halves of a pair of elements that are infinite or NaN, as ones in all of their bits: an exponent of
// all ones carries into the sign's place.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t EXP = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t ONE = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
  return ((((w & EXP) + ONE) & 0x80008000u) >> 15) * 0xffffu;
}

// Pair by pair the larger of a >= 0 and |b|, NaN where one is.
template <typename T>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r =
        __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// An output element `o` that also takes a value `v` that is not finite (16-bit patterns): v, or NaN where o is
// not finite and another.
template <typename T>
__device__ __forceinline__ uint32_t join_not_finite(uint32_t o, uint32_t v) {
  return not_finite<T>(o) && o != v ? 0x7fffu : v;
}

// Whether `ok` holds in all THREADS threads that meet at named barrier 1.
template <int THREADS>
__device__ __forceinline__ bool all_meet(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "n"(THREADS)
      : "memory");
  return all != 0;
}

template <typename T, int HEAD_DIM, bool IS_RAGGED>
__global__ void __launch_bounds__(PpCfg<T, HEAD_DIM>::THREADS, 1)
packed_prefill_tc_kernel(const __grid_constant__ PackedParams p) {
  using C = PpCfg<T, HEAD_DIM>;
  constexpr int KS = C::KSTAGES;
  constexpr int VS = C::VSTAGES;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;  // (a constant address: rounded up here, it and what follows from it cost registers in every role)
  // [ITEMS][INFO]: the item (s: -1 past the last), [5] a masked row may meet a value that is not finite
  int* infos = reinterpret_cast<int*>(sm + C::INFO_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  // Phases count over all items of the CTA.
  uint64_t* kfull = bars;                  // [KS] K of a block landed
  uint64_t* vfull = kfull + KS;            // [VS] V of a block may be multiplied
  uint64_t* vraw = vfull + VS;             // [VS] V of a block that some row does not see all of has landed
  // step n: P V of block n - 1, then Q K^T of block n.  One commit per step and tile frees K of
  // block n and V of block n - 1.
  uint64_t* done = vraw + VS;              // [DONE] both tiles' MMAs of a step have completed
  uint64_t* sfull = done + C::DONE;        // [tile] S of the tile's next block is in TMEM
  uint64_t* pfull = sfull + TC_TILES;      // [tile][half] P of 64 keys of that block is written (128 arrivals)
  uint64_t* pvhalf = pfull + 2 * TC_TILES; // [tile] P V of the first 64 keys of that block has completed
                                           // (EARLY: of the block)
  uint64_t* sfree = pvhalf + TC_TILES;     // [tile] EARLY: S of the block is done with (128 arrivals)
  uint64_t* pvdone = sfree + TC_TILES;     // [tile] the last P V of the tile's item has completed
  uint64_t* lready = pvdone + TC_TILES;    // [tile] the sums of the item's weights are stored (128 arrivals)
  uint64_t* ofree = lready + TC_TILES;     // [tile] the sums and O of the item are read (128 arrivals)
  uint64_t* qbar = ofree + TC_TILES;       // [tile] Q of the tile's next item landed
  uint64_t* drain = qbar + TC_TILES;       // [tile] every MMA issued has completed
  uint64_t* turn = drain + TC_TILES;       // [tile] its MMA warp may issue the next step
  uint64_t* ifull = turn + TC_TILES;       // [ITEMS] an item is published
  uint64_t* begun = ifull + C::ITEMS;      // the loads of an item come to its last three blocks
  uint64_t* cbar = begun + 1;              // the answer about another CTA landed
  float* sums = reinterpret_cast<float*>(sm + C::SUM_OFF);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::SLOT_OFF);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int tt = p.tile_tokens;

  // What needs no input is set up while the kernel before this one ends.
  if (warp == C::MMA_WARP && lane == 0) {
    for (int i = 0; i < KS; ++i) mbar_init(&kfull[i], 1);
    for (int i = 0; i < VS; ++i) mbar_init(&vfull[i], 1);
    for (int i = 0; i < VS; ++i) mbar_init(&vraw[i], 1);
    for (int i = 0; i < C::DONE; ++i) mbar_init(&done[i], TC_TILES);
    for (int i = 0; i < TC_TILES; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[2 * i], TC_ROWS);
      mbar_init(&pfull[2 * i + 1], TC_ROWS);
      mbar_init(&pvhalf[i], 1);
      mbar_init(&sfree[i], TC_ROWS);
      mbar_init(&pvdone[i], 2);
      mbar_init(&lready[i], TC_ROWS);
      mbar_init(&ofree[i], C::SIDE);
      mbar_init(&qbar[i], 1);
      mbar_init(&drain[i], 1);
      mbar_init(&turn[i], 1);
    }
    for (int i = 0; i < C::ITEMS; ++i) mbar_init(&ifull[i], 1);
    mbar_init(begun, 1);
    mbar_init(cbar, 1);
    fence_mbar_init();
    tma_prefetch_map(&p.tmap_q);
    tma_prefetch_map(&p.tmap_k);
    tma_prefetch_map(&p.tmap_v);
  }
  // Rows of the tiles that a group leaves over are no query's: zeros, whose scores need no care.
  if (tt * G < TC_ROWS) {
#pragma unroll 1
    for (int i = tt * G * 8 + static_cast<int>(threadIdx.x); i < TC_ROWS * 8; i += C::THREADS)
      for (int b = 0; b < TC_TILES * C::DBOX; ++b) *reinterpret_cast<uint4*>(sm + b * C::QATOM + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  grid_dependency_wait();
  // Tensor memory after the wait, and the next kernel only after that: a CTA that held it and waited for a kernel whose
  // CTAs still want theirs on the same SM would never end, nor would they.
  if (warp == 0) {
    tmem_alloc(tslot, C::TMEM_COLS);
    allow_dependent_launch();
  }

  PackedItem it;
  ListPlace known;
  const bool found_one = find_packed_item<IS_RAGGED>(p, make_uint3(blockIdx.x, blockIdx.y, blockIdx.z), it, known);
  const bool aligned = (smem_addr(smem_raw) & 1023u) == 0;  // (as declared)
  if (!found_one || !aligned) {
    if (found_one) write_nan_rows<T, HEAD_DIM>(p, it, threadIdx.x, C::THREADS);
    __syncwarp();
    if (warp == 0) tmem_dealloc(*tslot, C::TMEM_COLS);
    return;
  }
  auto load_q = [&](const PackedItem& i, int u) {  // one thread
    mbar_arrive_expect_tx(&qbar[u], C::DBOX * tt * G * 128);
    for (int db = 0; db < C::DBOX; ++db)
      tma_load_3d(sm + u * C::QBYTES + db * C::QATOM, &p.tmap_q, db * BOX_DIMS, i.kvh * G, i.q0 + i.ta + u * tt, &qbar[u]);
  };
  auto publish = [&](const PackedItem& i, int k) {  // one thread
    int* f = infos + (k % C::ITEMS) * C::INFO;
    f[0] = i.s, f[1] = i.kvh, f[2] = i.ta, f[3] = i.q0, f[4] = i.qlen, f[5] = 0;
    mbar_arrive(&ifull[k % C::ITEMS]);
  };
  // Item k of the CTA, published.
  auto item = [&](int k) -> PackedItem {
    const volatile int* f = infos + (k % C::ITEMS) * C::INFO;
    PackedItem i;
    i.s = f[0], i.kvh = f[1], i.ta = f[2], i.q0 = f[3], i.qlen = f[4];
    return i;
  };
  // Waits for it; false past the last (or when the warp of the items gave up).
  auto has_item = [&](int k) -> bool {
    return __all_sync(kFullMask, tc_wait(&ifull[k % C::ITEMS], (k / C::ITEMS) & 1)) &&
           *const_cast<const volatile int*>(infos + (k % C::ITEMS) * C::INFO) >= 0;
  };
  auto read_item = [&](int k, PackedItem& i) -> bool {
    if (!has_item(k)) return false;
    i = item(k);
    return true;
  };

  if (warp == C::MMA_WARP && lane == 0) {
    for (int u = 0; u < it.tiles(tt); ++u) load_q(it, u);
    publish(it, 0);
    if (it.blocks(tt) <= C::ASK_AT_ONCE) ask_for_cta(sm + C::RESP_OFF, cbar);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp >= C::SIDE_WARP && warp < C::MMA_WARP) {
    // ------------------------------------------------ the cache write and the outputs
    set_max_regs<false, C::SIDE_REGS>();
    const int tid = threadIdx.x - C::SIDE_WARP * 32;
    constexpr int U = HEAD_DIM / 8;  // 16-byte units of a row
    // The item's own tokens' rows into the pools: 2 U lanes take the key's and the value's units of a token, eight
    // tokens of theirs on the way at a time.
    auto write_cache = [&](const PackedItem& i) {
      constexpr int AT_ONCE = 8;
      constexpr int STEP = C::SIDE / (2 * U);  // tokens apart
      const int end = i.kend(tt) - i.ta;
      int me = tid;
      use_here(me);  // (what follows from it is not worth registers elsewhere)
      const int unit = me % U;
      const bool is_v = me / U & 1;
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
      const T* src = (is_v ? static_cast<const T*>(p.value) : static_cast<const T*>(p.key)) + (i.q0 + i.ta) * stride +
                     i.kvh * HEAD_DIM + unit * 8;
      uint4* dst = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache) + i.kvh * U + unit;
      const int64_t* slots = p.slot_mapping + i.q0 + i.ta;
#pragma unroll 1
      for (int t0 = me / (2 * U); t0 < end; t0 += AT_ONCE * STEP) {
        uint4 v[AT_ONCE];
        int64_t slot[AT_ONCE];
#pragma unroll
        for (int a = 0; a < AT_ONCE; ++a) {
          const int t = t0 + a * STEP;
          slot[a] = t < end ? __ldg(slots + t) : -1;
          if (t < end) v[a] = __ldg(reinterpret_cast<const uint4*>(src + t * stride));
        }
#pragma unroll
        for (int a = 0; a < AT_ONCE; ++a)
          if (slot[a] >= 0 && slot[a] < p.num_slots) dst[slot[a] * p.num_kv_heads * U] = v[a];
      }
    };
    // O / l of tile u of item k: a row per thread
    const uint32_t tO = tmem + C::O_COL + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    uint32_t opar = 0;  // parities of lready and pvdone, a bit per tile
    auto outputs = [&](const PackedItem& i, int k, int u) {
      const bool done_ok = __all_sync(kFullMask, tc_wait(&lready[u], opar >> u & 1)) &&
                           __all_sync(kFullMask, tc_wait(&pvdone[u], opar >> u & 1));
      opar ^= 1u << u;
      tc_fence_after_sync();
      const float inv = done_ok ? 1.f / sums[u * TC_ROWS + tid] : NAN;
      const bool fix = *const_cast<const volatile int*>(infos + (k % C::ITEMS) * C::INFO + 5);
      // A thread holds one row, and rows of different tokens are far apart in `out`: four lanes exchange their
      // 16-byte units, so that a store writes 64 bytes of each of eight rows.
      int row = tid;
      use_here(row);
      const int t0 = i.ta + u * tt;
      const int t_end = i.tile_end(u, tt);
      uint4* base = static_cast<uint4*>(p.out) + (static_cast<size_t>(i.q0 + t0) * p.num_heads + i.kvh * G) * U;
      uint32_t at[4];  // 16-byte units from there (below 128 tokens x 2^20 heads x 16); ~0: past the tile's last token
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int rr = (row & ~3) + y;
        const int q = rr * p.inv_g >> 16;  // (rows past the tile's last token count as the next one's)
        at[y] = t0 + q < t_end ? static_cast<uint32_t>(q * p.num_heads + rr - q * G) * U + (row & 3) : ~0u;
      }
#pragma unroll 1
      for (int c = 0; c < HEAD_DIM; c += 32) {
        uint32_t o[32];
        tmem_ld16(tO + 256 * u + c, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
        tmem_ld16(tO + 256 * u + c + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
        tmem_wait_ld();
        if (c + 32 == HEAD_DIM) {  // all of O is read
          tc_fence_before_sync();
          mbar_arrive(&ofree[u]);
        }
        uint4 unit[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t w[4];
#pragma unroll
          for (int d = 0; d < 4; ++d)
            w[d] = pack2<T>(__uint_as_float(o[8 * y + 2 * d]) * inv, __uint_as_float(o[8 * y + 2 * d + 1]) * inv);
          unit[y] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        transpose4(unit, row);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (at[y] != ~0u) base[at[y] + c / 8] = unit[y];
      }
      if (fix) {  // rare: the row takes the values that are not finite among the keys that entered as 0
        __syncwarp();
        const int q = row * p.inv_g >> 16;
        uint32_t* o = reinterpret_cast<uint32_t*>(base + (static_cast<size_t>(q) * p.num_heads + row - q * G) * U);
#pragma unroll 1
        for (int key = t0 + q < t_end ? i.ta + 1 : INT32_MAX; key <= t0 + q; ++key) {
          const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.value) + (i.q0 + key) * p.v_stride +
                                                                i.kvh * HEAD_DIM);
#pragma unroll 1
          for (int d = 0; d < HEAD_DIM / 2; ++d) {
            const uint32_t w = __ldg(v + d);
            const uint32_t m = not_finite<T>(w);
            if (m == 0) continue;
            const uint32_t x = o[d];
            const uint32_t lo = m & 0xffffu ? join_not_finite<T>(x & 0xffffu, w & 0xffffu) : x & 0xffffu;
            const uint32_t hi = m >> 16 ? join_not_finite<T>(x >> 16, w >> 16) : x >> 16;
            o[d] = lo | hi << 16;
          }
        }
      }
    };
    bool go = true;
#pragma unroll 1
    for (int k = 0; go; ++k) {
      if (p.slot_mapping) write_cache(it);
#pragma unroll 1
      for (int u = 0; u < it.tiles(tt); ++u) outputs(it, k, u);
      go = all_meet<C::SIDE>(read_item(k + 1, it));  // (the warps go on or give up together)
    }
    tc_fence_before_sync();
    __syncthreads();
    return;
  }

  if (warp >= C::MMA_WARP) {
    set_max_regs<false, C::MMA_REGS>();
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFullMask, tc_wait(bar, parity)) != 0; };
    if (warp < C::ITEM_WARP) {
      // ---------------------------------------------- MMA issue: warp u, tile u
      // The whole warp runs the loop and one elected lane issues: every value stays uniform, so descriptors
      // sit in uniform registers.
      const int u = __shfl_sync(kFullMask, warp - C::MMA_WARP, 0);
      const uint64_t dq = umma_desc_sw128(smem_addr(sm + u * C::QBYTES), 16, 1024);    // Q, K-major
      const uint64_t dk = umma_desc_sw128(smem_addr(sm + C::K_OFF), 16, 1024);         // K, K-major
      const uint64_t dv = umma_desc_sw128(smem_addr(sm + C::V_OFF), C::KATOM, 1024);   // V, MN-major
      const uint32_t tS = tmem + 256 * u;
      const uint32_t tP = tS + C::P_COL;
      const uint32_t tO = tS + C::O_COL;
      // stages of the next block's K and of the current one's V, parities of the phases
      int kslot = 0, vslot = 0, dslot = 0;
      uint32_t kpar = 0, vpar = 0, spar = 0, ppar = 0, qpar = 0, tpar = u ^ 1;
      uint32_t opar = 0;
      bool was = false;                // the tile had an item before
      bool q_open = it.tiles(tt) > u;  // Q was asked for and not waited for
      // Three barriers at once, a lane each: the waits cost a hundred cycles together, not each.
      // (A test, not a wait that suspends: that one sleeps past the completion of one lane's
      // barrier while another lane's is open.)  The limit is some seconds.
      auto wait3 = [&](uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t* b2, uint32_t p2) -> bool {
        uint64_t* b = lane == 0 ? b0 : lane == 1 ? b1 : b2;
        const uint32_t par = lane == 0 ? p0 : lane == 1 ? p1 : p2;
#pragma unroll 1
        for (int i = 0; i < 1 << 26; ++i)
          if (__all_sync(kFullMask, mbar_test(b, par))) return true;
        return false;
      };
      auto qk = [&]() {
        const uint64_t kj = umma_desc_add(dk, kslot * C::KBYTES);
#pragma unroll
        for (int ks = 0; ks < HEAD_DIM / 16; ++ks) {
          const uint32_t off = (ks >> 2) * C::QATOM + ((ks & 3) << 5);
          const uint32_t koff = (ks >> 2) * C::KATOM + ((ks & 3) << 5);
          umma_f16_elect(tS, umma_desc_add(dq, off), umma_desc_add(kj, koff), C::ID_S, ks > 0);
        }
      };
      uint32_t fpar = 0;  // EARLY: of sfree
      auto first_qk = [&]() -> bool {  // of an item
        const bool busy = C::EARLY && was;  // (S of the tile's item before)
        if (!wait3(&qbar[u], qpar, busy ? &sfree[u] : &qbar[u], busy ? fpar : qpar, &kfull[kslot], kpar)) return false;
        fpar ^= busy;
        tc_fence_after_sync();
        qpar ^= 1;
        q_open = false;
        qk();
        umma_commit_elect(&sfull[u]);
        return true;
      };
      auto end_step = [&]() {
        umma_commit_elect(&done[dslot]);
        dslot = dslot + 1 == C::DONE ? 0 : dslot + 1;
        kpar ^= kslot + 1 == KS;
        kslot = kslot + 1 == KS ? 0 : kslot + 1;
      };
      // The tiles' MMAs take turns, so that one tile's run under the other's softmax.  (Not EARLY: there the softmax
      // warps of both tiles have work all the time.)
      auto pass_turn = [&]() {
        if (lane == 0) mbar_arrive(&turn[u ^ 1]);
        __syncwarp();
      };
      // P V of the current block in the tile's turn, and Q K^T of the next one; first: the item's
      // first block, last: the tile's last one
      auto step = [&](bool first, bool last) -> bool {
        if constexpr (C::EARLY) {
          if (!last) {
            if (!wait3(&sfree[u], fpar, &sfree[u], fpar, &kfull[kslot], kpar)) return false;
            fpar ^= 1;
            tc_fence_after_sync();
            qk();
            umma_commit_elect(&sfull[u]);
            spar ^= 1;
          }
        }
        uint64_t* const go = C::EARLY ? &vfull[vslot] : &turn[u];
        if (!wait3(go, C::EARLY ? vpar : tpar, &vfull[vslot], vpar, &pfull[2 * u], ppar)) return false;
        tpar ^= 1;
        if (first) {  // O of the tile's item before is read
          if (was && !wait3(&ofree[u], opar, &ofree[u], opar, &ofree[u], opar)) return false;
          opar ^= was;
          was = true;
        }
        tc_fence_after_sync();
        const uint64_t vj = umma_desc_add(dv, vslot * C::KBYTES);
        // the first 64 keys while the softmax writes the weights of the others
#pragma unroll
        for (int kk = 0; kk < TC_KEYS / 32; ++kk)  // 16 keys = 8 columns of P
          umma_f16_ts_elect(tO, tP + 8 * kk, umma_desc_add(vj, kk * 2048), C::ID_PV, !first || kk > 0);
        if constexpr (!C::EARLY) umma_commit_elect(&pvhalf[u]);
        uint64_t* p1 = &pfull[2 * u + 1];
        const bool k_too = !C::EARLY && !last;
        if (!wait3(p1, ppar, p1, ppar, k_too ? &kfull[kslot] : p1, k_too ? kpar : ppar)) return false;
        ppar ^= 1;
        tc_fence_after_sync();
#pragma unroll
        for (int kk = TC_KEYS / 32; kk < TC_KEYS / 16; ++kk)
          umma_f16_ts_elect(tO, tP + 8 * kk, umma_desc_add(vj, kk * 2048), C::ID_PV, true);
        if constexpr (C::EARLY) {
          umma_commit_elect(&pvhalf[u]);
        } else {
          if (!last) qk();
          pass_turn();
        }
        if (last) {
          if (lane == 0) mbar_arrive(&pvdone[u]);
          umma_commit_elect(&pvdone[u]);
        } else if (!C::EARLY) {
          umma_commit_elect(&sfull[u]);
          spar ^= 1;
        }
        return true;
      };
      // a step of the item in which the tile has no block: at the pace of the other tile
      auto no_step = [&]() -> bool {
        if (!wait3(C::EARLY ? &vfull[vslot] : &turn[u], C::EARLY ? vpar : tpar, &vfull[vslot], vpar, &vfull[vslot], vpar))
          return false;
        tpar ^= 1;
        if constexpr (!C::EARLY) pass_turn();
        return true;
      };
      auto next_v = [&]() {
        vpar ^= vslot + 1 == VS;
        vslot = vslot + 1 == VS ? 0 : vslot + 1;
      };
      int nb, nblk;  // blocks of the tile and of the item
      auto lengths = [&](const PackedItem& i) {
        nb = __shfl_sync(kFullMask, i.tile_blocks(u, tt), 0);
        nblk = __shfl_sync(kFullMask, i.blocks(tt), 0);
      };
      lengths(it);
      bool ok = nb == 0 || first_qk();
      if (ok) end_step();
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        // all blocks but the item's last
#pragma unroll 1
        for (int j = 0; j + 1 < nblk; ++j) {
          ok = j < nb ? step(j == 0, j + 1 == nb) : no_step();
          if (!ok) break;
          end_step();
          next_v();
        }
        if (!ok) break;
        // the last one, and Q K^T of the next item's first
        const bool more = has_item(k + 1);
        const int last_nb = nb, last = nblk - 1;
        if (more) lengths(item(k + 1));
        if (more && nb > 0) {
          if (last_nb > 0) ok = wait(&sfull[u], spar);  // the tile's last S is there: its Q has been read
          if (!ok) break;
          if (lane == 0) load_q(item(k + 1), u);
          q_open = true;
          __syncwarp();
        }
        ok = last < last_nb ? step(last == 0, true) : no_step();
        if (!ok) break;
        if (last_nb > 0) spar ^= 1;
        if (!more) break;
        if (nb > 0) {
          ok = first_qk();
          if (!ok) break;
        }
        end_step();
        next_v();
      }
      umma_commit_elect(&drain[u]);  // every MMA finishes before the TMEM is released
      wait(&drain[u], 0);
      if (q_open) wait(&qbar[u], qpar);  // (after a wait ran out)
      tc_fence_before_sync();
    } else if (warp == C::ITEM_WARP) {
      // ---------------------------------------------- items, and values that rows must not meet
      int asked = 0;                                 // answers that were taken
      bool open = it.blocks(tt) <= C::ASK_AT_ONCE;  // one is on its way
      auto ask = [&]() {
        if (lane == 0) {
          fence_proxy_async_smem();
          ask_for_cta(sm + C::RESP_OFF, cbar);
        }
        open = true;
      };
      // A weight of 0 times a value that is not finite must not occur.  In blocks that some rows do not see all of,
      // keys past the item's last become zeros; what is not finite in keys that some tokens see and others do
      // not enters as 0, and the rows that see it take it at the end.
      constexpr int U = HEAD_DIM / 8;  // 16-byte units of a row
      auto make_safe = [&](uint8_t* stage, int key0, int ta, int kend) -> bool {  // whether something was not finite
        uint32_t any = 0;
#pragma unroll 1
        for (int x = (max(0, ta + 1 - key0) & ~31) | lane; x < TC_KEYS; x += 32) {  // a row per lane
          const int key = key0 + x;
          if (key <= ta) continue;
          uint8_t* row = stage + x * 128;
          if (key >= kend) {
#pragma unroll
            for (int y = 0; y < U; ++y)  // (from different units on: no bank conflict)
              *reinterpret_cast<uint4*>(row + (y >> 3) * C::KATOM + ((y + x) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            continue;
          }
          uint32_t top = 0;  // the largest magnitudes of the row's pairs, NaN above all: one instruction a pair
#pragma unroll
          for (int y = 0; y < U; ++y) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + (y >> 3) * C::KATOM + ((y + x) & 7) * 16);
            top = max_abs<T>(max_abs<T>(max_abs<T>(max_abs<T>(top, w.x), w.y), w.z), w.w);
          }
          if (not_finite<T>(top) == 0) continue;
#pragma unroll 1
          for (int y = 0; y < U; ++y) {
            uint4* at = reinterpret_cast<uint4*>(row + (y >> 3) * C::KATOM + ((y + x) & 7) * 16);
            const uint4 w = *at;
            const uint4 m = make_uint4(not_finite<T>(w.x), not_finite<T>(w.y), not_finite<T>(w.z), not_finite<T>(w.w));
            const uint32_t bad = m.x | m.y | m.z | m.w;
            if (bad) *at = make_uint4(w.x & ~m.x, w.y & ~m.y, w.z & ~m.z, w.w & ~m.w);
            any |= bad;
          }
        }
        return any != 0;
      };
      // Whichever comes first: a block of V to look through, or an item to find because the loads come to the end of
      // the last one.  (Found at once it would be taken from CTAs that are free sooner.)
      int found = 1, begins = 0;    // items published, starts of loads taken
      int at = 0, n0 = 0;           // the item whose values are next, and the blocks of those before
      int j = it.first_masked();    // its next block
      uint32_t seen = 0;            // parities of vraw
      bool more = true, ok = true;
      PackedItem now = it;          // item `at`
      uint64_t idle = 0;            // since when there is nothing to do
#pragma unroll 1
      while (more || at < found) {
        bool did = false;
        if (at < found) {
          const int slot = (n0 + j) % VS;
          if (__all_sync(kFullMask, mbar_test(&vraw[slot], seen >> slot & 1))) {
            seen ^= 1u << slot;
            if (make_safe(sm + C::V_OFF + slot * C::KBYTES, j * TC_KEYS, now.ta, now.kend(tt)))
              *const_cast<volatile int*>(infos + (at % C::ITEMS) * C::INFO + 5) = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&vfull[slot]);
            if (++j == now.blocks(tt)) {
              n0 += j;
              if (++at < found) {
                now = item(at);
                j = now.first_masked();
              }
            }
            did = true;
          }
        }
        if (more && __all_sync(kFullMask, mbar_test(begun, begins & 1))) {
          ++begins;
          did = true;
          if (!open) ask();
          for (;;) {
            if (!wait(cbar, asked & 1)) {
              ok = false;
              break;
            }
            ++asked;
            uint3 id;
            more = cta_given(sm + C::RESP_OFF, id);
            open = false;
            __syncwarp();  // every lane has read the answer
            if (!more) {
              it.s = -1;
              break;
            }
            const bool has = find_packed_item<IS_RAGGED>(p, id, it, known);
            if (!has || it.blocks(tt) <= C::ASK_AT_ONCE) ask();
            if (has) break;
          }
          if (!ok) break;
          if (lane == 0) {
            publish(it, found);
            if (more)
              for (int u = 0; u < it.tiles(tt); ++u)  // Q is loaded late, when its place is free: from L2 then
                for (int db = 0; db < C::DBOX; ++db)
                  tma_prefetch_3d(&p.tmap_q, db * BOX_DIMS, it.kvh * G, it.q0 + it.ta + u * tt);
          }
          __syncwarp();
          if (more && at == found++) {
            now = it;
            j = now.first_masked();
          }
        }
        if (did) {
          idle = 0;
        } else if (idle == 0) {
          idle = global_timer_ns();
        } else if (__any_sync(kFullMask, global_timer_ns() - idle > WAIT_LIMIT_NS)) {
          ok = false;
          break;
        } else {
          __nanosleep(32);
        }
      }
      if (!ok) {  // a wait ran out: no more items, and NaN in what was asked for
        uint3 id;
        if (open && wait(cbar, asked & 1) && cta_given(sm + C::RESP_OFF, id) && find_packed_item<IS_RAGGED>(p, id, it, known))
          write_nan_rows<T, HEAD_DIM>(p, it, lane, 32);
        it.s = -1;
        if (more && lane == 0) publish(it, found);
      }
    } else {
      // ---------------------------------------------- loads of K and V
      bool go = true;
      int n = 0;  // blocks asked for, over all items
      uint32_t raw = 0, rawpar = 0;  // per stage of V: its last copy reports to vraw; the parity of the next that does
#pragma unroll 1
      for (int k = 0; go; ++k) {
        const int nblk = it.blocks(tt);
        const int jm = it.first_masked();
#pragma unroll 1
        for (int j = 0; j < nblk; ++j, ++n) {
          const int kslot = n % KS;
          const int vslot = n % VS;
          // K's stage is free after step n - KS, V's after step n - VS + 1
          const int step = max(n - KS, n - VS + 1);
          if (step >= 0 && !wait(&done[step % C::DONE], (step / C::DONE) & 1)) {
            go = false;
            break;
          }
          raw &= ~(1u << vslot);
          if (j >= jm) raw |= 1u << vslot, rawpar ^= 1u << vslot;
          if (lane == 0) {
            if (j == max(0, nblk - 3)) mbar_arrive(begun);
            uint64_t* vb = j < jm ? &vfull[vslot] : &vraw[vslot];
            mbar_arrive_expect_tx(&kfull[kslot], C::KBYTES);
            for (int db = 0; db < C::DBOX; ++db)
              tma_load_3d(sm + C::K_OFF + kslot * C::KBYTES + db * C::KATOM, &p.tmap_k, db * BOX_DIMS, it.kvh,
                          it.q0 + j * TC_KEYS, &kfull[kslot]);
            mbar_arrive_expect_tx(vb, C::KBYTES);
            for (int db = 0; db < C::DBOX; ++db)
              tma_load_3d(sm + C::V_OFF + vslot * C::KBYTES + db * C::KATOM, &p.tmap_v, db * BOX_DIMS, it.kvh,
                          it.q0 + j * TC_KEYS, vb);
          }
          __syncwarp();
        }
        go = go && read_item(k + 1, it);
      }
      // the copies in flight land before the shared memory is released
      for (int x = max(0, n - KS); x < n; ++x) wait(&kfull[x % KS], (x / KS) & 1);
      for (int x = max(0, n - VS); x < n; ++x) {
        const int vslot = x % VS;
        if (raw >> vslot & 1) wait(&vraw[vslot], (rawpar >> vslot & 1) ^ 1);
        else wait(&vfull[vslot], (x / VS) & 1);
      }
    }
    __syncthreads();
    return;
  }
  // ------------------------------------------------ softmax: warps 4 u .. 4 u + 3 run tile u
  set_max_regs<true, C::SOFT_REGS>();
  const int u = warp >> 2;
  const int r = 32 * (warp & 3) + lane;
  const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t tS = tmem + 256 * u + lane_off;
  const uint32_t tP = tS + C::P_COL;
  const uint32_t tO = tS + C::O_COL;
  auto token_of = [&](int row) { return row * p.inv_g >> 16; };  // of the tile
  const int own_t = token_of(r);
  const int least_t = token_of(r & ~31);
  const int most_t = token_of(r | 31);
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(kFullMask, tc_wait(bar, parity));
  };
  // A negative `scale` turns the order of the scores around: the largest product is then
  // the smallest score times the (negative) factor.
  const float a = p.scale_log2;
  const bool neg = a < 0.f;
  const float hidden = neg ? INFINITY : -INFINITY;
  const uint64_t a2 = pack_f32x2(a);
  auto further = [&](float x, float y) { return neg ? fminf(x, y) : fmaxf(x, y); };  // (of NaN and y: y)
  auto is_wide = [&](float bias) { return !(fabsf(bias) <= C::WIDE); };  // (also where t a is infinite or t is `hidden`)
  // What weights measured from t0 are multiplied by to be measured from t1.
  auto moved = [&](float t0, float t1) -> float {
    const float b0 = C::MID - rounded_up(t0 * a), b1 = C::MID - rounded_up(t1 * a);
    const bool w0 = is_wide(b0), w1 = is_wide(b1);
    return ex2(w0 ? (w1 ? (t0 - t1) * a : fmaf(t0, a, b1 - C::MID)) : w1 ? fmaf(-t1, a, C::MID - b0) : b1 - b0);
  };
  uint32_t spar = 0, opar = 0;  // parities of the tile's blocks, of its items' outputs
  bool stored = false;
#pragma unroll 1
  for (int k = 0;; ++k) {
    int left, seen;  // the tile's blocks to come; the keys of the block that all its rows see, minus one
    int tiles;
    {
      const PackedItem i = item(k);
      tiles = i.tiles(tt);
      left = i.tile_blocks(u, tt);
      seen = i.ta + u * tt;
    }
    float t_used = hidden, l = 0.f;  // the score that weights are measured from (`hidden`: no score yet), their sum
    float bias = 0.f;                // EARLY: the exponents' offset (0: no score yet)
    uint32_t x[TC_KEYS];  // the block's raw scores, later its weights
    auto load_half = [&](int h) {
#pragma unroll
      for (int c = TC_HALF * h; c < TC_HALF * (h + 1); c += 16) tmem_ld16(tS + c, *reinterpret_cast<uint32_t(*)[16]>(&x[c]));
      tmem_wait_ld();  // (at once: a register that a load still fills must not meet a branch)
    };
    // Hides the scores v of 16 keys, of which the first kv + 1 are visible.
    auto hide = [&](uint32_t* v, int kv) {
      const uint32_t m = kv < 0 ? 0u : kv > 15 ? ~0u : (2u << kv) - 1u;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!(m >> i & 1u)) v[i] = __float_as_uint(hidden);
    };
    // The score to take off first, and the exponent's offset, of a row that is measured from t_used.
    auto offsets = [&](float& off, float& bias) {
      const bool none = t_used == hidden;
      const float b = C::MID - rounded_up(t_used * a);
      const bool wide = !none && is_wide(b);
      off = wide ? t_used : 0.f;
      bias = none ? 0.f : wide ? C::MID : b;
    };
    // The weights of a half from its scores in TMEM, measured from t_used, 16 at a time, and their sums as the unrolled
    // code adds them: rows that need no care get the same bits.  (P goes over scores that were read, or beside them.)
    auto reweigh = [&](int h, int seen, uint64_t (&sum2)[2]) {
      uint32_t v[16];
      const int own = seen + own_t - TC_HALF * h;
      float off, bias;
      offsets(off, bias);
#pragma unroll 1
      for (int c = 0; c < TC_HALF; c += 16) {
        tmem_ld16(tS + TC_HALF * h + c, v);
        tmem_wait_ld();
        hide(v, own - c);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p0 = ex2(fmaf(__uint_as_float(v[2 * i]) - off, a, bias));
          const float p1 = ex2(fmaf(__uint_as_float(v[2 * i + 1]) - off, a, bias));
          sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(__float_as_uint(p0), __float_as_uint(p1)));
          w[i] = pack2<T>(p0, p1);
        }
        tmem_st8(tP + 32 * h + c / 2, w);
      }
    };
    // The weights of a half once more, those of the rows with `low` measured from the maximum of their scores, and O
    // and l after them; returns the row's sum.  Rare: a row's sum came out above the limit, or its scores are wide (then
    // its sum said nothing).
    auto again = [&](int h, int low, int seen) -> float {
      if (h == 1) {  // the first half's P V adds to O at this time
        wait(&pvhalf[u], spar ^ 1);
        tc_fence_after_sync();
      }
      uint32_t v[16];
      const int own = seen + own_t - TC_HALF * h;
      float top = t_used;
#pragma unroll 1
      for (int c = 0; c < TC_HALF; c += 16) {
        tmem_ld16(tS + TC_HALF * h + c, v);
        tmem_wait_ld();
        hide(v, own - c);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = further(top, __uint_as_float(v[i]));
      }
      if (t_used != hidden && is_wide(C::MID - rounded_up(t_used * a))) low = (top - t_used) * a > TC_RESCALE_LOG2;
      if (__any_sync(kFullMask, low)) {  // (never at an item's first scores, when O is still the last item's)
        const float f = low ? moved(t_used, top) : 1.f;
        if (low) t_used = top;
        l *= f;
#pragma unroll 1
        for (int c = 0; c < HEAD_DIM; c += 16) {
          tmem_ld16(tO + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
          tmem_st16(tO + c, v);
        }
      }
      uint64_t sum2[2] = {0, 0};
      reweigh(h, seen, sum2);
      const float2 s2 = unpack_f32x2(add_f32x2(sum2[0], sum2[1]));
      return s2.x + s2.y;
    };
#pragma unroll 1
    for (; left > 0; --left, seen -= TC_KEYS) {
      wait(&sfull[u], spar);
      spar ^= 1;
      tc_fence_after_sync();
      if constexpr (C::EARLY) {
        // All scores at once.  Their place is free for the next block's when the first half's weights are done: until then
        // a warp may have to weigh them once more.  (Given free as soon as they were loaded, before there was such a
        // case, 8 x 2048 tokens took 168 us; now 164.)
        load_half(0);
        load_half(1);
        if (seen + least_t < TC_KEYS - 1) {  // a key here may lie past some row of the warp
#pragma unroll
          for (int c = 0; c < TC_KEYS; c += 16)
            if (seen + least_t < c + 15) hide(x + c, seen + own_t - c);
        }
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) e[c] = __uint_as_float(x[c]);
        if (!neg) {
#pragma unroll
          for (int i = 4; i < TC_KEYS - 4; i += 8)
#pragma unroll
            for (int c = 0; c < 4; ++c) e[c] = fmaxf(fmaxf(e[c], __uint_as_float(x[i + c])), __uint_as_float(x[i + 4 + c]));
#pragma unroll
          for (int c = 0; c < 4; ++c) e[c] = fmaxf(e[c], __uint_as_float(x[TC_KEYS - 4 + c]));
          e[0] = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
        } else {
#pragma unroll
          for (int i = 4; i < TC_KEYS; i += 4)
#pragma unroll
            for (int c = 0; c < 4; ++c) e[c] = fminf(e[c], __uint_as_float(x[i + c]));
          e[0] = fminf(fminf(e[0], e[1]), fminf(e[2], e[3]));
        }
        // Weights are measured from another score at the first block and when the row maximum has grown by more than
        // 2^8; O and l then scale by f.
        const float top = e[0];
        const bool far = (top - t_used) * a > TC_RESCALE_LOG2;  // (a row without a score yet: by an infinity)
        int none = t_used == hidden;                            // nothing in O yet (opaque as below)
        use_here(none);
        const bool need = far && !none;
        const float b_new = C::MID - rounded_up(top * a);
        float f = need ? ex2(b_new - bias) : 1.f;
        if (far) bias = b_new;
        const bool wide = is_wide(bias);
        const uint64_t b2 = pack_f32x2(bias);
        bool wide_rows = false;
        uint64_t sum2[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 32 * h; i < 32 * h + 32; ++i) {
            const float2 t = unpack_f32x2(fma_f32x2(pack_f32x2(x[2 * i], x[2 * i + 1]), a2, b2));
            const float p0 = ex2(t.x), p1 = ex2(t.y);
            sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(__float_as_uint(p0), __float_as_uint(p1)));
            x[i] = pack2<T>(p0, p1);  // (its place was consumed)
          }
          if (h == 0) {
            wait(&pvhalf[u], spar);  // P V of the block before: it has read P and O stands
            tc_fence_after_sync();
            bool scale_o = false;
            if (__any_sync(kFullMask, need || wide)) {
              scale_o = __any_sync(kFullMask, need);
              wide_rows = __any_sync(kFullMask, wide);
              if (wide_rows && need) f = moved(t_used, top);
            }
            if (far) t_used = top;
            if (scale_o) {
#pragma unroll 1
              for (int c = 0; c < HEAD_DIM; c += 8) {  // (eight at a time: the scores hold registers)
                uint32_t o8[8];
                tmem_ld8(tO + c, o8);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) o8[i] = __float_as_uint(__uint_as_float(o8[i]) * f);
                tmem_st8(tO + c, o8);
              }
            }
            if (wide_rows) {  // rare: the weights of both halves once more
              sum2[0] = sum2[1] = 0;
              reweigh(0, seen, sum2);
              reweigh(1, seen, sum2);
              tmem_wait_st();
              tc_fence_before_sync();
              mbar_arrive(&sfree[u]);
              mbar_arrive(&pfull[2 * u]);
              mbar_arrive(&pfull[2 * u + 1]);
              break;
            }
            tc_fence_before_sync();
            mbar_arrive(&sfree[u]);
          }
          tmem_st16(tP + 32 * h, &x[32 * h]);
          tmem_st16(tP + 32 * h + 16, &x[32 * h + 16]);
          tmem_wait_st();
          tc_fence_before_sync();
          mbar_arrive(&pfull[2 * u + h]);
        }
        const float2 s2 = unpack_f32x2(add_f32x2(sum2[0], sum2[1]));
        l = fmaf(l, f, s2.x + s2.y);
      } else {
        // Half of the keys at a time, so that the first weights are on their way to the MMA while the second half is
        // at work.  The exponent's offset stays where it is as long as the weights' own sum says that they fit:
        // the maximum of a half is looked for at the first scores, and where its weights came out too large.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t* y = x + TC_HALF * h;
          if (h == 1 && seen + most_t < TC_HALF) {  // nobody of the warp sees a key of the second half
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = 0u;
            tmem_st16(tP + 32, &y[0]);
            tmem_st16(tP + 48, &y[0]);
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive(&pfull[2 * u + 1]);
            continue;
          }
          load_half(h);
          if (seen + least_t < TC_HALF * (h + 1) - 1) {  // a key here may lie past some row of the warp
#pragma unroll
            for (int c = 0; c < TC_HALF; c += 16)
              if (seen + least_t < TC_HALF * h + c + 15) hide(y + c, seen + own_t - TC_HALF * h - c);
          }
          float bias = C::MID - rounded_up(t_used * a);
          bool wide = is_wide(bias);
          if (__any_sync(kFullMask, wide)) {
            // (an opaque truth value: folded into the selection below, `t_used == hidden ? max(t_used, x) : t_used` has
            // come out as max(t_used, x))
            int none = t_used == hidden;
            use_here(none);
            if (__any_sync(kFullMask, none)) {  // a row's first scores
              float e[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) e[c] = __uint_as_float(y[c]);
#pragma unroll
              for (int i = 4; i < TC_HALF; i += 4)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  e[c] = neg ? fminf(e[c], __uint_as_float(y[i + c])) : fmaxf(e[c], __uint_as_float(y[i + c]));
              const float top = neg ? fminf(fminf(e[0], e[1]), fminf(e[2], e[3])) : fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
              // (a row that sees no key here stays without)
              if (none) t_used = further(t_used, top);
              bias = C::MID - rounded_up(t_used * a);
              none = t_used == hidden;
            }
            if (none) bias = 0.f;  // (no key seen yet)
            wide = is_wide(bias);
          }
          const uint64_t b2 = pack_f32x2(bias);
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < TC_HALF / 2; ++i) {
            const float2 t = unpack_f32x2(fma_f32x2(pack_f32x2(y[2 * i], y[2 * i + 1]), a2, b2));
            const float p0 = ex2(t.x), p1 = ex2(t.y);
            sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(__float_as_uint(p0), __float_as_uint(p1)));
            y[i] = pack2<T>(p0, p1);  // (its place was consumed)
          }
          const float2 s2 = unpack_f32x2(add_f32x2(sum2[0], sum2[1]));
          float sum = s2.x + s2.y;
          if (__any_sync(kFullMask, wide || sum > C::LIMIT)) {
            sum = again(h, sum > C::LIMIT, seen);
          } else {  // P in the half's 32 columns, over scores that are in registers
            tmem_st16(tP + 32 * h, &y[0]);
            tmem_st16(tP + 32 * h + 16, &y[16]);
          }
          l += sum;
          tmem_wait_st();
          tc_fence_before_sync();
          mbar_arrive(&pfull[2 * u + h]);
        }
      }
    }
    // the sums for the warps of the outputs, which have read the last item's
    if (u < tiles) {
      if (stored) {
        wait(&ofree[u], opar);
        opar ^= 1;
      }
      stored = true;
      sums[u * TC_ROWS + r] = ok ? l : NAN;
      mbar_arrive(&lready[u]);
    }
    if (!has_item(k + 1)) break;
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
}

// x as [rows][heads][HEAD_DIM] with rows of `stride` elements: boxes of 64 dims x `box_heads` x `box_rows`, 128-byte
// swizzled.
template <typename T>
cudaError_t make_rows_map(CUtensorMap* map, const void* x, int head_dim, int heads, int64_t rows, int64_t stride, int box_heads,
                          int box_rows) {
  EncodeTiledFn enc = nullptr;
  const cudaError_t e = encode_fn(&enc);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {BOX_DIMS, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estride[3] = {1, 1, 1};
  const CUresult r = enc(map, tma_dtype<T>(), 3, const_cast<void*>(x), dims, strides, box, estride,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int HEAD_DIM>
cudaError_t launch_packed_prefill_t(const PackedPrefillArgs& a, cudaStream_t stream) {
  using C = PpCfg<T, HEAD_DIM>;
  PackedParams p;
  const int group = a.num_heads / a.num_kv_heads;
  p.tile_tokens = TC_ROWS / group;
  cudaError_t e = make_rows_map<T>(&p.tmap_q, a.q, HEAD_DIM, a.num_heads, a.num_rows, a.q_stride, group, p.tile_tokens);
  if (e == cudaSuccess)
    e = make_rows_map<T>(&p.tmap_k, a.key, HEAD_DIM, a.num_kv_heads, a.num_rows, a.k_stride, 1, TC_KEYS);
  if (e == cudaSuccess)
    e = make_rows_map<T>(&p.tmap_v, a.value, HEAD_DIM, a.num_kv_heads, a.num_rows, a.v_stride, 1, TC_KEYS);
  if (e != cudaSuccess) return e;
  p.out = a.out;
  p.key = a.key;
  p.value = a.value;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.slot_mapping = a.slot_mapping;
  p.num_slots = a.num_slots;
  p.query_start_loc = a.query_start_loc;
  p.num_seqs = a.num_seqs;
  p.num_rows = a.num_rows;
  p.max_query_len = a.max_query_len;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = group;
  p.inv_g = 65536 / group + 1;
  const int pair_tokens = TC_TILES * p.tile_tokens;
  p.pair_magic = ~uint64_t{0} / pair_tokens + 1;  // (2^64 is no multiple of it or ends in zeros: either way rounded up)
  p.pairs = (a.max_query_len + pair_tokens - 1) / pair_tokens;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  // a factor of 0 would turn a masked score (an infinity) into NaN; 2^-149 makes 0 of every score
  if (p.scale_log2 == 0.f) p.scale_log2 = 1.401298464324817e-45f;
  // A grid over (sequence, pair) is mostly empty where one sequence is long and the others are short, and an empty
  // CTA takes half a microsecond of an SM: the list of all pairs is searched instead where the grid is much longer.
  // A search takes 2.6 us per 1000 sequences, so the more of them, the longer.  Measured, list against grid, one
  // prompt beside others: 2048, 63 of one token (ratio 22) 30 against 59 us; 8192, 2000 of 20 (96) 653 against
  // 3366; 1024, 4000 of one (16; here the grid) 1479 against 1432; 2000, 4000 of 100 (12; the grid) 7400 against 3266.
  const int64_t listed = a.num_rows / pair_tokens + static_cast<int64_t>(a.num_seqs);
  const int64_t boxed = static_cast<int64_t>(p.pairs) * a.num_seqs;
  const int64_t ratio = a.num_seqs > 256 ? a.num_seqs / 128 : 2;
  const bool ragged = boxed > ratio * listed && listed * a.num_kv_heads <= INT32_MAX;
  p.longest_first = p.pairs <= 65535;
  cudaLaunchConfig_t cfg = {};
  if (ragged) {
    cfg.gridDim = dim3(static_cast<unsigned>(listed * a.num_kv_heads));
  } else if (p.longest_first) {
    cfg.gridDim = dim3(a.num_kv_heads, a.num_seqs, p.pairs);
  } else {
    cfg.gridDim = dim3(p.pairs, a.num_kv_heads, a.num_seqs);
  }
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> smem_set[2];
  auto kern = ragged ? packed_prefill_tc_kernel<T, HEAD_DIM, true> : packed_prefill_tc_kernel<T, HEAD_DIM, false>;
  e = ensure_smem(kern, C::SMEM_BYTES, smem_set[ragged]);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

}  // namespace pa
