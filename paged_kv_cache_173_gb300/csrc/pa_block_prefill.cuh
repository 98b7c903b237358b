// pa_block_prefill.cuh -- prefill over block-scaled E4M3 pools on the tcgen05
// tensor cores.
//
//  block_prefill_tc_kernel  one CTA per SM; an item of work is a pair of query
//                           tiles of a (KV head, sequence), a tile 128 rows
//                           (128 / G new tokens x G heads).  Q K^T and P V in
//                           tensor memory (S 128 and O 128 columns per tile, P
//                           over S), one softmax thread per row with the block's
//                           128 scores in registers.
//
// The bound is the tensor cores: 4 x 128 x 128 x d multiply-adds per pair and 128
// keys, 2050 cycles at d = 128.  What kept them waiting, and what stands against it:
//  - The codes do not fit a kind::f16 MMA.  Four producer warps read them from the
//    pools (16 codes per lane and load, one block of 128 keys ahead, held in
//    registers while the stage is in use), widen them exactly to float16 and store
//    them in the swizzled layout that a TMA box of 16-bit rows would leave.
//  - A tile's chain (scores, softmax, weights, P V, next scores) takes longer than
//    its MMAs.  Two tiles alternate, an MMA warp for each, in turns, so that one
//    tile's MMAs run under the other's softmax.
//  - The start and the end of a pair (first loads, last outputs) took as long as
//    five blocks of keys when each pair had its own CTA.  A CTA goes on to the next
//    pair that has not started, and its producers, Q loads and first MMAs overlap
//    the outputs of the last pair.
//  - 128 scores per softmax thread leave few registers for the rest.  The launch's
//    512 x 128 registers are shared out by role, so that nothing is spilled in a loop.
// Measured through graph replays (fp16, 32/8 heads of 128, blocks of 16): 8 prompts of
// 2048 tokens 231 us, 2 of 16384 2998 us (0.77 of the measured peak), 16 x 512 on 16384
// cached 1551 us; bf16, 16 chunks of 509 on 1536 cached 205 us.  Before the codes were
// multiplied by a part of the value scale: 226, 2955, 1535 and 203 us; and before that, with
// one CTA per pair and one MMA warp for both tiles: 282, 3005, 1584 and 230 us.
//
// The mathematics of the scales.  The value scale of a block b is split,
// v_b = 2^(ref + 3) 2^kappa_b 2^r_b, with 2^ref the power of two of the largest scale
// among the item's first 128 keys.  2^kappa_b, -15 <= kappa_b <= 7, multiplies the
// widened codes: exact, and below 2^16.  What is left, 0 <= r_b < 1 for scales of 2^-12
// to 2^10 times 2^ref (0 for powers of two) and the rest beyond, moves into the exponent of
// the weight of key i:
//   w_i = 2^(s_i + r_b - M),   out = 2^(ref + 3) sum w_i 2^kappa_b code_i / sum w_i 2^-r_b,
// one fused multiply-add per score (key scale and r_b of its 16-key chunk), one
// multiply per chunk for the sum.  So over 22 powers of two a block's scale says
// nothing about the float16 weights of the others.  (With all of v_b in the exponent
// 16384 keys behind one by 10 nats whose block's scale is 2^11 times theirs came out 40%
// short.)  The largest weight is 2^7 to 2^15: the running maximum M moves when it has
// grown by 2^8, and stays 7 below; a weight is off by 2^-32 of the largest at most.
// r_b is held to -64 and more, and above 36 makes NaN of the item: within a spread of
// 2^100 neither a weight that counts in the sum nor the sum leaves float32.  So a value
// scale below 2^-76 times 2^ref reads as that, one of 2^47 times 2^ref is refused, and
// one below 2^-64 reads as 2^-64.
// (The multiplications, and the scales that the producers load for them, take 1 to 2.6%
// of the launch.  ref from the largest scale of all of the item's blocks, looked up
// by the warp of the scales one item ahead, took 3 to 5%: the next item is
// known too late for it.)
//
// bfloat16 queries: the softmax thread of a row scales it in shared memory by
// the power of two that brings its largest element to [2^14, 2^15) and writes
// it back as float16 (see load_q_frags_scaled); all MMAs run in float16, so P
// needs no residual.
//
// The method: causal multi-query attention over a paged cache ("in-depth
// reading", section 5.1, item 5), online softmax of "vLLM PagedAttention
// source walk-through", section 3.4.
#pragma once

#include "pa_block.cuh"
#include "pa_prefill.cuh"
#include "pa_tc.cuh"

namespace pa {

namespace {

struct BlockPrefillParams {
  CUtensorMap tmap_q;  // as PrefillTcParams
  void* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int max_blocks_per_seq;
  int num_heads;
  int num_kv_heads;
  int group;
  int log2_g;  // group = 1 << log2_g: it divides 128
  int log2_b;  // block_size = 1 << log2_b
  int num_blocks;
  int pairs;
  int tile_tokens;
  // grid order: (KV head, sequence, pair) or, longest_first = 0, (pair, KV head, sequence).  Ragged
  // kernels: one dimension, KV head and place in the list of all sequences' pairs, longest first.
  int longest_first;
  int num_seqs;
  float scale_log2;
  float least_factor;  // kLeastFactor with the sign of scale_log2
};

// Shared memory of one CTA: Q of both tiles, the K and V rings of widened
// codes, the scales of the V ring's blocks, the barriers.
template <int HEAD_DIM>
struct BpCfg {
  // Warps: two warpgroups of softmax, one of producers, and one of MMA issue (a warp per tile),
  // items and scales (one warp) and one idle warp.
  static constexpr int SOFT = TC_TILES * TC_ROWS;  // softmax threads
  static constexpr int PROD_WARP = SOFT / 32;
  static constexpr int PROD_WARPS = 4;
  static constexpr int PROD = PROD_WARPS * 32;
  static constexpr int MMA_WARP = PROD_WARP + PROD_WARPS;
  static constexpr int ITEM_WARP = MMA_WARP + TC_TILES;
  static constexpr int THREADS = SOFT + PROD + 128;
  // (d = 64 holds half the codes per producer; with the split of d = 128 it took 189 us, not 185)
  static constexpr int SOFT_REGS = HEAD_DIM == 64 ? 168 : 160;
  static constexpr int PROD_REGS = HEAD_DIM == 64 ? 112 : 120;
  static constexpr int MMA_REGS = HEAD_DIM == 64 ? 64 : 72;
  // what the warpgroups hold is what the block was launched with
  static_assert(SOFT * SOFT_REGS + PROD * PROD_REGS + 128 * MMA_REGS <= THREADS * 128, "registers");
  static constexpr int DBOX = HEAD_DIM / BOX_DIMS;
  static constexpr int QATOM = TC_ROWS * 128;
  static constexpr int QBYTES = DBOX * QATOM;
  static constexpr int KATOM = TC_KEYS * 128;
  static constexpr int KBYTES = DBOX * KATOM;
  static constexpr int CHUNKS = TC_KEYS / CHUNK;
  static constexpr int SMEM_MAX = 227 * 1024;
  static constexpr int RESERVE = 1024 + 2048;  // base alignment slack, scales, barriers
  static constexpr int STAGES_FIT = (SMEM_MAX - RESERVE - TC_TILES * QBYTES) / KBYTES;
  static constexpr int KSTAGES = STAGES_FIT / 2 < 4 ? STAGES_FIT / 2 : 4;
  static constexpr int VSTAGES = STAGES_FIT - KSTAGES < 4 ? STAGES_FIT - KSTAGES : 4;
  static_assert(KSTAGES >= 2 && VSTAGES >= 2, "the rings do not fit");
  static constexpr int K_OFF = TC_TILES * QBYTES;
  static constexpr int V_OFF = K_OFF + KSTAGES * KBYTES;
  static constexpr int SC_OFF = V_OFF + VSTAGES * KBYTES;  // [2 * GROUP][CHUNKS] float4
  static constexpr int GROUP = 4;  // blocks whose scales one warp loads together, a lane per 16-key chunk
  static_assert(GROUP * CHUNKS == 32, "one chunk per lane");
  static constexpr int INFO_OFF = SC_OFF + 2 * GROUP * CHUNKS * 16;
  static constexpr int ITEMS = 4;  // ring of published work items
  static constexpr int INFO = 12;  // words of an item
  static constexpr int RESP_OFF = INFO_OFF + ITEMS * INFO * 4;
  static constexpr int BAR_OFF = RESP_OFF + 16;
  static constexpr int DONE = VSTAGES;  // ring of completed steps
  static_assert(KSTAGES <= VSTAGES, "a step's commit is waited for before its place is used again");
  static constexpr int NBARS = KSTAGES + VSTAGES + DONE + 8 * TC_TILES + ITEMS + 5;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int LAYOUT_BYTES = SLOT_OFF + 16;
  static constexpr int SMEM_BYTES = LAYOUT_BYTES + 1024;
  static_assert(SMEM_BYTES <= SMEM_MAX, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ID_S = umma_idesc_f16(TC_ROWS, TC_KEYS, false, false);
  static constexpr uint32_t ID_PV = umma_idesc_f16(TC_ROWS, HEAD_DIM, false, true);
};

__device__ __forceinline__ uint4 ldg128(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// 2^-100: the least size of the factor that a raw score (below 2^33) is multiplied by; it makes 0 of
// every score.
constexpr float kLeastFactor = 7.888609052210118e-31f;

constexpr float kMidWeight = 7.f;  // log2 of the largest weight when the running maximum has just moved
constexpr int kLeastRest = -64;    // of a value scale's powers of two
constexpr int kMostRest = 36;

// The bits of a value scale for a maximum; what is no scale does not count.
__device__ __forceinline__ int scale_bits(float v) { return v <= kFloatMax ? __float_as_int(v) : 0; }
// The exponent of a value scale: that of 2^-64 for smaller ones (and negative ones, which make NaN elsewhere).
__device__ __forceinline__ int value_exp(float v) { return (max(__float_as_int(v), (127 - 64) << 23) >> 23) - 127; }
// ref by the largest bits over the first 128 keys; of values around 1 where those are all zero.
__device__ __forceinline__ int ref_exp(int bits) {
  const int e = value_exp(__int_as_float(bits));
  return e > -64 ? e : -8;
}
// The power of two of a value scale that multiplies the codes: 448 * 2^7 < 65504, and
// 2^-9 * 2^-15 is float16's smallest step.
__device__ __forceinline__ int kappa(int e, int ref) { return min(max(e - ref - 3, -15), 7); }

// Two float16 times two.
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 codes widened to float16: two 16-byte units.
__device__ __forceinline__ void widen16(const uint4& c, uint4& a, uint4& b) {
  e4m3x4_to_half2x2(c.x, a.x, a.y);
  e4m3x4_to_half2x2(c.y, a.z, a.w);
  e4m3x4_to_half2x2(c.z, b.x, b.y);
  e4m3x4_to_half2x2(c.w, b.z, b.w);
}

// ---------------------------------------------------------------- work items
// An item is a pair of query tiles of one (sequence, KV head).  A CTA starts with
// the item of its own grid index and then takes over CTAs that have not started
// yet, one at a time: cancelling one hands over its index.

struct PrefillItem {
  int s, kvh;
  int ta;    // first new token of tile 0
  int q0;    // row of the sequence's first new token
  int qlen;  // its new tokens
  int base;  // its tokens before them

  __device__ __forceinline__ int tiles(int tt) const { return ta + tt < qlen ? 2 : 1; }
  // one past tile u's last new token, and the key blocks that it meets
  __device__ __forceinline__ int tile_end(int u, int tt) const { return min(qlen, ta + (u + 1) * tt); }
  __device__ __forceinline__ int tile_blocks(int u, int tt) const {
    return u < tiles(tt) ? (base + tile_end(u, tt) + TC_KEYS - 1) / TC_KEYS : 0;
  }
  __device__ __forceinline__ int kend(int tt) const { return base + tile_end(1, tt); }  // the keys' end
  __device__ __forceinline__ int blocks(int tt) const { return (kend(tt) + TC_KEYS - 1) / TC_KEYS; }
};

// The pairs of query tiles of sequence i (0 past the last).
__device__ __forceinline__ int pairs_of(const BlockPrefillParams& p, int i) {
  if (i >= p.num_seqs) return 0;
  const int n = __ldg(p.query_start_loc + i + 1) - __ldg(p.query_start_loc + i);
  return n <= 0 ? 0 : min(((n - 1) >> (8 - p.log2_g)) + 1, p.pairs);
}

// Place `at` of the list of all sequences' pairs, the pairs of highest number first and those of
// one number in the sequences' order: (pair, sequence), or false past the last.  The whole warp
// searches; C(x), the pairs numbered above x, is the sum over the sequences of max(0, pairs - 1 - x).
__device__ __forceinline__ bool ragged_item(const BlockPrefillParams& p, int at, int& pair, int& s) {
  const int lane = threadIdx.x & 31;
  auto above = [&](int x) {
    int n = 0;
    for (int i = lane; i < p.num_seqs; i += 32) n += max(0, pairs_of(p, i) - 1 - x);
    return __reduce_add_sync(FULL_MASK, n);
  };
  if (at >= above(-1)) return false;
  int lo = 0, hi = p.pairs - 1;  // the least x with C(x) <= at
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (above(mid) <= at) hi = mid;
    else lo = mid + 1;
  }
  int rank = at - above(lo);
  for (int i = 0; i < p.num_seqs; i += 32) {
    const unsigned has = __ballot_sync(FULL_MASK, pairs_of(p, i + lane) > lo);
    const int n = __popc(has);
    if (rank < n) {
      pair = lo;
      s = i + static_cast<int>(__fns(has, 0, rank + 1));
      return true;
    }
    rank -= n;
  }
  return false;
}

// The item of a grid index, by whole warps: 0 nothing to do, 1 work, -1 a context length that cannot be.
template <bool IS_RAGGED>
__device__ __forceinline__ int find_item(const BlockPrefillParams& p, uint3 id, PrefillItem& it) {
  int pair;
  if constexpr (IS_RAGGED) {
    it.kvh = id.x % p.num_kv_heads;
    if (!ragged_item(p, id.x / p.num_kv_heads, pair, it.s)) return 0;
  } else {
    const bool lf = p.longest_first;
    pair = p.pairs - 1 - static_cast<int>(lf ? id.z : id.x);  // the longest pairs start first
    it.kvh = lf ? id.x : id.y;
    it.s = lf ? id.y : id.z;
  }
  it.q0 = __ldg(p.query_start_loc + it.s);
  it.qlen = __ldg(p.query_start_loc + it.s + 1) - it.q0;
  const int ctx = __ldg(p.context_lens + it.s);
  it.base = ctx - it.qlen;
  it.ta = 2 * pair * p.tile_tokens;
  if (it.ta >= it.qlen) return 0;
  return ctx < it.qlen || ctx > (p.max_blocks_per_seq << p.log2_b) ? -1 : 1;
}

// NaN in the rows of an item, by `n` threads.
template <typename T, int HEAD_DIM>
__device__ __forceinline__ void write_nan_rows(const BlockPrefillParams& p, const PrefillItem& it, int i, int n) {
  constexpr int U = HEAD_DIM / 8;
  const uint32_t v = pack2<T>(NAN, NAN);
  const int rows = (it.tile_end(1, p.tile_tokens) - it.ta) << p.log2_g;
#pragma unroll 1
  for (; i < rows * U; i += n) {
    const int r = i / U;
    T* row = static_cast<T*>(p.out) + (static_cast<size_t>(it.q0 + it.ta + (r >> p.log2_g)) * p.num_heads +
                                       it.kvh * p.group + (r & (p.group - 1))) * HEAD_DIM;
    reinterpret_cast<uint4*>(row)[i % U] = make_uint4(v, v, v, v);
  }
}

// The bytes of a word of codes that are NaN, as 0x80 each.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

template <typename T, int HEAD_DIM, bool IS_RAGGED>
__global__ void __launch_bounds__(BpCfg<HEAD_DIM>::THREADS, 1)
block_prefill_tc_kernel(const __grid_constant__ BlockPrefillParams p) {
  using C = BpCfg<HEAD_DIM>;
  constexpr bool BF16 = !std::is_same<T, __half>::value;
  constexpr int DO = HEAD_DIM;
  constexpr int KS = C::KSTAGES;
  constexpr int VS = C::VSTAGES;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float4* scales = reinterpret_cast<float4*>(sm + C::SC_OFF);
  // [ITEMS][INFO]: the item (s: -1 past the last), [6] a bad block or scale was met, [7] a masked row may meet a NaN
  // value, [8] ref
  int* infos = reinterpret_cast<int*>(sm + C::INFO_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  // Phases count over all items of the CTA.
  uint64_t* kfull = bars;                  // [KS] K of a block is widened (128 arrivals)
  uint64_t* vfull = kfull + KS;            // [VS] V of a block is widened (128 arrivals)
  // step n: P V of block n - 1, then Q K^T of block n.  One commit per step and tile frees K of
  // block n and V of block n - 1.
  uint64_t* done = vfull + VS;             // [DONE] both tiles' MMAs of a step have completed
  uint64_t* sfull = done + C::DONE;        // [tile] S of the tile's next block is in TMEM
  uint64_t* pfull = sfull + TC_TILES;      // [tile][half] P of 64 keys of that block is written (128 arrivals)
  uint64_t* pvdone = pfull + 2 * TC_TILES; // [tile] the last P V of the tile's item has completed
  uint64_t* qbar = pvdone + TC_TILES;      // [tile] Q of the tile's next item landed
  uint64_t* qready = qbar + TC_TILES;      // [tile] bfloat16: it is float16 now (128 arrivals)
  uint64_t* drain = qready + TC_TILES;     // [tile] every MMA issued has completed
  uint64_t* turn = drain + TC_TILES;       // [tile] its MMA warp may issue the next step
  uint64_t* ifull = turn + TC_TILES;      // [ITEMS] an item is published
  uint64_t* scfull = ifull + C::ITEMS;     // [2] a group of scales is stored
  uint64_t* scfree = scfull + 2;           // [2] it is read (one arrival per softmax warp)
  uint64_t* cbar = scfree + 2;             // the answer about another CTA landed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::SLOT_OFF);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int tt = p.tile_tokens;

  grid_dependency_wait();  // the cache write before this launch has finished

  PrefillItem it;
  const int found = find_item<IS_RAGGED>(p, make_uint3(blockIdx.x, blockIdx.y, blockIdx.z), it);
  if (found <= 0) {
    if (found < 0) write_nan_rows<T, HEAD_DIM>(p, it, threadIdx.x, C::THREADS);
    allow_dependent_launch();
    return;
  }
  auto load_q = [&](const PrefillItem& i, int u) {  // one thread
    mbar_arrive_expect_tx(&qbar[u], C::QBYTES);
    for (int db = 0; db < C::DBOX; ++db)
      tma_load_3d(sm + u * C::QBYTES + db * C::QATOM, &p.tmap_q, db * BOX_DIMS, i.kvh * G, i.q0 + i.ta + u * tt, &qbar[u]);
  };
  auto publish = [&](const PrefillItem& i, int k) {  // one thread
    int* f = infos + (k % C::ITEMS) * C::INFO;
    f[0] = i.s, f[1] = i.kvh, f[2] = i.ta, f[3] = i.q0, f[4] = i.qlen, f[5] = i.base, f[6] = 0, f[7] = 0;
    mbar_arrive(&ifull[k % C::ITEMS]);
  };
  // Item k of the CTA, published.
  auto item = [&](int k) -> PrefillItem {
    const volatile int* f = infos + (k % C::ITEMS) * C::INFO;
    PrefillItem i;
    i.s = f[0], i.kvh = f[1], i.ta = f[2], i.q0 = f[3], i.qlen = f[4], i.base = f[5];
    return i;
  };
  // Waits for it; false past the last (or when the MMA warp gave up).
  auto has_item = [&](int k) -> bool {
    return __all_sync(FULL_MASK, tc_wait(&ifull[k % C::ITEMS], (k / C::ITEMS) & 1)) &&
           *const_cast<const volatile int*>(infos + (k % C::ITEMS) * C::INFO) >= 0;
  };
  auto read_item = [&](int k, PrefillItem& i) -> bool {
    if (!has_item(k)) return false;
    i = item(k);
    return true;
  };

  if (warp == C::MMA_WARP && lane == 0) {
    for (int i = 0; i < KS; ++i) mbar_init(&kfull[i], C::PROD);
    for (int i = 0; i < VS; ++i) mbar_init(&vfull[i], C::PROD);
    for (int i = 0; i < C::DONE; ++i) mbar_init(&done[i], TC_TILES);
    for (int i = 0; i < TC_TILES; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[2 * i], TC_ROWS);
      mbar_init(&pfull[2 * i + 1], TC_ROWS);
      mbar_init(&pvdone[i], 2);
      mbar_init(&qbar[i], 1);
      mbar_init(&qready[i], TC_ROWS);
      mbar_init(&drain[i], 1);
      mbar_init(&turn[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&scfull[i], 1);
      mbar_init(&scfree[i], C::SOFT / 32);
    }
    for (int i = 0; i < C::ITEMS; ++i) mbar_init(&ifull[i], 1);
    mbar_init(cbar, 1);
    fence_mbar_init();
    for (int u = 0; u < it.tiles(tt); ++u) load_q(it, u);
    publish(it, 0);
    ask_for_cta(sm + C::RESP_OFF, cbar);
  }
  if (warp >= C::PROD_WARP && warp < C::MMA_WARP) {
    // ------------------------------------------------ producers: K, then V of each block
    set_max_regs<false, C::PROD_REGS>();
    const int pw = warp - C::PROD_WARP;
    constexpr int NG = 16 / C::PROD_WARPS;  // the warp's groups of 8 rows of a block
    constexpr int HALVES = HEAD_DIM / 64;               // 64-code halves of a row
    const int r8 = lane >> 2;  // four lanes per row: 64 codes of it per load
    const int c = lane & 3;
    const unsigned row_bytes = p.num_kv_heads * HEAD_DIM;
    const int bmask = (1 << p.log2_b) - 1;
    auto rg = [&](int i) { return pw + C::PROD_WARPS * i; };
    uint4 kd[NG][HALVES], vd[NG][HALVES];
    // (scaled: times `by`, two float16)
    auto store = [&](const uint4 (&d)[HALVES], uint8_t* stage, int r, bool scaled, uint32_t by) {
      uint8_t* drow = stage + r * 128;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        uint4 a, b;
        widen16(d[h], a, b);
        if (scaled) {
          a = make_uint4(mul_half2(a.x, by), mul_half2(a.y, by), mul_half2(a.z, by), mul_half2(a.w, by));
          b = make_uint4(mul_half2(b.x, by), mul_half2(b.y, by), mul_half2(b.z, by), mul_half2(b.w, by));
        }
        // unit u of row r sits at u ^ (r % 8): the eight lanes of two rows write eight different units
        *reinterpret_cast<uint4*>(drow + h * C::KATOM + (((2 * c) ^ (r & 7)) << 4)) = a;
        *reinterpret_cast<uint4*>(drow + h * C::KATOM + (((2 * c + 1) ^ (r & 7)) << 4)) = b;
      }
    };
    bool go = true;
    int n = 0;  // blocks stored, over all items
#pragma unroll 1
    for (int k = 0; go; ++k) {
      const int kend = it.kend(tt);
      const int nblk = it.blocks(tt);
      const int full = it.base + it.ta;  // every row of the item sees the keys up to this one
      const int32_t* bt = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
      const unsigned head = it.kvh * HEAD_DIM + c * 16;
      // lane i: the physical block of row group i % 16 (8 rows lie in one pool block)
      auto fetch = [&](int j) { return __ldg(bt + (min(j * TC_KEYS + (lane & 15) * 8, kend - 1) >> p.log2_b)); };
      // the ids in hand, checked: never read outside the pool (the warp of the scales, which meets
      // every id, makes NaN of the item's outputs)
      auto checked = [&](int id) {
        use_here(id);
        return static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks) ? id : 0;
      };
      auto load = [&](uint4 (&d)[HALVES], const uint8_t* pool, int phys, int key) {
        // (slots fit 31 bits)
        const uint8_t* src = pool + (static_cast<size_t>((static_cast<unsigned>(phys) << p.log2_b) + (key & bmask)) * row_bytes + head);
#pragma unroll
        for (int h = 0; h < HALVES; ++h)  // rows past the item's last key are zeros: 0 x NaN must not occur
          d[h] = key < kend ? ldg128(src + h * 64) : make_uint4(0u, 0u, 0u, 0u);
      };
      int ids = checked(fetch(0));
      int next = fetch(min(1, nblk - 1));
      // the value scale of row group lane % 16, as long ahead of its use as the codes
      auto scale_of = [&]() { return __ldg(p.v_scales + static_cast<size_t>(ids) * p.num_kv_heads + it.kvh); };
      float vs = scale_of();
      int ref = 0;
      auto phys = [&](int g) { return __shfl_sync(FULL_MASK, ids, g & 15); };
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        load(kd[i], p.k_cache, phys(rg(i)), rg(i) * 8 + r8);
        load(vd[i], p.v_cache, phys(rg(i)), rg(i) * 8 + r8);
      }
      // (the first block's rows are on their way while the barriers and the tensor memory are set up)
      if (k == 0) __syncthreads();
#pragma unroll 1
      for (int j = 0; j < nblk; ++j, ++n) {
        const int kslot = n % KS;
        const int vslot = n % VS;
        // K's stage is free after step n - KS, V's after step n - VS + 1
        const int step = max(n - KS, n - VS + 1);
        if (step >= 0 && !__all_sync(FULL_MASK, tc_wait(&done[step % C::DONE], (step / C::DONE) & 1))) {
          go = false;
          break;
        }
        // (waited for where the ids are: behind the loads below it would wait for those, too)
        use_here(vs);
        if (j == 0) ref = ref_exp(__reduce_max_sync(FULL_MASK, scale_bits(vs)));
        const int kap = kappa(value_exp(vs), ref);
        ids = checked(next);
        next = fetch(min(j + 2, nblk - 1));  // a whole block before their use
        vs = scale_of();
        uint8_t* kdst = sm + C::K_OFF + kslot * C::KBYTES;
        uint8_t* vdst = sm + C::V_OFF + vslot * C::KBYTES;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          store(kd[i], kdst, rg(i) * 8 + r8, false, 0u);
          if (j + 1 < nblk) load(kd[i], p.k_cache, phys(rg(i)), (j + 1) * TC_KEYS + rg(i) * 8 + r8);
        }
        fence_proxy_async_smem();  // the widened rows become visible to the tensor core
        mbar_arrive(&kfull[kslot]);
        if ((j + 1) * TC_KEYS - 1 > full) {
          // some row does not see some key here: its weight is 0, and 0 x NaN must not occur.
          // NaN values enter as 0; the rows that see them get their NaN at the end.
          uint32_t any = 0;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
  #pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              uint32_t* w = reinterpret_cast<uint32_t*>(&vd[i][h]);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t m = nan_codes(w[x]);
                any |= m;
                w[x] &= ~((m >> 7) * 0xffu);
              }
            }
          }
          if (any) *const_cast<volatile int*>(infos + (k % C::ITEMS) * C::INFO + 7) = 1;
        }
        const uint32_t two = (kap > -15 ? (kap + 15) << 10 : 1 << 9) * 0x10001u;  // 2^kappa twice, as float16
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          store(vd[i], vdst, rg(i) * 8 + r8, true, __shfl_sync(FULL_MASK, two, rg(i) & 15));
          if (j + 1 < nblk) load(vd[i], p.v_cache, phys(rg(i)), (j + 1) * TC_KEYS + rg(i) * 8 + r8);
        }
        fence_proxy_async_smem();
        mbar_arrive(&vfull[vslot]);
      }
      go = go && read_item(k + 1, it);
    }
    __syncthreads();
    allow_dependent_launch();
    return;
  }
  if (warp == 0) tmem_alloc(tslot, C::TMEM_COLS);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp >= C::MMA_WARP) {
    set_max_regs<false, C::MMA_REGS>();
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(FULL_MASK, tc_wait(bar, parity)) != 0; };
    if (warp < C::ITEM_WARP) {
      // ---------------------------------------------- MMA issue: warp u, tile u
      // A warp per tile: one for both spent 3100 cycles a step in its waits and issues.  The whole warp runs the loop and one elected lane
      // issues: every value stays uniform, so descriptors sit in uniform registers (with one lane
      // in a branch of its own the 16 MMAs of a tile and block took 2000 cycles to issue).
      const int u = __shfl_sync(FULL_MASK, warp - C::MMA_WARP, 0);
      const uint64_t dq = umma_desc_sw128(smem_addr(sm + u * C::QBYTES), 16, 1024);    // Q, K-major
      const uint64_t dk = umma_desc_sw128(smem_addr(sm + C::K_OFF), 16, 1024);         // K, K-major
      const uint64_t dv = umma_desc_sw128(smem_addr(sm + C::V_OFF), C::KATOM, 1024);   // V, MN-major
      const uint32_t tP = tmem + 256 * u;
      const uint32_t tO = tP + 128;
      // stages of the next block's K and of the current one's V, parities of the phases
      int kslot = 0, vslot = 0, dslot = 0;
      uint32_t kpar = 0, vpar = 0, spar = 0, ppar = 0, qpar = 0, tpar = u ^ 1;
      // Three barriers at once, a lane each: the waits cost a hundred cycles together, not each.
      // (A test, not a wait that suspends: that one sleeps past the completion of one lane's
      // barrier while another lane's is open.)  The limit is some seconds.
      auto wait3 = [&](uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t* b2, uint32_t p2) -> bool {
        uint64_t* b = lane == 0 ? b0 : lane == 1 ? b1 : b2;
        const uint32_t par = lane == 0 ? p0 : lane == 1 ? p1 : p2;
#pragma unroll 1
        for (int i = 0; i < 1 << 26; ++i)
          if (__all_sync(FULL_MASK, mbar_test(b, par))) return true;
        return false;
      };
      auto qk = [&]() {
        const uint64_t kj = umma_desc_add(dk, kslot * C::KBYTES);
#pragma unroll
        for (int ks = 0; ks < HEAD_DIM / 16; ++ks) {
          const uint32_t off = (ks >> 2) * C::QATOM + ((ks & 3) << 5);
          const uint32_t koff = (ks >> 2) * C::KATOM + ((ks & 3) << 5);
          umma_f16_elect(tP, umma_desc_add(dq, off), umma_desc_add(kj, koff), C::ID_S, ks > 0);
        }
      };
      auto first_qk = [&]() -> bool {  // of an item
        uint64_t* q = BF16 ? &qready[u] : &qbar[u];
        if (!wait3(q, qpar, q, qpar, &kfull[kslot], kpar)) return false;
        tc_fence_after_sync();
        qpar ^= 1;
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
      // The tiles' MMAs take turns, so that one tile's run under the other's softmax: issued as
      // they become ready, the two tiles' interleave, end together and leave the tensor cores idle
      // while both wait for weights (2 x 16384: 3244 us against 2973).
      auto pass_turn = [&]() {
        if (lane == 0) mbar_arrive(&turn[u ^ 1]);
        __syncwarp();
      };
      // P V of the current block in the tile's turn, and Q K^T of the next one; first: the item's
      // first block, last: the tile's last one
      auto step = [&](bool first, bool last) -> bool {
        if (!wait3(&turn[u], tpar, &vfull[vslot], vpar, &pfull[2 * u], ppar)) return false;
        tpar ^= 1;
        tc_fence_after_sync();
        const uint64_t vj = umma_desc_add(dv, vslot * C::KBYTES);
        // the first 64 keys while the softmax writes the weights of the others
#pragma unroll
        for (int kk = 0; kk < TC_KEYS / 32; ++kk)  // 16 keys = 8 columns of P
          umma_f16_ts_elect(tO, tP + 8 * kk, umma_desc_add(vj, kk * 2048), C::ID_PV, !first || kk > 0);
        uint64_t* p1 = &pfull[2 * u + 1];
        if (!wait3(p1, ppar, p1, ppar, last ? p1 : &kfull[kslot], last ? ppar : kpar)) return false;
        ppar ^= 1;
        tc_fence_after_sync();
#pragma unroll
        for (int kk = TC_KEYS / 32; kk < TC_KEYS / 16; ++kk)
          umma_f16_ts_elect(tO, tP + 8 * kk, umma_desc_add(vj, kk * 2048), C::ID_PV, true);
        if (!last) qk();
        pass_turn();
        if (last) {
          if (lane == 0) mbar_arrive(&pvdone[u]);
          umma_commit_elect(&pvdone[u]);
        } else {
          umma_commit_elect(&sfull[u]);
          spar ^= 1;
        }
        return true;
      };
      // a step of the item in which the tile has no block: at the pace of the other tile
      auto no_step = [&]() -> bool {
        if (!wait3(&turn[u], tpar, &vfull[vslot], vpar, &vfull[vslot], vpar)) return false;
        tpar ^= 1;
        pass_turn();
        return true;
      };
      auto next_v = [&]() {
        vpar ^= vslot + 1 == VS;
        vslot = vslot + 1 == VS ? 0 : vslot + 1;
      };
      int nb, nblk;  // blocks of the tile and of the item
      auto lengths = [&](const PrefillItem& i) {
        nb = __shfl_sync(FULL_MASK, i.tile_blocks(u, tt), 0);
        nblk = __shfl_sync(FULL_MASK, i.blocks(tt), 0);
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
      tc_fence_before_sync();
    } else if (warp == C::ITEM_WARP) {
      // ---------------------------------------------- items and scales
      // Items are asked for one ahead of their use, and published at once.
      int asked = 0, published = 1;
      bool open = true;  // an answer is on its way
      auto next_item = [&](PrefillItem& i) -> bool {
        while (open) {
          if (!wait(cbar, asked & 1)) {
            open = false;
            break;
          }
          ++asked;
          uint3 id;
          open = cta_given(sm + C::RESP_OFF, id);
          __syncwarp();  // every lane has read the answer
          if (!open) break;
          if (lane == 0) {
            fence_proxy_async_smem();
            ask_for_cta(sm + C::RESP_OFF, cbar);
          }
          const int f = find_item<IS_RAGGED>(p, id, i);
          if (f < 0) write_nan_rows<T, HEAD_DIM>(p, i, lane, 32);
          if (f > 0) return true;
        }
        return false;
      };
      // Scales of the blocks' 16-key chunks, four blocks (a lane per chunk) at a time, one such
      // group ahead of the softmax.
      bool ok = true;
#pragma unroll 1
      for (int g = 0, n = 0; ok; ++n) {
        const int32_t* bt = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
        const int nblk = it.blocks(tt);
        const int kend = it.kend(tt);
        int ref = 0;
#pragma unroll 1
        for (int b = 0; b < nblk; b += C::GROUP, ++g) {
          // (chunks past the item's last key repeat the last one: their keys are masked)
          const int phys = __ldg(bt + (min(b * TC_KEYS + lane * CHUNK, kend - 1) >> p.log2_b));
          const bool in = static_cast<unsigned>(phys) < static_cast<unsigned>(p.num_blocks);
          const size_t at = static_cast<size_t>(in ? phys : 0) * p.num_kv_heads + it.kvh;
          const float sk = __ldg(p.k_scales + at);
          const float sv = __ldg(p.v_scales + at);
          if (b == 0) {  // as the producers have it
            ref = ref_exp(__reduce_max_sync(FULL_MASK, lane < C::CHUNKS ? scale_bits(sv) : 0));
            if (lane == 0) *const_cast<volatile int*>(infos + (n % C::ITEMS) * C::INFO + 8) = ref;
          }
          // what 2^kappa leaves of the value scale: 2^rest times a mantissa
          const int e = value_exp(sv);
          const int rest = max(e - ref - 3 - kappa(e, ref), kLeastRest);
          const float mant = sv >= 5.421010862427522e-20f ? __int_as_float((__float_as_int(sv) & 0x7fffff) | 0x3f800000) : 1.f;
          // (the item is published, which clears this flag: the first one before the set-up barrier)
          if (!(in && sk >= 0.f && sk <= kFloatMax && sv >= 0.f && sv <= kFloatMax && rest <= kMostRest))
            *const_cast<volatile int*>(infos + (n % C::ITEMS) * C::INFO + 6) = 1;
          // (a factor of 0 would turn a masked score (-inf) into NaN; bfloat16: see `factor`)
          float a = sk * p.scale_log2;
          if constexpr (!BF16) a = fabsf(a) >= kLeastFactor ? a : p.least_factor;
          const float4 v = make_float4(a, rest + (mant == 1.f ? 0.f : __log2f(mant)), pow2f(-rest) * __frcp_rn(mant), 0.f);
          ok = g < 2 || wait(&scfree[g & 1], ((g >> 1) - 1) & 1);
          if (!ok) break;
          scales[(g & 1) * 32 + lane] = v;
          __syncwarp();
          if (lane == 0) mbar_arrive(&scfull[g & 1]);
        }
        if (!ok || !next_item(it)) break;
        if (lane == 0) publish(it, published);
        __syncwarp();
        ++published;
      }
      if (!ok && open && wait(cbar, asked & 1)) {  // a wait ran out: NaN in what was asked for
        uint3 id;
        if (cta_given(sm + C::RESP_OFF, id) && find_item<IS_RAGGED>(p, id, it) != 0)
          write_nan_rows<T, HEAD_DIM>(p, it, lane, 32);
      }
      it.s = -1;
      if (lane == 0) publish(it, published);
    }
    __syncthreads();
    allow_dependent_launch();
    return;
  }
  // ------------------------------------------------ softmax: warps 4 u .. 4 u + 3 run tile u
  set_max_regs<true, C::SOFT_REGS>();
  const int u = warp >> 2;
  const int r = 32 * (warp & 3) + lane;
  const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t tS = tmem + 256 * u + lane_off;
  const uint32_t tO = tS + 128;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(FULL_MASK, tc_wait(bar, parity));
  };
  // What changes from block to block and item to item, in one register (x[] below takes 128, and
  // a spilled register makes every arrival wait for local memory: 282 -> 370 us): [2:0] the
  // item's number, [4:3] the block's place in its group of scales, [6:5] the group's number,
  // parities of [7] the tile's blocks, [8] its items, [9] its Q.
  uint32_t st = 0;
  // bfloat16: Q of the tile's next item as float16, each row scaled by a power of two whose
  // inverse is returned
  auto convert_q = [&](const PrefillItem& i) -> float {
    if (u >= i.tiles(tt)) return 1.f;
    wait(&qbar[u], (st >> 9) & 1);
    st ^= 1u << 9;
    float f = 1.f, back = 1.f;
    if (ok) {
      uint4* row = reinterpret_cast<uint4*>(sm + u * C::QBYTES + r * 128);
      constexpr int AT = C::QATOM / 16;
      float amax = 0.f;
#pragma unroll 4
      for (int x = 0; x < HEAD_DIM / 8; ++x) {
        const uint4 v = row[(x >> 3) * AT + ((x + lane) & 7)];  // lanes start at different units: no bank conflict
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 z = unpack_bf162(w[y]);
          amax = fmaxf(amax, fmaxf(fabsf(z.x), fabsf(z.y)));
        }
      }
      const int e = min(14 - ((__float_as_int(amax) >> 23) - 127), 126);
      f = pow2f(e);
      back = pow2f(-e);
#pragma unroll 4
      for (int x = 0; x < HEAD_DIM / 8; ++x) {
        uint4* at = row + (x >> 3) * AT + ((x + lane) & 7);
        const uint4 v = *at;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 z = unpack_bf162(w[y]);
          o[y] = pack_half2(z.x * f, z.y * f);
        }
        *at = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&qready[u]);
    return back;
  };
  // A negative `scale` turns the order of the scores around: the largest product is then
  // the smallest score times the (negative) factor.
  const bool neg = p.scale_log2 < 0.f;
  const float hidden = neg ? INFINITY : -INFINITY;
  float qinv = 1.f;  // bfloat16: undoes the row's scaling
  // The factor of a chunk's raw scores.  A row's own power of two (down to 2^-126, for a row of
  // zeros) can bring the product to 0, which a masked score (-inf) must not meet: 2^-100 is added, of
  // the factor's sign.  It is lost in factors above 2^-76, and smaller ones make 0 of every score anyway.
  // (16 chunks of 509 on 1536: 205.4 us, by a maximum behind the multiplication 207.5 us.)
  auto factor = [&](float a) -> float { return BF16 ? fmaf(a, qinv, p.least_factor) : a; };
  auto next_group = [&]() {  // the warp has read its group of scales
    __syncwarp();
    if (lane == 0) mbar_arrive(&scfree[(st >> 5) & 1]);
    st = (st & ~(15u << 3)) | ((st + (1u << 5)) & (3u << 5));
  };
  if constexpr (BF16) qinv = convert_q(it);
#pragma unroll 1
  for (;;) {
    int left, seen;  // the tile's blocks to come; the keys of the block that all its rows see, minus one
    {
      const PrefillItem i = item(st & 7);
      left = i.tile_blocks(u, tt);
      seen = i.base + i.ta + u * tt;
    }
    float m_used = -INFINITY, l = 0.f;  // log2 units, the rest of the value scale's exponent included
    uint32_t x[TC_KEYS];  // the block's raw scores, later its weights
#pragma unroll 1
    for (; left > 0; --left, seen -= TC_KEYS) {
      if ((st & (3u << 3)) == 0) wait(&scfull[(st >> 5) & 1], (st >> 6) & 1);
      wait(&sfull[u], (st >> 7) & 1);
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < TC_KEYS / 16; ++c) tmem_ld16(tS + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&x[16 * c]));
      tmem_wait_ld();
      if (seen < TC_KEYS - 1) {  // a key here may lie past some row of the tile
        const int own = seen + (r >> p.log2_g);  // (rows past the item's end are not written)
        const int all = seen + ((r & ~31) >> p.log2_g);
#pragma unroll
        for (int c = 0; c < TC_KEYS; c += 16) {
          if (c + 15 <= all) continue;  // the whole warp sees the chunk
          const int k = own - c;  // visible keys of the chunk, minus one
          const uint32_t m = k < 0 ? 0u : k > 15 ? ~0u : (2u << k) - 1u;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!(m >> i & 1u)) x[c + i] = __float_as_uint(hidden);
        }
      }
      // the row's maximum: per chunk of raw scores (the factor is the same), then one fma each
      const float4* sc = scales + ((st >> 3) & 7u) * C::CHUNKS;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c) {
        float e = __uint_as_float(x[16 * c]);
        if (!neg) {
#pragma unroll
          for (int i = 1; i < 15; i += 2)
            e = fmaxf(fmaxf(e, __uint_as_float(x[16 * c + i])), __uint_as_float(x[16 * c + i + 1]));
          e = fmaxf(e, __uint_as_float(x[16 * c + 15]));
        } else {
#pragma unroll
          for (int i = 1; i < 16; ++i) e = fminf(e, __uint_as_float(x[16 * c + i]));
        }
        mx = fmaxf(mx, fmaf(e, factor(sc[c].x), sc[c].y));
      }
      const float m_new = fmaxf(m_used, rounded_up(mx));  // (a row that sees no key here keeps its own: the other is NaN)
      // The exponent's offset moves at the first block and when the row maximum has grown
      // by more than 2^8; O and l then scale by f.
      const bool none = m_used == -INFINITY;  // nothing in O yet
      const bool need = !none && m_new > m_used + TC_RESCALE_LOG2;
      const float f = need ? ex2(m_used - m_new) : 1.f;
      if (none || need) m_used = m_new;
      const float bias = m_used == -INFINITY ? 0.f : kMidWeight - m_used;  // a row that has seen no key yet
      if (__any_sync(FULL_MASK, need)) {
#pragma unroll 1
        for (int c = 0; c < DO; c += 8) {  // (eight at a time: the scores hold 128 registers)
          uint32_t o8[8];
          tmem_ld8(tO + c, o8);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) o8[i] = __float_as_uint(__uint_as_float(o8[i]) * f);
          tmem_st8(tO + c, o8);
        }
      }
      l *= f;
      // the weights, half of the keys at a time: P in the half's first 32 columns; l takes each
      // chunk's sum divided by the rest of its value scale
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 4 * h; c < 4 * h + 4; ++c) {
          const float4 s4 = sc[c];
          const uint64_t a2 = pack_f32x2(factor(s4.x));
          const uint64_t b2 = pack_f32x2(s4.y + bias);
          uint64_t sum2 = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 t = unpack_f32x2(fma_f32x2(pack_f32x2(x[16 * c + 2 * i], x[16 * c + 2 * i + 1]), a2, b2));
            const float p0 = ex2(t.x), p1 = ex2(t.y);
            sum2 = add_f32x2(sum2, pack_f32x2(__float_as_uint(p0), __float_as_uint(p1)));
            x[8 * c + i] = pack_half2(p0, p1);  // (its place was consumed: 8 c + i <= 16 c + 2 i)
          }
          const float2 s2 = unpack_f32x2(sum2);
          l = fmaf(s2.x + s2.y, s4.z, l);
        }
        tmem_st16(tS + 32 * h, &x[32 * h]);
        tmem_st16(tS + 32 * h + 16, &x[32 * h + 16]);
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&pfull[2 * u + h]);
      }
      st ^= 1u << 7;
      if ((st & (3u << 3)) == (3u << 3) || left == 1) {
        next_group();
      } else {
        st += 1u << 3;
      }
    }
    const PrefillItem i = item(st & 7);  // (read again: held over the loop it would cost registers there)
    const volatile int* flags = infos + (st % C::ITEMS) * C::INFO + 6;
    // groups of scales that only the other tile needs
    for (int b = (i.tile_blocks(u, tt) + C::GROUP - 1) / C::GROUP * C::GROUP; b < i.blocks(tt); b += C::GROUP) {
      wait(&scfull[(st >> 5) & 1], (st >> 6) & 1);
      next_group();
    }
    st = (st & ~7u) | ((st + 1) & 7u);
    float qinv_next = 1.f;
    if constexpr (BF16) {  // before the outputs: the next item's first MMAs wait for nothing else
      if (has_item(st & 7)) qinv_next = convert_q(item(st & 7));
    }
    // ------------------------------------------------ O / l
    if (u < i.tiles(tt)) {
      wait(&pvdone[u], (st >> 8) & 1);
      st ^= 1u << 8;
      tc_fence_after_sync();
      const float inv = !ok || flags[0] ? NAN : 8.f / l * pow2f(flags[2]);
      const bool nans = flags[1];
      // A thread holds one row, and rows of different tokens are far apart in `out`: four lanes
      // exchange their 16-byte units, so that a store writes 64 bytes of each of eight rows (a
      // thread's own 32 bytes a store took 229 us against 227).  The loop is short because its code runs
      // once per item: unrolled it waited for instructions (235 us).
      int row = r;
      use_here(row);  // (what follows from it is not worth registers in the blocks' loop)
      const int t0 = i.ta + u * tt;
      const int t_end = i.tile_end(u, tt);
      const int t = t0 + (row >> p.log2_g);
      T* at[4];
      bool on[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int rr = (row & ~3) + x;
        on[x] = t0 + (rr >> p.log2_g) < t_end;
        at[x] = static_cast<T*>(p.out) + (static_cast<size_t>(i.q0 + t0 + (rr >> p.log2_g)) * p.num_heads + i.kvh * G +
                                          (rr & (G - 1))) * HEAD_DIM + 8 * (row & 3);
      }
#pragma unroll 1
      for (int c = 0; c < DO; c += 32) {
        uint32_t o[32];
        tmem_ld16(tO + c, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
        tmem_ld16(tO + c + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
        tmem_wait_ld();
#pragma unroll
        for (int d = 0; d < 16; ++d)
          o[d] = pack2<T>(__uint_as_float(o[2 * d]) * inv, __uint_as_float(o[2 * d + 1]) * inv);
        if (nans && t < t_end) {  // rare: look for the NaN values that the row sees among the item's last blocks
          uint32_t mask = 0;
#pragma unroll 1
          for (int key = (i.base + i.ta + 1) / TC_KEYS * TC_KEYS; key <= i.base + t; ++key) {
            const int phys = __ldg(p.block_tables + static_cast<size_t>(i.s) * p.max_blocks_per_seq + (key >> p.log2_b));
            if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) continue;  // NaN all over already
            const uint32_t* v = reinterpret_cast<const uint32_t*>(
                p.v_cache + ((((static_cast<size_t>(phys) << p.log2_b) + (key & ((1 << p.log2_b) - 1))) * p.num_kv_heads +
                              i.kvh) * HEAD_DIM + c));
#pragma unroll 1
            for (int y = 0; y < 8; ++y) {
              const uint32_t m = nan_codes(__ldg(v + y));
              mask |= (((m >> 7) & 1u) | ((m >> 14) & 2u) | ((m >> 21) & 4u) | ((m >> 28) & 8u)) << (4 * y);
            }
          }
#pragma unroll
          for (int d = 0; d < 16; ++d)
            o[d] |= (mask >> (2 * d) & 1u ? 0x7fffu : 0u) | (mask >> (2 * d) & 2u ? 0x7fff0000u : 0u);
        }
        uint4 unit[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) unit[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        transpose4(unit, row);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (on[x]) *reinterpret_cast<uint4*>(at[x] + c) = unit[x];
      }
    }
    qinv = qinv_next;
    if (!has_item(st & 7)) break;
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
  allow_dependent_launch();
}

template <typename T, int HEAD_DIM>
cudaError_t launch_block_prefill_t(const BlockPrefillArgs& b, cudaStream_t stream) {
  using C = BpCfg<HEAD_DIM>;
  const PrefillArgs& a = b.a;
  cudaError_t e = cudaSuccess;
  BlockPrefillParams p;
  const int group = a.num_heads / a.num_kv_heads;
  e = make_q_map<T>(&p.tmap_q, a.q, HEAD_DIM, a.num_heads, group, a.num_rows);
  if (e != cudaSuccess) return e;
  p.out = a.out;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scales = b.k_scales;
  p.v_scales = b.v_scales;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start_loc = a.query_start_loc;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = group;
  p.log2_g = __builtin_ctz(static_cast<unsigned>(group));
  p.log2_b = __builtin_ctz(static_cast<unsigned>(a.block_size));
  p.num_blocks = a.num_blocks;
  p.tile_tokens = TC_ROWS / group;
  const int tiles = (a.max_query_len + p.tile_tokens - 1) / p.tile_tokens;
  p.pairs = (tiles + TC_TILES - 1) / TC_TILES;
  p.scale_log2 = a.scale * 1.4426950408889634f + 0.f;  // a scale of -0 becomes +0: the sign decides what masks a score
  p.least_factor = copysignf(kLeastFactor, p.scale_log2);
  if (p.pairs == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  // Over all sequences and heads longest first leaves the shortest CTAs for the end (8 prompts
  // of 2048: 339 -> 295 us; 16 chunks of 509 on 1536: 245 -> 230 us; 2 prompts of 16384: 3147 ->
  // 3098 us).  Where most of the context is cached the pairs are nearly equal, and pairs of one
  // head that run together share its K and V in L2 (16 x 512 on 16384: 1574 us against 1673).
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
  // A grid over (sequence, pair) is mostly empty where one sequence brings many new tokens and the
  // others few, and an empty CTA takes a quarter of a microsecond of an SM.  The list of all pairs
  // is searched instead (a prompt of 8192 beside 255 sequences of 1 new token on 1000: 1057 -> 668
  // us; one of 2048 beside 63 of 1 on 2000: 167 -> 136 us), where the grid would be more than twice
  // its length: below that the search costs more (64 sequences of 1 to 4096 new tokens: 2330 us by
  // the grid, 2526 us by the list).
  const int64_t listed = a.num_rows / (2 * p.tile_tokens) + static_cast<int64_t>(a.num_seqs);
  const int64_t boxed = static_cast<int64_t>(p.pairs) * a.num_seqs;
  p.num_seqs = a.num_seqs;
  const bool ragged = boxed > 2 * listed && a.num_seqs <= 1024 && listed * a.num_kv_heads <= INT32_MAX;
  p.longest_first = cap <= 8 * static_cast<int64_t>(a.max_query_len) && p.pairs <= 65535;
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
  auto kern = ragged ? block_prefill_tc_kernel<T, HEAD_DIM, true> : block_prefill_tc_kernel<T, HEAD_DIM, false>;
  e = ensure_smem(kern, C::SMEM_BYTES, smem_set[ragged]);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

}  // namespace pa
