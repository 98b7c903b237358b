// pa_block_prefill.cuh -- prefill over block-scaled E4M3 pools on the tcgen05
// tensor cores.
//
//  block_prefill_tc_kernel  the pipeline of paged_prefill_tc_kernel
//                           (pa_prefill_tc.cuh): one CTA per (pair of query
//                           tiles, KV head, sequence), tiles of 128 rows
//                           (128 / G new tokens x G heads), Q K^T and P V in
//                           tensor memory, one softmax thread per row.
//
// What differs is the way in: the codes do not fit a kind::f16 MMA, so four
// producer warps read them from the pools (16 codes per lane and load, one
// block of 128 keys ahead, held in registers while the stage is in use), widen
// them exactly to float16 and store them in the swizzled layout that a TMA box
// of 16-bit rows would leave.  Two warps carry K, two V.
//
// The mathematics of the scales is that of pa_block_decode.cuh: with v_b the
// value scale of the block of key i,
//   w_i = 2^(s_i + log2 v_b - M),   out = sum w_i code_i / sum w_i / v_b,
// one fused multiply-add per score (key scale and log2 v_b of its 16-key chunk),
// one multiply per chunk for the sum.  A value scale below 2^-64 reads as 2^-64.
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
  int by_length;  // grid order: 1: (KV head, sequence, pair), 0: (pair, KV head, sequence)
  float scale_log2;
};

// Shared memory of one CTA: Q of both tiles, the K and V rings of widened
// codes, the scales of the V ring's blocks, the barriers.
template <int HEAD_DIM>
struct BpCfg {
  static constexpr int SOFT = TC_TILES * TC_ROWS;  // softmax threads
  static constexpr int MMA_WARP = SOFT / 32;
  static constexpr int PROD_WARP = MMA_WARP + 1;
  static constexpr int PROD_WARPS = 3;  // twelve warps in all: three per scheduler, 168 registers a thread
  static constexpr int PROD = PROD_WARPS * 32;
  static constexpr int THREADS = SOFT + 32 + PROD;
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
  static constexpr int SC_OFF = V_OFF + VSTAGES * KBYTES;  // [VSTAGES][CHUNKS] float4
  static constexpr int BAR_OFF = SC_OFF + VSTAGES * CHUNKS * 16;
  static constexpr int DONE = KSTAGES > VSTAGES ? KSTAGES : VSTAGES;  // ring of completed steps
  static constexpr int NBARS = KSTAGES + VSTAGES + DONE + 4 * TC_TILES + 3;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int LAYOUT_BYTES = SLOT_OFF + 16;
  static constexpr int SMEM_BYTES = LAYOUT_BYTES + 1024;
  static_assert(SMEM_BYTES <= SMEM_MAX, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ID_S = umma_idesc_f16(TC_ROWS, TC_KEYS, false, false);
  static constexpr uint32_t ID_PV = umma_idesc_f16(TC_ROWS, HEAD_DIM, false, true);
};

__device__ __forceinline__ uint4 ldg128(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// What is computed from x is computed after this point.  A value loaded an
// iteration ahead would otherwise be turned into an address right behind its
// load, and the warp would wait there.
__device__ __forceinline__ void use_here(int& x) { asm volatile("" : "+r"(x)); }
__device__ __forceinline__ void use_here(float& x) { asm volatile("" : "+f"(x)); }

// 16 codes widened to float16: two 16-byte units.
__device__ __forceinline__ void widen16(const uint4& c, uint4& a, uint4& b) {
  e4m3x4_to_half2x2(c.x, a.x, a.y);
  e4m3x4_to_half2x2(c.y, a.z, a.w);
  e4m3x4_to_half2x2(c.z, b.x, b.y);
  e4m3x4_to_half2x2(c.w, b.z, b.w);
}

// Pairs of float32 in one 64-bit register pair: one instruction for both.
__device__ __forceinline__ uint64_t pack_f32x2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack_f32x2(float x) { return pack_f32x2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The MMAs and the commit of pa_ptx.cuh issued by one elected lane of a warp that
// runs them together.
__device__ __forceinline__ void umma_f16_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u));
}
__device__ __forceinline__ void umma_f16_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                  bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u));
}
__device__ __forceinline__ void umma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}

template <typename T, int HEAD_DIM>
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  uint64_t* kfull = bars;                  // [KS] K of a block is widened (96 arrivals)
  uint64_t* vfull = kfull + KS;            // [VS] V of a block is widened (96 arrivals)
  // step i of the MMA warp: P V of block i - 1, then Q K^T of block i, of both tiles.  One
  // commit per step frees K of block i and V of block i - 1.
  uint64_t* done = vfull + VS;             // [DONE] the MMAs of a step have completed
  uint64_t* sfull = done + C::DONE;        // [tile] S of the tile's next block is in TMEM, its scales in `scales`
  uint64_t* pfull = sfull + TC_TILES;      // [tile][half] P of 64 keys of that block is written (128 arrivals)
  uint64_t* pvdone = pfull + 2 * TC_TILES; // [tile] the tile's last P V has completed
  uint64_t* qbar = pvdone + TC_TILES;      // Q of both tiles landed
  uint64_t* qready = qbar + 1;             // bfloat16: Q is float16 now (256 arrivals)
  uint64_t* drain = qready + 1;            // every MMA issued has completed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::SLOT_OFF);
  volatile int* flags = reinterpret_cast<volatile int*>(sm + C::SLOT_OFF + 4);  // [0] bad block or scale, [1] timeout

  // the longest pairs start first
  const int pair = p.pairs - 1 - static_cast<int>(p.by_length ? blockIdx.z : blockIdx.x);
  const int kvh = p.by_length ? blockIdx.x : blockIdx.y;
  const int s = p.by_length ? blockIdx.y : blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int H = p.num_heads;
  const int tt = p.tile_tokens;

  grid_dependency_wait();  // the cache write before this launch has finished

  const int q0 = __ldg(p.query_start_loc + s);
  const int qlen = __ldg(p.query_start_loc + s + 1) - q0;
  const int ctx = __ldg(p.context_lens + s);
  const int cap = p.max_blocks_per_seq << p.log2_b;
  const int ta = 2 * pair * tt;  // first new token of tile 0
  if (ta >= qlen) {
    allow_dependent_launch();
    return;
  }
  const int ntiles = ta + tt < qlen ? 2 : 1;
  const bool ctx_bad = ctx < qlen || ctx > cap;
  const int base = ctx - qlen;
  auto tile_end = [&](int u) { return min(qlen, ta + (u + 1) * tt); };
  auto tile_blocks = [&](int u) { return ctx_bad ? 0 : (base + tile_end(u) + TC_KEYS - 1) / TC_KEYS; };
  const int kend = ctx_bad ? 0 : base + tile_end(ntiles - 1);  // the K/V stream's last key + 1
  const int nblk = tile_blocks(ntiles - 1);

  if (warp == C::MMA_WARP && lane == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&kfull[i], C::PROD);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&vfull[i], C::PROD);
    }
    for (int i = 0; i < C::DONE; ++i) mbar_init(&done[i], 1);
    for (int i = 0; i < TC_TILES; ++i) {
      mbar_init(&sfull[i], 2);
      mbar_init(&pfull[2 * i], TC_ROWS);
      mbar_init(&pfull[2 * i + 1], TC_ROWS);
      mbar_init(&pvdone[i], 1);
    }
    mbar_init(qbar, 1);
    mbar_init(qready, C::SOFT);
    mbar_init(drain, 1);
    flags[0] = 0;
    flags[1] = 0;
    fence_mbar_init();
    if (nblk > 0) {
      mbar_arrive_expect_tx(qbar, ntiles * C::QBYTES);
      for (int u = 0; u < ntiles; ++u)
        for (int db = 0; db < C::DBOX; ++db)
          tma_load_3d(sm + u * C::QBYTES + db * C::QATOM, &p.tmap_q, db * BOX_DIMS, kvh * G, q0 + ta + u * tt, qbar);
    }
  }
  if (warp >= C::PROD_WARP) {
    // ------------------------------------------------ producers: K, then V of each block
    const int pw = warp - C::PROD_WARP;
    if (nblk == 0) {
      __syncthreads();
    } else {
      constexpr int RG = 16;                              // groups of 8 rows per block
      constexpr int NG = (RG + C::PROD_WARPS - 1) / C::PROD_WARPS;  // a warp's, at most
      constexpr int HALVES = HEAD_DIM / 64;               // 64-code halves of a row
      const int32_t* bt = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
      const int r8 = lane >> 2;  // four lanes per row: 64 codes of it per load
      const int c = lane & 3;
      const size_t row_bytes = static_cast<size_t>(p.num_kv_heads) * HEAD_DIM;
      const uint8_t* khead = p.k_cache + static_cast<size_t>(kvh) * HEAD_DIM + c * 16;
      const uint8_t* vhead = p.v_cache + static_cast<size_t>(kvh) * HEAD_DIM + c * 16;
      const int bmask = (1 << p.log2_b) - 1;
      // the warp's groups of K and of V: 6 + 5, 5 + 5 and 5 + 6
      auto kg = [&](int i) { return pw + C::PROD_WARPS * i; };
      auto vg = [&](int i) { return C::PROD_WARPS - 1 - pw + C::PROD_WARPS * i; };
      int kph[NG], vph[NG];  // physical block of each row group (8 rows lie in one pool block)
      // (a group past the last one is clamped, and not used)
      auto fetch_k = [&](int j) {
#pragma unroll
        for (int i = 0; i < NG; ++i) kph[i] = __ldg(bt + (min(j * TC_KEYS + kg(i) * 8, kend - 1) >> p.log2_b));
      };
      auto fetch_v = [&](int j) {
#pragma unroll
        for (int i = 0; i < NG; ++i) vph[i] = __ldg(bt + (min(j * TC_KEYS + vg(i) * 8, kend - 1) >> p.log2_b));
      };
      uint4 kd[NG][HALVES], vd[NG][HALVES];
      bool bad = false;
      auto load = [&](uint4 (&d)[HALVES], const uint8_t* head, int phys, int key) {
        use_here(phys);
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
          bad = true;  // never read outside the pool; the tiles' outputs become NaN
          phys = 0;
        }
        const uint8_t* src = head + ((static_cast<size_t>(phys) << p.log2_b) + (key & bmask)) * row_bytes;
#pragma unroll
        for (int h = 0; h < HALVES; ++h)  // rows past the stream's last key are zeros: 0 x NaN must not occur
          d[h] = key < kend ? ldg128(src + h * 64) : make_uint4(0u, 0u, 0u, 0u);
      };
      auto store = [&](const uint4 (&d)[HALVES], uint8_t* stage, int r) {
        uint8_t* drow = stage + r * 128;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          uint4 a, b;
          widen16(d[h], a, b);
          // unit u of row r sits at u ^ (r % 8): the eight lanes of two rows write eight different units
          *reinterpret_cast<uint4*>(drow + h * C::KATOM + (((2 * c) ^ (r & 7)) << 4)) = a;
          *reinterpret_cast<uint4*>(drow + h * C::KATOM + (((2 * c + 1) ^ (r & 7)) << 4)) = b;
        }
      };
      fetch_k(0);
      fetch_v(0);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (kg(i) < RG) load(kd[i], khead, kph[i], kg(i) * 8 + r8);
        if (vg(i) < RG) load(vd[i], vhead, vph[i], vg(i) * 8 + r8);
      }
      fetch_k(min(1, nblk - 1));
      fetch_v(min(1, nblk - 1));
      // (the first block's rows are on their way while the barriers and the tensor memory are set up)
      __syncthreads();
      for (int j = 0; j < nblk; ++j) {
        const int kslot = j % KS;
        const int vslot = j % VS;
        // K's stage is free after step j - KS, V's after step j - VS + 1
        const int step = max(j - KS, j - VS + 1);
        if (step >= 0 && !__all_sync(FULL_MASK, tc_wait(&done[step % C::DONE], (step / C::DONE) & 1))) {
          flags[1] = 1;
          break;
        }
        uint8_t* kdst = sm + C::K_OFF + kslot * C::KBYTES;
        uint8_t* vdst = sm + C::V_OFF + vslot * C::KBYTES;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if (kg(i) >= RG) continue;
          store(kd[i], kdst, kg(i) * 8 + r8);
          if (j + 1 < nblk) load(kd[i], khead, kph[i], (j + 1) * TC_KEYS + kg(i) * 8 + r8);
        }
        fence_proxy_async_smem();  // the widened rows become visible to the tensor core
        mbar_arrive(&kfull[kslot]);
        fetch_k(min(j + 2, nblk - 1));  // a whole block before their use
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if (vg(i) >= RG) continue;
          store(vd[i], vdst, vg(i) * 8 + r8);
          if (j + 1 < nblk) load(vd[i], vhead, vph[i], (j + 1) * TC_KEYS + vg(i) * 8 + r8);
        }
        fence_proxy_async_smem();
        mbar_arrive(&vfull[vslot]);
        fetch_v(min(j + 2, nblk - 1));
      }
      if (bad) flags[0] = 1;  // read after the barrier below
    }
    // the producers meet the softmax warps at their two barriers
    __syncthreads();
    __syncthreads();
    allow_dependent_launch();
    return;
  }
  if (warp == 0) tmem_alloc(tslot, C::TMEM_COLS);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp == C::MMA_WARP) {
    // ------------------------------------------------ MMA issue
    // The whole warp runs this loop and one elected lane issues: every value stays uniform, so
    // descriptors sit in uniform registers (with one lane in a branch of its own each MMA paid
    // for moving its operands there, and the 16 MMAs of a tile and block took 2000 cycles to issue).
    if (nblk > 0) {
      int nbt[TC_TILES];
      for (int u = 0; u < TC_TILES; ++u) nbt[u] = u < ntiles ? tile_blocks(u) : 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(FULL_MASK, tc_wait(bar, parity)) != 0; };
      int k_seen = -1;
      auto wait_k = [&](int j) -> bool {
        if (j <= k_seen) return true;
        if (!wait(&kfull[j % KS], (j / KS) & 1)) return false;
        k_seen = j;
        tc_fence_after_sync();
        return true;
      };
      const uint64_t dq = umma_desc_sw128(smem_addr(sm), 16, 1024);                    // Q, K-major
      const uint64_t dk = umma_desc_sw128(smem_addr(sm + C::K_OFF), 16, 1024);         // K, K-major
      const uint64_t dv = umma_desc_sw128(smem_addr(sm + C::V_OFF), C::KATOM, 1024);   // V, MN-major
      auto qk = [&](int u, int j) {
        const uint64_t qu = umma_desc_add(dq, u * C::QBYTES);
        const uint64_t kj = umma_desc_add(dk, (j % KS) * C::KBYTES);
#pragma unroll
        for (int ks = 0; ks < HEAD_DIM / 16; ++ks) {
          const uint32_t off = (ks >> 2) * C::QATOM + ((ks & 3) << 5);
          const uint32_t koff = (ks >> 2) * C::KATOM + ((ks & 3) << 5);
          umma_f16_elect(tmem + 256 * u, umma_desc_add(qu, off), umma_desc_add(kj, koff), C::ID_S, ks > 0);
        }
        if (lane == 0) mbar_arrive(&sfull[u]);
        umma_commit_elect(&sfull[u]);
      };
      // Scales of each block's 16-key chunks, lanes 0-7: read two blocks before their use, their
      // physical block's id three before.  Row b % VS is free for block b once the softmax of
      // block b - VS is over, which this warp has waited for.  (A producer warp that carried the
      // scales too waited for its latest row loads at each, 900 cycles a block.)
      const int32_t* bt = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
      float sk = 0.f, sv = 0.f;
      int sph = 0;
      auto scale_fetch = [&](int j) {
        if (lane < C::CHUNKS) sph = __ldg(bt + (min(j * TC_KEYS + lane * CHUNK, kend - 1) >> p.log2_b));
      };
      auto scale_load = [&]() {  // (chunks past the stream repeat its last one: their keys are masked)
        use_here(sph);
        if (lane < C::CHUNKS) {
          const bool in = static_cast<unsigned>(sph) < static_cast<unsigned>(p.num_blocks);
          const size_t at = static_cast<size_t>(in ? sph : 0) * p.num_kv_heads + kvh;
          sk = __ldg(p.k_scales + at);
          sv = __ldg(p.v_scales + at);
        }
      };
      auto scale_store = [&](int j) {
        use_here(sk);
        use_here(sv);
        if (lane < C::CHUNKS) {
          if (!(sk >= 0.f && sk <= kFloatMax && sv >= 0.f && sv <= kFloatMax)) flags[0] = 1;
          // a factor of 0 would turn a masked score (-inf) into NaN: 2^-120 makes 0 of every score
          float a = sk * p.scale_log2;
          a = fabsf(a) >= 7.52316384526264e-37f ? a : copysignf(7.52316384526264e-37f, p.scale_log2);
          const float lv = __log2f(fmaxf(sv, 5.421010862427522e-20f));  // at least 2^-64
          scales[(j % VS) * C::CHUNKS + lane] = make_float4(a, lv, ex2(-lv), 0.f);
        }
        __syncwarp();  // lane 0's next arrival on sfull releases them
      };
      static_assert(VS >= 3, "two blocks' scales ahead");
      scale_fetch(0);
      scale_load();
      scale_fetch(1);
      scale_store(0);
      scale_load();
      scale_fetch(2);
      bool ok = wait(BF16 ? qready : qbar, 0) && wait_k(0);
      if (ok) {
        for (int u = 0; u < ntiles; ++u) qk(u, 0);
        umma_commit_elect(&done[0]);
      }
      if (nblk > 1) scale_store(1);
      scale_load();
      scale_fetch(3);
      for (int j = 0; ok && j < nblk; ++j) {
        const int vslot = j % VS;
        bool have_v = false;
        for (int u = 0; u < ntiles; ++u) {
          // while the last tile's weights are awaited, and while the producers are quiet: behind
          // the commit below their loads crowd the queue, and this warp's waited 900 cycles
          if (u == ntiles - 1 && j + 2 < nblk) {
            scale_store(j + 2);
            scale_load();
            scale_fetch(j + 4);
          }
          if (j >= nbt[u]) continue;
          ok = wait(&pfull[2 * u], j & 1) && (have_v || wait(&vfull[vslot], (j / VS) & 1));
          if (!ok) break;
          have_v = true;
          tc_fence_after_sync();
          const uint64_t vj = umma_desc_add(dv, vslot * C::KBYTES);
          const uint32_t tP = tmem + 256 * u;
          const uint32_t tO = tP + 128;
          // the first 64 keys while the softmax writes the weights of the others
#pragma unroll
          for (int kk = 0; kk < TC_KEYS / 32; ++kk)  // 16 keys = 8 columns of P
            umma_f16_ts_elect(tO, tP + 8 * kk, umma_desc_add(vj, kk * 2048), C::ID_PV, j > 0 || kk > 0);
          ok = wait(&pfull[2 * u + 1], j & 1);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int kk = TC_KEYS / 32; kk < TC_KEYS / 16; ++kk)
            umma_f16_ts_elect(tO, tP + 8 * kk, umma_desc_add(vj, kk * 2048), C::ID_PV, true);
          if (j + 1 < nbt[u]) {
            ok = wait_k(j + 1);
            if (!ok) break;
            qk(u, j + 1);
          } else {
            umma_commit_elect(&pvdone[u]);
          }
        }
        if (!ok) break;
        umma_commit_elect(&done[(j + 1) % C::DONE]);
      }
      if (!ok) flags[1] = 1;
      umma_commit_elect(drain);  // every MMA finishes before the TMEM is released
      if (!wait(drain, 0)) flags[1] = 1;
    }
  } else {
    // ------------------------------------------------ softmax: warps 4 u .. 4 u + 3 run tile u
    const int u = warp >> 2;
    const int r = 32 * (warp & 3) + lane;
    const bool tile_on = u < ntiles;
    const int t0 = ta + u * tt;
    const int t = t0 + (r >> p.log2_g);
    const bool rv = tile_on && t < tile_end(u);
    const int pos = rv ? base + t : -1;
    const int nb = tile_on ? tile_blocks(u) : 0;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + 256 * u + lane_off;
    const uint32_t tO = tS + 128;
    float m_used = -INFINITY, l = 0.f;  // log2 units, the value scale's exponent included
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(FULL_MASK, tc_wait(bar, parity));
    };
    float qinv = 1.f;  // bfloat16: undoes the row's scaling
    if constexpr (BF16) {
      if (nblk > 0) {
        wait(qbar, 0);
        if (ok && tile_on) {
          uint4* row = reinterpret_cast<uint4*>(sm + u * C::QBYTES + r * 128);
          constexpr int AT = C::QATOM / 16;
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < HEAD_DIM / 8; ++i) {
            const uint4 v = row[(i >> 3) * AT + ((i + lane) & 7)];  // lanes start at different units: no bank conflict
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = unpack_bf162(w[k]);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          const int e = min(14 - ((__float_as_int(amax) >> 23) - 127), 126);
          const float f = pow2f(e);
          qinv = pow2f(-e);
#pragma unroll
          for (int i = 0; i < HEAD_DIM / 8; ++i) {
            uint4* at = row + (i >> 3) * AT + ((i + lane) & 7);
            const uint4 v = *at;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x2 = unpack_bf162(w[k]);
              o[k] = pack_half2(x2.x * f, x2.y * f);
            }
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(qready);
      }
    }
    // A negative `scale` turns the order of the scores around: the largest product is then
    // the smallest score times the (negative) factor.
    const bool neg = p.scale_log2 < 0.f;
    const float hidden = neg ? INFINITY : -INFINITY;
    uint32_t x[TC_KEYS];  // the block's raw scores, later its weights
    for (int j = 0; j < nb; ++j) {
      wait(&sfull[u], j & 1);
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < TC_KEYS / 16; ++c) tmem_ld16(tS + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&x[16 * c]));
      tmem_wait_ld();
      const int k0 = j * TC_KEYS;
      if (k0 + TC_KEYS - 1 > base + t0) {  // a key here may lie past some row of the tile
#pragma unroll
        for (int c = 0; c < TC_KEYS; ++c)
          if (k0 + c > pos) x[c] = __float_as_uint(hidden);
      }
      // the row's maximum: per chunk of raw scores (the factor is the same), then one fma each
      const float4* sc = scales + (j % VS) * C::CHUNKS;
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
        mx = fmaxf(mx, fmaf(e, BF16 ? sc[c].x * qinv : sc[c].x, sc[c].y));
      }
      const float m_new = fmaxf(m_used, mx);
      // The exponent's offset moves at the first block and when the row maximum has grown
      // by more than 2^8; O and l then scale by f.
      const bool need = j > 0 && m_new > m_used + TC_RESCALE_LOG2;
      const float f = need ? ex2(m_used - m_new) : 1.f;
      if (j == 0 || need) m_used = m_new;
      const float bias = m_used == -INFINITY ? 0.f : -m_used;  // a row that has seen no key yet
      if (__any_sync(FULL_MASK, need)) {
#pragma unroll 1
        for (int c = 0; c < DO; c += 16) {
          uint32_t o16[16];
          tmem_ld16(tO + c, o16);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o16[i] = __float_as_uint(__uint_as_float(o16[i]) * f);
          tmem_st16(tO + c, o16);
        }
      }
      l *= f;
      // the weights, half of the keys at a time: P in the half's first 32 columns; l takes each
      // chunk's sum divided by its value scale
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 4 * h; c < 4 * h + 4; ++c) {
          const float4 s4 = sc[c];
          const uint64_t a2 = pack_f32x2(BF16 ? s4.x * qinv : s4.x);
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
    }
    // ------------------------------------------------ O / l
    if (nb > 0) wait(&pvdone[u], 0);
    const bool have = ok && nb > 0;
    if (!ok) flags[1] = 1;
    __syncthreads();  // the other warps' flags are visible past this point
    tc_fence_after_sync();
    // O / l through the tile's Q rows in shared memory (its MMAs are over): a thread holds one
    // row, and rows of different tokens are far apart in `out`, so writing them from here
    // would touch 32 lines per store.  A warp turns its own 32 rows (6300 -> 1900 cycles per CTA).
    const float inv = (!have || ctx_bad || flags[0] || flags[1]) ? NAN : 1.f / l;
    if (nb > 0) {
      uint8_t* qrow = sm + u * C::QBYTES + r * 128;
#pragma unroll 1
      for (int h = 0; h < DO / 64; ++h) {  // one 64-dim atom at a time
        uint32_t o[64];
        if (have) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld16(tO + 64 * h + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&o[16 * c]));
          tmem_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w4[i] = have ? pack2<T>(__uint_as_float(o[8 * c + 2 * i]) * inv, __uint_as_float(o[8 * c + 2 * i + 1]) * inv)
                         : pack2<T>(NAN, NAN);
          *reinterpret_cast<uint4*>(qrow + h * C::QATOM + ((c ^ (r & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      }
      __syncwarp();
    }
    if (tile_on) {  // rows in order, DO / 8 lanes of 16 bytes each
      constexpr int U = DO / 8;
      constexpr int RPI = 32 / U;
      const int unit = lane % U;
      const int rw = 32 * (warp & 3);
      const int t_end = tile_end(u);
#pragma unroll 4
      for (int i = 0; i < 32 / RPI; ++i) {
        const int rr = rw + i * RPI + lane / U;
        const int tr = t0 + (rr >> p.log2_g);
        if (tr < t_end) {
          const uint4 v = nb > 0 ? *reinterpret_cast<const uint4*>(sm + u * C::QBYTES + rr * 128 + (unit >> 3) * C::QATOM +
                                                                   (((unit & 7) ^ (rr & 7)) << 4))
                                 : make_uint4(pack2<T>(NAN, NAN), pack2<T>(NAN, NAN), pack2<T>(NAN, NAN), pack2<T>(NAN, NAN));
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) +
                                    (static_cast<size_t>(q0 + tr) * H + kvh * G + (rr & (G - 1))) * HEAD_DIM + unit * 8) = v;
        }
      }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
    allow_dependent_launch();
    return;
  }
  // the MMA warp meets the softmax warps at their two barriers
  tc_fence_before_sync();
  __syncthreads();
  __syncthreads();
  allow_dependent_launch();
}

template <typename T, int HEAD_DIM>
cudaError_t launch_block_prefill_t(const BlockPrefillArgs& b, cudaStream_t stream) {
  using C = BpCfg<HEAD_DIM>;
  const PrefillArgs& a = b.a;
  auto kern = block_prefill_tc_kernel<T, HEAD_DIM>;
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = ensure_smem(kern, C::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
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
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (p.pairs == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  // Over all sequences and heads longest first leaves the shortest CTAs for the end (8 prompts
  // of 2048: 339 -> 295 us; 16 chunks of 509 on 1536: 245 -> 230 us; 2 prompts of 16384: 3147 ->
  // 3098 us).  Where most of the context is cached the pairs are nearly equal, and pairs of one
  // head that run together share its K and V in L2 (16 x 512 on 16384: 1574 us against 1673).
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
  p.by_length = cap <= 8 * static_cast<int64_t>(a.max_query_len) && p.pairs <= 65535;
  cfg.gridDim = p.by_length ? dim3(a.num_kv_heads, a.num_seqs, p.pairs) : dim3(p.pairs, a.num_kv_heads, a.num_seqs);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

}  // namespace pa
