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
  int log2_b;  // block_size = 1 << log2_b
  int num_blocks;
  int pairs;
  int tile_tokens;
  float scale_log2;
};

// Shared memory of one CTA: Q of both tiles, the K and V rings of widened
// codes, the scales of the V ring's blocks, the barriers.
template <int HEAD_DIM>
struct BpCfg {
  static constexpr int SOFT = TC_TILES * TC_ROWS;  // softmax threads
  static constexpr int MMA_WARP = SOFT / 32;
  static constexpr int PROD_WARP = MMA_WARP + 1;  // K: two warps, then V: two
  static constexpr int PROD = 64;                 // producer threads of K, and of V
  static constexpr int THREADS = SOFT + 32 + 2 * PROD;
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
  static constexpr int NBARS = 2 * KSTAGES + 3 * VSTAGES + 3 * TC_TILES + 3;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int LAYOUT_BYTES = SLOT_OFF + 16;
  static constexpr int SMEM_BYTES = LAYOUT_BYTES + 1024;
  static_assert(SMEM_BYTES <= SMEM_MAX, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ID_S = umma_idesc_f16(TC_ROWS, TC_KEYS, false, false);
  static constexpr uint32_t ID_PV = umma_idesc_f16(TC_ROWS, HEAD_DIM, false, true);
};

__device__ __forceinline__ uint4 ldg128(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// 16 codes widened to float16: two 16-byte units.
__device__ __forceinline__ void widen16(const uint4& c, uint4& a, uint4& b) {
  e4m3x4_to_half2x2(c.x, a.x, a.y);
  e4m3x4_to_half2x2(c.y, a.z, a.w);
  e4m3x4_to_half2x2(c.z, b.x, b.y);
  e4m3x4_to_half2x2(c.w, b.z, b.w);
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
  uint64_t* kfull = bars;                  // [KS] K of a block is widened (64 arrivals)
  uint64_t* kempty = kfull + KS;           // [KS] that block's Q K^T (both tiles) is done
  uint64_t* vfull = kempty + KS;           // [VS] V of a block is widened (64 arrivals)
  uint64_t* vempty = vfull + VS;           // [VS] that block's P V (both tiles) is done
  uint64_t* scfull = vempty + VS;          // [VS] the scales of the block are in `scales`
  uint64_t* sfull = scfull + VS;           // [tile] S of the tile's next block is in TMEM
  uint64_t* pfull = sfull + TC_TILES;      // [tile] P of that block is written (128 arrivals)
  uint64_t* pvdone = pfull + TC_TILES;     // [tile] the tile's P V of that block has completed
  uint64_t* qbar = pvdone + TC_TILES;      // Q of both tiles landed
  uint64_t* qready = qbar + 1;             // bfloat16: Q is float16 now (256 arrivals)
  uint64_t* drain = qready + 1;            // every MMA issued has completed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::SLOT_OFF);
  volatile int* flags = reinterpret_cast<volatile int*>(sm + C::SLOT_OFF + 4);  // [0] bad block or scale, [1] timeout

  const int pair = p.pairs - 1 - static_cast<int>(blockIdx.x);  // the longest pairs start first
  const int kvh = blockIdx.y;
  const int s = blockIdx.z;
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
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&vfull[i], C::PROD);
      mbar_init(&vempty[i], 1);
      mbar_init(&scfull[i], 1);
    }
    for (int i = 0; i < TC_TILES; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], TC_ROWS);
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
  if (warp == 0) tmem_alloc(tslot, C::TMEM_COLS);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp >= C::PROD_WARP) {
    // ------------------------------------------------ producers: K, then V
    const bool is_v = warp >= C::PROD_WARP + 2;
    const int w2 = (warp - C::PROD_WARP) & 1;
    const int ns = is_v ? VS : KS;
    uint64_t* fullb = is_v ? vfull : kfull;
    uint64_t* emptyb = is_v ? vempty : kempty;
    const uint8_t* pool = is_v ? p.v_cache : p.k_cache;
    uint8_t* ring = sm + (is_v ? C::V_OFF : C::K_OFF);
    if (nblk > 0) {
      constexpr int RG = 8;                   // groups of 8 rows per warp and block
      constexpr int HALVES = HEAD_DIM / 64;   // 64-code halves of a row
      const int32_t* bt = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
      const int r8 = lane >> 2;  // four lanes per row: 64 codes of it per load
      const int c = lane & 3;
      const size_t row_bytes = static_cast<size_t>(p.num_kv_heads) * HEAD_DIM;
      const uint8_t* head = pool + static_cast<size_t>(kvh) * HEAD_DIM + c * 16;
      const int bmask = (1 << p.log2_b) - 1;
      int ph[RG];  // physical block of each row group of a block of keys (8 rows lie in one pool block)
      auto fetch = [&](int j) {
#pragma unroll
        for (int i = 0; i < RG; ++i) ph[i] = __ldg(bt + (min(j * TC_KEYS + (i * 2 + w2) * 8, kend - 1) >> p.log2_b));
      };
      uint4 data[RG][HALVES];
      auto load = [&](int j, int i) {
        int phys = ph[i];
        const int key = j * TC_KEYS + (i * 2 + w2) * 8 + r8;
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
          flags[0] = 1;  // never read outside the pool; the tiles' outputs become NaN
          phys = 0;
        }
        const uint8_t* src = head + ((static_cast<size_t>(phys) << p.log2_b) + (key & bmask)) * row_bytes;
#pragma unroll
        for (int h = 0; h < HALVES; ++h)  // rows past the stream's last key are zeros: 0 x NaN must not occur
          data[i][h] = key < kend ? ldg128(src + h * 64) : make_uint4(0u, 0u, 0u, 0u);
      };
      // scales of the block's 16-key chunks: lanes 0-7 of the first V warp
      const bool side = is_v && w2 == 0;
      float sk = 0.f, sv = 0.f;
      auto side_load = [&](int j) {
        if (side && lane < C::CHUNKS) {
          const int key = j * TC_KEYS + lane * CHUNK;
          sk = 0.f;
          sv = 1.f;
          if (key < kend) {
            const int phys = __ldg(bt + (key >> p.log2_b));
            if (static_cast<unsigned>(phys) < static_cast<unsigned>(p.num_blocks)) {
              const size_t at = static_cast<size_t>(phys) * p.num_kv_heads + kvh;
              sk = __ldg(p.k_scales + at);
              sv = __ldg(p.v_scales + at);
            }
          }
        }
      };
      fetch(0);
#pragma unroll
      for (int i = 0; i < RG; ++i) load(0, i);
      side_load(0);
      fetch(min(1, nblk - 1));
      for (int j = 0; j < nblk; ++j) {
        const int slot = j % ns;
        if (j >= ns && !__all_sync(FULL_MASK, tc_wait(&emptyb[slot], ((j / ns) - 1) & 1))) {
          flags[1] = 1;
          break;
        }
        if (side) {
          if (lane < C::CHUNKS) {
            if (!(sk >= 0.f && sk <= kFloatMax && sv >= 0.f && sv <= kFloatMax)) flags[0] = 1;
            const float v = fmaxf(sv, 5.421010862427522e-20f);  // 2^-64
            scales[slot * C::CHUNKS + lane] = make_float4(sk * p.scale_log2, __log2f(v), __frcp_rn(v), 0.f);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&scfull[slot]);
        }
        uint8_t* dst = ring + slot * C::KBYTES;
#pragma unroll
        for (int i = 0; i < RG; ++i) {
          const int r = (i * 2 + w2) * 8 + r8;
          uint8_t* drow = dst + r * 128;
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            uint4 a, b;
            widen16(data[i][h], a, b);
            // unit u of row r sits at u ^ (r % 8): the eight lanes of two rows write eight different units
            *reinterpret_cast<uint4*>(drow + h * C::KATOM + (((2 * c) ^ (r & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(drow + h * C::KATOM + (((2 * c + 1) ^ (r & 7)) << 4)) = b;
          }
          if (j + 1 < nblk) load(j + 1, i);
        }
        if (j + 1 < nblk) {
          side_load(j + 1);
          fetch(min(j + 2, nblk - 1));
        }
        fence_proxy_async_smem();  // the widened rows become visible to the tensor core
        mbar_arrive(&fullb[slot]);
      }
    }
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------ MMA issue (lane 0), as paged_prefill_tc_kernel
    if (lane == 0 && nblk > 0) {
      int nbt[TC_TILES];
      for (int u = 0; u < TC_TILES; ++u) nbt[u] = u < ntiles ? tile_blocks(u) : 0;
      int k_seen = -1;
      auto wait_k = [&](int j) -> bool {
        if (j <= k_seen) return true;
        if (!tc_wait(&kfull[j % KS], (j / KS) & 1)) return false;
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
          umma_f16(tmem + 256 * u, umma_desc_add(qu, off), umma_desc_add(kj, koff), C::ID_S, ks > 0);
        }
        umma_commit(&sfull[u]);
      };
      bool ok = tc_wait(BF16 ? qready : qbar, 0) && wait_k(0);
      if (ok) {
        for (int u = 0; u < ntiles; ++u) qk(u, 0);
        umma_commit(&kempty[0]);
      }
      for (int j = 0; ok && j < nblk; ++j) {
        const int vslot = j % VS;
        bool have_v = false;
        for (int u = 0; u < ntiles; ++u) {
          if (j >= nbt[u]) continue;
          if (!tc_wait(&pfull[u], j & 1)) {
            ok = false;
            break;
          }
          if (!have_v) {
            if (!tc_wait(&vfull[vslot], (j / VS) & 1)) {
              ok = false;
              break;
            }
            have_v = true;
          }
          tc_fence_after_sync();
          const uint64_t vj = umma_desc_add(dv, vslot * C::KBYTES);
          const uint32_t tP = tmem + 256 * u;
          const uint32_t tO = tP + 128;
#pragma unroll
          for (int kk = 0; kk < TC_KEYS / 16; ++kk)  // 16 keys = 8 columns of P
            umma_f16_ts(tO, tP + 64 * (kk >> 2) + 8 * (kk & 3), umma_desc_add(vj, kk * 2048), C::ID_PV, j > 0 || kk > 0);
          umma_commit(&pvdone[u]);
          if (j + 1 < nbt[u]) {
            if (!wait_k(j + 1)) {
              ok = false;
              break;
            }
            qk(u, j + 1);
          }
        }
        if (!ok) break;
        umma_commit(&vempty[vslot]);
        if (j + 1 < nblk) umma_commit(&kempty[(j + 1) % KS]);
      }
      if (!ok) flags[1] = 1;
      umma_commit(drain);  // every MMA finishes before the TMEM is released
      if (!tc_wait(drain, 0)) flags[1] = 1;
    }
  } else {
    // ------------------------------------------------ softmax: warps 4 u .. 4 u + 3 run tile u
    const int u = warp >> 2;
    const int r = 32 * (warp & 3) + lane;
    const bool tile_on = u < ntiles;
    const int t0 = ta + u * tt;
    const int t = t0 + r / G;
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
    float x[TC_HALF];  // base-2 scores of one half of the block's keys, value exponent added; masked ones -inf
    auto load_half = [&](int j, int h) {
      uint32_t v[TC_HALF / 16][16];
#pragma unroll
      for (int c = 0; c < TC_HALF / 16; ++c) tmem_ld16(tS + TC_HALF * h + 16 * c, v[c]);
      tmem_wait_ld();
      const float4* sc = scales + (j % VS) * C::CHUNKS + 4 * h;
#pragma unroll
      for (int c = 0; c < TC_HALF / 16; ++c) {
        const float4 f = sc[c];
        const float a = BF16 ? f.x * qinv : f.x;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[16 * c + i] = fmaf(__uint_as_float(v[c][i]), a, f.y);
      }
      const int k0 = j * TC_KEYS + TC_HALF * h;
      if (k0 + TC_HALF - 1 > base + t0) {  // a key here may lie past some row of the tile
#pragma unroll
        for (int c = 0; c < TC_HALF; ++c)
          if (k0 + c > pos) x[c] = -INFINITY;
      }
    };
    auto half_max = [&]() {
      float mq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mq[i] = x[i];
#pragma unroll
      for (int c = 4; c < TC_HALF; ++c) mq[c & 3] = fmaxf(mq[c & 3], x[c]);
      return fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
    };
    // the weights of the half in x, written as P over the half's first 32 columns; returns
    // their sum, each chunk's divided by its value scale
    auto half_weights = [&](int j, int h, float bias) {
      uint32_t w[TC_HALF / 2];
      const float4* sc = scales + (j % VS) * C::CHUNKS + 4 * h;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < TC_HALF / 16; ++c) {
        float ls[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p0 = ex2(x[16 * c + 2 * i] + bias);
          const float p1 = ex2(x[16 * c + 2 * i + 1] + bias);
          ls[i & 1] += p0 + p1;
          w[8 * c + i] = pack_half2(p0, p1);
        }
        sum = fmaf(ls[0] + ls[1], sc[c].z, sum);
      }
      tmem_st16(tS + TC_HALF * h, w);
      tmem_st16(tS + TC_HALF * h + 16, w + 16);
      return sum;
    };
    for (int j = 0; j < nb; ++j) {
      wait(&scfull[j % VS], (j / VS) & 1);
      wait(&sfull[u], j & 1);
      tc_fence_after_sync();
      load_half(j, 0);
      float mx = half_max();
      load_half(j, 1);  // half 1 stays in x for its weights
      mx = fmaxf(mx, half_max());
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
      float lsum = half_weights(j, 1, bias);
      load_half(j, 0);
      lsum += half_weights(j, 0, bias);
      l = l * f + lsum;
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&pfull[u]);
    }
    // ------------------------------------------------ O / l
    if (nb > 0) wait(&pvdone[u], (nb - 1) & 1);
    const bool have = ok && nb > 0;
    if (!ok) flags[1] = 1;
    __syncthreads();  // the other warps' flags are visible past this point
    tc_fence_after_sync();
    const float inv = (!have || ctx_bad || flags[0] || flags[1]) ? NAN : 1.f / l;
    T* dst = static_cast<T*>(p.out) + (static_cast<size_t>(q0 + t) * H + kvh * G + r % G) * HEAD_DIM;
#pragma unroll
    for (int c = 0; c < DO; c += 16) {
      uint32_t o16[16];
      if (have) {  // warp-uniform
        tmem_ld16(tO + c, o16);
        tmem_wait_ld();
      }
      if (rv) {
        uint32_t w8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w8[i] = have ? pack2<T>(__uint_as_float(o16[2 * i]) * inv, __uint_as_float(o16[2 * i + 1]) * inv)
                       : pack2<T>(NAN, NAN);
        *reinterpret_cast<uint4*>(dst + c) = make_uint4(w8[0], w8[1], w8[2], w8[3]);
        *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w8[4], w8[5], w8[6], w8[7]);
      }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
    allow_dependent_launch();
    return;
  }
  // the MMA and producer warps meet the softmax warps at their two barriers
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
  p.log2_b = __builtin_ctz(static_cast<unsigned>(a.block_size));
  p.num_blocks = a.num_blocks;
  p.tile_tokens = TC_ROWS / group;
  const int tiles = (a.max_query_len + p.tile_tokens - 1) / p.tile_tokens;
  p.pairs = (tiles + TC_TILES - 1) / TC_TILES;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (p.pairs == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.pairs, a.num_kv_heads, a.num_seqs);
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
