// pa_block_decode.cuh -- decode attention with side data per (block, KV head):
// E4M3 pools whose scale is one float per (block, KV head), and tables of
// blocks per (sequence, KV head) (block-sparse decode, over those pools or over
// 16-bit ones).  Included by one translation unit per query type and use.
//
//  block_decode_kernel   the pipeline of paged_decode_kernel (pa_decode.cuh):
//                        one CTA per (KV head, partition, sequence), each warp
//                        streams 16-token chunks through a private ring of TMA
//                        stages; clusters split a sequence when the pairs do
//                        not fill the GPU.
//
// HBM bounds it: 2 d bytes per token and KV head.  64 sequences of 128 to 2048
// tokens, 32/8 heads of 128: 146 MB in 29.7 us (4.9 TB/s; the start, and the tail of
// the longest sequences, are most of the rest); 32 of 8192, 64/8 heads: 538 MB in
// 84 us (6.4 TB/s).  With a table per head the 128-byte rows of a block lie 1 KB
// apart and their neighbours are not wanted: 101 MB in about 24 us, by 256 CTAs on
// 304 places.  One sequence of 485 tokens: 4.7 us, latency.  (Graph replays.)
//
// The mathematics of the scales.  Block b of a sequence holds the keys
// ks_b * code and the values v_b * code.  With s_i the base-2 score of token i
// (scale * log2(e) * ks_b * q . code_i) and p_i = 2^(s_i - m), m a running maximum,
//
//   out = sum_b v_b (sum_{i in b} p_i code_i) / sum_i p_i.
//
// The weights of a 16-token chunk, which has one value scale, meet its codes in
// MMAs of their own, and the products join the accumulators by a float32
// multiply-add with v_b: what one block's scale is says nothing about the weights
// of another, and the denominator is the sum of the weights.  (With v_b in the
// weight's exponent, 2^(s_i + log2 v_b - M), the MMAs accumulate on, but a block of
// large values that a sequence hardly attends to pushes the weights of all others
// towards float16's end: 131072 keys behind one by 12 nats whose block's scale is
// 2^8 times theirs came out 5% short.)
//
// A weight is float16: m lies 15 below the largest score, so the largest weight is
// 2^15, and every weight above 2^-29 of it has 11 bits, a smaller one is off by
// 2^-40 of it at most.  The sum adds the weights unrounded, in float32.  The
// accumulators carry v_b 2^-39 and a merge the sums times 2^-39 (the weights' 2^15
// and room for 2^24 tokens of the largest scale); value scales from 2^-87 on keep
// all bits.
//
// Queries enter the MMAs as float16 beside the widened codes (exact in
// float16).  A bfloat16 query row is first scaled by the power of two that
// brings its largest element to [2^14, 2^15): exact for every element within
// 2^-28 of the largest, and within 2^-39 of the largest's size below that; the
// inverse multiplies the scores in float32.
#pragma once

#include "pa_block.cuh"
#include "pa_decode.cuh"

namespace pa {

namespace {

constexpr float kTopWeight = 15.f;                         // log2 of the largest weight: float16 ends at 2^16
constexpr float kValueUnit = 1.8189894035458565e-12f;      // 2^-39: the accumulators' unit
constexpr float kValueUnitInv = 549755813888.f;            // 2^39

struct BlockDecodeParams {
  CUtensorMap tmap_k;  // as DecodeParams: [N*B rows][Hk][d], 16-row boxes
  CUtensorMap tmap_v;
  void* out;
  const void* q;
  const float* k_scales;  // [N][Hk]; null for 16-bit pools
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_o;
  float* ws_m;
  float* ws_l;
  int max_blocks_per_seq;
  int num_heads;
  int num_kv_heads;
  int group;
  int block_size;
  int chunks_per_block_log2;
  int num_blocks;
  int partition_chunks;
  int max_num_partitions;
  int num_seqs;
  float scale_log2;  // scale * log2(e)
};

// Query fragments for E4M3 keys (the order of load_q_frags_e4m3) as float16,
// and inv[nt] = the factor that undoes row nt * 8 + lane / 4's scaling.
template <typename T, int HEAD_DIM, int NT>
__device__ __forceinline__ void load_q_frags_scaled(uint32_t (&qf)[HEAD_DIM / 16][NT][2], float (&inv)[NT],
                                                    const void* q, int s, int H, int kvh, int G, int lane) {
  load_q_frags_e4m3<HEAD_DIM, NT>(qf, q, s, H, kvh, G, G, lane);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    inv[nt] = 1.f;
    if constexpr (!std::is_same<T, __half>::value) {
      float amax = 0.f;
#pragma unroll
      for (int ks = 0; ks < HEAD_DIM / 16; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = unpack_bf162(qf[ks][nt][j]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 2));
      const int x = (__float_as_int(amax) >> 23) - 127;  // -127 for zeros and subnormals
      const int e = min(14 - x, 126);
      const float f = pow2f(e);
      inv[nt] = pow2f(-e);
#pragma unroll
      for (int ks = 0; ks < HEAD_DIM / 16; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 v = unpack_bf162(qf[ks][nt][j]);
          qf[ks][nt][j] = pack_half2(v.x * f, v.y * f);
        }
    }
  }
}

// The scales of one chunk's keys and values, the latter in the accumulators' unit.
struct ChunkScale {
  float ks;
  float vs;
  bool bad;  // a scale that is negative, infinite or NaN

  __device__ __forceinline__ void set(float k, float v) {
    bad = !(k >= 0.f && k <= kFloatMax && v >= 0.f && v <= kFloatMax);
    ks = k;
    vs = v * kValueUnit;
  }
};

// softmax_step (pa_decode.cuh) with a scale per chunk: sl[nt][j] is the
// base-2 factor of query nt * 8 + 2c + j without the key scale.  acc.m lies
// kTopWeight below the largest score.  P^T enters as float16; the running sum
// adds the weights unrounded.
template <int HEAD_DIM, int NT, int NSUB>
__device__ __forceinline__ void softmax_step_scaled(WarpAcc<HEAD_DIM, NT>& acc, const float (&sacc)[NSUB][NT][4],
                                                    const int (&valid)[NSUB], const float (&sl)[NT][2],
                                                    const ChunkScale (&cs)[NSUB], int lane,
                                                    uint32_t (&pb)[NSUB][NT][2]) {
  constexpr int KSTEPS = HEAD_DIM / 16;
  const int g = lane >> 2;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float x[NSUB][4];
#pragma unroll
    for (int sb = 0; sb < NSUB; ++sb) {
      const bool v0 = g < valid[sb];
      const bool v1 = g + 8 < valid[sb];
      const float f0 = sl[nt][0] * cs[sb].ks, f1 = sl[nt][1] * cs[sb].ks;
      x[sb][0] = v0 ? sacc[sb][nt][0] * f0 : -INFINITY;
      x[sb][1] = v0 ? sacc[sb][nt][1] * f1 : -INFINITY;
      x[sb][2] = v1 ? sacc[sb][nt][2] * f0 : -INFINITY;
      x[sb][3] = v1 ? sacc[sb][nt][3] * f1 : -INFINITY;
    }
    float mx0 = fmaxf(x[0][0], x[0][2]);
    float mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
    for (int sb = 1; sb < NSUB; ++sb) {
      mx0 = fmaxf(mx0, fmaxf(x[sb][0], x[sb][2]));
      mx1 = fmaxf(mx1, fmaxf(x[sb][1], x[sb][3]));
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, off));
    }
    const float mn0 = fmaxf(acc.m[nt][0], rounded_up(mx0) - kTopWeight);
    const float mn1 = fmaxf(acc.m[nt][1], rounded_up(mx1) - kTopWeight);
    const float cr0 = ex2(acc.m[nt][0] - mn0);
    const float cr1 = ex2(acc.m[nt][1] - mn1);
    const bool grew = __any_sync(FULL_MASK, (mn0 != acc.m[nt][0]) | (mn1 != acc.m[nt][1]));
    acc.m[nt][0] = mn0;
    acc.m[nt][1] = mn1;
    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
    for (int sb = 0; sb < NSUB; ++sb) {
      const float p0 = ex2(x[sb][0] - mn0), p1 = ex2(x[sb][1] - mn1);  // token g
      const float p2 = ex2(x[sb][2] - mn0), p3 = ex2(x[sb][3] - mn1);  // token g + 8
      sum0 += p0 + p2;
      sum1 += p1 + p3;
      pb[sb][nt][0] = movmatrix_trans(pack_half2(p0, p1));  // P^T tokens 0-7 as the B fragment
      pb[sb][nt][1] = movmatrix_trans(pack_half2(p2, p3));  // P^T tokens 8-15
    }
    acc.l[nt][0] = fmaf(acc.l[nt][0], cr0, sum0);
    acc.l[nt][1] = fmaf(acc.l[nt][1], cr1, sum1);
    if (grew) {  // a running maximum moved: rescale the accumulators
#pragma unroll
      for (int dm = 0; dm < KSTEPS; ++dm) {
        acc.o[dm][nt][0] *= cr0;
        acc.o[dm][nt][1] *= cr1;
        acc.o[dm][nt][2] *= cr0;
        acc.o[dm][nt][3] *= cr1;
      }
    }
  }
}

// O^T += vs * V^T P^T over one chunk's codes: pv_e4m3 (pa_decode.cuh) with the
// chunk's products apart from the accumulators until they are scaled: NT * d / 4
// multiply-adds a lane and chunk (with all of the scale in the exponent 64 sequences
// of 128 to 2048 tokens took 29.4 us, now 29.7; 32 of 8192 82.5 and 84.0 us; d = 256, 32
// of 128 to 4096, 36.7 and 38.0 us; split-K of 32 K to 131 K, the sparse steps and one of
// 485 tokens as long as now).
template <int HEAD_DIM, int NT, int ROW_BYTES, bool MASK>
__device__ __forceinline__ void pv_e4m3_scaled(WarpAcc<HEAD_DIM, NT>& acc, const uint32_t (&pb)[NT][2], uint32_t vaddr,
                                               uint32_t tok, uint32_t uo, uint32_t mlo, uint32_t mhi, float vs) {
  constexpr int UNITS = ROW_BYTES / 16;
  constexpr int BOXB = CHUNK * ROW_BYTES;
#pragma unroll
  for (int u = 0; u < HEAD_DIM / 16; u += 2) {
    uint32_t r[4];  // tokens 0-7 / 8-15 of unit u, then of unit u + 1
    ldsm_x4_trans(r, vaddr + (u / UNITS) * BOXB + swizzled<ROW_BYTES>(tok, (u % UNITS) + uo));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[4];  // (tok 2c, 2c+1) at dim 2g, at dim 2g+1; then tokens 2c+8, 2c+9
      e4m3x4_to_half2x2(__byte_perm(r[2 * h], 0u, 0x3120), a[0], a[1]);
      e4m3x4_to_half2x2(__byte_perm(r[2 * h + 1], 0u, 0x3120), a[2], a[3]);
      if constexpr (MASK) {
        a[0] &= mlo;
        a[1] &= mlo;
        a[2] &= mhi;
        a[3] &= mhi;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16_16816(t, a, pb[nt][0], pb[nt][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.o[u + h][nt][i] = fmaf(t[i], vs, acc.o[u + h][nt][i]);
      }
    }
  }
}

// One or two chunks of a stage (NSUB): scores, softmax step, P V.  Chunks
// before the last are full.
template <int HEAD_DIM, int NT, int ROW_BYTES, int NSUB>
__device__ __forceinline__ void attend_scaled(WarpAcc<HEAD_DIM, NT>& acc, const uint32_t (&qf)[HEAD_DIM / 16][NT][2],
                                              uint32_t kb, uint32_t chunk_bytes, uint32_t half_bytes, int valid_last,
                                              const float (&sl)[NT][2], const ChunkScale (&cs)[NSUB], int lane) {
  const uint32_t tok = e4m3_tok(lane), uo = e4m3_uo(lane);
  float sacc[NSUB][NT][4];
  int valid[NSUB];
#pragma unroll
  for (int sb = 0; sb < NSUB; ++sb) {
    qk_e4m3<HEAD_DIM, NT, ROW_BYTES>(sacc[sb], qf, kb + sb * chunk_bytes, tok, uo);
    valid[sb] = sb == NSUB - 1 ? valid_last : CHUNK;
  }
  uint32_t pb[NSUB][NT][2];
  softmax_step_scaled<HEAD_DIM, NT, NSUB>(acc, sacc, valid, sl, cs, lane, pb);
  uint32_t mlo, mhi;
  v_masks(valid_last, lane, mlo, mhi);
#pragma unroll
  for (int sb = 0; sb < NSUB - 1; ++sb)
    pv_e4m3_scaled<HEAD_DIM, NT, ROW_BYTES, false>(acc, pb[sb], kb + sb * chunk_bytes + half_bytes, tok, uo, mlo, mhi,
                                                   cs[sb].vs);
  const uint32_t vb = kb + (NSUB - 1) * chunk_bytes + half_bytes;
  if (valid_last == CHUNK) {
    pv_e4m3_scaled<HEAD_DIM, NT, ROW_BYTES, false>(acc, pb[NSUB - 1], vb, tok, uo, mlo, mhi, cs[NSUB - 1].vs);
  } else {  // the last chunk of the sequence
    pv_e4m3_scaled<HEAD_DIM, NT, ROW_BYTES, true>(acc, pb[NSUB - 1], vb, tok, uo, mlo, mhi, cs[NSUB - 1].vs);
  }
}

// CTA shapes: warps, stages per warp, 16-token chunks per stage, and the CTAs
// per SM that the registers are bounded for (0: unbounded).  Measured on one GPU
// through graph replays, E4M3 pools, beside the shapes of the pool-scaled decode
// (DecodeShape: 4 warps x 2 stages x 2 chunks up to d = 128):
// (The figures compare shapes of one kernel, before the products were scaled apart.)
//  - single launch, d = 128, groups up to 8: 8 x 2 x 1.  A CTA that walks a long
//    sequence alone is paced by its warps' chains, and eight of them halve its
//    share of each (64 sequences of 128 to 2048 tokens, 32/8 heads: 31.2 -> 29.3
//    us; 32 x 8192, 64/8 heads: 91.1 -> 83.5 us; 8 x 1 x 2: 30.5 and 88.3 us).
//    d = 64: 8 x 2 x 2 (64 x 128 to 4096 tokens: 44.1 -> 29.7 us).  At d = 256 and for
//    groups of 16 the accumulators leave no room for more warps (36.5 us against
//    38.2 to 50.9; 104.5 us against 110 to 134).
//  - split-K, whose CTAs cover a partition: many small CTAs overlap their
//    beginnings and ends.  d = 128: 2 x 2 x 2, six per SM (32 K to 131 K tokens, 512
//    per partition: 139.8 -> 129.4 us); groups of 16: 2 x 2 x 1 (227 -> 175 us);
//    d = 256: 2 x 2 x 1 (82.5 -> 80.0 us), five per SM now (6: 84.6 us, 5: 82.8 us).
template <int HEAD_DIM, int NT, int ELEM, int KIND, bool PER_HEAD>
struct BlockShape {
  using Base = DecodeShape<HEAD_DIM, ELEM, KIND>;
  static constexpr bool FP8 = ELEM == 1;
  static constexpr bool WIDE = FP8 && KIND == KIND_SINGLE && NT == 1 && HEAD_DIM <= 128;
  static constexpr bool SMALL = FP8 && KIND == KIND_SPLITK && HEAD_DIM >= 128;
  static constexpr int WARPS = WIDE ? 8 : SMALL ? 2 : Base::WARPS;
  static constexpr int STAGES = WIDE || SMALL ? 2 : Base::STAGES;
  static constexpr int CPS = FP8 && (HEAD_DIM == 64 || (HEAD_DIM == 128 && !WIDE && (!SMALL || NT == 1))) ? 2 : 1;
  static constexpr int MIN_CTAS = WIDE ? 2 : SMALL ? (NT == 1 && HEAD_DIM < 256 ? 6 : 5) : 0;
};
// Tokens of table capacity per CTA of a cluster, at least (a context of 485: 6.0 us
// with 512, 4.9 us with 128).
constexpr int kClusterTokens = 128;

// DecodeCfg with the shape's chunks per stage.
template <typename Shape, int HEAD_DIM, int NT, int ELEM>
struct BlockCfg : DecodeCfg<HEAD_DIM, NT, Shape::WARPS, Shape::STAGES, ELEM> {
  using Base = DecodeCfg<HEAD_DIM, NT, Shape::WARPS, Shape::STAGES, ELEM>;
  static constexpr int CPS = Shape::CPS;
  static constexpr int STAGE_BYTES = CPS * Base::CHUNK_BYTES;
  static constexpr int RING_BYTES = Shape::WARPS * Shape::STAGES * STAGE_BYTES;
  static_assert(RING_BYTES >= (kLongestFirstMax + 1) * 4, "the longest-first ranking fits in the ring");
  static constexpr int SMEM_BYTES =
      1024 + Base::BAR_BYTES + (RING_BYTES > Base::TAIL_BYTES ? RING_BYTES : Base::TAIL_BYTES);
};

// KV: E4M3 (block scales), or T (16-bit pools; PER_HEAD only).  PER_HEAD: the
// table row and the context length belong to (sequence, KV head).  MODE as
// decode_cta: MODE_GRID, MODE_CLUSTER or MODE_LONGEST_FIRST.
template <typename T, typename KV, int HEAD_DIM, int NT, int KIND, int MODE, bool PER_HEAD>
__global__ void __launch_bounds__(BlockShape<HEAD_DIM, NT, kElemBytes<KV>, KIND, PER_HEAD>::WARPS * 32,
                                  BlockShape<HEAD_DIM, NT, kElemBytes<KV>, KIND, PER_HEAD>::MIN_CTAS)
    block_decode_kernel(const __grid_constant__ BlockDecodeParams p) {
  using Shape = BlockShape<HEAD_DIM, NT, kElemBytes<KV>, KIND, PER_HEAD>;
  constexpr int WARPS = Shape::WARPS;
  constexpr int STAGES = Shape::STAGES;
  constexpr bool CLUSTER = MODE == MODE_CLUSTER;
  constexpr bool LONGEST = MODE == MODE_LONGEST_FIRST;
  static_assert(!(LONGEST && PER_HEAD), "sparse batches are not ranked");
  constexpr bool FP8 = kIsFp8<KV>;
  using Cfg = BlockCfg<Shape, HEAD_DIM, NT, kElemBytes<KV>>;
  constexpr int KSTEPS = HEAD_DIM / 16;
  constexpr int GMAX = Cfg::GMAX;
  constexpr int CPS = Cfg::CPS;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint8_t* ring = smem + Cfg::BAR_BYTES;

  const int kvh = blockIdx.x;
  const int part = blockIdx.y;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int H = p.num_heads;

  grid_dependency_wait();

  const int cap = p.max_blocks_per_seq * p.block_size;
  int s = static_cast<int>(blockIdx.z);
  int ctx;
  if constexpr (LONGEST) {  // as decode_cta: CTA z takes the sequence of rank z
    int* lens = reinterpret_cast<int*>(ring);
    int* pick = lens + kLongestFirstMax;
    const int S = p.num_seqs;
    for (int t = threadIdx.x; t < S; t += WARPS * 32) lens[t] = __ldg(p.context_lens + t);
    __syncthreads();
    for (int t = threadIdx.x; t < S; t += WARPS * 32) {
      const int ct = lens[t];
      int rank = 0;
      for (int j = 0; j < S; ++j) {
        const int cj = lens[j];
        rank += (cj > ct) | ((cj == ct) & (j < t));
      }
      if (rank == s) *pick = t;
    }
    __syncthreads();
    s = *pick;
    ctx = lens[s];
    __syncthreads();
  } else {
    ctx = __ldg(p.context_lens + (PER_HEAD ? static_cast<size_t>(s) * p.num_kv_heads + kvh : static_cast<size_t>(s)));
  }
  const int cpb_log2 = p.chunks_per_block_log2;
  const int table_chunks = p.max_blocks_per_seq << cpb_log2;
  const bool ctx_bad = ctx < 0 || ctx > cap;
  const int nchunks = ctx_bad ? 0 : (ctx + CHUNK - 1) / CHUNK;
  const int nclu = CLUSTER ? static_cast<int>(gridDim.y) : 1;
  const int c0 = CLUSTER ? static_cast<int>((static_cast<int64_t>(part) * nchunks) / nclu) : part * p.partition_chunks;
  const int cmax = CLUSTER ? static_cast<int>((static_cast<int64_t>(part + 1) * nchunks) / nclu)
                           : min(c0 + p.partition_chunks, table_chunks);
  const int first = c0 + warp;
  const int nk_cap = first < cmax ? (cmax - first + WARPS - 1) / WARPS : 0;

  uint32_t qf[KSTEPS][NT][2];
  float sl[NT][2];  // base-2 score factor of queries nt * 8 + 2c, + 1
  if constexpr (FP8) {
    float inv[NT];
    load_q_frags_scaled<T, HEAD_DIM, NT>(qf, inv, p.q, s, H, kvh, G, lane);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        sl[nt][j] = std::is_same<T, __half>::value
                        ? p.scale_log2
                        : p.scale_log2 * __shfl_sync(FULL_MASK, inv[nt], (2 * (lane & 3) + j) << 2);
  } else {
    load_q_frags<HEAD_DIM, NT>(qf, p.q, s, H, kvh, G, G, lane);
  }

  // ---- block-table window, as decode_cta; beside it the window's scales.
  //      Stages are consumed at most STAGES * CPS <= 32 chunks after they are
  //      issued, so a consumed chunk lies in the current or the last window.
  const int32_t* bt =
      p.block_tables +
      (PER_HEAD ? static_cast<size_t>(s) * p.num_kv_heads + kvh : static_cast<size_t>(s)) * p.max_blocks_per_seq;
  auto win_load = [&](int kbase) -> int {
    const int k = kbase + lane;
    if (k >= nk_cap) return 0;
    return __ldg(bt + ((first + k * WARPS) >> cpb_log2));
  };
  static_assert(STAGES * CPS <= 32, "the scale windows cover the chunks in flight");
  int win_cur = win_load(0);
  int win_nxt = win_load(32);
  float ks_cur = 0.f, vs_cur = 0.f, ks_last = 0.f, vs_last = 0.f;
  int win_index = 0;
  auto scales_load = [&]() {  // the current window's; entries past the context may be any number
    if constexpr (FP8) {
      const bool in = static_cast<unsigned>(win_cur) < static_cast<unsigned>(p.num_blocks);
      const size_t at = static_cast<size_t>(in ? win_cur : 0) * p.num_kv_heads + kvh;
      ks_cur = __ldg(p.k_scales + at);
      vs_cur = __ldg(p.v_scales + at);
    }
  };

  uint64_t* wbar = bars + warp * STAGES;
  uint8_t* wring = ring + warp * STAGES * Cfg::STAGE_BYTES;
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&wbar[i], 1);
    fence_mbar_init();
  }
  __syncwarp();

  const int nparts = CLUSTER ? nclu : (nchunks + p.partition_chunks - 1) / p.partition_chunks;
  if (nchunks == 0) {  // empty: zeros; impossible length: NaN.  Written once.
    if (part == 0) {
      const T v = to_elem<T>(ctx_bad ? NAN : 0.f);
      T* o = static_cast<T*>(p.out) + (static_cast<size_t>(s) * H + kvh * G) * HEAD_DIM;
      for (int i = threadIdx.x; i < G * HEAD_DIM; i += WARPS * 32) o[i] = v;
    }
    allow_dependent_launch();
    return;  // in a cluster every CTA takes this exit together
  }
  if (!CLUSTER && part >= nparts) {
    allow_dependent_launch();
    return;
  }
  const bool single = !CLUSTER && nparts == 1;
  const int c1 = CLUSTER ? cmax : min(c0 + p.partition_chunks, nchunks);
  const int nk = first < c1 ? (c1 - first + WARPS - 1) / WARPS : 0;
  const bool empty = CLUSTER && c1 <= c0;  // a short sequence: nothing for this CTA

  const int nst = (nk + CPS - 1) / CPS;
  int issued = 0;
  bool bad = false;

  auto issue_next = [&]() {
    const int it = issued;
    const int slot = it % STAGES;
    const int nload = min(CPS, nk - it * CPS);
    uint8_t* dst = wring + slot * Cfg::STAGE_BYTES;
    if (lane == 0) mbar_arrive_expect_tx(&wbar[slot], nload * Cfg::CHUNK_BYTES);
#pragma unroll
    for (int j = 0; j < CPS; ++j) {
      const int k = it * CPS + j;
      if (j > 0 && k >= nk) break;  // warp-uniform
      if (k > 0 && (k & 31) == 0) {
        win_cur = win_nxt;
        win_nxt = win_load(k + 32);
        ks_last = ks_cur;
        vs_last = vs_cur;
        scales_load();
        ++win_index;
      }
      int phys = __shfl_sync(FULL_MASK, win_cur, k & 31);
      if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
        bad = true;  // never read outside the pool; the result becomes NaN
        phys = 0;
      }
      const int ch = first + k * WARPS;
      const int row0 = (ch & ((1 << cpb_log2) - 1)) * CHUNK;
      if (lane == 0) {
        uint8_t* cd = dst + j * Cfg::CHUNK_BYTES;
        const int y = phys * p.block_size + row0;
#pragma unroll
        for (int b = 0; b < Cfg::DBOX; ++b) {
          tma_load_3d(cd + b * Cfg::BOX_B, &p.tmap_k, b * Cfg::BOX_ELEMS, kvh, y, &wbar[slot]);
          tma_load_3d(cd + Cfg::HALF_BYTES + b * Cfg::BOX_B, &p.tmap_v, b * Cfg::BOX_ELEMS, kvh, y, &wbar[slot]);
        }
      }
    }
    ++issued;
  };

#pragma unroll 1
  for (int i = 0; i < STAGES && i < nst; ++i) issue_next();
  if (nst > 0) scales_load();  // the first window's, behind its copies (no window moves before)

  WarpAcc<HEAD_DIM, NT> acc;
  acc.reset();

  auto chunk_scale = [&](int k) {
    ChunkScale c;
    const bool cur = (k >> 5) == win_index;
    c.set(__shfl_sync(FULL_MASK, cur ? ks_cur : ks_last, k & 31), __shfl_sync(FULL_MASK, cur ? vs_cur : vs_last, k & 31));
    bad |= c.bad;
    return c;
  };

  int consumed = 0;
  bool timed_out = false;
#pragma unroll 1
  for (; consumed < nst; ++consumed) {
    const int it = consumed;
    const int slot = it % STAGES;
    const bool ok = mbar_wait_bounded(&wbar[slot], (it / STAGES) & 1, WAIT_LIMIT_NS);
    if (!__all_sync(FULL_MASK, ok)) {  // a warp-uniform decision
      timed_out = true;
      break;
    }
    const int k0 = it * CPS;
    const int ch = first + k0 * WARPS;
    const int valid = min(CHUNK, ctx - ch * CHUNK);
    const uint32_t stage = smem_addr(wring + slot * Cfg::STAGE_BYTES);
    if constexpr (FP8) {
      if (CPS == 2 && k0 + 1 < nk) {
        const int valid2 = min(CHUNK, ctx - (ch + WARPS) * CHUNK);
        const ChunkScale cs[2] = {chunk_scale(k0), chunk_scale(k0 + 1)};
        attend_scaled<HEAD_DIM, NT, Cfg::ROW_BYTES, 2>(acc, qf, stage, Cfg::CHUNK_BYTES, Cfg::HALF_BYTES, valid2, sl,
                                                       cs, lane);
      } else {
        const ChunkScale cs[1] = {chunk_scale(k0)};
        attend_scaled<HEAD_DIM, NT, Cfg::ROW_BYTES, 1>(acc, qf, stage, Cfg::CHUNK_BYTES, Cfg::HALF_BYTES, valid, sl,
                                                       cs, lane);
      }
    } else {
      attend_chunk<T, HEAD_DIM, NT>(acc, qf, stage, Cfg::HALF_BYTES, valid, p.scale_log2, lane);
    }
    fence_proxy_async_smem();  // this lane's reads of the slot precede the refill's writes
    __syncwarp();
    if (issued < nst) issue_next();
  }

  if (timed_out) {
    bad = true;
    for (int k = consumed; k < issued; ++k)
      (void)mbar_wait_bounded(&wbar[k % STAGES], (k / STAGES) & 1, WAIT_LIMIT_NS);
  }

  reduce_warp_sums<HEAD_DIM, NT>(acc);

  __syncthreads();  // every warp is done with its ring: reuse it for the merge
  float* mo = reinterpret_cast<float*>(ring);
  float* mm = mo + WARPS * GMAX * Cfg::MO_PITCH;
  float* ml = mm + WARPS * GMAX;
  int* mbad = reinterpret_cast<int*>(ml + WARPS * GMAX);
  store_warp_state<HEAD_DIM, NT, FP8>(acc, mo + warp * GMAX * Cfg::MO_PITCH, mm + warp * GMAX, ml + warp * GMAX,
                                      Cfg::MO_PITCH, lane);
  if (lane == 0) mbad[warp] = bad ? 1 : 0;
  __syncthreads();

  bool any_bad = false;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) any_bad |= mbad[w] != 0;

  for (int idx = threadIdx.x; idx < G * HEAD_DIM; idx += WARPS * 32) {
    const int head = idx / HEAD_DIM;
    const int d = idx - head * HEAD_DIM;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, mm[w * GMAX + head]);
    float L = 0.f, O = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = ex2(mm[w * GMAX + head] - M);  // warps without chunks: 2^-inf = 0
        L += ml[w * GMAX + head] * f;
        O += mo[(w * GMAX + head) * Cfg::MO_PITCH + d] * f;
      }
    }
    // no positive sum: a cluster CTA without chunks (weight 0), or NaN scores
    const bool none = !(L > 0.f) && !empty;
    const float r = any_bad || none ? NAN : (empty ? 0.f : FP8 ? O / L * kValueUnitInv : O / L);
    const float Lm = FP8 ? L * kValueUnit : L;  // a merge adds r times this: at most 1 in 2^24 tokens
    const size_t qrow = static_cast<size_t>(s) * H + kvh * G + head;
    if (CLUSTER) {
      float* cta = reinterpret_cast<float*>(ring + Cfg::CTA_OFFSET);
      cta[head * HEAD_DIM + d] = r;
      if (d == 0) {
        cta[GMAX * HEAD_DIM + head] = any_bad || none ? 0.f : M;
        cta[GMAX * HEAD_DIM + GMAX + head] = any_bad || none ? 1.f : Lm;
      }
    } else if (single) {
      static_cast<T*>(p.out)[qrow * HEAD_DIM + d] = to_elem<T>(r);
    } else {
      const size_t row = qrow * p.max_num_partitions + part;
      p.ws_o[row * HEAD_DIM + d] = r;
      if (d == 0) {
        p.ws_m[row] = any_bad || none ? 0.f : M;
        p.ws_l[row] = any_bad || none ? 1.f : Lm;
      }
    }
  }

  if constexpr (CLUSTER) {  // as decode_cta: merge the cluster's results through distributed shared memory
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    float* cta = reinterpret_cast<float*>(ring + Cfg::CTA_OFFSET);
    const int rank = static_cast<int>(cluster.block_rank());
    for (int idx = rank * (WARPS * 32) + threadIdx.x; idx < G * HEAD_DIM; idx += nclu * WARPS * 32) {
      const int head = idx / HEAD_DIM;
      const int d = idx - head * HEAD_DIM;
      float M = -INFINITY;
      for (int r = 0; r < nclu; ++r) {
        const float* peer = cluster.map_shared_rank(cta, r);
        M = fmaxf(M, peer[GMAX * HEAD_DIM + head]);
      }
      float L = 0.f, O = 0.f;
      for (int r = 0; r < nclu; ++r) {
        const float* peer = cluster.map_shared_rank(cta, r);
        const float w = peer[GMAX * HEAD_DIM + GMAX + head] * ex2(peer[GMAX * HEAD_DIM + head] - M);
        L += w;
        O += w * peer[head * HEAD_DIM + d];
      }
      static_cast<T*>(p.out)[(static_cast<size_t>(s) * H + kvh * G + head) * HEAD_DIM + d] = to_elem<T>(O / L);
    }
    cluster.sync();  // no CTA leaves while the others still read its shared memory
  }
  allow_dependent_launch();
}

// ================================================================ launchers
// Tensor maps over the pools.  Dense launches use make_pool_map, whose copies ask
// L2 for 256 bytes around each row: the neighbouring head's row, which a
// neighbouring CTA reads.  With a table per KV head the neighbour usually wants
// another block, so one-byte rows of 128 bytes ask for 128 (16 sequences, 96 of
// 125 to 1024 blocks of 32 tokens each: 138 -> 104 MB read).  Maps of recent pools
// are kept as in make_pool_map: a map depends on nothing but its arguments.
template <typename KV, int HEAD_DIM, bool PER_HEAD>
struct PoolMaps {
  static cudaError_t make(CUtensorMap* map, const void* pool, int num_kv_heads, int64_t rows) {
    if constexpr (!PER_HEAD || HEAD_DIM * kElemBytes<KV> >= 256) {
      return make_pool_map<KV, HEAD_DIM>(map, pool, num_kv_heads, rows);
    } else {
      struct Entry {
        CUtensorMap map;
        const void* pool;
        int64_t rows;
        int heads;
      };
      constexpr int kEntries = 16;
      thread_local Entry cache[kEntries];
      thread_local int next = 0;
      for (const Entry& e : cache)
        if (e.pool != nullptr && e.pool == pool && e.rows == rows && e.heads == num_kv_heads) {
          *map = e.map;
          return cudaSuccess;
        }
      EncodeTiledFn enc = nullptr;
      const cudaError_t err = encode_fn(&enc);
      if (err != cudaSuccess) return err;
      using Cfg = DecodeCfg<HEAD_DIM, 1, 1, 1, kElemBytes<KV>>;
      constexpr int ELEM = kElemBytes<KV>;
      const cuuint64_t dims[3] = {static_cast<cuuint64_t>(HEAD_DIM), static_cast<cuuint64_t>(num_kv_heads),
                                  static_cast<cuuint64_t>(rows)};
      const cuuint64_t strides[2] = {static_cast<cuuint64_t>(HEAD_DIM) * ELEM,
                                     static_cast<cuuint64_t>(num_kv_heads) * HEAD_DIM * ELEM};
      const cuuint32_t box[3] = {Cfg::BOX_ELEMS, 1, CHUNK};
      const cuuint32_t estride[3] = {1, 1, 1};
      const CUresult r =
          enc(map, tma_dtype<KV>(), 3, const_cast<void*>(pool), dims, strides, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              Cfg::ROW_BYTES == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              HEAD_DIM * ELEM >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
      cache[next] = Entry{*map, pool, rows, num_kv_heads};
      next = (next + 1) % kEntries;
      return cudaSuccess;
    }
  }
};

template <typename T, typename KV, int HEAD_DIM, int NT, int MODE, int KIND, bool PER_HEAD>
cudaError_t launch_block_decode_t(const BlockDecodeArgs& a, cudaStream_t stream) {
  constexpr bool CLUSTER = MODE == MODE_CLUSTER;
  constexpr int ELEM = kElemBytes<KV>;
  using Shape = BlockShape<HEAD_DIM, NT, ELEM, KIND, PER_HEAD>;
  constexpr int WARPS = Shape::WARPS;
  using Cfg = BlockCfg<Shape, HEAD_DIM, NT, ELEM>;
  auto kern = block_decode_kernel<T, KV, HEAD_DIM, NT, KIND, MODE, PER_HEAD>;
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = ensure_smem(kern, Cfg::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  BlockDecodeParams p;
  const int64_t pool_rows = static_cast<int64_t>(a.num_blocks) * a.block_size;
  using Maps = PoolMaps<KV, HEAD_DIM, PER_HEAD>;
  e = Maps::make(&p.tmap_k, a.k_cache, a.num_kv_heads, pool_rows);
  if (e != cudaSuccess) return e;
  e = Maps::make(&p.tmap_v, a.v_cache, a.num_kv_heads, pool_rows);
  if (e != cudaSuccess) return e;
  p.out = a.out;
  p.q = a.q;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  const size_t rows = ws_rows(a.num_seqs, a.num_heads, a.max_num_partitions);
  p.ws_o = a.ws;
  p.ws_m = a.ws ? a.ws + rows * HEAD_DIM : nullptr;
  p.ws_l = a.ws ? a.ws + rows * HEAD_DIM + rows : nullptr;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_heads / a.num_kv_heads;
  p.block_size = a.block_size;
  p.chunks_per_block_log2 = __builtin_ctz(static_cast<unsigned>(a.block_size / CHUNK));
  p.num_blocks = a.num_blocks;
  p.partition_chunks = a.partition_size / CHUNK;
  p.max_num_partitions = a.max_num_partitions;
  p.num_seqs = a.num_seqs;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_kv_heads, CLUSTER ? a.cluster_size : a.max_num_partitions, a.num_seqs);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (CLUSTER) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = a.cluster_size;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Resident CTAs of the single launch on the device (SMs x CTAs per SM), cached
// per device.
template <typename T, typename KV, int HEAD_DIM, int NT, bool PER_HEAD>
cudaError_t block_decode_slots(int* slots) {
  constexpr int ELEM = kElemBytes<KV>;
  using Shape = BlockShape<HEAD_DIM, NT, ELEM, KIND_SINGLE, PER_HEAD>;
  constexpr int WARPS = Shape::WARPS;
  using Cfg = BlockCfg<Shape, HEAD_DIM, NT, ELEM>;
  static std::atomic<int> cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_acquire);
    if (c > 0) {
      *slots = c;
      return cudaSuccess;
    }
  }
  auto kern = block_decode_kernel<T, KV, HEAD_DIM, NT, KIND_SINGLE, MODE_GRID, PER_HEAD>;
  static std::atomic<uint64_t> smem_set{0};
  e = ensure_smem(kern, Cfg::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  int sms = 0, per_sm = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, WARPS * 32, Cfg::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  *slots = sms * (per_sm > 0 ? per_sm : 1);
  if (dev < 64) cache[dev].store(*slots, std::memory_order_release);
  return cudaSuccess;
}

// As launch_decode_auto: one CTA per (sequence, KV head) when those fill the
// resident slots (longest first when they need one second wave), else
// clusters of up to 8 CTAs per pair.  Split-K (a workspace): the plain grid.
template <typename T, typename KV, int HEAD_DIM, int NT, bool PER_HEAD>
cudaError_t launch_block_decode_auto(const BlockDecodeArgs& a, cudaStream_t stream) {
  if constexpr (!PER_HEAD) {
    if (a.ws != nullptr) return launch_block_decode_t<T, KV, HEAD_DIM, NT, MODE_GRID, KIND_SPLITK, false>(a, stream);
  }
  int slots = 0;
  cudaError_t e = block_decode_slots<T, KV, HEAD_DIM, NT, PER_HEAD>(&slots);
  if (e != cudaSuccess) return e;
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
  const int64_t k = std::min<int64_t>(slots / pairs, (cap + kClusterTokens - 1) / kClusterTokens);
  BlockDecodeArgs b = a;
  b.cluster_size = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, k)));
  if (b.cluster_size > 1) return launch_block_decode_t<T, KV, HEAD_DIM, NT, MODE_CLUSTER, KIND_SINGLE, PER_HEAD>(b, stream);
  if constexpr (!PER_HEAD) {
    if (pairs > slots && pairs <= 2 * static_cast<int64_t>(slots) && a.num_seqs <= kLongestFirstMax)
      return launch_block_decode_t<T, KV, HEAD_DIM, NT, MODE_LONGEST_FIRST, KIND_SINGLE, false>(b, stream);
  }
  return launch_block_decode_t<T, KV, HEAD_DIM, NT, MODE_GRID, KIND_SINGLE, PER_HEAD>(b, stream);
}

template <typename T, typename KV, bool PER_HEAD>
cudaError_t launch_block_decode_typed(const BlockDecodeArgs& a, cudaStream_t stream) {
  const bool two = a.num_heads / a.num_kv_heads > 8;
  switch (a.head_dim) {
    case 64:
      return two ? launch_block_decode_auto<T, KV, 64, 2, PER_HEAD>(a, stream)
                 : launch_block_decode_auto<T, KV, 64, 1, PER_HEAD>(a, stream);
    case 128:
      return two ? launch_block_decode_auto<T, KV, 128, 2, PER_HEAD>(a, stream)
                 : launch_block_decode_auto<T, KV, 128, 1, PER_HEAD>(a, stream);
    case 256: return two ? cudaErrorInvalidValue : launch_block_decode_auto<T, KV, 256, 1, PER_HEAD>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace pa
