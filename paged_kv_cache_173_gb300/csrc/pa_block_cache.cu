// pa_block_cache.cu -- side data kept per (block, KV head): the cache write
// into E4M3 pools with one scale per (block, KV head), the key bounds of the
// block selection, and the selection itself.
//
//  block_write_kernel   block_size / 16 warps per (run of new tokens in a block, KV head, K or V)
//  key_bounds_kernel    the same per (run of new tokens in a block, KV head)
//  block_score_kernel   one warp per (32 blocks of a sequence, KV head)
//  select_kernel        one CTA per (sequence, KV head)
//
// "PagedAttention: when the KV cache meets OS paging", section 6, stacks
// compression on the block abstraction; the block is the unit here for the
// scales and for the selection.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_block.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// The block of a slot, -1 for padding and slots outside the pool (num_slots < 2^31).
__device__ __forceinline__ int slot_block(int64_t slot, int num_slots, int log2_b) {
  return static_cast<uint64_t>(slot) < static_cast<uint64_t>(num_slots) ? static_cast<int>(slot) >> log2_b : -1;
}

// ---------------------------------------------------------- runs of new tokens
// The new tokens of one block stand next to each other in slot_mapping: a run.
// A CTA looks at a stretch of tokens for one KV head and hands each run that
// begins there to a group of block_size / 16 warps; warp g of the group holds
// the run's tokens 16 g .. 16 g + 15 in registers, so every element is read
// once, whatever the block size.  (8 prompts of 2048 tokens, 8 KV heads of 128,
// blocks of 16, bf16: 19.3 us for the write, 10.0 us for the bounds; one warp per
// run that walked its tokens twice took 153 and 135 us.)
constexpr int kRunRows = 16;      // tokens a warp holds
constexpr int kMaxStretch = 128;  // tokens a CTA looks at, at most
constexpr int kMaxGroup = 16;     // warps per group at most: 256-token blocks

struct RunParams {
  const int64_t* slot_mapping;
  int num_slots;  // num_blocks * block_size
  int num_tokens;
  int num_kv_heads;
  int block_size;
  int log2_b;
  int stretch;  // tokens per CTA
};

// The first tokens of the runs that begin in a CTA's stretch, by 32 tokens: one
// warp looks at each 32.
struct RunList {
  int count[kMaxStretch / 32];
  int start[kMaxStretch / 32][32];

  __device__ __forceinline__ void find(const RunParams& p, int t0) {
    const int lane = threadIdx.x & 31;
    const int i = threadIdx.x >> 5;
    if (i < kMaxStretch / 32) {
      const int x = 32 * i + lane;
      const int t = t0 + x;
      const bool in = x < p.stretch && t < p.num_tokens;
      const int blk = in ? slot_block(__ldg(p.slot_mapping + t), p.num_slots, p.log2_b) : -1;
      const int prev = in && t > 0 ? slot_block(__ldg(p.slot_mapping + t - 1), p.num_slots, p.log2_b) : -1;
      const bool first = blk >= 0 && blk != prev;
      const unsigned mask = __ballot_sync(kFull, first);
      if (first) start[i][__popc(mask & ((1u << lane) - 1u))] = t;
      if (lane == 0) count[i] = __popc(mask);
    }
    __syncthreads();
  }
  // The first token of run k, -1 past the last.
  __device__ __forceinline__ int get(int k) const {
#pragma unroll
    for (int i = 0; i < kMaxStretch / 32; ++i) {
      const int c = count[i];
      if (k < c) return start[i][k];
      k -= c;
    }
    return -1;
  }
  __device__ __forceinline__ int total() const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kMaxStretch / 32; ++i) n += count[i];
    return n;
  }
};

// Lane r < 16: the offset in the block of the run's token (first + r), -1 if it
// belongs to another block.  `first`: the warp's first token, `blk` the run's block.
__device__ __forceinline__ int row_offset(const RunParams& p, int first, int blk, int lane) {
  const int t = first + lane;
  if (lane >= kRunRows || t >= p.num_tokens) return -1;
  const int64_t slot = __ldg(p.slot_mapping + t);
  return slot_block(slot, p.num_slots, p.log2_b) == blk ? static_cast<int>(slot & (p.block_size - 1)) : -1;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A warp's 16 rows of one KV head: lane i holds 16-byte unit i % U of row (32 / U) j + i / U.
template <int HEAD_DIM>
struct RowTile {
  static constexpr int U = HEAD_DIM / 8;              // units per row
  static constexpr int RPI = 32 / U;                  // rows per load
  static constexpr int N = kRunRows / RPI;            // loads
  uint4 v[N];  // zeros in rows that hold no token of the run

  // `rows`: the tensor as units, `first`: the warp's first token, off16: row_offset of each
  // lane, `whole`: every row holds a token.
  __device__ __forceinline__ void load(const uint4* rows, int first, int num_kv_heads, int h, int off16, bool whole,
                                       int lane) {
    const int64_t pitch = static_cast<int64_t>(num_kv_heads) * U;
    const uint4* at = rows + (first + lane / U) * pitch + static_cast<int64_t>(h) * U + lane % U;
    if (whole) {  // warp-uniform
#pragma unroll
      for (int j = 0; j < N; ++j, at += RPI * pitch) v[j] = __ldg(at);
      return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int r = j * RPI + lane / U;
      v[j] = __shfl_sync(kFull, off16, r) >= 0 ? __ldg(at + static_cast<int64_t>(j) * RPI * pitch) : make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // The largest |element| over finite elements.  16-bit floats order like their
  // bits, so the maximum runs on packed pairs; a non-finite element, the only
  // case that needs a look at each, shows in it.
  template <typename T>
  __device__ __forceinline__ float finite_amax(bool* all_finite) const {
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      m = max_u16x2(m, v[j].x & 0x7fff7fffu);
      m = max_u16x2(m, v[j].y & 0x7fff7fffu);
      m = max_u16x2(m, v[j].z & 0x7fff7fffu);
      m = max_u16x2(m, v[j].w & 0x7fff7fffu);
    }
    uint32_t top = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
    *all_finite = top < kInf;
    if (top >= kInf) {  // warp-uniform
      m = 0u;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
          m = max(m, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
        }
      }
      top = __reduce_max_sync(kFull, m);
    }
    return unpack2<T>(top).x;
  }
};

// Asks L2 for the rows of one head that a CTA's stretch holds, while the runs are found: the
// slots, the list and the rows are three waits in turn (write of 8 x 2048 tokens 22.7 -> 19.3 us;
// the bounds, whose keys the write beside them has just brought into L2, lose 0.4 us by it).
template <int HEAD_DIM>
__device__ __forceinline__ void prefetch_rows(const uint4* rows, const RunParams& p, int t0, int h) {
  constexpr int LINES = HEAD_DIM / 64;  // 128-byte lines of a row
  if (p.stretch < kRunRows) return;
  for (int i = threadIdx.x; i < p.stretch * LINES; i += blockDim.x) {
    const int64_t t = t0 + i / LINES;
    if (t >= p.num_tokens) break;
    const uint4* at = rows + (t * p.num_kv_heads + h) * (HEAD_DIM / 8) + i % LINES * 8;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
  }
}

// 256 threads for blocks of up to 128 tokens (8 groups of one warp ... one of 8), 512
// for 256.  A warp's rows take 32 registers at d = 128, so 64 in all let 32 warps share an SM.
constexpr int run_min_ctas(int head_dim, int threads) { return (head_dim > 128 ? 512 : 1024) / threads; }

struct BlockWriteParams {
  RunParams r;
  const uint4* key;
  const uint4* value;
  uint2* k_cache;  // 8 codes per unit
  uint2* v_cache;
  float* k_scales;
  float* v_scales;
};

// 8 elements times k (DIVIDE: over k) as 8 codes.
template <typename T, bool DIVIDE>
__device__ __forceinline__ uint2 to_codes8(const uint4& v, float k) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = unpack2<T>(w[i]);
    f = DIVIDE ? make_float2(__fdiv_rn(f.x, k), __fdiv_rn(f.y, k)) : make_float2(f.x * k, f.y * k);
    c[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 8 codes moved to another scale: value(code) * ratio, rounded to float32, then to a code.
__device__ __forceinline__ uint2 move_codes8(const uint2& v, float ratio) {
  const uint32_t in[2] = {v.x, v.y};
  uint32_t out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t lo, hi;
    e4m3x4_to_half2x2(in[j], lo, hi);
    const float2 a = unpack_half2(lo), b = unpack_half2(hi);
    const uint32_t c0 = __nv_cvt_float2_to_fp8x2(make_float2(a.x * ratio, a.y * ratio), __NV_SATFINITE, __NV_E4M3);
    const uint32_t c1 = __nv_cvt_float2_to_fp8x2(make_float2(b.x * ratio, b.y * ratio), __NV_SATFINITE, __NV_E4M3);
    out[j] = c0 | (c1 << 16);
  }
  return make_uint2(out[0], out[1]);
}

// Grid (stretch, KV head, K or V).  The write is a copy that shrinks: 3 bytes
// moved per element, so HBM bounds prompts (101 MB in 19.3 us: 5.2 TB/s; the rows are
// held in registers between the maximum and the codes, which leaves 32 warps per SM)
// and latency bounds single tokens (64 of them 2.8 us).
template <typename T, int HEAD_DIM, int THREADS>
__global__ void __launch_bounds__(THREADS, run_min_ctas(HEAD_DIM, THREADS)) block_write_kernel(const __grid_constant__ BlockWriteParams p) {
  using Tile = RowTile<HEAD_DIM>;
  __shared__ RunList runs;
  __shared__ float sh_amax[kMaxGroup];
  __shared__ int sh_starts[kMaxGroup];
  grid_dependency_wait();
  allow_dependent_launch();
  const RunParams& rp = p.r;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int gw_log2 = rp.log2_b - 4;  // 2^gw_log2 = block_size / kRunRows warps per group
  const int gw = 1 << gw_log2;
  const int groups = (THREADS / 32) >> gw_log2;
  const int g = warp >> gw_log2;
  const int wg = warp & (gw - 1);
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int t0 = blockIdx.x * rp.stretch;
  const uint4* src = is_v ? p.value : p.key;
  prefetch_rows<HEAD_DIM>(src, rp, t0, h);
  runs.find(rp, t0);
  const int nruns = runs.total();
  uint2* cache = is_v ? p.v_cache : p.k_cache;
  float* scales = is_v ? p.v_scales : p.k_scales;
  for (int k0 = 0; k0 < nruns; k0 += groups) {  // the same trips for every warp
    const int t = runs.get(k0 + g);
    const bool on = t >= 0;
    const int blk = on ? slot_block(__ldg(rp.slot_mapping + t), rp.num_slots, rp.log2_b) : 0;
    const int first = t + wg * kRunRows;
    const int off16 = on ? row_offset(rp, first, blk, lane) : -1;
    float* scale = scales + (static_cast<int64_t>(blk) * rp.num_kv_heads + h);
    // 16 tokens in consecutive slots
    const int off0 = __shfl_sync(kFull, off16, 0);
    const bool whole = __all_sync(kFull, lane >= kRunRows || (off0 >= 0 && off16 == off0 + lane));
    Tile tile;
    tile.load(src, first, rp.num_kv_heads, h, off16, whole, lane);
    const float was = on ? *scale : 0.f;
    bool finite;
    float amax = tile.template finite_amax<T>(&finite);
    int starts = __any_sync(kFull, off16 == 0);
    if (gw > 1) {
      if (lane == 0) {
        sh_amax[warp] = amax;
        sh_starts[warp] = starts;
      }
      __syncthreads();
      for (int i = g * gw; i < (g + 1) * gw; ++i) {
        amax = fmaxf(amax, sh_amax[i]);
        starts |= sh_starts[i];
      }
    }
    const float need = pow2f(scale_exp(amax));
    const float old = !starts && was > 0.f && was <= kFloatMax ? was : 0.f;
    const float s = fmaxf(old, need);
    const int pitch = rp.num_kv_heads * Tile::U;  // units between slots
    uint2* rows = cache + static_cast<int64_t>(blk << rp.log2_b) * pitch + h * Tile::U + lane % Tile::U;
    if (on && old > 0.f && s > old) {  // the block's other codes move to the new scale
      const float ratio = __fdiv_rn(old, s);
#pragma unroll 4
      for (int o = wg * kRunRows + lane / Tile::U; o < (wg + 1) * kRunRows; o += Tile::RPI)
        rows[static_cast<int64_t>(o) * pitch] = move_codes8(rows[static_cast<int64_t>(o) * pitch], ratio);
    }
    // the moved codes before the new ones (which may share rows with them), every
    // read of the scale before its write
    if (gw > 1) {
      __syncthreads();
    } else {
      __syncwarp();
    }
    const int bits = __float_as_int(s);
    const bool pow2 = (bits & 0x7fffff) == 0 && bits <= (126 + 127) << 23 && bits >= 1 << 23;
    if (pow2) {  // uniform over the group: a multiplication by the exact inverse
      const float inv = pow2f(127 - (bits >> 23));
      if (whole) {
        uint2* at = rows + static_cast<int64_t>(off0 + lane / Tile::U) * pitch;
        const int64_t step = static_cast<int64_t>(Tile::RPI) * pitch;
#pragma unroll
        for (int j = 0; j < Tile::N; ++j, at += step) *at = to_codes8<T, false>(tile.v[j], inv);
      } else {
#pragma unroll
        for (int j = 0; j < Tile::N; ++j) {
          const int off = __shfl_sync(kFull, off16, j * Tile::RPI + lane / Tile::U);
          if (off >= 0) rows[static_cast<int64_t>(off) * pitch] = to_codes8<T, false>(tile.v[j], inv);
        }
      }
    } else {  // a scale from elsewhere
#pragma unroll 1
      for (int j = 0; j < kRunRows; j += Tile::RPI) {
        const int r = j + lane / Tile::U;
        const int off = __shfl_sync(kFull, off16, r);
        if (off >= 0)
          rows[static_cast<int64_t>(off) * pitch] =
              to_codes8<T, true>(__ldg(src + (static_cast<int64_t>(first + r) * rp.num_kv_heads + h) * Tile::U + lane % Tile::U), s);
      }
    }
    if (on && wg == 0 && lane == 0) *scale = s;
  }
}

struct KeyBoundsParams {
  RunParams r;
  const uint4* key;
  int8_t* bounds;
  int32_t* exps;
};

// lo (up = false): floor(v / 2^e); hi: ceil.  Codes stay in [-127, 127].
__device__ __forceinline__ int bound_code(float v, float inv, bool up) {
  const float x = v * inv;
  const float r = up ? ceilf(x) : floorf(x);
  return static_cast<int>(fminf(fmaxf(r, -127.f), 127.f));
}

// Packed minimum and maximum of 16-bit floats without NaN.
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// NaN halves of a packed pair replaced by `with` (both halves of it).
template <typename T>
__device__ __forceinline__ uint32_t nan2(uint32_t w, uint32_t with) {
  constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  uint32_t r = w;
  if ((w & 0x7fffu) > kInf) r = (r & 0xffff0000u) | (with & 0xffffu);
  if (((w >> 16) & 0x7fffu) > kInf) r = (r & 0xffffu) | (with & 0xffff0000u);
  return r;
}

// Grid (stretch, KV head).  Reads 2 bytes per element and writes 2 per channel
// and block: HBM bounds prompts (36 MB in 10.0 us), latency single tokens (64: 2.9 us).
template <typename T, int HEAD_DIM, int THREADS>
__global__ void __launch_bounds__(THREADS, run_min_ctas(HEAD_DIM, THREADS)) key_bounds_kernel(const __grid_constant__ KeyBoundsParams p) {
  using Tile = RowTile<HEAD_DIM>;
  constexpr int U = Tile::U;
  constexpr uint32_t kPosInf = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t kNegInf = kPosInf | 0x80008000u;
  __shared__ RunList runs;
  __shared__ float sh_amax[kMaxGroup];
  __shared__ int sh_starts[kMaxGroup];
  __shared__ uint4 sh_lo[kMaxGroup][U], sh_hi[kMaxGroup][U];
  grid_dependency_wait();
  allow_dependent_launch();
  const RunParams& rp = p.r;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int gw_log2 = rp.log2_b - 4;  // 2^gw_log2 = block_size / kRunRows warps per group
  const int gw = 1 << gw_log2;
  const int groups = (THREADS / 32) >> gw_log2;
  const int g = warp >> gw_log2;
  const int wg = warp & (gw - 1);
  const int h = blockIdx.y;
  const int t0 = blockIdx.x * rp.stretch;
  runs.find(rp, t0);
  const int nruns = runs.total();
  for (int k0 = 0; k0 < nruns; k0 += groups) {  // the same trips for every warp
    const int t = runs.get(k0 + g);
    const bool on = t >= 0;
    const int blk = on ? slot_block(__ldg(rp.slot_mapping + t), rp.num_slots, rp.log2_b) : 0;
    const int first = t + wg * kRunRows;
    const int off16 = on ? row_offset(rp, first, blk, lane) : -1;
    const int64_t at = static_cast<int64_t>(blk) * rp.num_kv_heads + h;
    const bool whole = __all_sync(kFull, off16 >= 0 || lane >= kRunRows);  // 16 tokens of the run
    Tile tile;
    tile.load(p.key, first, rp.num_kv_heads, h, off16, whole, lane);
    // the block's bounds as they are, on the lanes that will write them
    const bool writer = on && wg == 0 && lane < U;
    uint2* lo_at = reinterpret_cast<uint2*>(p.bounds + at * 2 * HEAD_DIM) + lane % U;
    uint2* hi_at = lo_at + HEAD_DIM / 8;
    uint2 old_lo = make_uint2(0u, 0u), old_hi = make_uint2(0u, 0u);
    int was = kMinBoundExp;
    if (writer) {
      old_lo = *lo_at;
      old_hi = *hi_at;
      was = p.exps[at];
    }
    bool finite;
    float amax = tile.template finite_amax<T>(&finite);
    int starts = __any_sync(kFull, off16 == 0);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = kPosInf;
      hi[i] = kNegInf;
    }
    if (finite && whole) {
#pragma unroll
      for (int j = 0; j < Tile::N; ++j) {
        const uint32_t w[4] = {tile.v[j].x, tile.v[j].y, tile.v[j].z, tile.v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = min2<T>(lo[i], w[i]);
          hi[i] = max2<T>(hi[i], w[i]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < Tile::N; ++j) {
        if (__shfl_sync(kFull, off16, j * Tile::RPI + lane / U) < 0) continue;
        const uint32_t w[4] = {tile.v[j].x, tile.v[j].y, tile.v[j].z, tile.v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = min2<T>(lo[i], nan2<T>(w[i], kNegInf));  // NaN: the widest bound
          hi[i] = max2<T>(hi[i], nan2<T>(w[i], kPosInf));
        }
      }
    }
#pragma unroll
    for (int o = U; o < 32; o <<= 1)  // over the lanes that hold the same channels
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = min2<T>(lo[i], __shfl_xor_sync(kFull, lo[i], o));
        hi[i] = max2<T>(hi[i], __shfl_xor_sync(kFull, hi[i], o));
      }
    if (gw > 1) {
      if (lane == 0) {
        sh_amax[warp] = amax;
        sh_starts[warp] = starts;
      }
      if (lane < U) {
        sh_lo[warp][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        sh_hi[warp][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
      __syncthreads();
      if (wg == 0) {
        for (int i = g * gw + 1; i < (g + 1) * gw; ++i) {
          amax = fmaxf(amax, sh_amax[i]);
          starts |= sh_starts[i];
          const uint4 l = sh_lo[i][lane % U], u = sh_hi[i][lane % U];
          const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            lo[x] = min2<T>(lo[x], lw[x]);
            hi[x] = max2<T>(hi[x], uw[x]);
          }
        }
      }
      __syncthreads();  // the shared rows are read before the next trip writes them
    }
    if (writer) {
      const int old_e = starts ? kMinBoundExp : was;
      const int e = max(bound_exp(amax), old_e);
      const int shift = min(e - old_e, 31);
      const float inv = pow2f(-e);
      uint32_t cl[2] = {0u, 0u}, ch[2] = {0u, 0u};
      const uint32_t ol[2] = {old_lo.x, old_lo.y}, oh[2] = {old_hi.x, old_hi.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 l = unpack2<T>(lo[i]), u = unpack2<T>(hi[i]);
        const float lf[2] = {l.x, l.y}, uf[2] = {u.x, u.y};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c = 2 * i + x;  // the lane's channel
          int a = bound_code(lf[x], inv, false);
          int b = bound_code(uf[x], inv, true);
          if (!starts) {  // nested floors: moving a bound to a larger step is a shift
            const int la = static_cast<int8_t>(ol[c >> 2] >> ((c & 3) * 8));
            const int lb = static_cast<int8_t>(oh[c >> 2] >> ((c & 3) * 8));
            a = min(a, la >> shift);
            b = max(b, -((-lb) >> shift));
          }
          cl[c >> 2] |= (static_cast<uint32_t>(a) & 0xffu) << ((c & 3) * 8);
          ch[c >> 2] |= (static_cast<uint32_t>(b) & 0xffu) << ((c & 3) * 8);
        }
      }
      *lo_at = make_uint2(cl[0], cl[1]);
      *hi_at = make_uint2(ch[0], ch[1]);
      if (lane == 0) p.exps[at] = e;
    }
  }
}

// ================================================================ selection
struct SelectParams {
  int32_t* sel_tables;
  int32_t* sel_lens;
  const void* q;
  const int8_t* bounds;
  const int32_t* exps;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* scores;
  int64_t pitch;
  int max_blocks;
  int num_heads;
  int num_kv_heads;
  int group;
  int block_size;
  int num_blocks;
  int max_selected;
  int num_first;
  int num_last;
};

// ---------------------------------------------------------------- scores
// With lo <= hi, max(qi lo, qi hi) is qi hi for qi >= 0 and qi lo otherwise, so
// the scores of 16 blocks for up to 8 query heads are one matrix product of
// depth 2 d: [lo | hi] (16 x 2d) times [min(qi, 0) | max(qi, 0)]^T (2d x heads).
// The codes and the whole-number queries are exact in float16, every product is
// below 2^15 and every partial sum below 2^23, so float16 MMAs with float32
// accumulators give the integer I exactly, in whatever order they add.
// (One warp per block on integer units took 189 us for selection and sparse
// decode of 4 sequences of 43 K to 115 K tokens, 8 KV heads of 128.)
//
// HBM bounds it: 2 d bytes per (block, KV head) against about 220 warp
// instructions per 4 KB.  A warp holds 16 blocks of one KV head, straight from
// global memory in the MMA's layout (lane (g, c) reads 16-byte units c, c + 4,
// ... of rows g and g + 8; a unit's four words are four k-steps); neighbouring
// warps take neighbouring heads, whose rows of a block are neighbours in memory.
// Tiles of 16 blocks per warp, behind one preparation of the queries, and warps per CTA
// (five CTAs per SM by registers).  2 x 4 beside 4 x 8 at three CTAs: selection 22.2 ->
// 20.2 us (4 sequences of 43 K to 115 K tokens, blocks of 16) and 20.3 -> 14.6 us (16 of
// 4 K to 32 K, blocks of 32); 4 x 4: 19.5 and 17.4 us.
constexpr int kScoreTiles = 2;
constexpr int kScoreWarps = 4;

// Four codes of one word as two pairs of float16: code + 128 + 1024 by bytes, minus 1152.
__device__ __forceinline__ void codes4_to_half(uint32_t w, uint32_t& a, uint32_t& b) {
  const uint32_t x = w ^ 0x80808080u;
  const uint32_t lo = __byte_perm(x, 0x64646464u, 0x4140), hi = __byte_perm(x, 0x64646464u, 0x4342);
  const uint32_t k = 0x64806480u;  // 1152
  const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&lo), *reinterpret_cast<const __half2*>(&k));
  const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&hi), *reinterpret_cast<const __half2*>(&k));
  a = *reinterpret_cast<const uint32_t*>(&ra);
  b = *reinterpret_cast<const uint32_t*>(&rb);
}

// x / 2^f as a whole number in [-255, 255]; NaN counts as 0.
__device__ __forceinline__ float whole(float x, float inv) {
  return fminf(fmaxf(rintf(x == x ? x * inv : 0.f), -255.f), 255.f);
}

template <typename T, int HEAD_DIM, int NT>
__global__ void __launch_bounds__(kScoreWarps * 32, HEAD_DIM * NT <= 128 ? 5 : 1) block_score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int UH = HEAD_DIM / 64;  // 16-byte units per lane and half (lo or hi) of a row
  constexpr int STEPS = UH * 4;      // k-steps per half
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2;
  const int c = lane & 3;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kScoreWarps + (threadIdx.x >> 5);
  const int s = blockIdx.y;
  const int kvh = static_cast<int>(wid % p.num_kv_heads);
  const int64_t b0 = wid / p.num_kv_heads * (16 * kScoreTiles);
  if (b0 >= p.max_blocks) return;
  const int ctx = __ldg(p.context_lens + s);
  const int32_t* bt = p.block_tables + static_cast<int64_t>(s) * p.max_blocks;

  // tile t's rows g and g + 8: physical blocks (-1: outside the pool), codes, exponents
  uint4 code[2][2 * UH];
  int phys[2], ex[2];
  auto table = [&](int t, int (&ph)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t b = b0 + 16 * t + 8 * r + g;  // entries past the context may be any number
      ph[r] = t < kScoreTiles && b < p.max_blocks ? __ldg(bt + b) : 0;
    }
  };
  auto load = [&](const int (&ph)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool in = static_cast<unsigned>(ph[r]) < static_cast<unsigned>(p.num_blocks);
      const int64_t at = static_cast<int64_t>(in ? ph[r] : 0) * p.num_kv_heads + kvh;
      const uint4* row = reinterpret_cast<const uint4*>(p.bounds + at * 2 * HEAD_DIM);
#pragma unroll
      for (int i = 0; i < 2 * UH; ++i) code[r][i] = __ldg(row + (i / UH) * (HEAD_DIM / 16) + (i % UH) * 4 + c);
      ex[r] = __ldg(p.exps + at);
      phys[r] = in ? 0 : -1;
    }
  };
  // the table's entries, which do not depend on the context length, before it is looked at
  int ph_next[2], ph_last[2];
  table(0, ph_next);
  table(1, ph_last);
  if (ctx <= 0 || ctx > static_cast<int64_t>(p.max_blocks) * p.block_size) return;
  const int n = (ctx + p.block_size - 1) / p.block_size;
  if (n <= p.max_selected || b0 >= n) return;  // every block is kept, or none is here
  load(ph_next);
  ph_next[0] = ph_last[0];
  ph_next[1] = ph_last[1];

  // the queries: column g of tile nt is head kvh * G + nt * 8 + g; k-step (i, w) holds
  // channels 16 (c + 4 i) + 4 w .. + 3
  uint32_t qn[STEPS][NT][2], qp[STEPS][NT][2];
  int fe[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int j = nt * 8 + g;
    const bool on = j < p.group;
    const uint4* q = reinterpret_cast<const uint4*>(
        static_cast<const T*>(p.q) + (static_cast<int64_t>(s) * p.num_heads + kvh * p.group + (on ? j : 0)) * HEAD_DIM);
    uint32_t w[STEPS][2];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < UH; ++i) {
      const uint4 u0 = __ldg(q + (c + 4 * i) * 2), u1 = __ldg(q + (c + 4 * i) * 2 + 1);
      const uint32_t e[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[4 * i + k / 2][k & 1] = on ? e[k] : 0u;
        const float2 f = unpack2<T>(w[4 * i + k / 2][k & 1]);
        amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    fe[nt] = query_exp(amax);
    const float inv = pow2f(-fe[nt]);
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 f = unpack2<T>(w[k][x]);
        const float a = whole(f.x, inv), b = whole(f.y, inv);
        qn[k][nt][x] = pack_half2(fminf(a, 0.f), fminf(b, 0.f));
        qp[k][nt][x] = pack_half2(fmaxf(a, 0.f), fmaxf(b, 0.f));
      }
  }

  float* out = p.scores + (static_cast<int64_t>(s) * p.num_kv_heads + kvh) * p.pitch;
#pragma unroll 1
  for (int t = 0; t < kScoreTiles && b0 + 16 * t < n; ++t) {
    float acc[2][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][nt][i] = acc[1][nt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * UH; ++i) {
      const uint32_t w0[4] = {code[0][i].x, code[0][i].y, code[0][i].z, code[0][i].w};
      const uint32_t w1[4] = {code[1][i].x, code[1][i].y, code[1][i].z, code[1][i].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a[4];
        codes4_to_half(w0[w], a[0], a[2]);
        codes4_to_half(w1[w], a[1], a[3]);
        const int k = (i % UH) * 4 + w;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t* q = i < UH ? qn[k][nt] : qp[k][nt];
          mma_f16_16816(acc[i & 1][nt], a, q[0], q[1]);
        }
      }
    }
    const int bad[2] = {phys[0], phys[1]}, e2[2] = {ex[0], ex[1]};
    if (t + 1 < kScoreTiles && b0 + 16 * (t + 1) < n) {
      load(ph_next);
      table(t + 2, ph_next);
    }
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // accumulators 0, 1: row g, heads 2c, 2c + 1; 2, 3: row g + 8
        const int f = __shfl_sync(kFull, fe[nt], (2 * c + j) << 2);
        if (nt * 8 + 2 * c + j < p.group) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float v = acc[0][nt][2 * r + j] + acc[1][nt][2 * r + j];
            best[r] = fmaxf(best[r], v * pow2f(min(max(f + e2[r], -100), 100)));
          }
        }
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = fmaxf(best[r], __shfl_xor_sync(kFull, best[r], 1));
      best[r] = fmaxf(best[r], __shfl_xor_sync(kFull, best[r], 2));
      const int64_t b = b0 + 16 * t + 8 * r + g;
      // a block outside the pool is selected, so that the decode meets it and gives NaN
      if (c == 0 && b < n) out[b] = bad[r] < 0 ? INFINITY : best[r];
    }
  }
}

// ---------------------------------------------------------------- the k best
// A float's bits as an unsigned number of the same order.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, KV head).  The smallest kept key is found by counting:
// the range of the keys is cut into 1024 buckets, the keys in each are counted
// (integer atomics in shared memory: the counts, and so the result, do not
// depend on their order), and the bucket that holds the last kept key becomes
// the next range, until its keys are all kept or all equal.  The range starts at
// the row's own minimum and maximum, because the scores of one row share their
// leading bits: counting by leading bits would put most keys in one bucket, and
// comparing all keys with three trial values per two bits took 16 us.  Ten bits
// a round: at most four rounds, usually two.
// Latency bounds it (5 to 6 us a launch): the scores of 8192 blocks are 32 KB.  Most of it is
// instructions of 32 warps, so keys that do not compete become 0 once, and what a thread keeps
// is a word of bits (sparse steps 30.7 -> 29.2 and 39.0 -> 37.1 us).  Ranking the last bucket's
// keys in place of further rounds, when 32 are left, took 1.2 us longer.
constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 8;  // per thread; rows of more than 8192 blocks are read again in each round
constexpr int kSelChunk = kSelThreads * kSelKeys;

// Inclusive sums over the CTA's threads in order; `sh` has one entry per warp and
// is free again after the next __syncthreads.
__device__ __forceinline__ int cta_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  const int w = sh[lane];
  const int before = __reduce_add_sync(kFull, lane < warp ? w : 0);
  *total = __reduce_add_sync(kFull, w);
  return before + inc;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int WARPS = kSelThreads / 32;
  static_assert(WARPS == 32, "one scan entry per lane");
  __shared__ int hist[kSelThreads];
  __shared__ int sh_scan[2][WARPS];
  __shared__ uint32_t sh_lo[WARPS], sh_hi[WARPS];
  __shared__ int sh_pick[3];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int kvh = blockIdx.x;
  const int s = blockIdx.y;
  const int64_t row = static_cast<int64_t>(s) * p.num_kv_heads + kvh;
  int32_t* out = p.sel_tables + row * p.max_selected;
  const int ctx = __ldg(p.context_lens + s);
  const bool bad = ctx < 0 || ctx > static_cast<int64_t>(p.max_blocks) * p.block_size;
  const int n = bad ? 0 : (ctx + p.block_size - 1) / p.block_size;
  const int32_t* bt = p.block_tables + static_cast<int64_t>(s) * p.max_blocks;
  const int k = min(n, p.max_selected);
  for (int i = k + threadIdx.x; i < p.max_selected; i += kSelThreads) out[i] = -1;
  if (threadIdx.x == 0) p.sel_lens[row] = bad ? -1 : ctx - (n - k) * p.block_size;
  if (n <= p.max_selected) {
    for (int i = threadIdx.x; i < n; i += kSelThreads) out[i] = __ldg(bt + i);
    return;
  }
  // the blocks that compete are [num_first, n - num_last) (not empty: n > max_selected)
  const int c0 = p.num_first, c1 = n - p.num_last;
  const float* sc = p.scores + row * p.pitch;
  uint32_t key[kSelKeys];
  auto load = [&](int chunk) {  // the thread's keys of chunk `chunk`, in index order
    const int i0 = chunk * kSelChunk + threadIdx.x * kSelKeys;
#pragma unroll
    for (int h = 0; h < kSelKeys / 4; ++h) {
      const int i = i0 + 4 * h;  // rows are padded to 4, so the vector stays in the row
      const float4 v = i < n ? *reinterpret_cast<const float4*>(sc + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      key[4 * h] = order_key(v.x);
      key[4 * h + 1] = order_key(v.y);
      key[4 * h + 2] = order_key(v.z);
      key[4 * h + 3] = order_key(v.w);
    }
    if (i0 < c0 || i0 + kSelKeys > c1) {  // no rival: 0, which no score gives (-infinity gives 0x7fffff)
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i)
        if (i0 + i < c0 || i0 + i >= c1) key[i] = 0u;
    }
  };
  const int chunks = (n + kSelChunk - 1) / kSelChunk;
  load(0);
  // the first chunk's table entries, on their way while the keys are counted (31.2 -> 30.7 and
  // 38.9 -> 38.0 us for the sparse steps of the two batches above)
  int ids[kSelKeys];
#pragma unroll
  for (int i = 0; i < kSelKeys; ++i) {
    const int x = threadIdx.x * kSelKeys + i;
    ids[i] = x < n ? __ldg(bt + x) : 0;
  }
  uint32_t lo = 0xffffffffu, hi = 0u;  // lo: less 1, so that 0 counts as the largest
  for (int ch = 0; ch < chunks; ++ch) {
    if (ch > 0) load(ch);
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      lo = min(lo, key[i] - 1u);
      hi = max(hi, key[i]);
    }
  }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
  if (lane == 0) {
    sh_lo[warp] = lo;
    sh_hi[warp] = hi;
  }
  hist[threadIdx.x] = 0;
  __syncthreads();
  lo = __reduce_min_sync(kFull, sh_lo[lane]) + 1u;
  hi = __reduce_max_sync(kFull, sh_hi[lane]);
  int need = k - p.num_first - p.num_last;  // competing blocks still to be kept among the keys in [lo, hi]
  int ties = n;                             // of the keys equal to lo in the end, how many are kept
  for (int round = 0; need > 0; ++round) {
    const int shift = max(0, 32 - __clz(hi - lo) - 10);
    for (int ch = 0; ch < chunks; ++ch) {
      if (chunks > 1) load(ch);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i)
        if (key[i] - lo <= hi - lo) atomicAdd(&hist[(key[i] - lo) >> shift], 1);  // (0 is past hi: lo >= 1)
    }
    __syncthreads();
    const int b = kSelThreads - 1 - threadIdx.x;  // the threads walk the buckets from the top
    const int count = hist[b];
    int total;
    const int upto = cta_scan(count, sh_scan[round & 1], &total);  // (its barrier: the buckets are read)
    hist[b] = 0;
    if (upto >= need && upto - count < need) {
      sh_pick[0] = b;
      sh_pick[1] = need - (upto - count);
      sh_pick[2] = count;
    }
    __syncthreads();
    need = sh_pick[1];
    lo += static_cast<uint32_t>(sh_pick[0]) << shift;
    hi = lo + ((1u << shift) - 1u);
    if (sh_pick[2] == need) break;  // every key from lo on is kept
    if (shift == 0) {               // equal keys: the first `need` of them
      ties = need;
      break;
    }
  }
  if (k == p.num_first + p.num_last) lo = 0xffffffffu;  // the forced blocks fill the row
  // kept in index order: forced blocks, keys above lo, and of those equal to lo the first `ties`
  int done = 0, tied = 0;
  for (int ch = 0; ch < chunks; ++ch) {
    if (chunks > 1) load(ch);
    const int i0 = ch * kSelChunk + threadIdx.x * kSelKeys;
    uint32_t kept = 0u, same = 0u;  // a bit per key
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      kept |= key[i] > lo ? 1u << i : 0u;
      same |= key[i] == lo ? 1u << i : 0u;
    }
    if (i0 < c0 || i0 + kSelKeys > c1) {
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i)
        if (i0 + i < n && (i0 + i < c0 || i0 + i >= c1)) kept |= 1u << i;
    }
    // prefix sums of (equal, others kept), 16 bits each: a chunk has 8192 keys
    const int v = __popc(same) | (__popc(kept) << 16);
    int total;
    __syncthreads();  // the previous use of the scan entries is over
    const int before = cta_scan(v, sh_scan[0], &total) - v;
    const int at = done + (before >> 16) + min(before & 0xffff, max(ties - tied, 0));
    for (int room = ties - tied - (before & 0xffff); same != 0u && room > 0; --room) {
      kept |= same & (0u - same);
      same &= same - 1u;
    }
    if (kept != 0u) {
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i)
        if (kept >> i & 1u) out[at + __popc(kept & ((1u << i) - 1u))] = ch == 0 ? ids[i] : __ldg(bt + i0 + i);
    }
    done += (total >> 16) + min(total & 0xffff, max(ties - tied, 0));
    tied += total & 0xffff;
  }
}

cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Tokens per CTA: enough CTAs to fill the GPU (1024 of them: 152 SMs, several
// each) before a CTA takes more than one token per group of warps, and at most
// kMaxStretch, which in a prompt holds one run per group.
RunParams run_params(const int64_t* slot_mapping, int num_tokens, int num_blocks, int block_size, int num_kv_heads,
                     int parts, int* threads) {
  RunParams r;
  r.slot_mapping = slot_mapping;
  r.num_slots = num_blocks * block_size;
  r.num_tokens = num_tokens;
  r.num_kv_heads = num_kv_heads;
  r.block_size = block_size;
  r.log2_b = __builtin_ctz(static_cast<unsigned>(block_size));
  const int gw = block_size / kRunRows;
  const int warps = gw > 8 ? gw : 8;
  *threads = warps * 32;
  const int64_t per_cta = static_cast<int64_t>(num_tokens) * num_kv_heads * parts / 1024;
  r.stretch = warps / gw;
  while (r.stretch < kMaxStretch && r.stretch < per_cta) r.stretch *= 2;
  return r;
}

template <typename P, typename K>
cudaError_t launch_runs(K kernel, const P& p, int num_kv_heads, int parts, int threads, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(dim3((p.r.num_tokens + p.r.stretch - 1) / p.r.stretch, num_kv_heads, parts),
                                            dim3(threads), stream, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int THREADS>
cudaError_t block_write_typed(const BlockWriteArgs& a, const BlockWriteParams& p, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_runs(block_write_kernel<T, 64, THREADS>, p, a.num_kv_heads, 2, THREADS, stream);
    case 128: return launch_runs(block_write_kernel<T, 128, THREADS>, p, a.num_kv_heads, 2, THREADS, stream);
    case 256: return launch_runs(block_write_kernel<T, 256, THREADS>, p, a.num_kv_heads, 2, THREADS, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <typename T, int THREADS>
cudaError_t key_bounds_typed(const KeyBoundsArgs& a, const KeyBoundsParams& p, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_runs(key_bounds_kernel<T, 64, THREADS>, p, a.num_kv_heads, 1, THREADS, stream);
    case 128: return launch_runs(key_bounds_kernel<T, 128, THREADS>, p, a.num_kv_heads, 1, THREADS, stream);
    case 256: return launch_runs(key_bounds_kernel<T, 256, THREADS>, p, a.num_kv_heads, 1, THREADS, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <typename T, int HEAD_DIM, int NT>
cudaError_t block_score_t(const SelectArgs& a, const SelectParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const int64_t stretches = (a.max_blocks_per_seq + 16 * kScoreTiles - 1) / (16 * kScoreTiles);
  const int64_t ctas = (stretches * a.num_kv_heads + kScoreWarps - 1) / kScoreWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(static_cast<unsigned>(ctas), a.num_seqs), dim3(kScoreWarps * 32), stream, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, block_score_kernel<T, HEAD_DIM, NT>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t block_score_typed(const SelectArgs& a, const SelectParams& p, cudaStream_t stream) {
  const bool two = p.group > 8;
  switch (a.head_dim) {
    case 64: return two ? block_score_t<T, 64, 2>(a, p, stream) : block_score_t<T, 64, 1>(a, p, stream);
    case 128: return two ? block_score_t<T, 128, 2>(a, p, stream) : block_score_t<T, 128, 1>(a, p, stream);
    case 256: return two ? cudaErrorInvalidValue : block_score_t<T, 256, 1>(a, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_block_write(const BlockWriteArgs& a, cudaStream_t stream) {
  BlockWriteParams p;
  int threads;
  p.r = run_params(a.slot_mapping, a.num_tokens, a.num_blocks, a.block_size, a.num_kv_heads, 2, &threads);
  p.key = static_cast<const uint4*>(a.key);
  p.value = static_cast<const uint4*>(a.value);
  p.k_cache = static_cast<uint2*>(a.k_cache);
  p.v_cache = static_cast<uint2*>(a.v_cache);
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  if (threads == 512)
    return a.dtype == PA_BF16 ? block_write_typed<__nv_bfloat16, 512>(a, p, stream)
                              : block_write_typed<__half, 512>(a, p, stream);
  return a.dtype == PA_BF16 ? block_write_typed<__nv_bfloat16, 256>(a, p, stream)
                            : block_write_typed<__half, 256>(a, p, stream);
}

cudaError_t launch_key_bounds(const KeyBoundsArgs& a, cudaStream_t stream) {
  KeyBoundsParams p;
  int threads;
  p.r = run_params(a.slot_mapping, a.num_tokens, a.num_blocks, a.block_size, a.num_kv_heads, 1, &threads);
  p.key = static_cast<const uint4*>(a.key);
  p.bounds = a.key_bounds;
  p.exps = a.bound_exps;
  if (threads == 512)
    return a.dtype == PA_BF16 ? key_bounds_typed<__nv_bfloat16, 512>(a, p, stream)
                              : key_bounds_typed<__half, 512>(a, p, stream);
  return a.dtype == PA_BF16 ? key_bounds_typed<__nv_bfloat16, 256>(a, p, stream)
                            : key_bounds_typed<__half, 256>(a, p, stream);
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t stream) {
  SelectParams p;
  p.sel_tables = a.sel_tables;
  p.sel_lens = a.sel_lens;
  p.q = a.q;
  p.bounds = a.key_bounds;
  p.exps = a.bound_exps;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.scores = a.scores;
  p.pitch = select_pitch(a.max_blocks_per_seq);
  p.max_blocks = a.max_blocks_per_seq;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_heads / a.num_kv_heads;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.max_selected = a.max_selected;
  p.num_first = a.num_first;
  p.num_last = a.num_last;
  cudaError_t e = cudaSuccess;
  if (a.max_blocks_per_seq > a.max_selected) {  // otherwise every block is kept
    e = a.dtype == PA_BF16 ? block_score_typed<__nv_bfloat16>(a, p, stream) : block_score_typed<__half>(a, p, stream);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(a.num_kv_heads, a.num_seqs), dim3(kSelThreads), stream, &attr);
  e = cudaLaunchKernelEx(&cfg, select_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
