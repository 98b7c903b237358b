// pa_block_cache.cu -- side data kept per (block, KV head): the cache write
// into E4M3 pools with one scale per (block, KV head), the key bounds of the
// block selection, and the selection itself.
//
//  block_write_kernel   one warp per (run of new tokens in a block, KV head, K or V)
//  key_bounds_kernel    one warp per (run of new tokens in a block, KV head)
//  block_score_kernel   one warp per (block of a sequence, KV head)
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

// The block of a slot, -1 for padding and slots outside the pool.
__device__ __forceinline__ int64_t slot_block(int64_t slot, int64_t num_slots, int log2_b) {
  return slot < 0 || slot >= num_slots ? -1 : slot >> log2_b;
}

// The run of token t: [t, returned end), the tokens from t on that go to t's
// block; empty when t continues the run of t - 1 or goes nowhere.
__device__ __forceinline__ int run_end(const int64_t* sm, int t, int num_tokens, int64_t num_slots, int log2_b,
                                       int64_t* blk) {
  *blk = slot_block(__ldg(sm + t), num_slots, log2_b);
  if (*blk < 0) return t;
  if (t > 0 && slot_block(__ldg(sm + t - 1), num_slots, log2_b) == *blk) return t;
  int e = t + 1;
  while (e < num_tokens && slot_block(__ldg(sm + e), num_slots, log2_b) == *blk) ++e;
  return e;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}

struct BlockWriteParams {
  const uint4* key;  // 8 elements per vector
  const uint4* value;
  uint2* k_cache;  // 8 codes per vector
  uint2* v_cache;
  float* k_scales;
  float* v_scales;
  const int64_t* slot_mapping;
  int64_t num_slots;
  int num_tokens;
  int num_kv_heads;
  int block_size;
  int log2_b;
  int row_vecs;  // head_dim / 8
};

template <typename T>
__global__ void __launch_bounds__(64) block_write_kernel(const __grid_constant__ BlockWriteParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int t = blockIdx.x;
  const int h = blockIdx.y;
  const bool is_v = threadIdx.x >= 32;
  const int lane = threadIdx.x & 31;
  int64_t blk;
  const int end = run_end(p.slot_mapping, t, p.num_tokens, p.num_slots, p.log2_b, &blk);
  if (end == t) return;
  const uint4* src = is_v ? p.value : p.key;
  uint2* pool = (is_v ? p.v_cache : p.k_cache) + blk * p.block_size * p.num_kv_heads * p.row_vecs;
  float* scale = (is_v ? p.v_scales : p.k_scales) + blk * p.num_kv_heads + h;
  const int rv = p.row_vecs;

  float amax = 0.f;
  bool starts = false;
  for (int i = t; i < end; ++i) {
    starts |= (__ldg(p.slot_mapping + i) & (p.block_size - 1)) == 0;
    const uint4* row = src + (static_cast<int64_t>(i) * p.num_kv_heads + h) * rv;
    for (int x = lane; x < rv; x += 32) {
      const uint4 v = __ldg(row + x);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<T>(w[j]);
        amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
    }
  }
  amax = warp_max(amax);
  const float need = pow2f(scale_exp(amax));
  float old = starts ? 0.f : *scale;
  if (!(old > 0.f && old <= kFloatMax)) old = 0.f;  // no scale to keep
  const float s = fmaxf(old, need);
  if (old > 0.f && s > old) {  // the block's other codes move to the new scale
    const float ratio = __fdiv_rn(old, s);
    for (int o = 0; o < p.block_size; ++o) {
      uint2* row = pool + (static_cast<int64_t>(o) * p.num_kv_heads + h) * rv;
      for (int x = lane; x < rv; x += 32) {
        const uint2 c = row[x];
        const uint32_t in[2] = {c.x, c.y};
        uint32_t out[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t lo, hi;
          e4m3x4_to_half2x2(in[j], lo, hi);
          const float2 a = unpack_half2(lo), b = unpack_half2(hi);
          out[j] = float_to_e4m3_sat(a.x * ratio) | (float_to_e4m3_sat(a.y * ratio) << 8) |
                   (float_to_e4m3_sat(b.x * ratio) << 16) | (static_cast<uint32_t>(float_to_e4m3_sat(b.y * ratio)) << 24);
        }
        row[x] = make_uint2(out[0], out[1]);
      }
    }
  }
  __syncwarp();  // the moved codes before the new ones, which may share their rows
  for (int i = t; i < end; ++i) {
    const int o = static_cast<int>(__ldg(p.slot_mapping + i) & (p.block_size - 1));
    const uint4* row = src + (static_cast<int64_t>(i) * p.num_kv_heads + h) * rv;
    uint2* dst = pool + (static_cast<int64_t>(o) * p.num_kv_heads + h) * rv;
    for (int x = lane; x < rv; x += 32) {
      const uint4 v = __ldg(row + x);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t c[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<T>(w[j]);
        const uint32_t c0 = float_to_e4m3_sat(__fdiv_rn(f.x, s));
        const uint32_t c1 = float_to_e4m3_sat(__fdiv_rn(f.y, s));
        c[j >> 1] |= (c0 | (c1 << 8)) << ((j & 1) * 16);
      }
      dst[x] = make_uint2(c[0], c[1]);
    }
  }
  if (lane == 0) *scale = s;
}

struct KeyBoundsParams {
  const void* key;
  int8_t* bounds;
  int32_t* exps;
  const int64_t* slot_mapping;
  int64_t num_slots;
  int num_tokens;
  int num_kv_heads;
  int block_size;
  int log2_b;
};

template <typename T>
__device__ __forceinline__ float elem_to_float(T x) {
  if constexpr (std::is_same<T, __half>::value) {
    return __half2float(x);
  } else {
    return __bfloat162float(x);
  }
}

// lo (up = false): floor(v / 2^e); hi: ceil.  Codes stay in [-127, 127].
__device__ __forceinline__ int bound_code(float v, float inv, bool up) {
  const float x = v * inv;
  const float r = up ? ceilf(x) : floorf(x);
  return static_cast<int>(fminf(fmaxf(r, -127.f), 127.f));
}

template <typename T, int HEAD_DIM>
__global__ void __launch_bounds__(32) key_bounds_kernel(const __grid_constant__ KeyBoundsParams p) {
  constexpr int N = HEAD_DIM / 32;
  grid_dependency_wait();
  allow_dependent_launch();
  const int t = blockIdx.x;
  const int h = blockIdx.y;
  const int lane = threadIdx.x;
  int64_t blk;
  const int end = run_end(p.slot_mapping, t, p.num_tokens, p.num_slots, p.log2_b, &blk);
  if (end == t) return;
  float lo[N], hi[N], amax = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  bool starts = false;
  for (int i = t; i < end; ++i) {
    starts |= (__ldg(p.slot_mapping + i) & (p.block_size - 1)) == 0;
    const T* row = static_cast<const T*>(p.key) + (static_cast<int64_t>(i) * p.num_kv_heads + h) * HEAD_DIM;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float f = elem_to_float(row[lane + 32 * j]);
      amax = fmaxf(amax, finite_abs(f));
      lo[j] = f == f ? fminf(lo[j], f) : -INFINITY;  // NaN: the widest bound
      hi[j] = f == f ? fmaxf(hi[j], f) : INFINITY;
    }
  }
  amax = warp_max(amax);
  int8_t* b = p.bounds + (blk * p.num_kv_heads + h) * 2 * HEAD_DIM;
  int32_t* ex = p.exps + blk * p.num_kv_heads + h;
  const int old_e = starts ? kMinBoundExp : *ex;
  const int e = max(bound_exp(amax), old_e);
  const int shift = min(e - old_e, 31);
  const float inv = pow2f(-e);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int c = lane + 32 * j;
    int l = bound_code(lo[j], inv, false);
    int u = bound_code(hi[j], inv, true);
    if (!starts) {  // nested floors: moving a bound to a larger step is a shift
      l = min(l, static_cast<int>(b[c]) >> shift);
      u = max(u, -((-static_cast<int>(b[HEAD_DIM + c])) >> shift));
    }
    b[c] = static_cast<int8_t>(l);
    b[HEAD_DIM + c] = static_cast<int8_t>(u);
  }
  __syncwarp();
  if (lane == 0) *ex = e;
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

template <typename T, int HEAD_DIM>
__global__ void __launch_bounds__(32) block_score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int N = HEAD_DIM / 32;
  grid_dependency_wait();
  const int b = blockIdx.x;
  const int kvh = blockIdx.y;
  const int s = blockIdx.z;
  const int lane = threadIdx.x;
  const int ctx = __ldg(p.context_lens + s);
  if (ctx <= 0 || static_cast<int64_t>(b) * p.block_size >= ctx) return;
  const int phys = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + b);
  float best = -INFINITY;
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
    best = INFINITY;  // selected, so that the decode meets it and gives NaN
  } else {
    const int8_t* bd = p.bounds + (static_cast<int64_t>(phys) * p.num_kv_heads + kvh) * 2 * HEAD_DIM;
    const int e = __ldg(p.exps + static_cast<int64_t>(phys) * p.num_kv_heads + kvh);
    for (int g = 0; g < p.group; ++g) {
      const T* q = static_cast<const T*>(p.q) + (static_cast<int64_t>(s) * p.num_heads + kvh * p.group + g) * HEAD_DIM;
      float f[N], amax = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        f[j] = elem_to_float(q[lane + 32 * j]);
        amax = fmaxf(amax, finite_abs(f[j]));
      }
      const int fe = query_exp(warp_max(amax));
      int sum = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float x = rintf(f[j] * pow2f(-fe));
        const int qi = x == x ? static_cast<int>(fminf(fmaxf(x, -255.f), 255.f)) : 0;
        const int c = lane + 32 * j;
        sum += max(qi * bd[c], qi * bd[HEAD_DIM + c]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
      const int x = min(max(fe + e, -100), 100);
      best = fmaxf(best, static_cast<float>(sum) * pow2f(x));
    }
  }
  if (lane == 0) p.scores[(static_cast<int64_t>(s) * p.num_kv_heads + kvh) * p.pitch + b] = best;
}

// A float's bits as an unsigned number of the same order.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 256;

__device__ __forceinline__ int block_sum(int v, int* sh) {
  __syncthreads();
  const int w = __reduce_add_sync(kFull, v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = w;
  __syncthreads();
  int t = 0;
  for (int i = 0; i < kSelThreads / 32; ++i) t += sh[i];
  return t;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ int sh[kSelThreads / 32];
  grid_dependency_wait();
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
  const float* sc = p.scores + row * p.pitch;
  auto key = [&](int i) -> uint32_t {
    if (i < p.num_first || i >= n - p.num_last) return 0xffffffffu;
    return order_key(sc[i]);
  };
  // the k-th largest key, bit by bit
  uint32_t kth = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = kth | (1u << bit);
    int c = 0;
    for (int i = threadIdx.x; i < n; i += kSelThreads) c += key(i) >= trial;
    if (block_sum(c, sh) >= k) kth = trial;
  }
  int above = 0;
  for (int i = threadIdx.x; i < n; i += kSelThreads) above += key(i) > kth;
  above = block_sum(above, sh);
  const int ties = k - above;  // of the keys equal to kth, the first ones
  int done = 0, tied = 0;
  for (int base = 0; base < n; base += kSelThreads) {
    const int i = base + threadIdx.x;
    const uint32_t x = i < n ? key(i) : 0u;
    const int gt = i < n && x > kth;
    const int eq = i < n && x == kth;
    const unsigned meq = __ballot_sync(kFull, eq);
    const unsigned below = (1u << (threadIdx.x & 31)) - 1u;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = __popc(meq);
    __syncthreads();
    int beq = tied, all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < (threadIdx.x >> 5)) beq += sh[w];
      all += sh[w];
    }
    const int take = gt || (eq && beq + __popc(meq & below) < ties);
    tied += all;
    const unsigned mt = __ballot_sync(kFull, take);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = __popc(mt);
    __syncthreads();
    int at = done;
    all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < (threadIdx.x >> 5)) at += sh[w];
      all += sh[w];
    }
    if (take) out[at + __popc(mt & below)] = __ldg(bt + i);
    done += all;
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

template <typename T>
cudaError_t key_bounds_typed(const KeyBoundsArgs& a, const KeyBoundsParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(a.num_tokens, a.num_kv_heads), dim3(32), stream, &attr);
  switch (a.head_dim) {
    case 64: return cudaLaunchKernelEx(&cfg, key_bounds_kernel<T, 64>, p);
    case 128: return cudaLaunchKernelEx(&cfg, key_bounds_kernel<T, 128>, p);
    case 256: return cudaLaunchKernelEx(&cfg, key_bounds_kernel<T, 256>, p);
    default: return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t block_score_typed(const SelectArgs& a, const SelectParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(a.max_blocks_per_seq, a.num_kv_heads, a.num_seqs), dim3(32), stream, &attr);
  switch (a.head_dim) {
    case 64: return cudaLaunchKernelEx(&cfg, block_score_kernel<T, 64>, p);
    case 128: return cudaLaunchKernelEx(&cfg, block_score_kernel<T, 128>, p);
    case 256: return cudaLaunchKernelEx(&cfg, block_score_kernel<T, 256>, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_block_write(const BlockWriteArgs& a, cudaStream_t stream) {
  BlockWriteParams p;
  p.key = static_cast<const uint4*>(a.key);
  p.value = static_cast<const uint4*>(a.value);
  p.k_cache = static_cast<uint2*>(a.k_cache);
  p.v_cache = static_cast<uint2*>(a.v_cache);
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.slot_mapping = a.slot_mapping;
  p.num_slots = static_cast<int64_t>(a.num_blocks) * a.block_size;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  p.block_size = a.block_size;
  p.log2_b = __builtin_ctz(static_cast<unsigned>(a.block_size));
  p.row_vecs = a.head_dim / 8;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(a.num_tokens, a.num_kv_heads), dim3(64), stream, &attr);
  const cudaError_t e = a.dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, block_write_kernel<__nv_bfloat16>, p)
                                           : cudaLaunchKernelEx(&cfg, block_write_kernel<__half>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_key_bounds(const KeyBoundsArgs& a, cudaStream_t stream) {
  KeyBoundsParams p;
  p.key = a.key;
  p.bounds = a.key_bounds;
  p.exps = a.bound_exps;
  p.slot_mapping = a.slot_mapping;
  p.num_slots = static_cast<int64_t>(a.num_blocks) * a.block_size;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  p.block_size = a.block_size;
  p.log2_b = __builtin_ctz(static_cast<unsigned>(a.block_size));
  const cudaError_t e = a.dtype == PA_BF16 ? key_bounds_typed<__nv_bfloat16>(a, p, stream)
                                           : key_bounds_typed<__half>(a, p, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
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
