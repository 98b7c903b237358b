// pa_block_prefill.cu -- prefill over block-scaled E4M3 pools.
//
//  block_prefill_row_kernel  one warp per (query row, head): the online softmax
//                            of "vLLM PagedAttention source walk-through",
//                            section 3.4, key by key
#include <cuda_runtime.h>

#include "pa_block.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

struct BlockPrefillParams {
  void* out;
  const void* q;
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
  int block_size;
  int num_blocks;
  float scale_log2;
};

__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
  uint32_t lo, hi;
  e4m3x4_to_half2x2(c, lo, hi);
  return unpack_half2(lo).x;
}

template <typename T, int HEAD_DIM>
__global__ void __launch_bounds__(32) block_prefill_row_kernel(const __grid_constant__ BlockPrefillParams p) {
  constexpr int N = HEAD_DIM / 32;
  const int i = blockIdx.x;
  const int h = blockIdx.y;
  const int s = blockIdx.z;
  const int lane = threadIdx.x;
  const int q0 = __ldg(p.query_start_loc + s);
  const int qlen = __ldg(p.query_start_loc + s + 1) - q0;
  if (i >= qlen) return;
  const int ctx = __ldg(p.context_lens + s);
  const bool ctx_bad = ctx < qlen || ctx > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  const int64_t row = (static_cast<int64_t>(q0) + i) * p.num_heads + h;
  const int kvh = h / (p.num_heads / p.num_kv_heads);
  float q[N], o[N], m = -INFINITY, l = 0.f;
  bool bad = ctx_bad;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    T x = static_cast<const T*>(p.q)[row * HEAD_DIM + lane + 32 * j];
    if constexpr (std::is_same<T, __half>::value) {
      q[j] = __half2float(x);
    } else {
      q[j] = __bfloat162float(x);
    }
    o[j] = 0.f;
  }
  const int last = ctx_bad ? -1 : ctx - qlen + i;
  for (int pos = 0; pos <= last; ++pos) {
    const int phys = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + pos / p.block_size);
    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
      bad = true;
      break;
    }
    const int64_t side = static_cast<int64_t>(phys) * p.num_kv_heads + kvh;
    const float ks = __ldg(p.k_scales + side), vs = __ldg(p.v_scales + side);
    bad |= !(ks >= 0.f && ks <= kFloatMax && vs >= 0.f && vs <= kFloatMax);
    const int64_t at = ((static_cast<int64_t>(phys) * p.block_size + pos % p.block_size) * p.num_kv_heads + kvh) * HEAD_DIM;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) dot += q[j] * e4m3_to_float(p.k_cache[at + lane + 32 * j]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float x = dot * (p.scale_log2 * ks);
    const float mn = fmaxf(m, x);
    const float f = ex2(m - mn), w = ex2(x - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = o[j] * f + w * vs * e4m3_to_float(p.v_cache[at + lane + 32 * j]);
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    static_cast<T*>(p.out)[row * HEAD_DIM + lane + 32 * j] = to_elem<T>(bad ? NAN : o[j] / l);
}

}  // namespace

cudaError_t launch_block_prefill(const BlockPrefillArgs& b, cudaStream_t stream) {
  const PrefillArgs& a = b.a;
  BlockPrefillParams p{a.out, a.q, static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache),
                       b.k_scales, b.v_scales, a.block_tables, a.context_lens, a.query_start_loc,
                       a.max_blocks_per_seq, a.num_heads, a.num_kv_heads, a.block_size, a.num_blocks,
                       a.scale * 1.4426950408889634f};
  const dim3 grid(a.max_query_len, a.num_heads, a.num_seqs);
  if (a.dtype == PA_BF16) {
    if (a.head_dim == 64)
      block_prefill_row_kernel<__nv_bfloat16, 64><<<grid, 32, 0, stream>>>(p);
    else
      block_prefill_row_kernel<__nv_bfloat16, 128><<<grid, 32, 0, stream>>>(p);
  } else {
    if (a.head_dim == 64)
      block_prefill_row_kernel<__half, 64><<<grid, 32, 0, stream>>>(p);
    else
      block_prefill_row_kernel<__half, 128><<<grid, 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace pa
