// pa_packed_prefill.cu -- causal attention over whole prompts in packed rows, which
// writes their keys and values into the pools too.
//
//  packed_prefill_kernel  one warp per (token, query head): the keys of its sequence
//                         up to its own, one after the other, with the running
//                         maximum and sum of the softmax in float32
#include <cuda_runtime.h>

#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

template <typename T, int HEAD_DIM>
__global__ void __launch_bounds__(256) packed_prefill_kernel(const __grid_constant__ PackedPrefillArgs p) {
  constexpr int PAIRS = HEAD_DIM / 64;  // 32-bit pairs of elements per lane
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= p.num_rows) return;
  int lo = 0, hi = p.num_seqs;  // the last sequence that starts at or before t
  while (lo < hi - 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.query_start_loc + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int start = max(0, __ldg(p.query_start_loc + lo));
  if (t < start || t >= __ldg(p.query_start_loc + lo + 1) || t - start >= p.max_query_len) return;
  const int group = p.num_heads / p.num_kv_heads;
  const int kvh = h / group;
  auto row = [&](const void* base, int64_t stride, int r, int head) {
    return reinterpret_cast<const uint32_t*>(static_cast<const T*>(base) + r * stride + head * HEAD_DIM) + lane;
  };
  if (p.slot_mapping && h == kvh * group) {
    const int64_t slot = __ldg(p.slot_mapping + t);
    if (slot >= 0 && slot < p.num_slots) {
      const int64_t at = (slot * p.num_kv_heads + kvh) * (HEAD_DIM / 2) + lane;
      for (int i = 0; i < PAIRS; ++i) {
        static_cast<uint32_t*>(p.k_cache)[at + 32 * i] = row(p.key, p.k_stride, t, kvh)[32 * i];
        static_cast<uint32_t*>(p.v_cache)[at + 32 * i] = row(p.value, p.v_stride, t, kvh)[32 * i];
      }
    }
  }
  float2 q[PAIRS], o[PAIRS];
  for (int i = 0; i < PAIRS; ++i) {
    q[i] = unpack2<T>(row(p.q, p.q_stride, t, h)[32 * i]);
    o[i] = make_float2(0.f, 0.f);
  }
  const float scale_log2 = p.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f;
  for (int u = start; u <= t; ++u) {
    float s = 0.f;
    for (int i = 0; i < PAIRS; ++i) {
      const float2 k = unpack2<T>(row(p.key, p.k_stride, u, kvh)[32 * i]);
      s = fmaf(q[i].x, k.x, fmaf(q[i].y, k.y, s));
    }
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= scale_log2;
    const float top = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : ex2(m - top);
    const float w = ex2(s - top);
    m = top;
    l = l * f + w;
    for (int i = 0; i < PAIRS; ++i) {
      const float2 v = unpack2<T>(row(p.value, p.v_stride, u, kvh)[32 * i]);
      o[i] = make_float2(fmaf(w, v.x, o[i].x * f), fmaf(w, v.y, o[i].y * f));
    }
  }
  uint32_t* out = static_cast<uint32_t*>(p.out) + (static_cast<int64_t>(t) * p.num_heads + h) * (HEAD_DIM / 2) + lane;
  for (int i = 0; i < PAIRS; ++i) out[32 * i] = pack2<T>(o[i].x / l, o[i].y / l);
}

template <typename T, int HEAD_DIM>
cudaError_t launch_t(const PackedPrefillArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.num_rows + 7) / 8, a.num_heads);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, packed_prefill_kernel<T, HEAD_DIM>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_prefill(const PackedPrefillArgs& a, cudaStream_t stream) {
  if (a.dtype == PA_BF16)
    return a.head_dim == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
  return a.head_dim == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
}

}  // namespace pa
