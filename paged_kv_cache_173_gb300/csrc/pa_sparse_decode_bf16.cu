// pa_sparse_decode_bf16.cu -- decode over per-KV-head block tables with __nv_bfloat16
// queries: 16-bit pools of the query type, or block-scaled E4M3 pools.
#include "pa_block_decode.cuh"
#include "pagedattn.h"

namespace pa {

cudaError_t launch_sparse_decode_bf16(const BlockDecodeArgs& a, cudaStream_t stream) {
  return a.kv_dtype == PA_FP8_E4M3 ? launch_block_decode_typed<__nv_bfloat16, E4M3, true>(a, stream)
                                   : launch_block_decode_typed<__nv_bfloat16, __nv_bfloat16, true>(a, stream);
}

}  // namespace pa
