// pa_sparse_decode_f16.cu -- decode over per-KV-head block tables with __half
// queries: 16-bit pools of the query type, or block-scaled E4M3 pools.
#include "pa_block_decode.cuh"
#include "pagedattn.h"

namespace pa {

cudaError_t launch_sparse_decode_f16(const BlockDecodeArgs& a, cudaStream_t stream) {
  return a.kv_dtype == PA_FP8_E4M3 ? launch_block_decode_typed<__half, E4M3, true>(a, stream)
                                   : launch_block_decode_typed<__half, __half, true>(a, stream);
}

}  // namespace pa
