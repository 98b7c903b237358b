// pa_block_decode_bf16.cu -- decode over block-scaled E4M3 pools with __nv_bfloat16
// queries (split-K partials go through the float reduce of pa_decode_bf16.cu).
#include "pa_block_decode.cuh"

namespace pa {

cudaError_t launch_block_decode_bf16(const BlockDecodeArgs& a, cudaStream_t stream) {
  return launch_block_decode_typed<__nv_bfloat16, E4M3, false>(a, stream);
}

}  // namespace pa
