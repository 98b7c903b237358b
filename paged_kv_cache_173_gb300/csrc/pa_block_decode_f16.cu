// pa_block_decode_f16.cu -- decode over block-scaled E4M3 pools with __half
// queries (split-K partials go through the float reduce of pa_decode_f16.cu).
#include "pa_block_decode.cuh"

namespace pa {

cudaError_t launch_block_decode_f16(const BlockDecodeArgs& a, cudaStream_t stream) {
  return launch_block_decode_typed<__half, E4M3, false>(a, stream);
}

}  // namespace pa
