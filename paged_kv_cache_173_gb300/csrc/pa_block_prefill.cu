// pa_block_prefill.cu -- prefill over block-scaled E4M3 pools with __half and
// __nv_bfloat16 queries.
#include "pa_block_prefill.cuh"
#include "pagedattn.h"

namespace pa {

cudaError_t launch_block_prefill(const BlockPrefillArgs& b, cudaStream_t stream) {
  if (b.a.dtype == PA_BF16)
    return b.a.head_dim == 64 ? launch_block_prefill_t<__nv_bfloat16, 64>(b, stream)
                              : launch_block_prefill_t<__nv_bfloat16, 128>(b, stream);
  return b.a.head_dim == 64 ? launch_block_prefill_t<__half, 64>(b, stream)
                            : launch_block_prefill_t<__half, 128>(b, stream);
}

}  // namespace pa
