// pa_packed_prefill.cu -- attention over packed prompts with __half and __nv_bfloat16 rows.
#include "pa_packed_prefill.cuh"
#include "pagedattn.h"

namespace pa {

cudaError_t launch_packed_prefill(const PackedPrefillArgs& a, cudaStream_t stream) {
  if (a.dtype == PA_BF16)
    return a.head_dim == 64 ? launch_packed_prefill_t<__nv_bfloat16, 64>(a, stream)
                            : launch_packed_prefill_t<__nv_bfloat16, 128>(a, stream);
  return a.head_dim == 64 ? launch_packed_prefill_t<__half, 64>(a, stream) : launch_packed_prefill_t<__half, 128>(a, stream);
}

}  // namespace pa
