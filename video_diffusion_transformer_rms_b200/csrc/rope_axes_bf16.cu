// bf16 instantiations of the multi-axis rotary kernels.
#include "rope_axes.cuh"

namespace sol {

cudaError_t launch_rope_axes_bf16(RopeArgs &a, RopeMode mode, bool half, cudaStream_t stream,
                                  int *ctas) {
  return half ? dispatch_mode<__nv_bfloat16, true>(a, mode, stream, ctas)
              : dispatch_mode<__nv_bfloat16, false>(a, mode, stream, ctas);
}

}  // namespace sol
