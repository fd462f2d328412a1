// Decode attention over the 4-bit cache [num_blocks, H, B, 5 D / 8].
#include "gather_kernel.cuh"
#include "pa.h"

namespace pa {

cudaError_t launch_decode_q4(int dtype, int D, const GatherArgs& a, int grid, cudaStream_t stream) {
  (void)grid;
  if (dtype == PA_F16)
    return D == 128 ? gk::launch_simple<__half, true, 128>(a, stream) : gk::launch_simple<__half, true, 64>(a, stream);
  return D == 128 ? gk::launch_simple<__nv_bfloat16, true, 128>(a, stream)
                  : gk::launch_simple<__nv_bfloat16, true, 64>(a, stream);
}

}  // namespace pa
