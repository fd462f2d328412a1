// Decode attention over the listed frames of a 16-bit cache [num_blocks, B, H, D].
#include "gather_kernel.cuh"
#include "pa.h"

namespace pa {

cudaError_t launch_decode_selected(int dtype, int D, const GatherArgs& a, const CUtensorMap& tk,
                                   const CUtensorMap& tv, int grid, cudaStream_t stream) {
  (void)tk;
  (void)tv;
  (void)grid;
  if (dtype == PA_F16)
    return D == 128 ? gk::launch_simple<__half, false, 128>(a, stream) : gk::launch_simple<__half, false, 64>(a, stream);
  return D == 128 ? gk::launch_simple<__nv_bfloat16, false, 128>(a, stream)
                  : gk::launch_simple<__nv_bfloat16, false, 64>(a, stream);
}

}  // namespace pa
