#include "prefill_window.cuh"

namespace pa {

cudaError_t launch_prefill_window_bf16(const PrefillArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                      int grid, cudaStream_t stream) {
  return prefill_window<__nv_bfloat16>(a, tq, tk, tv, grid, stream);
}

}  // namespace pa
