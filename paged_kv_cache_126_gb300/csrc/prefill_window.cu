// Attention of query chunks over a window and the first tokens (fp16 and bf16 caches, shared key heads).
#include "pa.h"
#include "prefill_kernel.cuh"

namespace pa {

cudaError_t launch_prefill_window(int dtype, const PrefillArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, int grid, cudaStream_t stream) {
  return dtype == PA_F16 ? pk::launch<__half, true>(a, tq, tk, tv, grid, stream)
                         : pk::launch<__nv_bfloat16, true>(a, tq, tk, tv, grid, stream);
}

}  // namespace pa
