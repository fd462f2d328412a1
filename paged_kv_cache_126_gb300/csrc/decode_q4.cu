// Decode attention over the 4-bit cache [num_blocks, H, B, 5 D / 8].
#include "gather_kernel.cuh"
#include "pa.h"

namespace pa {
namespace {

// Weights go to the tensor cores as two fp16 parts: one alone, off by 2^-12 of a weight, would add an error as large as a
// fp16 output's own rounding, and several times what fp32 sums leave to a bf16 output that the values cancel to near zero.
//
// 12 warps an SM, three on each scheduler, with one stage of 64 keys (168 registers, five or six of them spilled at
// D = 128): 64 sequences of 512 to 2048 tokens, 32 heads of 128 in fp16 (421 MB) take 95.9 us, 4.4 TB/s; 4 x 16384 in bf16
// (336 MB) 73.9 us, 4.5 TB/s.  16 warps (128 registers, spills) 98.8 us for the first, 10 and 8 warps 105 and 101 us; tiles of 16
// keys with 16 warps 108, of 32 keys with 12 warps 98 us.
template <typename T, int D>
cudaError_t by_group(const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, cudaStream_t stream,
                     int* workers) {
  using F = gk::Q4Format<T, D>;
  typename F::Maps maps;
  maps.k = tk;
  maps.v = tv;
  if (a.g <= 4) return gk::launch<F, 1, gk::kTwinColumns, gk::kEvery, 1, 4, 3>(a, maps, num_sms, stream, workers);
  if (a.g <= 8) return gk::launch<F, 1, gk::kTwoParts, gk::kEvery, 1, 4, 3>(a, maps, num_sms, stream, workers);
  return gk::launch<F, 2, gk::kTwoParts, gk::kEvery, 1, 4, 2>(a, maps, num_sms, stream, workers);
}

}  // namespace

cudaError_t launch_decode_q4(int dtype, int D, const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms,
                             cudaStream_t stream, int* workers) {
  if (dtype == PA_F16)
    return D == 128 ? by_group<__half, 128>(a, tk, tv, num_sms, stream, workers)
                    : by_group<__half, 64>(a, tk, tv, num_sms, stream, workers);
  return D == 128 ? by_group<__nv_bfloat16, 128>(a, tk, tv, num_sms, stream, workers)
                  : by_group<__nv_bfloat16, 64>(a, tk, tv, num_sms, stream, workers);
}

}  // namespace pa
