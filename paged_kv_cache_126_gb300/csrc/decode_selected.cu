// Decode attention over the listed frames of a 16-bit cache [num_blocks, B, H, D].
#include "pa.h"
#include "row_format.cuh"

namespace pa {
namespace {

// Bound by memory as it is read here, in pieces of one head's row (256 bytes, H rows apart): 64 of 1024 frames
// of 16 tokens for 4 x 32 heads (67 MB) take 19.5 us, 2048 of up to 65,536 tokens for 32 x 8 heads (184 MB) 43 us,
// 38 of them streaming at 4.8 TB/s.  Two to six stages, 4 to 16 warps an SM, boxes of 128- or 256-byte
// rows and every L2 promotion gave the same within 3 %.
//
// Weights in two parts of the cache's type, in the second copy of the queries where four or fewer share a head.
template <typename T, int D>
cudaError_t by_group(const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, cudaStream_t stream,
                     int* workers) {
  using F = gk::RowFormat<T, D>;
  typename F::Maps maps;
  maps.k = tk;
  maps.v = tv;
  if (a.g <= 4) return gk::launch<F, 1, gk::kTwinColumns, gk::kListed, 2, 4, 2>(a, maps, num_sms, stream, workers);
  if (a.g <= 8) return gk::launch<F, 1, gk::kTwoParts, gk::kListed, 2, 4, 2>(a, maps, num_sms, stream, workers);
  return gk::launch<F, 2, gk::kTwoParts, gk::kListed, 2, 4, 2>(a, maps, num_sms, stream, workers);
}

}  // namespace

cudaError_t launch_decode_selected(int dtype, int D, const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                                   int num_sms, cudaStream_t stream, int* workers) {
  if (dtype == PA_F16)
    return D == 128 ? by_group<__half, 128>(a, tk, tv, num_sms, stream, workers)
                    : by_group<__half, 64>(a, tk, tv, num_sms, stream, workers);
  return D == 128 ? by_group<__nv_bfloat16, 128>(a, tk, tv, num_sms, stream, workers)
                  : by_group<__nv_bfloat16, 64>(a, tk, tv, num_sms, stream, workers);
}

}  // namespace pa
