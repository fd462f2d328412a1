// Decode attention over the last tokens of each sequence and its first few, 16-bit cache [num_blocks, B, H, D].
#include "pa.h"
#include "row_format.cuh"

namespace pa {
namespace {

template <typename T, int D>
cudaError_t by_group(const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, cudaStream_t stream,
                     int* workers) {
  using F = gk::RowFormat<T, D, 2>;
  typename F::Maps maps;
  maps.k = tk;
  maps.v = tv;
  if (a.g <= 4) return gk::launch<F, 1, gk::kTwinColumns, gk::kWindow, 1, 4, 2>(a, maps, num_sms, stream, workers);
  if (a.g <= 8) return gk::launch<F, 1, gk::kTwoParts, gk::kWindow, 1, 4, 2>(a, maps, num_sms, stream, workers);
  return gk::launch<F, 2, gk::kTwoParts, gk::kWindow, 1, 4, 2>(a, maps, num_sms, stream, workers);
}

}  // namespace

cudaError_t launch_decode_window(int dtype, int D, const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                                 int num_sms, cudaStream_t stream, int* workers) {
  if (dtype == PA_F16)
    return D == 128 ? by_group<__half, 128>(a, tk, tv, num_sms, stream, workers)
                    : by_group<__half, 64>(a, tk, tv, num_sms, stream, workers);
  return D == 128 ? by_group<__nv_bfloat16, 128>(a, tk, tv, num_sms, stream, workers)
                  : by_group<__nv_bfloat16, 64>(a, tk, tv, num_sms, stream, workers);
}

}  // namespace pa
