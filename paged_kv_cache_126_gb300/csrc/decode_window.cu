// Decode attention over the last tokens of each sequence and its first few, 16-bit cache [num_blocks, B, H, D].
#include "pa.h"
#include "row_format.cuh"

namespace pa {
namespace {

// Bound by memory while it streams, in pieces of one head's row (256 bytes, H rows apart).  Tiles of 32 keys, one stage, 8 warps an SM: a window of
// 1024 tokens for 64 x 32 heads in fp16 (1015 MB) takes 157 to 161 us, 6.4 TB/s, of 4000 for 32 sequences of 100 to 65,536 tokens and 8
// heads in bf16 (304 MB) 56.3 us, one sequence of 20,000 9.7 us.  12 warps 162.6 and 58.1 us, tiles of 64 keys with 6 warps 164 and
// 59.8 us, of 16 keys with two stages 166 and 58.2 us (10.9 for the one sequence); boxes of 16 rows 158.9 where boxes of 8 took
// 156.6, copies issued by one lane 163.
template <typename T, int D>
cudaError_t by_group(const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, cudaStream_t stream,
                     int* workers) {
  using F = gk::RowFormat<T, D, 2>;
  typename F::Maps maps;
  maps.k = tk;
  maps.v = tv;
  constexpr int kBlocks = D == 64 ? 3 : 2;  // (of half as many bytes)
  if (a.g <= 4) return gk::launch<F, 1, gk::kTwinColumns, gk::kWindow, 1, 4, kBlocks>(a, maps, num_sms, stream, workers);
  if (a.g <= 8) return gk::launch<F, 1, gk::kTwoParts, gk::kWindow, 1, 4, kBlocks>(a, maps, num_sms, stream, workers);
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
