// Attention of query chunks over a window and the first tokens, shared key heads: which slots a launch has.
#pragma once

#include "prefill_kernel.cuh"

namespace pa {

template <typename T>
cudaError_t prefill_window(const PrefillArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                           cudaStream_t stream) {
  // the most tiles that T rows of S sequences are
  const int64_t tiles = a.T <= a.S ? a.T : (a.T - a.S) / pk::kBM + a.S;
  if (tiles * a.H <= grid) return pk::launch<T, pk::kSplit>(a, tq, tk, tv, grid, stream);
  if (a.g % 2 == 0) return pk::launch<T, pk::kHeads>(a, tq, tk, tv, grid, stream);
  return pk::launch<T, pk::kRows>(a, tq, tk, tv, grid, stream);
}

}  // namespace pa
