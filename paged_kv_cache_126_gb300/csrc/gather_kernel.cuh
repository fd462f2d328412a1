// Single-query attention over gathered keys: every token of a sequence held in the 4-bit
// cache, or the tokens of listed frames of a 16-bit cache.
//
// out = sum_j w_j v_j / sum_j w_j, w_j = exp(q . k_j * scale - m), in one pass with the
// running maximum m and sum per warp.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_kernel.cuh"
#include "pa_internal.h"

namespace pa {
namespace gk {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One block per (query head, sequence), a warp per token in turn, D / 32 elements a lane.
template <typename T, bool Q4, int D>
__global__ void __launch_bounds__(128) simple_kernel(const GatherArgs a) {
  constexpr int E = D / 32, W = D / 2 + D / 8;
  __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
  __shared__ int bad;
  const int s = blockIdx.y, hq = blockIdx.x, h = hq / a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int L = a.context_lens[s];
  if (L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks) * a.B) {
    if (threadIdx.x == 0) atomicOr(a.status, kDevBadLen);
    L = 0;
  }
  const int blocks = (L + a.B - 1) / a.B;
  const int count = a.selected ? min(a.K, blocks) : blocks;
  const T* q = static_cast<const T*>(a.q) + s * a.q_row + hq * D;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) {
    qv[i] = to_float(q[lane * E + i]);
    o[i] = 0.f;
  }
  for (int j = 0; j < count; ++j) {
    int e = j;
    if (a.selected) {
      e = a.selected[s * a.sel_seq + h * a.sel_head + j];
      if (e == -1) break;
    }
    const int frame = e >= 0 && e < blocks ? a.block_tables[s * a.bt_row + e] : -1;
    if (frame < 0 || frame >= a.num_blocks) {
      if (lane == 0) {
        atomicOr(a.status, kDevBadBlock);
        bad = 1;
      }
      break;
    }
    for (int i = warp; i < a.B && e * a.B + i < L; i += 4) {
      float k[E], v[E], x = 0.f;
      for (int y = 0; y < 2; ++y) {
        const unsigned char* base = y ? a.v_cache : a.k_cache;
        float* dst = y ? v : k;
        if (Q4) {
          const unsigned char* row = base + ((static_cast<int64_t>(frame) * a.H + h) * a.B + i) * W;
          const __half* par = reinterpret_cast<const __half*>(row + D / 2 + (lane * E / 32) * 4);
          for (int u = 0; u < E; ++u) {
            const int d = lane * E + u;
            const int n = (row[d >> 1] >> (4 * (d & 1))) & 15;
            dst[u] = __half2float(__hfma(__int2half_rn(n), par[0], par[1]));
          }
        } else {
          const T* row = reinterpret_cast<const T*>(base) + ((static_cast<int64_t>(frame) * a.B + i) * a.H + h) * D;
          for (int u = 0; u < E; ++u) dst[u] = to_float(row[lane * E + u]);
        }
      }
      for (int u = 0; u < E; ++u) x = fmaf(qv[u], k[u], x);
      for (int b = 16; b; b >>= 1) x += __shfl_xor_sync(kAll, x, b);
      x *= a.qk_scale_log2;
      const float mn = fmaxf(m, x), al = exp2f(m - mn), p = exp2f(x - mn);
      l = l * al + p;
      for (int u = 0; u < E; ++u) o[u] = o[u] * al + p * v[u];
      m = mn;
    }
  }
  sm_m[warp] = m;
  sm_l[warp] = l;
  for (int u = 0; u < E; ++u) sm_o[warp][lane * E + u] = o[u];
  __syncthreads();
  T* out = static_cast<T*>(a.out) + s * a.out_row + hq * D;
  for (int d = threadIdx.x; d < D; d += 128) {
    float mm = -INFINITY, ll = 0.f, oo = 0.f;
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm_m[w]);
    for (int w = 0; w < 4; ++w) {
      if (sm_l[w] == 0.f) continue;
      const float al = exp2f(sm_m[w] - mm);
      ll += al * sm_l[w];
      oo += al * sm_o[w][d];
    }
    out[d] = from_float<T>(bad || ll == 0.f ? 0.f : oo / ll);
  }
}

template <typename T, bool Q4, int D>
cudaError_t launch_simple(const GatherArgs& a, cudaStream_t stream) {
  simple_kernel<T, Q4, D><<<dim3(a.g * a.H, a.S), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gk
}  // namespace pa
