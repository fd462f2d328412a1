// Bounds of the keys of each frame, and the frames that a score from them selects.
//
// bounds[frame][h][0 / 1][d] = min / max over the frame's tokens of k[d].  For a query q and any
// key k of the frame, q . k <= sum_d max(q_d min_d, q_d max_d): the frame's score.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// One block per (position in the table, sequence), a thread per two elements of a token row.
template <typename T2>
__global__ void __launch_bounds__(256) block_bounds_kernel(const BoundsArgs a) {
  const int s = blockIdx.y;
  const int L = a.context_lens[s];
  const int first = a.first ? a.first[s] : 0;
  if (L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks) * a.B || first < 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.status, kDevBadLen);
    return;
  }
  const int pairs = a.H * a.D / 2;
  for (int j = first / a.B + blockIdx.x; j < (first < L ? (L + a.B - 1) / a.B : 0); j += gridDim.x) {
    const int frame = a.block_tables[s * a.bt_row + j];
    if (frame < 0 || frame >= a.num_blocks) {
      if (threadIdx.x == 0) atomicOr(a.status, kDevBadBlock);
      continue;
    }
    const int n = min(a.B, L - j * a.B);
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
      const T2* k = static_cast<const T2*>(a.k_cache) + static_cast<int64_t>(frame) * a.B * pairs + i;
      T2 lo = k[0], hi = k[0];
      for (int u = 1; u < n; ++u) {
        lo = __hmin2(lo, k[static_cast<int64_t>(u) * pairs]);
        hi = __hmax2(hi, k[static_cast<int64_t>(u) * pairs]);
      }
      const int h = i / (a.D / 2), d = i - h * (a.D / 2);
      T2* b = static_cast<T2*>(a.bounds) + (static_cast<int64_t>(frame) * a.H + h) * a.D + d;
      b[0] = lo;
      b[a.D / 2] = hi;
    }
  }
}

// A warp per (frame position, key head, sequence): scores [S, H, max_blocks].
template <typename T>
__global__ void __launch_bounds__(256) score_kernel(const SelectArgs a) {
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y, s = blockIdx.z;
  const int L = a.context_lens[s];
  if (L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks) * a.B) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.status, kDevBadLen);
    return;
  }
  const int blocks = (L + a.B - 1) / a.B, E = a.D / 32;
  for (int j = blockIdx.x * 8 + (threadIdx.x >> 5); j < blocks; j += gridDim.x * 8) {
    const int frame = a.block_tables[s * a.bt_row + j];
    float best = -INFINITY;
    if (frame < 0 || frame >= a.num_blocks) {
      if (lane == 0) atomicOr(a.status, kDevBadBlock);
    } else {
      const T* b = static_cast<const T*>(a.bounds) + (static_cast<int64_t>(frame) * a.H + h) * 2 * a.D;
      for (int g = 0; g < a.g; ++g) {
        const T* q = static_cast<const T*>(a.q) + s * a.q_row + (h * a.g + g) * a.D;
        float x[4];
        for (int u = 0; u < 4; ++u) {
          x[u] = 0.f;
          if (u >= E) continue;
          const int d = lane * E + u;
          const float qd = to_float(q[d]);
          x[u] = qd * to_float(qd >= 0.f ? b[a.D + d] : b[d]);
        }
        float y = E == 4 ? __fadd_rn(__fadd_rn(x[0], x[1]), __fadd_rn(x[2], x[3])) : __fadd_rn(x[0], x[1]);
        for (int o = 1; o < 32; o <<= 1) y = __fadd_rn(y, __shfl_xor_sync(kAll, y, o));
        best = fmaxf(best, y);
      }
    }
    if (lane == 0) a.scores[(static_cast<int64_t>(s) * a.H + h) * a.max_blocks + j] = best;
  }
}

// Keys whose unsigned order is the order of the floats; frames that are always kept come
// above all others.
__device__ __forceinline__ uint32_t rank_of(const SelectArgs& a, const float* scores, int j, int blocks) {
  if (j < a.keep_first || j >= blocks - a.keep_last) return 0xffffffffu;
  const uint32_t u = __float_as_uint(__fadd_rn(scores[j], 0.f));  // -0 ranks as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kTopThreads = 256;

__device__ __forceinline__ int block_scan(int v, int* total, int* warp_sums) {  // exclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kTopThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  return before + x - v;
}

// One block per (key head, sequence): the K largest ranks, found digit by digit.
__global__ void __launch_bounds__(kTopThreads) top_kernel(const SelectArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kTopThreads / 32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  const int h = blockIdx.x, s = blockIdx.y;
  int32_t* sel = a.selected + s * a.sel_seq + h * a.sel_head;
  int L = a.context_lens[s];
  if (L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks) * a.B) L = 0;
  const int blocks = (L + a.B - 1) / a.B;
  if (blocks <= a.K) {
    for (int j = threadIdx.x; j < a.K; j += kTopThreads) sel[j] = j < blocks ? j : -1;
    return;
  }
  const float* scores = a.scores + (static_cast<int64_t>(s) * a.H + h) * a.max_blocks;
  uint32_t prefix = 0, mask = 0;
  int need = a.K;  // how many of the ranks that match the prefix are taken
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kTopThreads) hist[i] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < blocks; j += kTopThreads) {
      const uint32_t r = rank_of(a, scores, j, blocks);
      if ((r & mask) == prefix) atomicAdd(&hist[(r >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int left = need, d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      sh_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      sh_need = left;
    }
    __syncthreads();
    prefix = sh_prefix;
    need = sh_need;
    mask |= 0xffu << shift;
  }
  int taken = 0, ties = 0;  // before this stretch of positions
  for (int j0 = 0; j0 < blocks; j0 += kTopThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t r = j < blocks ? rank_of(a, scores, j, blocks) : 0;
    const bool tie = j < blocks && r == prefix;
    int all;
    const int tie_at = ties + block_scan(tie, &all, warp_sums);
    ties += all;
    const bool take = j < blocks && (r > prefix || (tie && tie_at < need));
    const int at = taken + block_scan(take, &all, warp_sums);
    taken += all;
    if (take) sel[at] = j;
  }
}

}  // namespace

cudaError_t launch_block_bounds(int dtype, const BoundsArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const dim3 grid(a.max_blocks < 1 ? 1 : a.max_blocks < 64 ? a.max_blocks : 64, a.S);
  if (dtype == PA_F16)
    block_bounds_kernel<__half2><<<grid, 256, 0, stream>>>(a);
  else
    block_bounds_kernel<__nv_bfloat162><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_select_blocks(int dtype, const SelectArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const int chunks = (a.max_blocks + 7) / 8;
  const dim3 grid(chunks < 1 ? 1 : chunks < 64 ? chunks : 64, a.H, a.S);
  if (dtype == PA_F16)
    score_kernel<__half><<<grid, 256, 0, stream>>>(a);
  else
    score_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  top_kernel<<<dim3(a.H, a.S), kTopThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
