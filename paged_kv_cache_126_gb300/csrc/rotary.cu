// Cache append with the position rotation applied on the way (16- and 32-bit caches and
// the 4-bit cache), and the 4-bit cache read back as 16-bit rows.
//
// Rotation of a head's first R elements by the token's row of cos_sin: a pair (x1, x2)
// becomes (x1 cos - x2 sin, x2 cos + x1 sin), each product and sum rounded to fp32 by
// itself, so that a 4-bit code follows from the formula alone and not from which of the
// two products a fused multiply-add keeps exact.
//
// 4-bit group of 32 elements: offset = fp16(min), step = fp16((max - offset) / 15), code =
// round((x - offset) / step); 5 bits an element with its two fp16 numbers.
//
// A warp takes rows of one token: a row is V = D * elem / 16 lanes of one 16-byte vector
// each, so 32 / V rows at a time.  A lane's vector position never changes, so the token's
// cosines and sines are loaded once and stay in registers over all its rows.  A vector's
// partner (i + R/2) is another lane of the same row: shuffles bring it, and since a row
// is loaded by one warp before any of it is stored, q_out may be q.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ uint4 shfl4(const uint4& u, int lane) {
  return make_uint4(__shfl_sync(kAll, u.x, lane), __shfl_sync(kAll, u.y, lane), __shfl_sync(kAll, u.z, lane),
                    __shfl_sync(kAll, u.w, lane));
}

// Eight consecutive elements of one 4-bit row (element 0 at a multiple of 8): the word of
// codes for this lane; step and offset of the group, the same in its four lanes.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t* params) {
  constexpr float kTop = 65024.f;  // the top code is at most kTop (1 + 2^-10): finite in fp16
  bool finite = true;
  float v[8], lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    finite = finite && fabsf(x[i]) < INFINITY;  // false for NaN too
    v[i] = fminf(fmaxf(x[i], -kTop), kTop);
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(kAll, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, o));
    finite = __shfl_xor_sync(kAll, static_cast<int>(finite), o) && finite;
  }
  const __half off = __float2half_rn(lo);
  const float offf = __half2float(off);
  const __half step = __float2half_rn(__fmul_rn(__fsub_rn(hi, offf), 1.0f / 15.0f));
  const float stepf = __half2float(step);
  uint32_t word = 0;
  if (finite && stepf > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[i], offf), stepf)), 0.f), 15.f);
      word |= static_cast<uint32_t>(n) << (4 * i);
    }
  }
  const uint32_t s = finite ? __half_as_ushort(step) : 0x7fffu, b = finite ? __half_as_ushort(off) : 0x7fffu;
  *params = s | (b << 16);
  return word;
}

template <typename T, bool Q4>
__global__ void __launch_bounds__(256) rope_append_kernel(const RopeArgs a) {
  constexpr int N = Vec<T>::N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int V = a.D / N, rows_at_once = 32 / V;
  const int sub = lane / V, vec = lane - sub * V;
  const bool active = sub < rows_at_once;
  const int rv = a.R / N;           // rotated vectors of a row
  const bool rot = vec < rv && active;
  const int Hq = a.q ? a.Hq : 0;
  const int rows = Hq + 2 * a.H;
  const int64_t jobs = static_cast<int64_t>(a.T) * a.splits;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (job >= jobs) return;
  const int t = static_cast<int>(job / a.splits);
  const int split = static_cast<int>(job - static_cast<int64_t>(t) * a.splits);
  const int per = ((rows + a.splits - 1) / a.splits + rows_at_once - 1) / rows_at_once * rows_at_once;
  const int row0 = split * per, row1 = min(rows, row0 + per);

  int32_t slot = a.slots[t];
  if (slot >= a.num_slots) {
    if (lane == 0) atomicOr(a.status, kDevBadSlot);
    slot = -1;
  }
  float c[N], s[N];
  if (a.positions) {
    const int32_t pos = a.positions[t];
    if (pos < 0) return;
    if (pos >= a.P) {
      if (lane == 0) atomicOr(a.status, kDevBadPos);
      return;
    }
    if (rot) {
      const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.cs_row;
      if (!a.interleaved) {
        const int i0 = (vec < rv / 2 ? vec : vec - rv / 2) * N;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          c[i] = row[i0 + i];
          s[i] = row[a.R / 2 + i0 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          c[i] = row[vec * (N / 2) + i];
          s[i] = row[a.R / 2 + vec * (N / 2) + i];
        }
      }
    }
  }
  // the lane that holds the partner vector (half-split pairs)
  const int partner = rot && !a.interleaved ? (vec < rv / 2 ? lane + rv / 2 : lane - rv / 2) : lane;

  for (int r0 = row0; r0 < row1; r0 += rows_at_once) {
    const int r = r0 + sub;
    const bool live = active && r < row1;
    const bool is_q = r < Hq;
    const int h = is_q ? r : (r - Hq) % a.H;
    const bool is_k = !is_q && r < Hq + a.H;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live) {
      const T* src = is_q ? static_cast<const T*>(a.q) + t * a.q_row
                     : is_k ? static_cast<const T*>(a.k_new) + t * a.k_row
                            : static_cast<const T*>(a.v_new) + t * a.v_row;
      u = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * a.D + vec * N);
    }
    const uint4 w = shfl4(u, partner);
    float x[N];
    Vec<T>::unpack(u, x);
    const bool turn = rot && (is_q || is_k) && a.positions;
    if (turn) {
      float y[N];
      Vec<T>::unpack(w, y);
      if (!a.interleaved) {
        const bool first = vec < rv / 2;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float p = __fmul_rn(x[i], c[i]), o = __fmul_rn(y[i], s[i]);
          x[i] = first ? __fsub_rn(p, o) : __fadd_rn(p, o);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float x1 = x[2 * i], x2 = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(x1, c[i]), __fmul_rn(x2, s[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(x2, c[i]), __fmul_rn(x1, s[i]));
        }
      }
    }
    if (Q4 && sizeof(T) == 2) {
      // every lane takes part in the shuffles; groups are four lanes of one row
      uint32_t params;
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = x[i % N];
      const uint32_t word = quantise8(e, &params);
      if (live && !is_q) {
        if (slot >= 0) {
          const int W = a.D / 2 + a.D / 8;
          unsigned char* cache = is_k ? a.k_cache : a.v_cache;
          const int64_t frame = slot / a.B;
          unsigned char* dst = cache + ((frame * a.H + h) * a.B + (slot - frame * a.B)) * static_cast<int64_t>(W);
          *reinterpret_cast<uint32_t*>(dst + vec * 4) = word;
          if ((vec & 3) == 0) *reinterpret_cast<uint32_t*>(dst + a.D / 2 + vec) = params;
        }
        continue;
      }
    }
    if (!live) continue;
    const uint4 y = turn ? Vec<T>::pack(x) : u;
    if (is_q) {
      *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + t * a.qo_row + static_cast<int64_t>(h) * a.D + vec * N) = y;
    } else if (slot >= 0) {
      T* cache = reinterpret_cast<T*>(is_k ? a.k_cache : a.v_cache);
      *reinterpret_cast<uint4*>(cache + (static_cast<int64_t>(slot) * a.H + h) * a.D + vec * N) = y;
    }
  }
}

// Eight numbers of a 4-bit row from a word of codes and the group's step and offset.
__device__ __forceinline__ void values8(uint32_t word, uint32_t params, __half2 (&x)[4]) {
  const __half2 step = __half2half2(__ushort_as_half(static_cast<unsigned short>(params)));
  const __half2 off = __half2half2(__ushort_as_half(static_cast<unsigned short>(params >> 16)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 n = __halves2half2(__ushort2half_rn((word >> (8 * i)) & 15u), __ushort2half_rn((word >> (8 * i + 4)) & 15u));
    x[i] = __hfma2(n, step, off);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) read_q4_kernel(const ReadQ4Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int V = a.D / 8;
  const int W = a.D / 2 + a.D / 8;
  const int64_t total = static_cast<int64_t>(a.T) * 2 * a.H * V;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int vec = static_cast<int>(i % V);
    const int64_t row = i / V;
    const int h = static_cast<int>(row % a.H);
    const int64_t tk = row / a.H;
    const int t = static_cast<int>(tk >> 1);
    const bool is_v = tk & 1;
    const int32_t slot = a.slots[t];
    if (slot < 0) continue;
    if (slot >= a.num_slots) {
      atomicOr(a.status, kDevBadSlot);
      continue;
    }
    const int64_t frame = slot / a.B;
    const unsigned char* src =
        (is_v ? a.v_cache : a.k_cache) + ((frame * a.H + h) * a.B + (slot - frame * a.B)) * static_cast<int64_t>(W);
    const uint32_t word = *reinterpret_cast<const uint32_t*>(src + vec * 4);
    const uint32_t params = *reinterpret_cast<const uint32_t*>(src + a.D / 2 + (vec >> 2) * 4);
    __half2 x[4];
    values8(word, params, x);
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = __half22float2(x[j]);
      f[2 * j] = p.x;
      f[2 * j + 1] = p.y;
    }
    T* dst = (is_v ? static_cast<T*>(a.v_out) + t * a.vo_row : static_cast<T*>(a.k_out) + t * a.ko_row) +
             static_cast<int64_t>(h) * a.D + vec * 8;
    *reinterpret_cast<uint4*>(dst) = Vec<T>::pack(f);
  }
}

cudaError_t launch_pdl(const void* fn, int64_t grid, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_rope_append(int dtype, bool q4, RopeArgs a, int num_sms, cudaStream_t stream) {
  const int rows = (a.q ? a.Hq : 0) + 2 * a.H;
  a.splits = 1;
  const int64_t warps = static_cast<int64_t>(a.T) * a.splits;
  const int64_t grid = (warps + 7) / 8;
  (void)rows;
  (void)num_sms;
  void* args[1] = {&a};
  const void* fn = nullptr;
  if (q4)
    fn = dtype == PA_F16 ? reinterpret_cast<const void*>(&rope_append_kernel<__half, true>)
                         : reinterpret_cast<const void*>(&rope_append_kernel<__nv_bfloat16, true>);
  else
    fn = dtype == PA_F32   ? reinterpret_cast<const void*>(&rope_append_kernel<float, false>)
         : dtype == PA_F16 ? reinterpret_cast<const void*>(&rope_append_kernel<__half, false>)
                           : reinterpret_cast<const void*>(&rope_append_kernel<__nv_bfloat16, false>);
  return launch_pdl(fn, grid, args, stream);
}

cudaError_t launch_read_q4(int dtype, const ReadQ4Args& a, int num_sms, cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(a.T) * 2 * a.H * (a.D / 8);
  const int64_t want = (total + 255) / 256, most = 16LL * num_sms;
  ReadQ4Args b = a;
  void* args[1] = {&b};
  const void* fn = dtype == PA_F16 ? reinterpret_cast<const void*>(&read_q4_kernel<__half>)
                                   : reinterpret_cast<const void*>(&read_q4_kernel<__nv_bfloat16>);
  return launch_pdl(fn, want < most ? want : most, args, stream);
}

}  // namespace pa
