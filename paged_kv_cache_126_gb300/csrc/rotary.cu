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
// A warp takes rows of one token and one kind (query, key or value): a row is V = D * elem / 16
// lanes of one 16-byte vector each, so 32 / V rows at a time and kSteps such steps, whose loads
// are all issued before the first is used (one memory round trip for 2 KB a warp).  A lane's
// vector position never changes, so the token's cosines and sines are loaded once for all its
// rows.  A vector's partner (i + R/2) is another lane of the same row: shuffles bring it, and
// since a row is loaded by one warp before any of it is stored, q_out may be q.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSteps = 4;  // row steps a warp loads at once

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
  static constexpr bool kBf16 = false;
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
  static constexpr bool kBf16 = true;
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
  // round((x - off) / step) by a product with 1 / step: the product is within 2^-21 * 15 of the quotient, so
  // where it is further than 2^-15 from a border between two codes both round alike; a lane with a
  // value nearer than that divides.
  const bool coded = finite && stepf > 0.f;
  const float inv = coded ? __frcp_rn(stepf) : 0.f;
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded addend
  float half_way = 0.f, n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(v[i], offf), inv), 0.f), 15.f);
    n[i] = __fsub_rn(__fadd_rn(q, kRound), kRound);
    half_way = fmaxf(half_way, fabsf(__fsub_rn(q, n[i])));
  }
  if (half_way > 0.5f - 0x1p-15f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[i], offf), stepf)), 0.f), 15.f);
  }
  // four codes as one number below 2^16, exact in fp32
  const float a = fmaf(fmaf(fmaf(n[3], 16.f, n[2]), 16.f, n[1]), 16.f, n[0]) + 8388608.f;
  const float b = fmaf(fmaf(fmaf(n[7], 16.f, n[6]), 16.f, n[5]), 16.f, n[4]) + 8388608.f;
  const uint32_t st = finite ? __half_as_ushort(step) : 0x7fffu, of = finite ? __half_as_ushort(off) : 0x7fffu;
  *params = st | (of << 16);
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}

template <typename T, bool Q4>
__global__ void __launch_bounds__(256) rope_append_kernel(const RopeArgs a) {
  constexpr int N = Vec<T>::N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int V = a.D / N, at_once = 32 / V;
  const int sub = lane / V, vec = lane - sub * V;
  const int rv = a.R / N;           // rotated vectors of a row
  const int per = at_once * kSteps;
  const int cq = a.q ? (a.Hq + per - 1) / per : 0, ck = (a.H + per - 1) / per;  // warps of a token's queries, keys
  const int64_t job = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int jobs = cq + 2 * ck;
  if (job >= static_cast<int64_t>(a.T) * jobs) return;
  const int t = static_cast<int>(job / jobs);
  const int part = static_cast<int>(job - static_cast<int64_t>(t) * jobs);
  const bool is_q = part < cq, is_k = !is_q && part < cq + ck;
  const int h0 = (is_q ? part : is_k ? part - cq : part - cq - ck) * per + sub;  // first of this lane's rows
  const int heads = is_q ? a.Hq : a.H;
  const T* src = is_q ? static_cast<const T*>(a.q) + t * a.q_row
                 : is_k ? static_cast<const T*>(a.k_new) + t * a.k_row
                        : static_cast<const T*>(a.v_new) + t * a.v_row;
  src += static_cast<int64_t>(h0) * a.D + vec * N;
  uint4 u[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    u[i] = make_uint4(0, 0, 0, 0);
    if (sub < at_once && h0 + i * at_once < heads) u[i] = *reinterpret_cast<const uint4*>(src + i * at_once * a.D);
  }

  const int32_t pos = a.positions ? a.positions[t] : 0;
  int32_t slot = is_q ? 0 : a.slots[t];
  if (pos < 0) return;
  if (a.positions && pos >= a.P) {
    if (lane == 0) atomicOr(a.status, kDevBadPos);
    return;
  }
  if (slot >= a.num_slots) {
    if (lane == 0) atomicOr(a.status, kDevBadSlot);
    return;
  }
  if (slot < 0) return;
  const bool turn = a.positions && (is_q || is_k);
  const bool rot = turn && vec < rv && sub < at_once;
  const bool first = vec < rv / 2;
  float c[N] = {}, s[N] = {};
  if (rot) {
    const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.cs_row;
    if (!a.interleaved) {  // (c, s) of this vector's elements; the second half of a pair takes its partner with + s
      row += (first ? vec : vec - rv / 2) * N;
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(row + i), y = *reinterpret_cast<const float4*>(row + a.R / 2 + i);
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        c[i] = row[vec * (N / 2) + i];
        s[i] = row[a.R / 2 + vec * (N / 2) + i];
      }
    }
  }
  // the lane that holds the partner vector (half-split pairs)
  const int partner = rot && !a.interleaved ? (first ? lane + rv / 2 : lane - rv / 2) : lane;

  const int64_t frame = slot / a.B;
  const int W = a.D / 2 + a.D / 8;
  unsigned char* dst;  // of this lane's first row, and its distance to the next
  int64_t dist;
  if (is_q) {
    dst = reinterpret_cast<unsigned char*>(static_cast<T*>(a.q_out) + t * a.qo_row + static_cast<int64_t>(h0) * a.D + vec * N);
    dist = static_cast<int64_t>(at_once) * a.D * sizeof(T);
  } else if (!Q4) {
    dst = (is_k ? a.k_cache : a.v_cache) + ((static_cast<int64_t>(slot) * a.H + h0) * a.D + vec * N) * sizeof(T);
    dist = static_cast<int64_t>(at_once) * a.D * sizeof(T);
  } else {
    dst = (is_k ? a.k_cache : a.v_cache) + ((frame * a.H + h0) * a.B + (slot - frame * a.B)) * W;
    dist = static_cast<int64_t>(at_once) * a.B * W;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const bool live = sub < at_once && h0 + i * at_once < heads;
    if (!__any_sync(kAll, live)) break;
    float x[N];
    if (turn || (Q4 && !is_q)) Vec<T>::unpack(u[i], x);
    if (turn) {
      if (!a.interleaved) {
        float y[N];
        Vec<T>::unpack(shfl4(u[i], partner), y);
        if (rot) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float p = __fmul_rn(x[j], c[j]), o = __fmul_rn(y[j], s[j]);
            x[j] = first ? __fsub_rn(p, o) : __fadd_rn(p, o);
          }
        }
      } else if (rot) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float x1 = x[2 * j], x2 = x[2 * j + 1];
          x[2 * j] = __fsub_rn(__fmul_rn(x1, c[j]), __fmul_rn(x2, s[j]));
          x[2 * j + 1] = __fadd_rn(__fmul_rn(x2, c[j]), __fmul_rn(x1, s[j]));
        }
      }
    }
    if constexpr (Q4) {
      if (!is_q) {
        uint32_t params;
        const uint32_t word = quantise8(x, &params);  // groups are four lanes of one row
        if (live) {
          *reinterpret_cast<uint32_t*>(dst + vec * 4) = word;
          if ((vec & 3) == 0) *reinterpret_cast<uint32_t*>(dst + a.D / 2 + vec) = params;
        }
        dst += dist;
        continue;
      }
    }
    if (live) *reinterpret_cast<uint4*>(dst) = rot ? Vec<T>::pack(x) : u[i];
    dst += dist;
  }
}

// Eight numbers of a 4-bit row from a word of codes and the group's step and offset, as pairs of
// elements (0, 1), (2, 3), (4, 5), (6, 7).  A code in the low bits of 1024's mantissa (or bits 4..7 of
// 64's) is 1024 + n (64 + n), exactly.
__device__ __forceinline__ void values8(uint32_t word, uint32_t params, uint32_t (&x)[4]) {
  const __half2 step = __half2half2(__ushort_as_half(static_cast<unsigned short>(params)));
  const __half2 off = __half2half2(__ushort_as_half(static_cast<unsigned short>(params >> 16)));
  uint32_t y[4];  // elements (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = word >> (i & 2 ? 8 : 0);
    const uint32_t m = i & 1 ? (w & 0x00f000f0u) | 0x54005400u : (w & 0x000f000fu) | 0x64006400u;
    const __half2 bias = __half2half2(__ushort_as_half(i & 1 ? 0x5400 : 0x6400));
    const __half2 z = __hfma2(__hsub2(*reinterpret_cast<const __half2*>(&m), bias), step, off);
    y[i] = *reinterpret_cast<const uint32_t*>(&z);
  }
  x[0] = __byte_perm(y[0], y[1], 0x5410);
  x[1] = __byte_perm(y[2], y[3], 0x5410);
  x[2] = __byte_perm(y[0], y[1], 0x7632);
  x[3] = __byte_perm(y[2], y[3], 0x7632);
}

// A warp per token, cache and kSteps * 32 / V heads; a lane reads a word of codes and writes 16 bytes.
template <typename T>
__global__ void __launch_bounds__(256) read_q4_kernel(const ReadQ4Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int V = a.D / 8, at_once = 32 / V, sub = lane / V, vec = lane - sub * V;
  const int W = a.D / 2 + a.D / 8, per = at_once * kSteps, chunks = (a.H + per - 1) / per;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (job >= static_cast<int64_t>(a.T) * 2 * chunks) return;
  const int t = static_cast<int>(job / (2 * chunks));
  const int part = static_cast<int>(job - static_cast<int64_t>(t) * 2 * chunks);
  const bool is_v = part >= chunks;
  const int h0 = (is_v ? part - chunks : part) * per + sub;
  const int32_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (lane == 0) atomicOr(a.status, kDevBadSlot);
    return;
  }
  const int64_t frame = slot / a.B;
  const unsigned char* src = (is_v ? a.v_cache : a.k_cache) + ((frame * a.H + h0) * a.B + (slot - frame * a.B)) * W;
  uint32_t word[kSteps], params[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (h0 + i * at_once >= a.H) continue;
    const unsigned char* row = src + static_cast<int64_t>(i * at_once) * a.B * W;
    word[i] = *reinterpret_cast<const uint32_t*>(row + vec * 4);
    params[i] = *reinterpret_cast<const uint32_t*>(row + a.D / 2 + (vec >> 2) * 4);
  }
  T* dst = (is_v ? static_cast<T*>(a.v_out) + t * a.vo_row : static_cast<T*>(a.k_out) + t * a.ko_row) +
           static_cast<int64_t>(h0) * a.D + vec * 8;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (h0 + i * at_once >= a.H) continue;
    uint32_t x[4];
    values8(word[i], params[i], x);
    uint4 y = make_uint4(x[0], x[1], x[2], x[3]);
    if (Vec<T>::kBf16) {
      float f[8];
      Vec<__half>::unpack(y, f);
      y = Vec<__nv_bfloat16>::pack(f);
    }
    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i * at_once) * a.D) = y;
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

cudaError_t launch_rope_append(int dtype, bool q4, RopeArgs a, cudaStream_t stream) {
  const int at_once = 32 / (a.D * (dtype == PA_F32 ? 4 : 2) / 16), per = at_once * kSteps;
  const int64_t jobs = (a.q ? (a.Hq + per - 1) / per : 0) + 2 * static_cast<int64_t>((a.H + per - 1) / per);
  const int64_t grid = (a.T * jobs + 7) / 8;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
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

cudaError_t launch_read_q4(int dtype, ReadQ4Args a, cudaStream_t stream) {
  const int per = 32 / (a.D / 8) * kSteps;
  const int64_t grid = (static_cast<int64_t>(a.T) * 2 * ((a.H + per - 1) / per) + 7) / 8;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  void* args[1] = {&a};
  const void* fn = dtype == PA_F16 ? reinterpret_cast<const void*>(&read_q4_kernel<__half>)
                                   : reinterpret_cast<const void*>(&read_q4_kernel<__nv_bfloat16>);
  return launch_pdl(fn, grid, args, stream);
}

}  // namespace pa
