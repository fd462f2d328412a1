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
//
// Bound by memory: 16 chunks of 512 tokens, 32 query and 8 key heads of 128 in bf16 (206 MB) take
// 33.1 us, 6.2 TB/s; into the 4-bit cache (178 MB) 37.2 us, where the codes of keys and values take more instructions
// than all queries; read back (44 MB) 9.5 us.  A decode step of 64 tokens (3.2 MB) takes 2.6 us, a launch.
// 34.8 and 41.8 us without two fp32 numbers an instruction (32.6 and 36.6 when its products were fused into its sums); 37.0 and 44.7 where a block's four warps were parts of one token,
// whose kind and rows were then each lane's to compute.  Two steps a warp (44 us), six (34.3 us) and warps that
// stay and load their next rows meanwhile (51 us) were slower.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa.h"
#include "pa_internal.h"
#include "pair32.cuh"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSteps = 4;  // row steps a warp loads at once
// Small blocks: a block's place is free again as soon as its four warps are done (36.9 us where 256 threads took 39.6).
// Nine blocks an SM, 56 registers (one or two of the 16-bit append's spilled): 33.1 us for 16 chunks of 512 tokens; with fused
// products nine 32.6, eight 33.7, ten (more spills) 33.5.  The 4-bit append spills about 20 registers at nine and was not
// tried at fewer.
constexpr int kThreads = 128;
constexpr int kBlocks = 9;

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
__device__ __forceinline__ uint32_t quantise8(const float* x, uint32_t* params) {
  constexpr float kTop = 65024.f;  // the top code is at most kTop (1 + 2^-10): finite in fp16
  float lo = x[0], hi = x[0];
  uint64_t p[4], none2 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = pair(x[2 * i], x[2 * i + 1]);
    none2 = fma2(p[i], 0, none2);  // NaN once an element is not finite
  }
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  float none = both(none2).x + both(none2).y;
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(kAll, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, o));
    none += __shfl_xor_sync(kAll, none, o);
  }
  const bool finite = none == 0.f;
  // an element beyond +-kTop is coded like +-kTop: as 0 or 15
  const float bottom = fminf(fmaxf(lo, -kTop), kTop), top = fminf(fmaxf(hi, -kTop), kTop);
  const __half off = __float2half_rn(bottom);
  const float offf = __half2float(off);
  const __half step = __float2half_rn(__fmul_rn(__fsub_rn(top, offf), 1.0f / 15.0f));
  const float stepf = __half2float(step);
  // round((x - off) / step) by a product with 1 / step: four roundings and 2^-23 of the reciprocal leave it within
  // 15.5 * 6 * 2^-24 < 2^-17 of the quotient, so where it is further than 2^-16 from a border between two codes both
  // round alike.  Nearer ones (16-bit rows have many that lie on a border: a seventh of the steps of bf16 values)
  // are compared with it: the rest of n steps is exact, and a quotient that is not on the border does not
  // round to it, for step and border have 16 bits together.  The same path serves groups whose ends are not coded
  // as 0 and 15 by themselves.
  const bool coded = finite && stepf > 0.f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(stepf));
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded addend
  const uint64_t noff2 = pair(-offf, -offf), inv2 = pair(inv, inv), round2 = pair(kRound, kRound), back2 = pair(-kRound, -kRound);
  const uint64_t minus2 = pair(-1.f, -1.f);
  float half_way = 0.f;
  uint64_t n2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t = mul2(add2(p[i], noff2), inv2);  // (fused into the next sum or not: within the margin below)
    n2[i] = add2(add2(t, round2), back2);
    const float2 d = both(fma2(n2[i], minus2, t));
    half_way = fmaxf(half_way, fmaxf(fabsf(d.x), fabsf(d.y)));
  }
  const bool inside = fmaf(lo - offf, inv, 0.5f) > 0x1p-10f && fmaf(hi - offf, inv, -15.5f) < -0x1p-10f;
  if (!(half_way <= 0.5f - 0x1p-16f) || !inside || !coded) {
    const float half = 0.5f * stepf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = both(n2[i]);
      float n[2] = {f.x, f.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        n[k] = fminf(fmaxf(n[k], 0.f), 15.f);
        const float rest = fmaf(-n[k], stepf, __fsub_rn(x[2 * i + k], offf));
        const bool odd = __float_as_uint(n[k] + kRound) & 1u;
        if (rest > half || (rest == half && odd)) n[k] += 1.f;
        else if (rest < -half || (rest == -half && odd)) n[k] -= 1.f;
        n[k] = coded ? fminf(fmaxf(n[k], 0.f), 15.f) : 0.f;
      }
      n2[i] = pair(n[0], n[1]);
    }
  }
  // four codes as one number below 2^16, exact in fp32
  const uint64_t s256 = pair(256.f, 256.f);
  const float2 a = both(fma2(n2[1], s256, n2[0])), b = both(fma2(n2[3], s256, n2[2]));
  const float wa = fmaf(a.y, 16.f, a.x) + 8388608.f, wb = fmaf(b.y, 16.f, b.x) + 8388608.f;
  const uint32_t st = finite ? __half_as_ushort(step) : 0x7fffu, of = finite ? __half_as_ushort(off) : 0x7fffu;
  *params = st | (of << 16);
  return __byte_perm(__float_as_uint(wa), __float_as_uint(wb), 0x5410);
}

template <typename T, bool Q4>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_append_kernel(const RopeArgs a) {
  constexpr int N = Vec<T>::N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int V = a.V, at_once = a.at_once;
  const int sub = (lane * a.per_V) >> 16, vec = lane - sub * V;  // lane / V
  const int rv = a.R / N;           // rotated vectors of a row
  // the kind and the rows are the block's, so that what follows from them is computed once for all lanes
  const int part = blockIdx.x;
  const int t = static_cast<int>((blockIdx.z * gridDim.y + blockIdx.y) * (kThreads / 32) + (threadIdx.x >> 5));
  if (t >= a.T) return;
  const int cq = a.warps_q, ck = a.warps_k;
  const bool is_q = part < cq, is_k = !is_q && part < cq + ck;
  const int h0 = (is_q ? part : is_k ? part - cq : part - cq - ck) * at_once * kSteps + sub;  // first of this lane's rows
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
    if (!a.interleaved) {  // the first of a pair takes its partner with - sin, the second with + sin
      row += (first ? vec : vec - rv / 2) * N;
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(row + i), y = *reinterpret_cast<const float4*>(row + a.R / 2 + i);
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = first ? -s[i] : s[i];
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

  const int64_t frame = Q4 ? slot >> a.log2_B : 0;
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
  const auto steps = [&](auto turned_, auto coded_) {
    constexpr bool turned = decltype(turned_)::value, coded = decltype(coded_)::value;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const bool live = sub < at_once && h0 + i * at_once < heads;
      if (!__any_sync(kAll, live)) break;
      float x[N];
      if constexpr (turned || coded) Vec<T>::unpack(u[i], x);
      if constexpr (turned) {
        if (!a.interleaved) {
          float y[N];
          Vec<T>::unpack(shfl4(u[i], partner), y);
          if (rot) {
            const uint64_t none2 = pair(a.minus_zero, a.minus_zero);
#pragma unroll
            for (int j = 0; j < N; j += 2) {
              const float2 z = both(add2(rounded2(pair(x[j], x[j + 1]), pair(c[j], c[j + 1]), none2), rounded2(pair(y[j], y[j + 1]), pair(s[j], s[j + 1]), none2)));
              x[j] = z.x, x[j + 1] = z.y;
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
      if constexpr (coded) {
        uint32_t params;
        const uint32_t word = quantise8(x, &params);  // groups are four lanes of one row
        if (live) {
          *reinterpret_cast<uint32_t*>(dst + vec * 4) = word;
          if ((vec & 3) == 0) *reinterpret_cast<uint32_t*>(dst + a.D / 2 + vec) = params;
        }
      } else if (live) {
        if constexpr (turned) *reinterpret_cast<uint4*>(dst) = rot ? Vec<T>::pack(x) : u[i];
        else *reinterpret_cast<uint4*>(dst) = u[i];
      }
      dst += dist;
    }
  };
  const std::true_type yes{};
  const std::false_type no{};
  if constexpr (Q4) {
    if (is_q) steps(yes, no);
    else if (turn) steps(yes, yes);
    else steps(no, yes);
  } else {
    if (turn) steps(yes, no);
    else steps(no, no);
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
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const ReadQ4Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int at_once = a.D == 128 ? 2 : 4, sub = a.D == 128 ? lane >> 4 : lane >> 3, vec = a.D == 128 ? lane & 15 : lane & 7;
  const int W = a.D / 2 + a.D / 8, per = at_once * kSteps;
  const unsigned chunks = a.warps_k;
  const unsigned job = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (job >= a.T * 2 * chunks) return;
  const int t = static_cast<int>(job / (2 * chunks));
  const int part = static_cast<int>(job - t * 2 * chunks);
  const bool is_v = part >= static_cast<int>(chunks);
  const int h0 = (is_v ? part - static_cast<int>(chunks) : part) * per + sub;
  const int32_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (lane == 0) atomicOr(a.status, kDevBadSlot);
    return;
  }
  const int64_t frame = slot >> a.log2_B;
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

cudaError_t launch_pdl(const void* fn, dim3 grid, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

// warps that the rows of a token are split into
static int64_t warps_of(int64_t heads, int at_once) { return (heads + at_once * kSteps - 1) / (at_once * kSteps); }

bool rope_fits(const RopeArgs& a, int elem) {
  const int at_once = 32 / (a.D * elem / 16);
  return a.T * ((a.q ? warps_of(a.Hq, at_once) : 0) + 2 * warps_of(a.H, at_once)) <= INT32_MAX;
}

cudaError_t launch_rope_append(int dtype, bool q4, RopeArgs a, cudaStream_t stream) {
  a.V = a.D * (dtype == PA_F32 ? 4 : 2) / 16;
  a.at_once = 32 / a.V;
  a.warps_q = a.q ? static_cast<int>(warps_of(a.Hq, a.at_once)) : 0;
  a.warps_k = static_cast<int>(warps_of(a.H, a.at_once));
  a.per_V = 65536 / a.V + 1;
  a.minus_zero = -0.f;
  const int tokens = (a.T + kThreads / 32 - 1) / (kThreads / 32), rows = tokens < 65535 ? tokens : 65535;
  const dim3 grid(a.warps_q + 2 * a.warps_k, rows, (tokens + rows - 1) / rows);
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
  a.warps_k = static_cast<int>(warps_of(a.H, 32 / (a.D / 8)));
  const int64_t grid = (static_cast<int64_t>(a.T) * 2 * a.warps_k + kThreads / 32 - 1) / (kThreads / 32);
  void* args[1] = {&a};
  const void* fn = dtype == PA_F16 ? reinterpret_cast<const void*>(&read_q4_kernel<__half>)
                                   : reinterpret_cast<const void*>(&read_q4_kernel<__nv_bfloat16>);
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), args, stream);
}

}  // namespace pa
