// Append into the 8-bit cache [num_blocks, H, B, D], and its rows read back in 16 bits.
//
// A byte b stands for (b - 128) * step, one step for each (frame, head).  A frame that begins with the call's tokens takes
//     r = 127 / max |x|, cut to 8 leading bits;  step = 1 / r;  b = 128 + round-half-even(x r).
// x has at most 11 bits, so x r has at most 19 and is exact in fp32: the rounding to a whole number is the only one, and a code
// follows from the formula alone.  A frame that holds earlier tokens keeps its r, or halves it as often as the new
// tokens need to fit, and each earlier code n becomes round-half-even(n / 2^k).  Halvings are exact, and there are
// few of them: an earlier token is off by less than (1/2 + 1/4 + ...) final steps, however often the frame grows (a step that followed each new maximum
// would round every earlier code again at every one).
//
// A warp takes 16 rows of one frame and head, all in registers: their maximum, then their codes, one pass over the data.
// Frames of more than 16 tokens are as many warps of one block, which exchange their maxima.
//
// 16 chunks of 256 to 512 tokens, 8 heads of 128 in bf16 (50 MB): 8.9 us, 5.6 TB/s, 64 registers, of which D = 128 spills 4 to 16 bytes (87, none: 10.2 us); read back (50 MB)
// 7.5 us, 6.7 TB/s.  A decode step of 64 tokens, 32 heads in fp16: 4.0 us, three loads that wait for one another (lengths, table,
// step) behind a launch, 4.4 us with a warp a head; read back, up to 16 tokens of each frame (13 MB), 3.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 128;
constexpr float kLeast = 0x1p-60f, kMost = 0x1p60f;  // what a frame's largest element counts as: every product of r and x stays in fp32's range

template <typename T>
struct Bits;
template <>
struct Bits<__half> {
  static constexpr uint32_t kInf = 0x7c00;
  static constexpr bool kPastMost = false;  // whether an element may be above kMost
  __device__ __forceinline__ static float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
  __device__ __forceinline__ static float value(uint32_t bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); }
  // what is beyond fp16's largest number is that one (a code may stand for half a step more than its element); NaN stays
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    uint32_t h;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
    return h;
  }
};
template <>
struct Bits<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f80;
  static constexpr bool kPastMost = true;
  __device__ __forceinline__ static float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ __forceinline__ static float value(uint32_t bits) { return __uint_as_float(bits << 16); }
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// The codes of four elements as bytes: x r + 128 rounded in the low bits of 1.5 * 2^23.
__device__ __forceinline__ uint32_t codes4(float2 a, float2 b, float r) {
  constexpr float kRound = 12582912.f + 128.f;  // even, as 128 is: ties go to even codes
  const uint32_t c0 = __float_as_uint(fmaf(a.x, r, kRound)), c1 = __float_as_uint(fmaf(a.y, r, kRound));
  const uint32_t c2 = __float_as_uint(fmaf(b.x, r, kRound)), c3 = __float_as_uint(fmaf(b.y, r, kRound));
  return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
}
// The same of four earlier codes times 2^-k = p.
__device__ __forceinline__ uint32_t halved4(uint32_t w, float p) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = static_cast<float>((w >> (8 * i)) & 255u) - 128.f;
  return codes4(make_float2(f[0], f[1]), make_float2(f[2], f[3]), p);
}

// A frame that holds new tokens, of the call's u-th block: found by each warp for itself.
struct Unit {
  int s, L, first, row0;  // sequence, its tokens, its first new one and that token's row of k_new
  int j;                  // position in its table; < 0: none
};
// New tokens of a sequence that has the rows row0 .. end - 1; -1: a bad length or range.
__device__ __forceinline__ int new_tokens(const Append8Args& a, int L, int row0, int end) {
  if (!a.query_start) end = row0 + min(max(L, 0), 1);
  const bool bad = row0 < 0 || end < row0 || end > a.T || L < end - row0 ||
                   static_cast<int64_t>(L) > (static_cast<int64_t>(a.max_blocks) << a.log2_B);
  return bad ? -1 : end - row0;
}
// Numbers of units ascend with the sequences.  STEP: a unit is a row, that of a frame's first new token, the others are none.
// Else sequence s has the units from query_start[s] / B + 2 s on, as many as it can have frames.  The last sequence whose first unit
// is not behind u is searched 32 at a time, so that a call of many sequences is no slower for it.
template <bool STEP>
__device__ __forceinline__ int first_unit_of(const Append8Args& a, int s, int row0) {
  return STEP ? row0 : (row0 >> a.log2_B) + 2 * s;
}
template <bool STEP>
__device__ __forceinline__ Unit find_unit(const Append8Args& a, int u, int lane) {
  Unit x;
  x.j = -1;
  int n = 0, end = 0;
  x.s = u;
  if (!a.query_start) {
    x.row0 = u;
    x.L = a.context_lens[u];
  } else {
    int lo = 0, hi = a.S;
    if (STEP && u < a.S && a.query_start[u] == u && a.query_start[u + 1] == u + 1) lo = u, hi = u + 1;  // a decode step's rows
    while (hi - lo > 32) {
      const int step = (hi - lo + 31) >> 5, s = lo + lane * step;
      const unsigned upto = __ballot_sync(kAll, s < hi && first_unit_of<STEP>(a, s, a.query_start[min(s, a.S)]) <= u);
      lo += max(0, __popc(upto) - 1) * step;
      hi = min(hi, lo + step);
    }
    const int s = min(lo + lane, a.S - 1), row0 = a.query_start[s], L = a.context_lens[s];
    end = a.query_start[s + 1];
    const unsigned upto = __ballot_sync(kAll, lo + lane < hi && first_unit_of<STEP>(a, s, row0) <= u);
    const int f = max(0, __popc(upto) - 1);
    x.s = min(lo + f, a.S - 1);
    x.row0 = __shfl_sync(kAll, row0, f);
    x.L = __shfl_sync(kAll, L, f);
    end = __shfl_sync(kAll, end, f);
  }
  n = new_tokens(a, x.L, x.row0, end);
  if (n <= 0) return x;
  x.first = x.L - n;
  const int i = u - first_unit_of<STEP>(a, x.s, x.row0);
  if (STEP) {
    const int token = x.first + i;
    if (i >= 0 && i < n && (i == 0 || (token & (a.B - 1)) == 0)) x.j = token >> a.log2_B;
  } else {
    const int j = (x.first >> a.log2_B) + i;
    if (i >= 0 && j <= (x.L - 1) >> a.log2_B) x.j = j;
  }
  return x;
}

// How new elements whose largest magnitude has the bits `top` are coded in a frame; `begun`: it holds earlier tokens, with step `was`.
struct Coding {
  float r, step;
  int halvings;
  bool sound;
};
template <typename T>
__device__ __forceinline__ Coding coding(uint32_t top, bool begun, float was) {
  Coding x;
  x.r = 0.f;
  x.step = __uint_as_float(0x7fffffffu);
  x.halvings = 0;
  const float largest = fminf(fmaxf(Bits<T>::value(top), kLeast), kMost);
  // an earlier step that no append leaves is as good as NaN
  x.sound = top < Bits<T>::kInf && (!begun || (was >= 0x1p-67f && was <= 0x1p60f));
  if (!x.sound) return x;
  if (!begun) {
    x.r = __uint_as_float(__float_as_uint(__fdiv_rn(127.f, largest)) & 0xffff0000u);
    x.step = __frcp_rn(x.r);
    return x;
  }
  const uint32_t inv = __float_as_uint(__frcp_rn(was));
  x.r = __uint_as_float((inv + 0x7fffu + ((inv >> 16) & 1u)) & 0xffff0000u);  // to 8 bits: the r that step is one over
  const float over = largest * x.r;
  x.halvings = max(0, static_cast<int>(__float_as_uint(over) >> 23) - 133);  // over / 2^halvings is below 128
  if (__uint_as_float(__float_as_uint(over) - (static_cast<uint32_t>(x.halvings) << 23)) > 127.f) ++x.halvings;
  x.r = __uint_as_float(__float_as_uint(x.r) - (static_cast<uint32_t>(x.halvings) << 23));
  x.step = __uint_as_float(__float_as_uint(was) + (static_cast<uint32_t>(x.halvings) << 23));
  return x;
}
__device__ __forceinline__ float power_of_half(int k) { return __uint_as_float(static_cast<uint32_t>(127 - min(k, 30)) << 23); }

__device__ __forceinline__ uint32_t larger(uint32_t top2, const uint4& w) {  // of magnitudes as bits, two at a time
  return __vmaxu2(top2, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
}
template <typename T>
__device__ __forceinline__ uint2 codes8(uint4 w, const Coding& x, bool past_most) {
  if (!x.sound) return make_uint2(0x80808080u, 0x80808080u);
  float2 f[4] = {Bits<T>::unpack(w.x), Bits<T>::unpack(w.y), Bits<T>::unpack(w.z), Bits<T>::unpack(w.w)};
  if (Bits<T>::kPastMost && past_most) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = make_float2(fminf(fmaxf(f[k].x, -kMost), kMost), fminf(fmaxf(f[k].y, -kMost), kMost));
  }
  return make_uint2(codes4(f[0], f[1], x.r), codes4(f[2], f[3], x.r));
}
__device__ __forceinline__ void halve8(unsigned char* at, float p) {
  uint2 y = *reinterpret_cast<const uint2*>(at);
  y.x = halved4(y.x, p);
  y.y = halved4(y.y, p);
  *reinterpret_cast<uint2*>(at) = y;
}

// Items of one frame (a cache and a head each, keys before values): those of this block's warps where it is the frame's `part`-th.
template <typename T, int D>
__device__ __forceinline__ void append_items(const Append8Args& a, const Unit& x, int part, uint32_t* maxima) {
  constexpr int V = D / 8, kRows = 32 / V, kSteps = 16 / kRows;  // lanes of a row, rows a step, steps of 16 rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / V, vec = lane % V;
  const int item = part * (blockDim.x >> (5 + a.log2_slabs)) + (warp >> a.log2_slabs), slab = warp & ((1 << a.log2_slabs) - 1);
  const bool is_v = item >= a.H;
  const int h = is_v ? item - a.H : item;
  bool live = h < a.H;
  const int begin = x.j << a.log2_B;  // the frame's first token
  const int at = slab * 16 + sub;      // this lane's first row of it
  const int past = min(a.B, x.L - begin), from = max(0, x.first - begin);  // its rows from .. past - 1 are new
  const int frame = live ? a.block_tables[x.s * a.bt_row + x.j] : 0;

  uint4 w[kSteps];
  const T* src = static_cast<const T*>(is_v ? a.v_new : a.k_new) + (x.row0 + static_cast<int64_t>(begin) + at - x.first) * (is_v ? a.v_row : a.k_row) +
                 static_cast<int64_t>(h) * D + vec * 8;
  const int64_t step_row = kRows * (is_v ? a.v_row : a.k_row);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = at + i * kRows;
    w[i] = make_uint4(0, 0, 0, 0);
    if (live && row >= from && row < past) w[i] = *reinterpret_cast<const uint4*>(src + i * step_row);
  }
  if (live && (frame < 0 || frame >= a.num_blocks)) {
    if (lane == 0) atomicOr(a.status, kDevBadBlock);
    live = false;
  }
  float* step_at = (is_v ? a.v_scale : a.k_scale) + (live ? frame * (is_v ? a.vs_row : a.ks_row) + h : 0);
  const float was = live && from > 0 ? *step_at : 0.f;
  __syncwarp();  // each lane has the old step before one writes the new

  // the largest magnitude, as the bits of T: those of an infinity or more once an element is not finite
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) top2 = larger(top2, w[i]);
  uint32_t top = __reduce_max_sync(kAll, max(top2 & 0xffffu, top2 >> 16));
  if (a.log2_slabs > 0) {
    if (lane == 0) maxima[warp] = top;
    __syncthreads();  // (also: each warp has the old step before one writes the new)
    for (int i = 0; i < 1 << a.log2_slabs; ++i) top = max(top, maxima[(warp & ~((1 << a.log2_slabs) - 1)) + i]);
  }
  if (!live) return;

  const Coding c = coding<T>(top, from > 0, was);
  unsigned char* dst = (is_v ? a.v_cache : a.k_cache) + ((static_cast<int64_t>(frame) * a.H + h) * a.B + at) * D + vec * 8;
  const bool past_most = Bits<T>::value(top) > kMost;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = at + i * kRows;
    if (row >= from && row < past) *reinterpret_cast<uint2*>(dst + i * kRows * D) = codes8<T>(w[i], c, past_most);
  }
  if (c.halvings > 0) {
    const float p = power_of_half(c.halvings);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (at + i * kRows < from) halve8(dst + i * kRows * D, p);
  }
  if (slab == 0 && lane == 0 && (from == 0 || c.halvings > 0 || !c.sound)) *step_at = c.step;
}

// One new token in its frame, as in a decode step: a row of each head is all there is, so a warp takes kStepRows * 32 / V of
// them (64 tokens of 32 heads: 4.4 us with a warp a head).
constexpr int kStepRows = 4;
template <typename T, int D>
__device__ __forceinline__ void append_token(const Append8Args& a, const Unit& x, int part) {
  constexpr int V = D / 8, kRows = 32 / V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / V, vec = lane % V;
  if (warp >= kThreads / 32) return;  // (blocks are larger for frames of more than 64 tokens)
  const int first = (part * (kThreads / 32) + warp) * kRows * kStepRows + sub;  // this lane's first row, keys' before values'
  const int begin = x.j << a.log2_B, at = x.first - begin;
  const int frame = a.block_tables[x.s * a.bt_row + x.j];
  uint4 w[kStepRows];
  float was[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = first + i * kRows;
    const bool is_v = row >= a.H;
    const T* src = is_v ? static_cast<const T*>(a.v_new) + x.row0 * a.v_row : static_cast<const T*>(a.k_new) + x.row0 * a.k_row;
    w[i] = make_uint4(0, 0, 0, 0);
    if (row < 2 * a.H) w[i] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(is_v ? row - a.H : row) * D + vec * 8);
  }
  if (frame < 0 || frame >= a.num_blocks) {
    if (lane == 0) atomicOr(a.status, kDevBadBlock);
    return;
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = first + i * kRows;
    was[i] = 0.f;
    if (at > 0 && row < 2 * a.H) was[i] = row >= a.H ? a.v_scale[frame * a.vs_row + row - a.H] : a.k_scale[frame * a.ks_row + row];
  }
  __syncwarp();  // each lane has the old steps before one writes the new
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = first + i * kRows;
    uint32_t top = larger(0, w[i]);
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 1; o < V; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
    if (row >= 2 * a.H) continue;
    const bool is_v = row >= a.H;
    const int h = is_v ? row - a.H : row;
    const Coding c = coding<T>(top, at > 0, was[i]);
    unsigned char* rows = (is_v ? a.v_cache : a.k_cache) + (static_cast<int64_t>(frame) * a.H + h) * a.B * D + vec * 8;
    *reinterpret_cast<uint2*>(rows + at * D) = codes8<T>(w[i], c, Bits<T>::value(top) > kMost);
    if (c.halvings > 0) {
      const float p = power_of_half(c.halvings);
#pragma unroll 4
      for (int e = 0; e < at; ++e) halve8(rows + e * D, p);
    }
    if (vec == 0 && (at == 0 || c.halvings > 0 || !c.sound))
      (is_v ? a.v_scale + frame * a.vs_row : a.k_scale + frame * a.ks_row)[h] = c.step;
  }
}

// STEP: as many blocks a frame as append_token needs; a frame with more new tokens than one takes its items in turn.
template <typename T, int D, bool STEP>
__global__ void __launch_bounds__(512, 2) append8_kernel(const Append8Args a) {
  __shared__ uint32_t maxima[16];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int u = blockIdx.x / a.blocks_unit, part = blockIdx.x - u * a.blocks_unit;
  if (threadIdx.x < 32) {
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x; s < a.S; s += static_cast<int64_t>(gridDim.x) * 32) {
      const int row0 = a.query_start ? a.query_start[s] : static_cast<int>(s);
      if (new_tokens(a, a.context_lens[s], row0, a.query_start ? a.query_start[s + 1] : 0) < 0) atomicOr(a.status, kDevBadLen);
    }
  }
  const Unit x = find_unit<STEP>(a, u, threadIdx.x & 31);
  if (x.j < 0) return;  // (the whole block)
  if (!STEP) {
    append_items<T, D>(a, x, part, maxima);
  } else if (min((x.j + 1) << a.log2_B, x.L) - max(x.j << a.log2_B, x.first) == 1 && x.first >= x.j << a.log2_B) {
    append_token<T, D>(a, x, part);
  } else {
    const int items = blockDim.x >> (5 + a.log2_slabs);
    for (int i = part; i * items < 2 * a.H; i += a.blocks_unit) {
      append_items<T, D>(a, x, i, maxima);
      __syncthreads();  // the maxima are read
    }
  }
}

// A warp per token, cache and kSteps * 32 / V heads; a lane reads 8 bytes and writes 16.
constexpr int kReadSteps = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read8_kernel(const Read8Args a) {
  constexpr int V = D / 8, kAtOnce = 32 / V;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, sub = lane / V, vec = lane % V;
  const unsigned job = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), chunks = a.chunks;
  if (job >= 2 * chunks * a.T) return;
  const int t = static_cast<int>(job / (2 * chunks));
  int part = static_cast<int>(job - t * 2 * chunks);
  const bool is_v = part >= static_cast<int>(chunks);
  if (is_v) part -= chunks;
  const int h0 = part * kAtOnce * kReadSteps + sub;
  const int32_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (lane == 0) atomicOr(a.status, kDevBadSlot);
    return;
  }
  const int frame = slot >> a.log2_B;
  const unsigned char* src = (is_v ? a.v_cache : a.k_cache) + ((static_cast<int64_t>(frame) * a.H + h0) * a.B + (slot & (a.B - 1))) * D + vec * 8;
  const float* steps = (is_v ? a.v_scale : a.k_scale) + frame * (is_v ? a.vs_row : a.ks_row) + h0;
  T* dst = static_cast<T*>(is_v ? a.v_out : a.k_out) + t * (is_v ? a.vo_row : a.ko_row) + static_cast<int64_t>(h0) * D + vec * 8;
  uint2 w[kReadSteps];
  float step[kReadSteps];
#pragma unroll
  for (int i = 0; i < kReadSteps; ++i) {
    if (h0 + i * kAtOnce >= a.H) continue;
    w[i] = *reinterpret_cast<const uint2*>(src + static_cast<int64_t>(i * kAtOnce) * a.B * D);
    step[i] = steps[i * kAtOnce];
  }
#pragma unroll
  for (int i = 0; i < kReadSteps; ++i) {
    if (h0 + i * kAtOnce >= a.H) continue;
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // 2^23 + byte, exactly
      const uint32_t v = k < 2 ? w[i].x : w[i].y;
      const float f0 = __uint_as_float(__byte_perm(v, 0x4b000000u, k & 1 ? 0x7442 : 0x7440)) - 8388736.f;
      const float f1 = __uint_as_float(__byte_perm(v, 0x4b000000u, k & 1 ? 0x7443 : 0x7441)) - 8388736.f;
      y[k] = Bits<T>::pack(f0 * step[i], f1 * step[i]);
    }
    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i * kAtOnce) * D) = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

cudaError_t launch_pdl(const void* fn, unsigned grid, unsigned threads, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

// Threads of a block: 16 rows a warp, and a frame's in one block.
static int64_t append8_threads(int64_t B) { return B / 16 * 32 > kThreads ? B / 16 * 32 : kThreads; }

bool append8_fits(Append8Args* a) {
  a->log2_slabs = a->B > 16 ? a->log2_B - 4 : 0;
  a->step = a->T <= a->S;
  const int64_t threads = append8_threads(a->B);
  const int64_t rows = 32 / (a->D / 8) * kStepRows;  // of a warp of append_token
  const int64_t items = a->step ? kThreads / 32 * rows : threads / 32 >> a->log2_slabs;
  const int64_t blocks = (2 * static_cast<int64_t>(a->H) + items - 1) / items;
  // (a sequence's new tokens are in at most a B-th as many frames and two)
  const int64_t units = a->step ? a->T : a->T / a->B + 2 * static_cast<int64_t>(a->S);
  if (a->T / a->B + 2 * static_cast<int64_t>(a->S) > 1 << 25 || units > 1 << 25 || units * blocks > INT32_MAX) return false;
  a->units = static_cast<int32_t>(units);
  a->blocks_unit = static_cast<int32_t>(blocks);
  return true;
}

template <typename T>
static const void* append8_function(const Append8Args& a) {
  if (a.D == 128)
    return a.step ? reinterpret_cast<const void*>(&append8_kernel<T, 128, true>) : reinterpret_cast<const void*>(&append8_kernel<T, 128, false>);
  return a.step ? reinterpret_cast<const void*>(&append8_kernel<T, 64, true>) : reinterpret_cast<const void*>(&append8_kernel<T, 64, false>);
}

cudaError_t launch_append8(int dtype, const Append8Args& a, cudaStream_t stream) {
  void* args[1] = {const_cast<Append8Args*>(&a)};
  const void* fn = dtype == PA_F16 ? append8_function<__half>(a) : append8_function<__nv_bfloat16>(a);
  return launch_pdl(fn, static_cast<unsigned>(a.units) * a.blocks_unit, static_cast<unsigned>(append8_threads(a.B)), args, stream);
}

bool read8_fits(Read8Args* a) {
  const int64_t per = 32 / (a->D / 8) * kReadSteps, chunks = (a->H + per - 1) / per;
  a->chunks = static_cast<int32_t>(chunks);
  return 2 * chunks * a->T <= INT32_MAX;
}

cudaError_t launch_read8(int dtype, const Read8Args& a, cudaStream_t stream) {
  void* args[1] = {const_cast<Read8Args*>(&a)};
  const void* fn = dtype == PA_F16 ? (a.D == 128 ? reinterpret_cast<const void*>(&read8_kernel<__half, 128>)
                                                 : reinterpret_cast<const void*>(&read8_kernel<__half, 64>))
                                   : (a.D == 128 ? reinterpret_cast<const void*>(&read8_kernel<__nv_bfloat16, 128>)
                                                 : reinterpret_cast<const void*>(&read8_kernel<__nv_bfloat16, 64>));
  const int64_t jobs = 2 * static_cast<int64_t>(a.chunks) * a.T;
  return launch_pdl(fn, static_cast<unsigned>((jobs + kThreads / 32 - 1) / (kThreads / 32)), kThreads, args, stream);
}

}  // namespace pa
