// Bounds of the keys of each frame, and the frames that a score from them selects.
//
// bounds[frame][h][0 / 1][d] = min / max over the frame's tokens of k[d].  For a query q and any
// key k of the frame, q . k <= sum_d max(q_d min_d, q_d max_d): the frame's score.
//
// The bounds and the scores read memory once and compute little: both give consecutive ranges
// of their (sequence, frame, head) units to resident warps, found from the lengths on the
// device, and keep several 16-byte loads or copies a lane in flight.  The selection holds a list's
// ranks in registers, finds the K-th's neighbourhood with one histogram over the scores' range, and
// orders the few that share its bin.
//
// Measured: bounds of 16 prompts of 4096 tokens, 8 heads of 128 in bf16, frames of 32 (143 MB): 25.9 us, 5.5 TB/s;
// of the tail frames of 64 sequences 4.5 us.  Selection of 64 from 1024 frames for 4 x 32 heads (67 MB of bounds, in
// 512-byte pieces): 18.6 us; for 32 sequences of 100 to 65,536 tokens with 8 heads of 4 queries (43 MB): 20.3 us,
// bound by the instructions of four queries a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_internal.h"
#include "pair32.cuh"
#include "ranges.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ bool bad_len(int L, int max_blocks, int B) {
  return L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(max_blocks) * B;
}

__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Where unit x lies when sequence s has count(s) * per units: its sequence, and the unit's number in it.
// Every lane of the warp calls it; x < the total.  Units are numbered in int32 over the whole batch.
template <typename Count>
__device__ __forceinline__ int find_unit(int S, int per, int x, int lane, Count count, int* rest) {
  int before = 0;
  for (int s0 = 0; s0 < S; s0 += 32) {
    const int n = s0 + lane < S ? count(s0 + lane) : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned past = __ballot_sync(kAll, before + upto * per > x);
    if (past) {
      const int f = __ffs(past) - 1;
      *rest = x - before - (__shfl_sync(kAll, upto, f) - __shfl_sync(kAll, n, f)) * per;
      return s0 + f;
    }
    before += __shfl_sync(kAll, upto, 31) * per;
  }
  return -1;
}
template <typename Count>
__device__ __forceinline__ int all_units(int S, int per, int lane, Count count) {
  int total = 0;
  for (int s0 = 0; s0 < S; s0 += 32) total += __reduce_add_sync(kAll, s0 + lane < S ? count(s0 + lane) : 0);
  return total * per;
}
template <typename T2>
__device__ __forceinline__ uint32_t bits(T2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
template <typename T2>
__device__ __forceinline__ T2 pair_of(uint32_t x) { return *reinterpret_cast<const T2*>(&x); }

// ---- bounds -----------------------------------------------------------------------------------------
// A unit is one frame of one head: its rows, 32 * 8 / D at a time, as 16-byte vectors.  More units than warps: 25.9 us for
// the prompts where a range each took 27.2; the units of a step spread over all SMs: 4.5 us, by blocks 5.2.
constexpr int kBoundsWarps = 8;

template <typename T2, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(const BoundsArgs a) {
  constexpr int kRowLanes = D / 8, kRows = 32 / kRowLanes, kAhead = 8;
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int sub = lane / kRowLanes, vec = lane % kRowLanes;
  auto count = [&](int s) {  // frames to look at
    const int L = a.context_lens[s], first = a.first ? a.first[s] : 0;
    return bad_len(L, a.max_blocks, a.B) || first < 0 || first >= L ? 0 : (L + a.B - 1) / a.B - first / a.B;
  };
  const int total = all_units(a.S, a.H, lane, count);
  const int warps = gridDim.x * kBoundsWarps;
  const int id = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  if (id < a.S) {  // bad lengths are reported by one warp each
    for (int64_t s = id; s < a.S; s += warps)
      if (lane == 0 && (bad_len(a.context_lens[s], a.max_blocks, a.B) || (a.first && a.first[s] < 0)))
        atomicOr(a.status, kDevBadLen);
  }
  int x0, x1;
  if (total <= warps) {  // one each, over all SMs
    x0 = id, x1 = min(id + 1, total);
  } else {  // a range a block, its warps on neighbouring heads of a frame: together they read whole rows of tokens
    x0 = first_unit(total, gridDim.x, blockIdx.x), x1 = first_unit(total, gridDim.x, blockIdx.x + 1);
    const int warp = threadIdx.x >> 5;
    if (x1 - x0 <= warp) return;  // x0 + warp may pass int32
    x0 += warp;
  }
  if (x0 >= x1) return;
  int rest;
  int s = find_unit(a.S, a.H, x0, lane, count, &rest);
  int left = count(s) - rest / a.H, h = rest % a.H;
  int L = a.context_lens[s];
  int j = (L + a.B - 1) / a.B - left;
  for (int x = x0; x < x1; x += kBoundsWarps) {
    const int frame = a.block_tables[s * a.bt_row + j];
    if (frame < 0 || frame >= a.num_blocks) {
      if (lane == 0) atomicOr(a.status, kDevBadBlock);
    } else {
      const int n = min(a.B, L - j * a.B);
      const uint4* k = static_cast<const uint4*>(a.k_cache) + (static_cast<int64_t>(frame) * a.B * a.H + h) * kRowLanes + vec;
      const int64_t row = static_cast<int64_t>(a.H) * kRowLanes;
      T2 lo[4], hi[4];
      for (int i0 = 0; i0 < n; i0 += kAhead * kRows) {
        uint4 u[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) u[i] = __ldg(k + min(i0 + i * kRows + sub, n - 1) * row);  // the last row again behind it
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const T2 y = pair_of<T2>(w[v]);
            lo[v] = i0 == 0 && i == 0 ? y : __hmin2(lo[v], y);
            hi[v] = i0 == 0 && i == 0 ? y : __hmax2(hi[v], y);
          }
        }
      }
#pragma unroll
      for (int o = kRowLanes; o < 32; o <<= 1)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          lo[v] = __hmin2(lo[v], __shfl_xor_sync(kAll, lo[v], o));
          hi[v] = __hmax2(hi[v], __shfl_xor_sync(kAll, hi[v], o));
        }
      if (sub < 2) {  // the row's first lanes store the minima, the next the maxima
        uint32_t y[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = sub == 0 ? bits(lo[v]) : bits(hi[v]);
        static_cast<uint4*>(a.bounds)[((static_cast<int64_t>(frame) * a.H + h) * 2 + sub) * kRowLanes + vec] =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
    if (x1 - x <= kBoundsWarps) break;
    for (h += kBoundsWarps; h >= a.H; h -= a.H) {
      ++j;
      if (--left == 0) {
        do left = count(++s);
        while (left == 0);
        L = a.context_lens[s];
        j = (L + a.B - 1) / a.B - left;
      }
    }
  }
}

// ---- scores -----------------------------------------------------------------------------------------
// A unit is kRows * kAhead consecutive frames of one (sequence, head): a bounds row is D / 8 lanes, kRows
// frames lie side by side in a warp and kAhead deep.  Lanes copy their own 16 bytes of the next units to
// shared memory while they use this one's, so that what is on its way takes no registers and no barrier.  With q split
// into its positive and negative part (in shared memory) one product is zero and the other exact,
// so x_d = max(q_d min_d, q_d max_d) comes from a product and a fused multiply-add, for two elements in one
// instruction.  The order of the sum is a tree: eight elements in a lane (neighbours, their sums, the two
// halves), then lanes by xor 1, 2, 4, ...; the four frames of a lane are reduced together, each lane passing on half
// of what it holds, which adds the same pairs.  kQueries queries at a time; more queries read the unit's rows again from
// shared memory and their own numbers from the cache.
//
// Units on their way and blocks an SM, both kernels of a selection, 4 x 32 heads of 1024 frames and 32 x 8 heads of up to
// 2048: one query 4 and 3 (18.6, 16.7 us; 3 and 4: 18.3, 19.8, where the selection's blocks no longer fit beside
// them and start late; through registers 20.8, 18.1); two 5 and 2 (21.3, 18.7; 3 and 3 20.8, 19.6); four 2 and 3
// (22.4, 20.3; 4 and 2 25.2, 22.0; through registers 24.8, 21.0; one element an instruction 25.3, 24.6).
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 2 && __is_same(T, __half)) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ bool scored(const SelectArgs& a, int blocks) { return blocks > a.K; }

constexpr int kScoreWarps = 4;

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {  // zeros where not live
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}

// Where a warp is in the batch's units: a head's unit of a sequence that has `units` of them.
struct ScoreAt {
  int s, h, unit, units, blocks;
};

template <int D, int kQueries>
struct ScoreSmem {
  static constexpr int kRowLanes = D / 8, kAhead = 4;
  static constexpr int kStages = kQueries == 1 ? 4 : kQueries == 2 ? 5 : 2;
  static constexpr int kBlocks = kQueries == 2 ? 2 : 3;  // an SM
  uint4 rows[kScoreWarps][kStages][kAhead][2][32];  // each lane's 16 bytes of minima and of maxima
  // positive part of the queries (two vectors a lane), negative part, in pairs (e, e + 4)
  float4 q[kScoreWarps][kQueries][4][kRowLanes];
};

template <typename T, int D, int kQueries>
__global__ void __launch_bounds__(kScoreWarps * 32, 3) score_kernel(const SelectArgs a) {
  constexpr int kRowLanes = D / 8, kRows = 32 / kRowLanes, kAhead = 4, kUnit = kRows * kAhead;
  constexpr int kStages = ScoreSmem<D, kQueries>::kStages;
  extern __shared__ __align__(16) unsigned char smem[];
  ScoreSmem<D, kQueries>& sm = *reinterpret_cast<ScoreSmem<D, kQueries>*>(smem);
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kRowLanes, vec = lane % kRowLanes;
  auto count = [&](int s) {
    const int L = a.context_lens[s];
    const int blocks = bad_len(L, a.max_blocks, a.B) ? 0 : (L + a.B - 1) / a.B;
    return scored(a, blocks) ? (blocks + kUnit - 1) / kUnit : 0;
  };
  const int total = all_units(a.S, a.H, lane, count);
  const int warps = gridDim.x * kScoreWarps;
  const int id = warp * gridDim.x + blockIdx.x;
  const int workers = min(warps, total);
  if (id >= workers) return;
  const int x0 = first_unit(total, workers, id), x1 = first_unit(total, workers, id + 1);
  int rest;
  ScoreAt now;
  now.s = find_unit(a.S, a.H, x0, lane, count, &rest);
  now.units = count(now.s);
  now.h = rest / now.units, now.unit = rest % now.units;
  now.blocks = (a.context_lens[now.s] + a.B - 1) / a.B;
  ScoreAt then = now;  // of the next copies
  auto advance = [&](ScoreAt& at) {  // not behind the last unit
    if (++at.unit < at.units) return;
    at.unit = 0;
    if (++at.h == a.H) {
      at.h = 0;
      do at.units = count(++at.s);
      while (at.units == 0);
      at.blocks = (a.context_lens[at.s] + a.B - 1) / a.B;
    }
  };
  float4 (*qs)[4][kRowLanes] = sm.q[warp];
  auto load_q = [&](const T* base, int g0) {  // base: the head's first query
    __syncwarp();
    for (int g = sub; g < kQueries; g += kRows) {
      // a query behind the group's last is its last again: the largest score stays
      const T* q = base + min(g0 + g, a.g - 1) * D;
      float f[8];
      unpack8<T>(__ldg(reinterpret_cast<const uint4*>(q) + vec), f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[g][i][vec] = make_float4(fmaxf(f[2 * i], 0.f), fmaxf(f[2 * i + 4], 0.f), fmaxf(f[2 * i + 1], 0.f), fmaxf(f[2 * i + 5], 0.f));
        qs[g][2 + i][vec] = make_float4(fminf(f[2 * i], 0.f), fminf(f[2 * i + 4], 0.f), fminf(f[2 * i + 1], 0.f), fminf(f[2 * i + 5], 0.f));
      }
    }
    __syncwarp();
  };
  // 32 of the sequence's block ids, a lane each, read a unit before they are used
  int frame;
  auto read_ids = [&]() {
    const int j = (then.unit * kUnit & ~31) + lane;
    frame = j < then.blocks ? a.block_tables[then.s * a.bt_row + j] : -1;
  };
  // copies of the next unit's rows, and whether each of its frames has a good id
  auto copy = [&](int x, int stage) {
    uint32_t good = 0;
    if (x < x1) {
      const int j0 = then.unit * kUnit;
      if ((j0 & ~31) + lane < then.blocks && (frame < 0 || frame >= a.num_blocks)) {
        atomicOr(a.status, kDevBadBlock);
        frame = -1;
      }
      good = __ballot_sync(kAll, frame >= 0) >> (j0 & 31);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int f = __shfl_sync(kAll, frame, (j0 + i * kRows + sub) & 31);
        const uint4* b = static_cast<const uint4*>(a.bounds) + (static_cast<int64_t>(max(f, 0)) * a.H + then.h) * 2 * kRowLanes + vec;
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&sm.rows[warp][stage][i][0][lane]));
        copy16(to, b, f >= 0);
        copy16(to + 32 * 16, b + kRowLanes, f >= 0);
      }
      if (x + 1 < x1) {
        advance(then);
        if (then.unit == 0 || (then.unit * kUnit & 31) == 0) read_ids();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return good;
  };
  read_ids();
  uint32_t goods[kStages - 1];
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) goods[k] = copy(x0 + k, k);
  int stage = 0, ahead = kStages - 1;
  bool fresh = true;
  for (int x = x0; x < x1; ++x) {
    const T* its_q = static_cast<const T*>(a.q) + now.s * a.q_row + static_cast<int64_t>(now.h) * a.g * D;
    if (fresh && a.g <= kQueries) load_q(its_q, 0);
    const uint32_t good = goods[0];
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) goods[k] = goods[k + 1];
    goods[kStages - 2] = copy(x + kStages - 1, ahead);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");  // a lane reads what it has copied itself
    const uint4 (*rows)[2][32] = sm.rows[warp][stage];
    float best = -INFINITY;
    for (int g0 = 0; g0 < a.g; g0 += kQueries) {
      if (a.g > kQueries) load_q(its_q, g0);
      float y[kQueries][kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float l8[8], h8[8];
        unpack8<T>(rows[i][0][lane], l8);
        unpack8<T>(rows[i][1][lane], h8);
#pragma unroll
        for (int g = 0; g < kQueries; ++g) {
          uint64_t t[4];  // elements (e, e + 4)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(&qs[g][e / 2][vec]), n = *reinterpret_cast<const ulonglong2*>(&qs[g][2 + e / 2][vec]);
            t[e] = fma2(n.x, pair(l8[e], l8[e + 4]), mul2(p.x, pair(h8[e], h8[e + 4])));
            t[e + 1] = fma2(n.y, pair(l8[e + 1], l8[e + 5]), mul2(p.y, pair(h8[e + 1], h8[e + 5])));
          }
          const float2 z = both(add2(add2(t[0], t[1]), add2(t[2], t[3])));
          y[g][i] = __fadd_rn(z.x, z.y);
        }
      }
#pragma unroll
      for (int g = 0; g < kQueries; ++g) {
        // lane bits 0 and 1 choose which of the four frames a lane ends with
        const bool b0 = lane & 1, b1 = lane & 2;
        const float k0 = b0 ? y[g][1] : y[g][0], k1 = b0 ? y[g][3] : y[g][2];
        const float p0 = b0 ? y[g][0] : y[g][1], p1 = b0 ? y[g][2] : y[g][3];
        const float z0 = __fadd_rn(k0, __shfl_xor_sync(kAll, p0, 1)), z1 = __fadd_rn(k1, __shfl_xor_sync(kAll, p1, 1));
        float z = __fadd_rn(b1 ? z1 : z0, __shfl_xor_sync(kAll, b1 ? z0 : z1, 2));
#pragma unroll
        for (int o = 4; o < kRowLanes; o <<= 1) z = __fadd_rn(z, __shfl_xor_sync(kAll, z, o));
        best = fmaxf(best, z);
      }
    }
    const int at = (lane & 3) * kRows + sub;  // frame (b1, b0) = step 2 b1 + b0
    const int j = now.unit * kUnit + at;
    if ((vec & ~3) == 0 && j < now.blocks)
      a.scores[(static_cast<int64_t>(now.s) * a.H + now.h) * a.max_blocks + j] = good >> at & 1 ? best : -INFINITY;
    if (x + 1 < x1) advance(now);
    fresh = now.unit == 0;
    stage = stage + 1 < kStages ? stage + 1 : 0;
    ahead = ahead + 1 < kStages ? ahead + 1 : 0;
  }
}

// ---- selection --------------------------------------------------------------------------------------
// Numbers whose unsigned order is the order of the scores (-0 as 0); frames that are always kept come above
// all others.
__device__ __forceinline__ uint32_t rank_of(const SelectArgs& a, float score, int j, int blocks) {
  if (j < a.keep_first || j >= blocks - a.keep_last) return 0xffffffffu;
  const uint32_t u = __float_as_uint(__fadd_rn(score, 0.f));
  return max(u & 0x80000000u ? ~u : u | 0x80000000u, 1u);  // 0 is no frame's, not even one with a NaN score
}

__device__ __forceinline__ float score_of(uint32_t rank) {
  return __uint_as_float(rank & 0x80000000u ? rank & 0x7fffffffu : ~rank);
}

// Sum over the block of a value per thread before this one, and over all threads (64-bit: two counts side by side).
template <int kWarpsOf>
__device__ __forceinline__ uint64_t block_before(uint64_t own, uint64_t* total, uint64_t (&sums)[kWarpsOf]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  uint64_t all = lane < kWarpsOf ? sums[lane] : 0, before = 0;
#pragma unroll
  for (int o = 1; o < kWarpsOf; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kAll, all, o);
    if (lane >= o) all += y;
  }
  before = __shfl_sync(kAll, all, (warp + 31) & 31);
  *total = __shfl_sync(kAll, all, kWarpsOf - 1);
  return upto - own + (warp ? before : 0);
}

// One block per (sequence, head).  Thread t holds the ranks of frames t * R .. t * R + R - 1 in registers, so
// that thread order is frame order; lists longer than kThreads * R frames (LONG) are read again for each
// count.
//
// The kept frames are above all others.  The scores of the rest are put into bins, four a thread, that split their
// range evenly (a subtraction and a product, both monotonic, so a higher bin holds higher scores only); the
// bin with the last place is found by a scan from the top, all above it are taken, and the
// scores in it, a handful, are ordered by comparing each with each.  Where that does not hold (scores that are
// not finite or all the same, more than kTies of them in the bin, more kept frames than places, LONG), the
// K-th largest rank is found from its top bits down instead: the largest T such that at least K ranks
// are >= T, two bits a step, three counts packed into one sum.  That alone took 15 us for 256 lists of up
// to 2048 frames, all of it counting.
template <int kThreads, int R, bool LONG>
__global__ void __launch_bounds__(kThreads) top_kernel(const SelectArgs a) {
  constexpr int kWarpsOf = kThreads / 32, kBins = 4 * kThreads, kTies = kThreads;
  __shared__ uint64_t sums[2][kWarpsOf];
  __shared__ int4 bins[LONG ? 1 : kThreads];     // bin b at word kBins - 1 - b: a thread's four from the top down
  __shared__ uint2 tied[LONG ? 1 : kTies];       // (rank, frame) of the bin with the last place
  __shared__ uint8_t tied_in[LONG ? 1 : kTies];  // whether it is taken
  __shared__ int edge_bin, edge_need, n_tied;
  __shared__ uint32_t least[kWarpsOf], most[kWarpsOf];
  pdl_begin();
  const int h = blockIdx.x % a.H, s = blockIdx.x / a.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* sel = a.selected + s * a.sel_seq + h * a.sel_head;
  int L = a.context_lens[s];
  if (bad_len(L, a.max_blocks, a.B)) {
    if (threadIdx.x == 0) atomicOr(a.status, kDevBadLen);
    L = 0;
  }
  const int blocks = (L + a.B - 1) / a.B;
  if (!scored(a, blocks)) {
    for (int64_t j = threadIdx.x; j < a.K; j += kThreads) sel[j] = j < blocks ? static_cast<int>(j) : -1;  // K may be INT32_MAX
    for (int j = threadIdx.x; h == 0 && j < blocks; j += kThreads) {  // no score has looked at these
      const int frame = a.block_tables[s * a.bt_row + j];
      if (frame < 0 || frame >= a.num_blocks) atomicOr(a.status, kDevBadBlock);
    }
    return;
  }
  const float* scores = a.scores + (static_cast<int64_t>(s) * a.H + h) * a.max_blocks;
  const int mine = LONG ? (blocks + kThreads - 1) / kThreads : R;  // frames of a thread
  const int j0 = threadIdx.x * mine;
  constexpr uint32_t kKept = 0xffffffffu;
  uint32_t held[R];
  if constexpr (!LONG) {
#pragma unroll
    for (int i = 0; i < R; ++i) held[i] = j0 + i < blocks ? rank_of(a, scores[j0 + i], j0 + i, blocks) : 0;
    // ---- one histogram ----
    uint32_t lo = kKept, hi = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (held[i] != 0 && held[i] != kKept) {
        lo = min(lo, held[i]);
        hi = max(hi, held[i]);
      }
    lo = __reduce_min_sync(kAll, lo);
    hi = __reduce_max_sync(kAll, hi);
    if (lane == 0) {
      least[warp] = lo;
      most[warp] = hi;
    }
    bins[threadIdx.x] = make_int4(0, 0, 0, 0);
    if (threadIdx.x == 0) n_tied = 0;
    __syncthreads();
    lo = __reduce_min_sync(kAll, lane < kWarpsOf ? least[lane] : kKept);
    hi = __reduce_max_sync(kAll, lane < kWarpsOf ? most[lane] : 0);
    const float low = score_of(lo), span = score_of(hi) - low;
    const int kept = min(a.keep_first, blocks) + max(0, min(a.keep_last, blocks - a.keep_first));
    const int places = a.K - kept;  // for the others
    const float scale = kBins / span;
    if (lo < hi && span < INFINITY && scale < INFINITY && places > 0) {  // not so for NaN
      int* words = reinterpret_cast<int*>(bins);
      int word[R];  // of each frame's bin; -1: taken in any case, kBins: no frame
#pragma unroll
      for (int i = 0; i < R; ++i) {
        word[i] = held[i] == 0 ? kBins : held[i] == kKept ? -1 : max(0, kBins - 1 - static_cast<int>((score_of(held[i]) - low) * scale));
        if (word[i] >= 0 && word[i] < kBins) atomicAdd(words + word[i], 1);
      }
      __syncthreads();
      const int4 c = bins[threadIdx.x];
      uint64_t all;
      int left = places - static_cast<int>(block_before<kWarpsOf>(c.x + c.y + c.z + c.w, &all, sums[0]));
      if (left > 0 && left <= c.x + c.y + c.z + c.w) {
        int i = 0;
        if (c.x < left) left -= c.x, ++i;
        if (i == 1 && c.y < left) left -= c.y, ++i;
        if (i == 2 && c.z < left) left -= c.z, ++i;
        edge_bin = 4 * static_cast<int>(threadIdx.x) + i;
        edge_need = left;
      }
      __syncthreads();
      const int edge = edge_bin, need = edge_need;
      uint32_t take = 0;
      uint32_t slot = 0;  // which of this thread's frames are in the edge's bin, and where in `tied` they are
      int first_slot = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        take |= static_cast<uint32_t>(word[i] < edge) << i;
        slot |= static_cast<uint32_t>(word[i] == edge) << i;
      }
      if (slot) {
        first_slot = atomicAdd(&n_tied, __popc(slot));
        int at = first_slot;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (slot >> i & 1) {
            if (at < kTies) tied[at] = make_uint2(held[i], j0 + i);
            ++at;
          }
      }
      __syncthreads();
      const int ties = n_tied;
      if (ties <= kTies) {
        if (static_cast<int>(threadIdx.x) < ties) {
          const uint2 own = tied[threadIdx.x];
          int above = 0;
          for (int k = 0; k < ties; ++k) {
            const uint2 x = tied[k];
            above += x.x > own.x || (x.x == own.x && x.y < own.y);
          }
          tied_in[threadIdx.x] = above < need;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (slot >> i & 1) take |= static_cast<uint32_t>(tied_in[first_slot++]) << i;
        uint64_t total;
        int at = static_cast<int>(block_before<kWarpsOf>(__popc(take), &total, sums[1]));
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (take >> i & 1) sel[at++] = j0 + i;
        return;
      }
    }
  }
  // ---- bit by bit ----
  // calls f(rank, position) for each of this thread's frames; ranks of frames are above 0
  auto each = [&](auto f) {
    if (LONG) {
      for (int i = 0; i < mine && j0 + i < blocks; ++i) f(rank_of(a, scores[j0 + i], j0 + i, blocks), j0 + i);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) f(held[i], j0 + i);
    }
  };
  uint32_t T = 0;
  __syncthreads();
  for (int shift = 30, turn = 0; shift >= 0; shift -= 2, turn ^= 1) {
    const uint32_t step = 1u << shift;
    uint32_t c1 = 0, c2 = 0, c3 = 0;
    each([&](uint32_t r, int) {
      c1 += r >= T + step;
      c2 += r >= T + 2 * step;
      c3 += r >= T + 3 * step;
    });
    c1 = __reduce_add_sync(kAll, c1);
    c2 = __reduce_add_sync(kAll, c2);
    c3 = __reduce_add_sync(kAll, c3);
    // 21 bits a count: tables have at most 2^20 columns
    if (lane == 0) sums[turn][warp] = c1 | static_cast<uint64_t>(c2) << 21 | static_cast<uint64_t>(c3) << 42;
    __syncthreads();
    const uint64_t w = lane < kWarpsOf ? sums[turn][lane] : 0;
    c1 = __reduce_add_sync(kAll, static_cast<uint32_t>(w) & 0x1fffff);
    c2 = __reduce_add_sync(kAll, static_cast<uint32_t>(w >> 21) & 0x1fffff);
    c3 = __reduce_add_sync(kAll, static_cast<uint32_t>(w >> 42));
    const uint32_t K = a.K, hits = c3 >= K ? c3 : c2 >= K ? c2 : c1 >= K ? c1 : 0;
    T += c3 >= K ? 3 * step : c2 >= K ? 2 * step : c1 >= K ? step : 0;
    if (hits == K) {  // exactly K ranks from T on: they are the ranks above T - 1, whatever its other digits
      --T;
      break;
    }
  }
  // above T: all; equal to T: the first K - above
  uint32_t above = 0, equal = 0;
  each([&](uint32_t r, int) {
    above += r > T;
    equal += r == T;
  });
  uint64_t total;
  const uint64_t before = block_before<kWarpsOf>(above | static_cast<uint64_t>(equal) << 32, &total, sums[0]);
  const uint32_t need = a.K - static_cast<uint32_t>(total);
  uint32_t a0 = static_cast<uint32_t>(before), e0 = static_cast<uint32_t>(before >> 32);
  each([&](uint32_t r, int j) {
    if (r > T)
      sel[a0++ + min(e0, need)] = j;
    else if (r == T) {
      if (e0 < need) sel[a0 + e0] = j;
      ++e0;
    }
  });
}

cudaError_t launch_pdl(const void* fn, int64_t grid, int threads, void** args, cudaStream_t stream, int smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <typename F>
const void* ptr(F* f) { return reinterpret_cast<const void*>(f); }

// as many blocks as are resident, at most `most` an SM, and no more than there can be units
cudaError_t launch_resident(const void* fn, int threads, int64_t units, int num_sms, void** args, cudaStream_t stream, int smem = 0,
                            int most = 32) {
  int occ = 0;
  cudaError_t e = kernel_prep(fn, threads, smem, &occ);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  int64_t grid = static_cast<int64_t>(num_sms) * (occ < most ? occ : most);
  if (units < grid) grid = units < 1 ? 1 : units;
  return launch_pdl(fn, grid, threads, args, stream, smem);
}

}  // namespace

cudaError_t launch_block_bounds(int dtype, BoundsArgs a, int num_sms, cudaStream_t stream) {
  const void* fn = dtype == PA_F16 ? (a.D == 128 ? ptr(block_bounds_kernel<__half2, 128>) : ptr(block_bounds_kernel<__half2, 64>))
                                   : (a.D == 128 ? ptr(block_bounds_kernel<__nv_bfloat162, 128>) : ptr(block_bounds_kernel<__nv_bfloat162, 64>));
  void* args[1] = {&a};
  return launch_resident(fn, kBoundsWarps * 32, static_cast<int64_t>(a.S) * a.H * (a.max_blocks < 1 ? 1 : a.max_blocks), num_sms, args, stream);
}

template <typename T, int D, int kQueries>
static const void* score_kernel_of(int* smem, int* blocks) {
  *blocks = ScoreSmem<D, kQueries>::kBlocks;
  *smem = sizeof(ScoreSmem<D, kQueries>);
  return ptr(score_kernel<T, D, kQueries>);
}

template <typename T>
static const void* score_fn(int D, int g, int* smem, int* blocks) {
  if (D == 128) return g == 1 ? score_kernel_of<T, 128, 1>(smem, blocks) : g == 2 ? score_kernel_of<T, 128, 2>(smem, blocks) : score_kernel_of<T, 128, 4>(smem, blocks);
  return g == 1 ? score_kernel_of<T, 64, 1>(smem, blocks) : g == 2 ? score_kernel_of<T, 64, 2>(smem, blocks) : score_kernel_of<T, 64, 4>(smem, blocks);
}

cudaError_t launch_select_blocks(int dtype, SelectArgs a, int num_sms, cudaStream_t stream, int* launched) {
  void* args[1] = {&a};
  *launched = 0;
  if (a.max_blocks > a.K) {
    int smem, blocks;
    const void* fn = dtype == PA_F16 ? score_fn<__half>(a.D, a.g, &smem, &blocks) : score_fn<__nv_bfloat16>(a.D, a.g, &smem, &blocks);
    const cudaError_t e = launch_resident(fn, kScoreWarps * 32, static_cast<int64_t>(a.S) * a.H * ((a.max_blocks + 7) / 8), num_sms, args, stream, smem, blocks);
    if (e != cudaSuccess) return e;
    ++*launched;
  }
  // threads by the longest list that a table can hold: a rank a register, eight a thread
  const int n = a.max_blocks;
  const int64_t lists = static_cast<int64_t>(a.S) * a.H;
  ++*launched;
  if (n <= 1024) return launch_pdl(ptr(top_kernel<128, 8, false>), lists, 128, args, stream);
  if (n <= 2048) return launch_pdl(ptr(top_kernel<256, 8, false>), lists, 256, args, stream);
  if (n <= 4096) return launch_pdl(ptr(top_kernel<512, 8, false>), lists, 512, args, stream);
  if (n <= 16384) return launch_pdl(ptr(top_kernel<1024, 16, false>), lists, 1024, args, stream);
  return launch_pdl(ptr(top_kernel<1024, 16, true>), lists, 1024, args, stream);
}

}  // namespace pa
