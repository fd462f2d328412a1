// Single-query attention over gathered keys: every token of a sequence held in the 4-bit
// cache, or the tokens of listed frames of a 16-bit cache.
//
// For each sequence s and key head h, with the g query heads that share it:
//     out = sum_j w_j v_j / sum_j w_j,   w_j = exp2(q . k_j * scale * log2(e) - m),
// in one pass, m being a running maximum (less 7) that moves only when a score passes it by 2^8.
//
// Work.  A tile is up to four parts of 16 keys of one (s, h): its keys are one copy, its values another,
// and each is loaded again as soon as the warp has read it.  All tiles of the batch, numbered by
// sequence, head and position, are cut into one consecutive range per resident warp, equal to within
// a tile: every warp is its own worker with its own ring of shared-memory stages, and no barrier
// joins the warps of a block before they are done.  The cut follows from the lengths, which each warp
// reads on the device.  A (s, h) that lies in one range is written straight out.  One that is cut leaves
// a partial (max, sum, weighted values) per piece in the workspace, and the warp that brings the arrival
// counter to the number of pieces has its block join them (in groups of 16 where they are many),
// in order, so that results do not depend on timing.  What runs once a warp, the joins above all, is
// kept short in code rather than unrolled: instructions that are not in the cache cost more
// than the loads do (joins unrolled over four queries and sixteen pieces: 102 us for 64
// sequences of 512 .. 2048 tokens where the loop alone takes 87).
//
// Tensor cores (mma.sync m16n8k16): scores are C[16 keys x 8 queries] = K (A operand) times
// q^T (B), and the values O^T[16 elements x 8 queries] += V^T (A) times P (B).  Keys and
// elements, of which there are many, fill the 16 rows; the few queries need only 8 columns.
// P comes out of the score layout by one movmatrix per 8 x 8 and is never in memory.  With
// g <= 4 the queries stand twice, in columns 0..3 and 4..7, and the second copy carries what
// the first one's rounding of the weights to 16 bits left over: the second part is free.
// (tcgen05 takes its operands from shared memory or tensor memory: what codes stand for would have to be
// written there first, for tiles of which 1 to 16 of 128 rows hold a query.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "decode_kernel.cuh"
#include "pa_internal.h"
#include "ranges.h"

namespace pa {
namespace gk {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kGroup = 16;       // pieces of one (s, h) are joined in groups of this many workers
constexpr float kSlack = 8.f;    // how far (log2) a score may pass the running maximum
// Weights are 2^kRoom times what they stand for: at most 2^15, which fp16 holds, and as many more of a long context's small
// ones are above its least number, 2^-24.  (Many keys 2^-24 below one sink were off by half of themselves.)
constexpr float kRoom = 7.f;
constexpr float kLeast = -3.402823466e38f;  // a running maximum of no score yet: finite, so that a score of -inf weighs nothing

// How the second part of the weights gets to the tensor cores: in the second copy of the queries, or as another operand.
enum Parts { kTwinColumns, kTwoParts };

// ---- instructions -----------------------------------------------------------------------------
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 of 16-bit elements, transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

template <typename M>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y) { return as_u32(__floats2half2_rn(x, y)); }
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) { return as_u32(__floats2bfloat162_rn(x, y)); }
template <typename M>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[2]) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[1]) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds(uint32_t addr) {
  uint32_t w;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(addr));
  return w;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// four rows of a two-dimensional tensor, one after the other
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int r0, int r1, int r2, int r3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
      : "memory");
}

// ---- the cursor over a batch's tiles ------------------------------------------------------------
struct Cursor {
  int s, h, t;               // tile t of (s, h)
  int L, blocks, parts, tiles;  // of sequence s
};

__device__ __forceinline__ int checked_len(const GatherArgs& a, int s) {
  const int L = a.context_lens[s];
  return L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks) * a.B ? -1 : L;
}

// Parts of 16 keys of a sequence or list (16 slots of a listed frame, or two frames of 8); at least one.
template <bool SEL>
__device__ __forceinline__ int parts_of(const GatherArgs& a, int L) {
  if (!SEL) return parts16(L);
  const int n = min(a.K, (max(L, 0) + a.B - 1) >> a.log2_B);
  return max(1, a.B >= 16 ? n << (a.log2_B - 4) : (n + 1) >> 1);
}
template <bool SEL, int LOADS>
__device__ __forceinline__ int tiles_of(const GatherArgs& a, int L) {
  return (parts_of<SEL>(a, L) + LOADS - 1) / LOADS;
}

template <bool SEL, int LOADS>
__device__ __forceinline__ void enter_seq(const GatherArgs& a, Cursor& c) {
  const int L = checked_len(a, c.s);
  if (L < 0) atomicOr(a.status, kDevBadLen);
  c.L = max(L, 0);
  c.blocks = (c.L + a.B - 1) >> a.log2_B;
  c.parts = parts_of<SEL>(a, L);
  c.tiles = (c.parts + LOADS - 1) / LOADS;
}

// To the next (s, h).
template <bool SEL, int LOADS>
__device__ __forceinline__ void next_head(const GatherArgs& a, Cursor& c) {
  c.t = 0;
  if (++c.h < a.H) return;
  c.h = 0;
  if (++c.s < a.S) enter_seq<SEL, LOADS>(a, c);
}

// A part of a tile as the producer sees it: 16 keys, two halves of 8, each inside one frame.
struct TilePlan {
  int frame[2];   // < 0: nothing to load
  int row;        // first key's row in its frame (both halves of one frame: row, row + 8)
  int meta;       // keys of the halves (0..8 each) | 1 << 16 for a bad frame id
};

// Where the list of (s, h) ends, as far as it has been read (SEL).
struct List {
  int seen;    // entries read so far
  bool ended;
};

// Table position and frame of entry j of (s, h), one entry per lane: frame -1 bad, -2 none.  `list`: for SEL,
// entries [0, list.seen) have been read; j - lane is at or behind that.
__device__ __forceinline__ int checked_frame(const GatherArgs& a, const Cursor& c, int e) {
  int frame = e >= 0 && e < c.blocks ? a.block_tables[c.s * a.bt_row + e] : -1;
  if (frame < 0 || frame >= a.num_blocks) {
    atomicOr(a.status, kDevBadBlock);
    frame = -1;
  }
  return frame;
}

// Plans of the 32 parts t0 .. t0 + 31 of (s, h), one per lane.
template <bool SEL>
__device__ __forceinline__ TilePlan plan_tiles(const GatherArgs& a, const Cursor& c, int t0, int lane, List& list) {
  TilePlan p;
  const bool pairs = a.B < 16;             // a part is two frames of 8
  const int per = a.log2_B - 4;            // log2(parts of a frame)
  const int t = t0 + lane;
  const int j = pairs ? 2 * t : t >> per;  // first entry of this lane's part
  p.row = pairs ? 0 : (t & ((1 << per) - 1)) << 4;
  int e[2] = {j, j + 1};
  const int n = SEL ? min(a.K, c.blocks) : c.blocks;
  bool have[2] = {t < c.parts && j < n, t < c.parts && pairs && j + 1 < n};
  if (SEL) {
    const int32_t* entries = a.selected + c.s * a.sel_seq + c.h * a.sel_head;
    const int j0 = pairs ? 2 * t0 : t0 >> per;
    for (int b = list.seen; b < j0 && !list.ended; b += 32)  // entries of other warps' tiles
      list.ended = __any_sync(kAll, b + lane < j0 && entries[min(b + lane, n - 1)] == -1);
#pragma unroll
    for (int i = 0; i < 2; ++i) e[i] = have[i] && !list.ended ? entries[e[i]] : -1;
    const unsigned end0 = __ballot_sync(kAll, e[0] == -1), end1 = __ballot_sync(kAll, pairs && e[1] == -1);
    const unsigned upto = (2u << lane) - 1u, before = upto >> 1;  // lanes 0 .. lane, 0 .. lane - 1
    have[0] = (end0 & upto) == 0 && (end1 & before) == 0;
    have[1] = pairs && (end0 & upto) == 0 && (end1 & upto) == 0;
    list.ended = list.ended || end0 != 0 || end1 != 0;
    list.seen = max(list.seen, j0);
  }
  p.frame[0] = have[0] ? checked_frame(a, c, e[0]) : -2;
  p.frame[1] = pairs ? (have[1] ? checked_frame(a, c, e[1]) : -2) : p.frame[0];
  if (!pairs) e[1] = e[0];
  const int n0 = p.frame[0] >= 0 ? min(8, max(0, c.L - e[0] * a.B - p.row)) : 0;
  const int n1 = p.frame[1] >= 0 ? min(8, max(0, c.L - e[1] * a.B - (pairs ? 0 : p.row + 8))) : 0;
  p.meta = n0 | (n1 << 8) | (p.frame[0] == -1 || p.frame[1] == -1 ? 1 << 16 : 0);
  if (n0 == 0) p.frame[0] = -2;
  if (n1 == 0) p.frame[1] = -2;
  return p;
}

// ---- formats: how a tile is loaded and multiplied ------------------------------------------------
// 4-bit rows of D / 2 bytes of codes and D / 8 bytes of (step, offset) pairs.  A code n is made fp16 by
// putting it into the mantissa of 1024 (low bits) or 64 (bits 4..7): 1024 + n and 64 + n are exact, so is
// the difference, and one fused multiply-add with (step, offset) gives the number that the code
// stands for.  Two codes of a 32-bit word at a time: five logic operations and eight half2
// operations for eight codes.  Both kinds run at half rate (2 clocks a warp and scheduler), so the
// 16 + 10 clocks of eight codes, not memory, bound the decode: 66 % of the copy bandwidth for
// 4 x 16384 tokens.
//
// Rows of the score tile are keys in an order that spreads the reads over the banks (rows are 80 bytes, 20 banks):
// keys 0,12,2,14,4,8,6,10,1,13,3,15,5,9,7,11 for the 16-byte reads of K (rows r and r + 1 together)
// and the 8-byte reads of V (rows 2c).
// (w & mask) | magic in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "r"(mask), "r"(magic));
  return y;
}
__device__ __forceinline__ void codes8(uint32_t w, __half2 step, __half2 off, uint32_t (&x)[4]) {
  const __half2 k1024 = __half2half2(__ushort_as_half(0x6400)), k64 = __half2half2(__ushort_as_half(0x5400));
  const uint32_t w8 = w >> 8;
  const __half2 y0 = __hsub2(as_half2(and_or(w, 0x000f000fu, 0x64006400u)), k1024);
  const __half2 y1 = __hsub2(as_half2(and_or(w, 0x00f000f0u, 0x54005400u)), k64);
  const __half2 y2 = __hsub2(as_half2(and_or(w8, 0x000f000fu, 0x64006400u)), k1024);
  const __half2 y3 = __hsub2(as_half2(and_or(w8, 0x00f000f0u, 0x54005400u)), k64);
  x[0] = as_u32(__hfma2(y0, step, off));
  x[1] = as_u32(__hfma2(y1, step, off));
  x[2] = as_u32(__hfma2(y2, step, off));
  x[3] = as_u32(__hfma2(y3, step, off));
}

template <typename T, int D_>
struct Q4Format {
  using In = T;          // queries and outputs
  using M = __half;      // operands of the tensor cores
  static constexpr int D = D_;
  static constexpr bool kScaleQ = !std::is_same<T, __half>::value;  // queries to fp16 range, by head
  static constexpr int kRow = D / 2 + D / 8;
  static constexpr uint32_t kTile = 16 * kRow;
  static constexpr int kWordsK = D / 32, kWordsV = D / 64;  // words of codes a lane reads of a key

  // key of score row r; that of row r + 8 is kSecond further on
  static constexpr int kSecond = 1;
  __device__ __forceinline__ static int key_of(int r) { return (r & 1) ? ((r + 3) & 7) + 8 : r; }

  // The caches as rows of 16 tokens of one head (of 8 where a frame holds 8): four rows a copy.
  struct Maps {
    CUtensorMap k, v;
  };
  static constexpr int kLoads = 4;
  // What the lane that plans a part keeps of it.  A half without a key loads row 0, which is always there
  // and never counted, so that every tile brings the same number of bytes.
  struct Place {
    int row[2];
  };
  __device__ __forceinline__ static Place place(const GatherArgs& a, const TilePlan& p, int h) {
    const int per = a.B >= 16 ? a.log2_B - 4 : 0;
    Place x;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x.row[i] = p.frame[i] >= 0 ? static_cast<int>((static_cast<int64_t>(p.frame[i]) * a.H + h) << per) + (p.row >> 4) : 0;
    return x;
  }
  // All lanes: the keys (or values) of a tile whose parts were planned by lanes part .. part + kLoads - 1.  The barrier
  // expects `more` bytes besides; lane issuer(part) is the one that arrives.
  __device__ __forceinline__ static int issuer(int) { return 0; }
  __device__ __forceinline__ static void load(const GatherArgs& a, const CUtensorMap* map, const Place& x, int, int lane,
                                              int part, uint32_t dst, uint32_t bar, uint32_t more) {
    const int r0 = __shfl_sync(kAll, x.row[0], part), r1 = __shfl_sync(kAll, x.row[0], part + 1);
    const int r2 = __shfl_sync(kAll, x.row[0], part + 2), r3 = __shfl_sync(kAll, x.row[0], part + 3);
    if (a.B >= 16) {
      if (lane == 0) {
        dk::mbar_arrive_expect_tx(bar, kLoads * kTile + more);
        tma_gather4(dst, map, r0, r1, r2, r3, bar);
      }
    } else {
      const int s0 = __shfl_sync(kAll, x.row[1], part), s1 = __shfl_sync(kAll, x.row[1], part + 1);
      const int s2 = __shfl_sync(kAll, x.row[1], part + 2), s3 = __shfl_sync(kAll, x.row[1], part + 3);
      if (lane == 0) {
        dk::mbar_arrive_expect_tx(bar, kLoads * kTile + more);
        tma_gather4(dst, map, r0, s0, r1, s1, bar);
        tma_gather4(dst + 2 * kTile, map, r2, s2, r3, s3, bar);
      }
    }
  }

  // The elements of a query that load_q takes in lane column c: a run of D / 4.
  __device__ __forceinline__ static void read_q(const T* q, int c, bool on, float (&x)[D / 4]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (on) u = *reinterpret_cast<const uint4*>(q + c * (D / 4) + 8 * i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = unpack2<T>(w[j]);
        x[8 * i + 2 * j] = y.x;
        x[8 * i + 2 * j + 1] = y.y;
      }
    }
  }
  // B operands for the D / 16 score steps of lane (r, c)
  __device__ __forceinline__ static void load_q(const float (&q)[D / 4], int, uint32_t (&f)[D / 16][2]) {
#pragma unroll
    for (int w = 0; w < kWordsK; ++w) {
      const float* e = q + 8 * w;
      f[2 * w][0] = pack2<M>(e[0], e[4]);
      f[2 * w][1] = pack2<M>(e[1], e[5]);
      f[2 * w + 1][0] = pack2<M>(e[2], e[6]);
      f[2 * w + 1][1] = pack2<M>(e[3], e[7]);
    }
  }

  template <int NT>
  __device__ __forceinline__ static void scores(uint32_t kst, int r, int c,
                                                const uint32_t (&qf)[NT][D / 16][2], float (&acc)[NT][4]) {
    const uint32_t row0 = kst + key_of(r) * kRow, row1 = row0 + kSecond * kRow;
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    uint32_t w0[kWordsK], w1[kWordsK];
    lds(row0 + c * (D / 8), w0);
    lds(row1 + c * (D / 8), w1);
    const uint32_t group = D / 2 + (D == 128 ? 4 * c : 4 * (c >> 1));
    const uint32_t p0 = lds(row0 + group), p1 = lds(row1 + group);
    const __half2 s0 = as_half2(prmt(p0, p0, 0x1010)), o0 = as_half2(prmt(p0, p0, 0x3232));
    const __half2 s1 = as_half2(prmt(p1, p1, 0x1010)), o1 = as_half2(prmt(p1, p1, 0x3232));
#pragma unroll
    for (int w = 0; w < kWordsK; ++w) {
      uint32_t x[4], y[4];
      codes8(w0[w], s0, o0, x);
      codes8(w1[w], s1, o1, y);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma(acc[n], x[0], y[0], x[1], y[1], qf[n][2 * w][0], qf[n][2 * w][1], M());
        mma(acc[n], x[2], y[2], x[3], y[3], qf[n][2 * w + 1][0], qf[n][2 * w + 1][1], M());
      }
    }
  }

  // o[t] += V^T P for the D / 16 groups of 16 elements; p[part][n]: B operands of the weights
  template <int NT, int PARTS>
  __device__ __forceinline__ static void values(uint32_t vst, int r, int c, int meta, const uint32_t (&p)[PARTS][NT][2],
                                                float (&o)[D / 16][NT][4]) {
    const int key[4] = {key_of(2 * c), key_of(2 * c + 1), key_of(2 * c) + kSecond, key_of(2 * c + 1) + kSecond};
    uint32_t w[4][kWordsV], par[4];
    const uint32_t group = D / 2 + (D == 128 ? 4 * (r >> 1) : 4 * (r >> 2));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t row = vst + (i < 2 ? key[i] : key[i - 2] + kSecond) * kRow;
      lds(row + r * (D / 16), w[i]);
      par[i] = lds(row + group);
    }
    if (meta != 0x0808) {  // slots that hold no key: step and offset may be anything, the weight is 0
      const int n0 = meta & 255, n1 = (meta >> 8) & 255;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key[i] < 8 ? key[i] >= n0 : key[i] - 8 >= n1) par[i] = 0;
    }
    const __half2 sa = as_half2(prmt(par[0], par[1], 0x5410)), oa = as_half2(prmt(par[0], par[1], 0x7632));
    const __half2 sb = as_half2(prmt(par[2], par[3], 0x5410)), ob = as_half2(prmt(par[2], par[3], 0x7632));
#pragma unroll
    for (int y = 0; y < kWordsV; ++y)
#pragma unroll
      for (int z = 0; z < 2; ++z) {  // codes 0..3, 4..7 of the word
        uint32_t xa[4], xb[4];
        codes8(prmt(w[0][y], w[1][y], z ? 0x7632 : 0x5410), sa, oa, xa);
        codes8(prmt(w[2][y], w[3][y], z ? 0x7632 : 0x5410), sb, ob, xb);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
              mma(o[4 * y + 2 * z + u][n], xa[2 * u], xa[2 * u + 1], xb[2 * u], xb[2 * u + 1], p[q][n][0], p[q][n][1], M());
      }
  }
  // where lane row r stores its D / 8 elements of one query (o[t] holds elements 2 t and 2 t + 1 of a run)
  __device__ __forceinline__ static void store(float* row, int r, const float (&y)[D / 16][2]) {
#pragma unroll
    for (int t = 0; t < D / 16; t += 2)
      *reinterpret_cast<float4*>(row + r * (D / 8) + 2 * t) = make_float4(y[t][0], y[t][1], y[t + 1][0], y[t + 1][1]);
  }
  __device__ __forceinline__ static void store(T* row, int r, const float (&y)[D / 16][2]) {
#pragma unroll
    for (int t = 0; t < D / 16; t += 4)
      *reinterpret_cast<uint4*>(row + r * (D / 8) + 2 * t) =
          make_uint4(pack2<T>(y[t][0], y[t][1]), pack2<T>(y[t + 1][0], y[t + 1][1]), pack2<T>(y[t + 2][0], y[t + 2][1]),
                     pack2<T>(y[t + 3][0], y[t + 3][1]));
  }
};

// ---- the kernel -------------------------------------------------------------------------------------
// One query's sum of n partials, in order: partial k is slot first + 2 k, and first + e for k = 0.  Into the output
// row, or into slot `into` (>= 0).
struct Join {
  int64_t first, into;
  int e, n, s, h;
};
template <typename T, int D>
__device__ __forceinline__ void join_query(const GatherArgs& a, const Join& x, int col, int lane) {
  constexpr int E = D / 32, kDeep = 16;
  using V = typename std::conditional<E == 4, float4, float2>::type;
  float top = -INFINITY, sum = 0.f, y[E] = {};
  bool bad = false;
  const int64_t row = 2 * static_cast<int64_t>(a.g);  // rows of [g] between one piece and the next
  const int64_t at0 = x.first * a.g + col;
#pragma unroll 1
  for (int k0 = 0; k0 < x.n; k0 += kDeep) {
    const int m = min(kDeep, x.n - k0);
    float2 p = make_float2(-INFINITY, 0.f);
    if (lane < m) p = __ldcg(reinterpret_cast<const float2*>(a.ws_ml) + at0 + (k0 + lane) * row + (k0 + lane == 0 ? x.e * a.g : 0));
    V v[kDeep];
    int64_t at = at0 + k0 * row + (k0 == 0 ? x.e * a.g : 0);
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (u < m) v[u] = __ldcg(reinterpret_cast<const V*>(a.ws_o + at * D) + lane);
      if (u == 0) at = at0 + k0 * row;
      at += row;
    }
    bad = bad || __any_sync(kAll, p.y < 0.f);
    float t = p.y != 0.f ? p.x : -INFINITY;  // an empty piece has no maximum
#pragma unroll
    for (int o = 1; o < kDeep; o <<= 1) t = fmaxf(t, __shfl_xor_sync(kAll, t, o));
    t = fmaxf(__shfl_sync(kAll, t, 0), top);
    const float less = top == t ? 1.f : dk::ex2(top - t);
    top = t;
    const float mine = p.y != 0.f ? dk::ex2(p.x - top) : 0.f;
    sum = sum * less + mine * p.y;
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] *= less;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const float w = __shfl_sync(kAll, mine, u);
      if (w != 0.f) {
        const float* z = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = fmaf(w, z[i], y[i]);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (x.into >= 0) {
    float* p = a.ws_o + (x.into * a.g + col) * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = y[i];
    if (lane == 0) *reinterpret_cast<float2*>(a.ws_ml + (x.into * a.g + col) * 2) = make_float2(top, bad ? -1.f : sum);
    return;
  }
  const float inv = bad || !(sum != 0.f) ? 0.f : 1.f / sum;
  T* out = static_cast<T*>(a.out) + x.s * a.out_row + (static_cast<int64_t>(x.h) * a.g + col) * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; i += 2) *reinterpret_cast<uint32_t*>(out + i) = bad ? 0u : pack2<T>(y[i] * inv, y[i + 1] * inv);
}

// Raises a counter of `n` arrivals; whether this one was the last, which leaves it zero again.
__device__ __forceinline__ bool last_of(int32_t* cnt, int n, int lane) {
  __threadfence();
  __syncwarp();
  int before = 0;
  if (lane == 0) before = atomicAdd(cnt, 1);
  before = __shfl_sync(kAll, before, 0);
  if (before != n - 1) return false;
  __threadfence();
  if (lane == 0) *cnt = 0;
  return true;
}

// Where there are at least kFlat + 1 pieces, the last to arrive of each group of kGroup workers joins the group's, and the
// last group the groups.  A group can hold the end of one such (s, h) and the start of another: two counters and
// two partials a group.
// A piece of (s, h) that a warp leaves: workers w0 .. w1 hold one each.  state 0: none, 1: counted, 2: counted as the last.
struct Left {
  int s, h, w0, w1, state;
};

// The counter that worker w's piece raises, and to what.
__device__ __forceinline__ int32_t* arrivals(const GatherArgs& a, const Left& x, int w) {
  const int g = w / kGroup;
  return x.w1 - x.w0 < kFlat ? a.cnt + static_cast<int64_t>(x.s) * a.H + x.h
                             : a.cnt + static_cast<int64_t>(a.S) * a.H + 2 * g + (x.w0 >= g * kGroup ? 1 : 0);
}
__device__ __forceinline__ int arrivals_of(const Left& x, int w) {
  const int g = w / kGroup;
  return x.w1 - x.w0 < kFlat ? x.w1 - x.w0 + 1 : min(x.w1, (g + 1) * kGroup - 1) - max(x.w0, g * kGroup) + 1;
}

template <class F, int NT>
__host__ __device__ constexpr uint32_t stage_bytes() {  // a tile's keys, its values, and the queries of a (s, h) that begins with it
  return 2 * F::kLoads * F::kTile + 8 * NT * F::D * sizeof(typename F::In);
}
template <class F, int NT, int STAGES>
__host__ __device__ constexpr uint32_t warp_smem() {
  return STAGES * (stage_bytes<F, NT>() + 32);  // stages, then metas (4 bytes a part) and two mbarriers each
}

template <class F, int NT, int PARTS, bool SEL, int STAGES, int WARPS, int BLOCKS>
__global__ void __launch_bounds__(WARPS * 32, BLOCKS)
    gather_kernel(const GatherArgs a, const __grid_constant__ typename F::Maps maps) {
  using T = typename F::In;
  using M = typename F::M;
  constexpr int D = F::D;
  constexpr int kB = PARTS == kTwoParts ? 2 : 1;  // B operands of the weights
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int LOADS = F::kLoads;
  static_assert(LOADS <= 4, "a stage's metas are 16 bytes");
  constexpr uint32_t kKeys = LOADS * F::kTile, kStage = stage_bytes<F, NT>();
  const uint32_t stages = dk::smem_u32(smem) + warp * (STAGES * kStage);
  const uint32_t metas = dk::smem_u32(smem) + WARPS * (STAGES * kStage) + warp * STAGES * 32;  // [stage][4]
  const uint32_t bars = metas + STAGES * 16;  // [stage][2]: keys, values
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + WARPS * warp_smem<F, NT, STAGES>());
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < 2 * STAGES; ++i) dk::mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // this warp's range [b0, b1) of the batch's tiles
  int total = 0;
  int n = 0;  // tiles of sequence s0 + lane
  for (int s0 = 0; s0 < a.S; s0 += 32) {
    n = s0 + lane < a.S ? tiles_of<SEL, LOADS>(a, checked_len(a, s0 + lane)) : 0;
    total += __reduce_add_sync(kAll, n);
  }
  total *= a.H;  // the host has checked that all this stays in int32
  const int all_warps = gridDim.x * WARPS;
  const Cut cut = cut_tiles(total, a.S * a.H, all_warps, 16 * LOADS);
  const int id = warp * gridDim.x + blockIdx.x;  // few workers: spread over the blocks
  if (blockIdx.x >= cut.workers) return;
  const int b0 = cut.start(min(id, cut.workers));
  const int count = cut.start(min(id + 1, cut.workers)) - b0;  // 0: no worker

  Cursor cur;
  cur.s = cur.h = cur.t = 0;
  int before = 0;
  for (int s0 = 0; s0 < a.S && count > 0; s0 += 32) {
    if (a.S > 32) n = s0 + lane < a.S ? tiles_of<SEL, LOADS>(a, checked_len(a, s0 + lane)) : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned past = __ballot_sync(kAll, before + upto * a.H > b0);
    if (past) {
      const int f = __ffs(past) - 1;
      const int nf = __shfl_sync(kAll, n, f), uf = __shfl_sync(kAll, upto, f);
      const int rest = b0 - before - (uf - nf) * a.H;
      cur.s = s0 + f;
      cur.h = rest / nf;
      cur.t = rest - cur.h * nf;
      break;
    }
    before += __shfl_sync(kAll, upto, 31) * a.H;
  }
  enter_seq<SEL, LOADS>(a, cur);

  // The producer's place.  Lane i plans the parts i, i + 32, ... of a (s, h) and issues their copies itself.
  Cursor ahead = cur;
  List list = {0, false};
  int planned = -1;  // first part of the window of 32 that the lanes have planned; -1: none
  typename F::Place place;
  int plan_meta = 0;
  int issued = 0, issue_st = 0;
  auto issue_keys = [&]() {
    const int part = ahead.t * LOADS;
    if ((part & ~31) != planned) {
      planned = part & ~31;
      const TilePlan p = plan_tiles<SEL>(a, ahead, planned, lane, list);
      place = F::place(a, p, ahead.h);
      plan_meta = p.meta;
    }
    const int sub = lane - (part & 31);
    if (static_cast<unsigned>(sub) < LOADS)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(metas + issue_st * 16 + sub * 4), "r"(plan_meta) : "memory");
    // the first tile of a (s, h), or of this warp's part of it, brings the queries along
    const uint32_t dst = stages + issue_st * kStage, bar = bars + 16 * issue_st;
    const bool first = ahead.t == 0 || issued == 0;
    const uint32_t q_bytes = a.g * D * sizeof(T);
    F::load(a, &maps.k, place, ahead.h, lane, part & 31, dst, bar, first ? q_bytes : 0);
    if (first && lane == F::issuer(part & 31))
      bulk_load(dst + 2 * kKeys, static_cast<const T*>(a.q) + ahead.s * a.q_row + static_cast<int64_t>(ahead.h) * a.g * D, q_bytes, bar);
  };
  auto issue_values = [&]() {  // of the same tile, and on to the next
    F::load(a, &maps.v, place, ahead.h, lane, (ahead.t * LOADS) & 31, stages + issue_st * kStage + kKeys, bars + 16 * issue_st + 8, 0);
    if (++issue_st == STAGES) issue_st = 0;
    ++issued;
    if (++ahead.t == ahead.tiles && issued < count) {
      next_head<SEL, LOADS>(a, ahead);
      planned = -1;
      list.seen = 0;
      list.ended = false;
    }
  };
  for (int i = 0; i < STAGES && i < count; ++i) {
    issue_keys();
    issue_values();
  }
  __syncwarp();

  uint32_t qf[NT][D / 16][2];
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2], f[NT][2];
  Left(*left)[2] = reinterpret_cast<Left(*)[2]>(smem + WARPS * warp_smem<F, NT, STAGES>() + 16);  // side 0: begun before
  if (lane < 2) left[warp][lane].state = 0;
  __syncwarp();
  bool stuck = false;
  const float rest = PARTS == kTwinColumns ? (c >= 2 ? 1.f : 0.f) : 1.f;
  int st = 0, phase = 0;

  // A copy is stuck: let those in flight land (bounded) before the block retires.  Tile i's keys were waited
  // for last, or its values (then the keys of tile i + STAGES may be in flight too).
  auto drain = [&](int i, bool at_values) {
    const long long t0 = clock64();
    for (int j = i; j < issued + (at_values && issued < count ? 1 : 0); ++j) {
      const uint32_t bar = bars + 16 * (j % STAGES), ph = (j / STAGES) & 1;
      for (int b = j == i && at_values ? 1 : 0; b < (j < issued ? 2 : 1); ++b)
        while (!dk::mbar_try_wait(bar + 8 * b, ph) && clock64() - t0 < dk::kDrainCycles) {
        }
    }
  };

  for (int i = 0; i < count && !stuck;) {
    // a new (s, h): its queries, as columns r (and r - 4 with twin columns)
    const int first_t = cur.t;
    bool poison = false;
    if (!__all_sync(kAll, dk::mbar_wait(bars + 16 * st, phase, abort_flag, a.status))) {
      drain(i, false);
      stuck = true;
      break;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = PARTS == kTwinColumns ? (r & 3) : 8 * n + r;
      const T* q = reinterpret_cast<const T*>(smem + warp * (STAGES * kStage) + st * kStage + 2 * kKeys) + col * D;
      float x[D / 4], top = 0.f;
      F::read_q(q, c, col < a.g, x);
#pragma unroll
      for (int j = 0; j < D / 4; ++j) top = fmaxf(top, fabsf(x[j]));
      float back = a.qk_scale_log2;
      if (F::kScaleQ) {
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        // by 2^(14 - e) with top in [2^e, 2^(e+1)), at most 2^126: 8 bits of an element down to 2^-31 of top are exact in fp16;
        // zero and non-finite heads stay as they are
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int lift = top > 0.f && e < 128 ? min(14 - e, 126) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + lift) << 23);
#pragma unroll
        for (int j = 0; j < D / 4; ++j) x[j] *= up;
        back *= __uint_as_float(static_cast<uint32_t>(127 - lift) << 23);
      }
      F::load_q(x, c, qf[n]);
      f[n][0] = __shfl_sync(kAll, back, 8 * c);       // column 2c is lane row 2c
      f[n][1] = __shfl_sync(kAll, back, 8 * c + 4);
      m[n][0] = m[n][1] = kLeast;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
    }
    const int stop = min(count, i + cur.tiles - cur.t);
    cur.t += stop - i;
    for (; i < stop; ++i) {
      const uint32_t kst = stages + st * kStage, vst = kst + kKeys, bar = bars + 16 * st;
      if (!__all_sync(kAll, dk::mbar_wait(bar, phase, abort_flag, a.status))) {
        drain(i, false);
        stuck = true;
        break;
      }
      uint32_t meta[LOADS], full = 0x0808, any = 0;
      lds(metas + st * 16, meta);
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        full = full == 0x0808 ? meta[u] : full;  // 0x0808: every slot of every part holds a key
        any |= meta[u];
      }
      if (any >> 16) poison = true;
      float x[LOADS][NT][4];
      if (any & 0xffff) {
#pragma unroll
        for (int u = 0; u < LOADS; ++u) F::template scores<NT>(kst + u * F::kTile, r, c, qf, x[u]);
      }
      __syncwarp();
      const bool more = issued < count;
      if (more) issue_keys();
      if (any & 0xffff) {
        float over = -INFINITY, top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < LOADS; ++u) x[u][n][j] *= f[n][j & 1];
        if (full != 0x0808) {
          const int k0 = F::key_of(r), k1 = F::key_of(r) + F::kSecond;
#pragma unroll
          for (int u = 0; u < LOADS; ++u) {
            const int n0 = meta[u] & 255, n1 = (meta[u] >> 8) & 255;
            const bool in0 = k0 < 8 ? k0 < n0 : k0 - 8 < n1, in1 = k1 < 8 ? k1 < n0 : k1 - 8 < n1;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!(j < 2 ? in0 : in1)) x[u][n][j] = -INFINITY;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[n][j] = fmaxf(x[0][n][j], x[0][n][j + 2]);
#pragma unroll
            for (int u = 1; u < LOADS; ++u) top[n][j] = fmaxf(top[n][j], fmaxf(x[u][n][j], x[u][n][j + 2]));
            over = fmaxf(over, top[n][j] - m[n][j]);
          }
        if (__any_sync(kAll, over > kSlack + kRoom)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float t = top[n][j];
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) t = fmaxf(t, __shfl_xor_sync(kAll, t, s));
              const float now = fmaxf(m[n][j], t - kRoom);
              const float less = m[n][j] == now ? 1.f : dk::ex2(m[n][j] - now);
              m[n][j] = now;
              l[n][j] *= less;
#pragma unroll
              for (int u = 0; u < D / 16; ++u) {
                o[u][n][j] *= less;
                o[u][n][j + 2] *= less;
              }
            }
        }
      }
      if (!__all_sync(kAll, dk::mbar_wait(bar + 8, phase, abort_flag, a.status))) {
        drain(i, true);
        stuck = true;
        break;
      }
      if (any & 0xffff) {
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
          uint32_t p[kB][NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = dk::ex2(x[u][n][j] - m[n][j & 1]);
            l[n][0] += w[0] + w[2];
            l[n][1] += w[1] + w[3];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t hi = pack2<M>(w[2 * j], w[2 * j + 1]);
              // what the rounding leaves over: `rest` is 1 in the lanes that carry it, else 0
              const float2 back = unpack2<M>(hi);
              const uint32_t lo = pack2<M>(fmaf(-rest, back.x, w[2 * j]), fmaf(-rest, back.y, w[2 * j + 1]));
              if (PARTS == kTwoParts) p[kB - 1][n][j] = transpose8(lo);
              if (PARTS == kTwinColumns) hi = lo;
              p[0][n][j] = transpose8(hi);
            }
          }
          F::template values<NT, kB>(vst + u * F::kTile, r, c, full != 0x0808 ? meta[u] & 0xffff : 0x0808, p, o);
        }
      }
      __syncwarp();
      if (more) issue_values();
      if (++st == STAGES) st = 0, phase ^= 1;
    }
    if (stuck) break;  // nothing of this piece is written or counted

    {
      // ---- the end of a piece of (s, h) ----
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) l[n][j] += __shfl_xor_sync(kAll, l[n][j], s);
          if (PARTS == kTwinColumns) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              o[t][n][j] += __shfl_xor_sync(kAll, o[t][n][j], 2);
              o[t][n][j + 2] += __shfl_xor_sync(kAll, o[t][n][j + 2], 2);
            }
          }
        }
      const bool whole = first_t == 0 && cur.t == cur.tiles;
      const int64_t slot = 2 * static_cast<int64_t>(id) + (first_t == 0 ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 8 * n + 2 * c + j;
          if (col >= a.g || (PARTS == kTwinColumns && c >= 2)) continue;
          float inv = 1.f;
          if (whole) inv = poison || !(l[n][j] != 0.f) ? 0.f : 1.f / l[n][j];
          float y[D / 16][2];
#pragma unroll
          for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) y[t][hi] = poison ? 0.f : o[t][n][j + 2 * hi] * inv;
          if (whole) {
            F::store(static_cast<T*>(a.out) + cur.s * a.out_row + (static_cast<int64_t>(cur.h) * a.g + col) * D, r, y);
          } else {
            F::store(a.ws_o + (slot * a.g + col) * D, r, y);
            if (r == 0)
              *reinterpret_cast<float2*>(a.ws_ml + (slot * a.g + col) * 2) = make_float2(m[n][j], poison ? -1.f : l[n][j]);
          }
        }
      if (!whole) {
        // pieces are the workers w0 .. w1: the first's second partial, the others' first
        const int p0 = b0 + i - cur.t;  // the first tile of (s, h)
        Left x;
        x.s = cur.s;
        x.h = cur.h;
        x.w0 = cut.owner(p0);
        x.w1 = cut.owner(p0 + cur.tiles - 1);
        x.state = last_of(arrivals(a, x, id), arrivals_of(x, id), lane) ? 2 : 1;
        if (lane == 0) left[warp][first_t == 0 ? 1 : 0] = x;
      }
    }
    if (i < count) next_head<SEL, LOADS>(a, cur);
  }

  // The joins that fall to this block, a query a warp at a time; then those of groups.
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    __syncthreads();
    if (*abort_flag) return;
    bool groups = false;
#pragma unroll 1
    for (int k = 0; k < 2 * WARPS; ++k) {
      const Left x = left[k >> 1][k & 1];
      if (x.state != 2) continue;
      const bool many = x.w1 - x.w0 >= kFlat;
      const int of = (k >> 1) * gridDim.x + blockIdx.x;  // the worker whose piece it is
      Join j;
      j.s = x.s;
      j.h = x.h;
      j.into = -1;
      if (round == 0 && many) {
        const int g = of / kGroup, lo = max(x.w0, g * kGroup);
        j.first = 2 * static_cast<int64_t>(lo);
        j.e = lo == x.w0 ? 1 : 0;
        j.n = arrivals_of(x, of);
        j.into = 2 * all_warps + 2 * g + j.e;  // partials of groups follow those of workers
        groups = true;
      } else {
        j.first = round == 0 ? 2 * static_cast<int64_t>(x.w0) : 2 * static_cast<int64_t>(all_warps) + 2 * (x.w0 / kGroup);
        j.e = 1;
        j.n = round == 0 ? x.w1 - x.w0 + 1 : x.w1 / kGroup - x.w0 / kGroup + 1;
      }
#pragma unroll 1
      for (int col = (warp + k) % WARPS; col < a.g; col += WARPS) join_query<T, D>(a, j, col, lane);
    }
    if (!groups) return;
    __syncthreads();
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const Left x = left[warp][side];
      if (x.state != 2) continue;
      bool last = false;
      if (x.w1 - x.w0 >= kFlat)
        last = last_of(a.cnt + static_cast<int64_t>(x.s) * a.H + x.h, x.w1 / kGroup - x.w0 / kGroup + 1, lane);
      __syncwarp();
      if (lane == 0 && !last) left[warp][side].state = 0;
    }
  }
}

// Launches, or only reports the launch's warps where `query` is not null.
template <class F, int NT, int PARTS, bool SEL, int STAGES, int WARPS, int BLOCKS>
cudaError_t launch(const GatherArgs& a, const typename F::Maps& maps, int num_sms, cudaStream_t stream, int* query) {
  const void* fn = reinterpret_cast<const void*>(&gather_kernel<F, NT, PARTS, SEL, STAGES, WARPS, BLOCKS>);
  constexpr uint32_t smem = WARPS * (warp_smem<F, NT, STAGES>() + 2 * sizeof(Left)) + 16;  // + the abort flag
  int occ = 0;
  cudaError_t e = kernel_prep(fn, WARPS * 32, smem, &occ);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  const int grid = num_sms * (occ < BLOCKS ? occ : BLOCKS);
  if (query) {
    *query = grid * WARPS;
    return cudaSuccess;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gather_kernel<F, NT, PARTS, SEL, STAGES, WARPS, BLOCKS>, a, maps);
}

}  // namespace gk
}  // namespace pa
