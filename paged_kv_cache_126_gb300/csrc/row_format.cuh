// 16-bit caches [num_blocks, B, H, D] as tiles of the gathered decode.
#pragma once

#include "gather_kernel.cuh"

namespace pa {
namespace gk {

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(addr));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// 16-bit rows.  A half tile, 8 keys, is one TMA box [D / 64 column groups][8 rows][64 elements] with the
// 128-byte swizzle: row y of a column group keeps its 16-byte chunk x at x ^ y, so that the eight row
// addresses of an ldmatrix fall into different banks.
// L parts a tile.
template <typename T, int D_, int L = 1>
struct RowFormat {
  using In = T;
  using M = T;
  static constexpr int D = D_;
  static constexpr bool kScaleQ = false;
  static constexpr bool kSteps = false;
  static constexpr int kSecond = 8;
  static constexpr uint32_t kHalfTile = 8 * D * 2, kTile = 2 * kHalfTile;
  __device__ __forceinline__ static int key_of(int r) { return r; }

  struct Maps {
    CUtensorMap k, v;
  };
  static constexpr int kLoads = L;
  struct Place {
    int slot[2];     // first slot of each half; < 0: nothing to load
  };
  __device__ __forceinline__ static Place place(const GatherArgs& a, const TilePlan& p, int) {
    Place x;
    x.slot[0] = p.frame[0] >= 0 ? p.frame[0] * a.B + p.row : -1;
    x.slot[1] = p.frame[1] >= 0 ? p.frame[1] * a.B + p.row + (a.B >= 16 ? 8 : 0) : -1;
    return x;
  }
  __device__ __forceinline__ static int issuer(int part) { return part; }
  __device__ __forceinline__ static void load(const GatherArgs&, const CUtensorMap* map, const Place& x, int h, int lane,
                                              int part, uint32_t dst, uint32_t bar, uint32_t more) {
    if (L == 1) {
      if (lane != part) return;
      dk::mbar_arrive_expect_tx(bar, ((x.slot[0] >= 0) + (x.slot[1] >= 0)) * kHalfTile + more);
    } else {
      const bool mine = static_cast<unsigned>(lane - part) < L;
      const unsigned first = __ballot_sync(kAll, mine && x.slot[0] >= 0), second = __ballot_sync(kAll, mine && x.slot[1] >= 0);
      if (lane == part) dk::mbar_arrive_expect_tx(bar, (__popc(first) + __popc(second)) * kHalfTile + more);
      __syncwarp();
      if (!mine) return;
      dst += (lane - part) * kTile;
    }
    if (x.slot[0] >= 0) tma_load_4d(dst, map, 0, x.slot[0], 0, h, bar);
    if (x.slot[1] >= 0) tma_load_4d(dst + kHalfTile, map, 0, x.slot[1], 0, h, bar);
  }

  // the elements of a query that load_q takes in lane column c: 16 k + 2 c + {0, 1, 8, 9}
  __device__ __forceinline__ static void read_q(const T* q, int c, bool on, float (&x)[D / 4]) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float2 y = unpack2<T>(on ? *reinterpret_cast<const uint32_t*>(q + 8 * i + 2 * c) : 0u);
      x[2 * i] = y.x;
      x[2 * i + 1] = y.y;
    }
  }
  __device__ __forceinline__ static void load_q(const float (&q)[D / 4], int, uint32_t (&f)[D / 16][2]) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      f[k][0] = pack2<M>(q[4 * k], q[4 * k + 1]);
      f[k][1] = pack2<M>(q[4 * k + 2], q[4 * k + 3]);
    }
  }

  // A step of all parts, then the next: products that follow one another do not wait for one another's sums.
  template <int NT>
  __device__ __forceinline__ static void scores_tile(uint32_t kst, int r, int c, const uint32_t (&qf)[NT][D / 16][2],
                                                     float (&acc)[L][NT][4]) {
    const int lane = 4 * r + c, y = lane & 7, mat = lane >> 3;
    const uint32_t row = kst + (mat & 1) * kHalfTile + y * 128;  // matrices: keys 0..7, 8..15, then the next 8 elements
#pragma unroll
    for (int u = 0; u < L; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[u][n][0] = acc[u][n][1] = acc[u][n][2] = acc[u][n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int u = 0; u < L; ++u) {
        uint32_t x[4];
        ldmatrix4(row + u * kTile + (k >> 2) * 1024 + ((((k & 3) * 2 + (mat >> 1)) ^ y) << 4), x);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(acc[u][n], x[0], x[1], x[2], x[3], qf[n][k][0], qf[n][k][1], M());
      }
    }
  }

  template <int NT, int PARTS>
  __device__ __forceinline__ static void values(uint32_t vst, int r, int c, int meta, const uint32_t (&p)[PARTS][NT][2],
                                                float (&o)[D / 16][NT][4]) {
    const int lane = 4 * r + c, y = lane & 7, mat = lane >> 3;
    const uint32_t row = vst + (mat >> 1) * kHalfTile + y * 128;  // matrices: elements 0..7, 8..15 of keys 0..7, then of 8..15
    uint32_t keep0 = ~0u, keep1 = ~0u;
    if (meta != 0x0808) {  // slots that hold no key: any bits, and the weight is 0
      const int n0 = meta & 255, n1 = (meta >> 8) & 255;
      keep0 = (2 * c < n0 ? 0xffffu : 0u) | (2 * c + 1 < n0 ? 0xffff0000u : 0u);
      keep1 = (2 * c < n1 ? 0xffffu : 0u) | (2 * c + 1 < n1 ? 0xffff0000u : 0u);
      if (meta >> 20) {  // the first so many neither
        const int from0 = (meta >> 20) & 15, from1 = (meta >> 24) & 15;
        keep0 &= (2 * c >= from0 ? 0xffffu : 0u) | (2 * c + 1 >= from0 ? 0xffff0000u : 0u);
        keep1 &= (2 * c >= from1 ? 0xffffu : 0u) | (2 * c + 1 >= from1 ? 0xffff0000u : 0u);
      }
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      uint32_t x[4];
      ldmatrix4_trans(row + (t >> 2) * 1024 + ((((t & 3) * 2 + (mat & 1)) ^ y) << 4), x);
      x[0] &= keep0;
      x[1] &= keep0;
      x[2] &= keep1;
      x[3] &= keep1;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < PARTS; ++q) mma(o[t][n], x[0], x[1], x[2], x[3], p[q][n][0], p[q][n][1], M());
    }
  }
  // where lane row r stores its D / 8 elements of one query: r of every 8
  template <typename U>
  __device__ __forceinline__ static void store(U* row, int r, const float (&y)[D / 16][2]) {
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) dk::Chunk<U>::store1(row + 16 * t + 8 * hi + r, y[t][hi]);
  }
};

}  // namespace gk
}  // namespace pa
