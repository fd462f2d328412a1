// Decode attention over the 8-bit cache [num_blocks, H, B, D] with a step for each (frame, head): every token, or a window.
#include "gather_kernel.cuh"
#include "pa.h"

namespace pa {
namespace gk {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// A byte put into the mantissa of fp16's 1024 is 1024 + byte, exactly, and less 1152 the code itself, a whole number
// of -127 .. 127: two codes are one permutation and one half2 operation.  What a step multiplies are sums: the scores of a frame, in
// fp32, and a weight before it is split into its two fp16 parts.  For that the steps are taken as multiples of a power of two above
// all those seen so far (`unit` in the kernel), so that weights stay in fp16's range whatever the values' size.
//
// A tile's 16 rows are one TMA box with a swizzle, chunks of 16 bytes exchanged by the row (128-byte rows: x ^ (row & 7)), so that
// the 16-byte reads of keys (a row's chunks 2 c and 2 c + 1, rows r) and of values (chunk r of rows 2 c) fall into different banks.
template <typename T, int D_>
struct Q8Format {
  using In = T;
  using M = __half;
  static constexpr int D = D_;
  static constexpr bool kScaleQ = !std::is_same<T, __half>::value;
  static constexpr bool kSteps = true;
  static constexpr int kSecond = 8;
  static constexpr uint32_t kTile = 16 * D, kHalfTile = 8 * D;
  __device__ __forceinline__ static int key_of(int r) { return r; }

  struct Maps {
    CUtensorMap k, v;
  };
  static constexpr int kLoads = 4;
  struct Place {
    int at[2];  // (frame, head) of each half; < 0: nothing to load
    int row;
  };
  __device__ __forceinline__ static Place place(const GatherArgs& a, const TilePlan& p, int h) {
    Place x;
    x.at[0] = p.frame[0] >= 0 ? p.frame[0] * a.H + h : -1;
    x.at[1] = p.frame[1] >= 0 ? p.frame[1] * a.H + h : -1;
    if (a.B >= 16) x.at[0] = max(x.at[0], x.at[1]);  // one box
    x.row = p.row;
    return x;
  }
  __device__ __forceinline__ static int issuer(int part) { return part; }
  __device__ __forceinline__ static void load(const GatherArgs& a, const CUtensorMap* map, const Place& x, int, int lane,
                                              int part, uint32_t dst, uint32_t bar, uint32_t more) {
    const bool mine = static_cast<unsigned>(lane - part) < kLoads, pairs = a.B < 16;
    const unsigned first = __ballot_sync(kAll, mine && x.at[0] >= 0), second = __ballot_sync(kAll, mine && pairs && x.at[1] >= 0);
    if (lane == part)
      dk::mbar_arrive_expect_tx(bar, (pairs ? kHalfTile * (__popc(first) + __popc(second)) : kTile * __popc(first)) + more);
    __syncwarp();
    if (!mine) return;
    dst += (lane - part) * kTile;
    if (x.at[0] >= 0) tma_load_3d(dst, map, 0, x.row, x.at[0], bar);
    if (pairs && x.at[1] >= 0) tma_load_3d(dst + kHalfTile, map, 0, x.row, x.at[1], bar);
  }

  // the elements of a query that load_q takes in lane column c: a run of D / 4
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
  __device__ __forceinline__ static void load_q(const float (&q)[D / 4], int, uint32_t (&f)[D / 16][2]) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      f[k][0] = pack2<M>(q[4 * k], q[4 * k + 1]);
      f[k][1] = pack2<M>(q[4 * k + 2], q[4 * k + 3]);
    }
  }

  // two bytes of w, by the selector, as the codes they are
  __device__ __forceinline__ static uint32_t codes2(uint32_t w, uint32_t sel) {
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    return as_u32(__hsub2(as_half2(prmt(w, 0x64646464u, sel)), bias));
  }
  // where chunk x of 16 bytes of a row stands
  __device__ __forceinline__ static uint32_t chunk(int row, int x) {
    return D == 128 ? row * 128 + ((x ^ (row & 7)) << 4) : row * 64 + ((x ^ ((row >> 1) & 3)) << 4);
  }

  // A step of all parts, then the next: products that follow one another do not wait for one another's sums (a part after the other:
  // 1170 clocks of a warp alone).
  template <int NT>
  __device__ __forceinline__ static void scores_tile(uint32_t kst, int r, int c, const uint32_t (&qf)[NT][D / 16][2],
                                                     float (&acc)[kLoads][NT][4]) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[u][n][0] = acc[u][n][1] = acc[u][n][2] = acc[u][n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t w0[kLoads][4], w1[kLoads][4];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        lds(kst + u * kTile + chunk(r, c * (D / 64) + j), w0[u]);
        lds(kst + u * kTile + chunk(r + 8, c * (D / 64) + j), w1[u]);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const uint32_t a0 = codes2(w0[u][w], 0x4140), a1 = codes2(w1[u][w], 0x4140);
          const uint32_t a2 = codes2(w0[u][w], 0x4342), a3 = codes2(w1[u][w], 0x4342);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(acc[u][n], a0, a1, a2, a3, qf[n][4 * j + w][0], qf[n][4 * j + w][1], M());
        }
    }
  }

  // Slots that hold no key hold some whole number, which the weight 0 takes out.  A part's codes are read while the part before
  // is multiplied; with more than 8 queries there are no registers for that (69.6 us, read ahead 70.6).
  template <int NT, int PARTS>
  __device__ __forceinline__ static void values_tile(uint32_t vst, int r, int c, const uint32_t (&p)[kLoads][PARTS][NT][2],
                                                     float (&o)[D / 16][NT][4]) {
    constexpr int W = D / 32;  // words of codes a lane reads of a key
    constexpr int kAhead = NT == 1;
    uint32_t w[1 + kAhead][4][W];
    auto read = [&](int u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 2 * c + (i & 1) + (i >> 1) * 8;
        lds(vst + u * kTile + (D == 128 ? chunk(key, r) : chunk(key, r >> 1) + (r & 1) * 8), w[u & kAhead][i]);
      }
    };
    if (kAhead) read(0);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (u + kAhead < kLoads) read(u + kAhead);
      const uint32_t(&x)[4][W] = w[u & kAhead];
#pragma unroll
      for (int y = 0; y < W; ++y)
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // elements 4 y + 2 z and the next: of two keys, then of the two 8 further on
          const uint32_t lo = prmt(x[0][y], x[1][y], z ? 0x7362 : 0x5140), hi = prmt(x[2][y], x[3][y], z ? 0x7362 : 0x5140);
          const uint32_t a0 = codes2(lo, 0x4140), a1 = codes2(lo, 0x4342), a2 = codes2(hi, 0x4140), a3 = codes2(hi, 0x4342);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) mma(o[2 * y + z][n], a0, a1, a2, a3, p[u][q][n][0], p[u][q][n][1], M());
        }
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
          make_uint4(pack_out<T, true>(y[t][0], y[t][1]), pack_out<T, true>(y[t + 1][0], y[t + 1][1]),
                     pack_out<T, true>(y[t + 2][0], y[t + 2][1]), pack_out<T, true>(y[t + 3][0], y[t + 3][1]));
  }
};

}  // namespace gk

namespace {

// Bound by memory while it streams.  8 warps an SM, two on each scheduler, one stage of 64 keys (heads of 128: 216 registers with up to 4
// queries a key head, 218 with up to 8, 255 and 20 to 40 bytes of spill stores with more): 64 sequences of
// 512 to 2048 tokens, 32 heads of 128 in fp16 (674 MB) take 110 us, 6.1 TB/s; 4 x 16384 in bf16 (538 MB) 85 to 87 us, 6.25 TB/s, of which
// about 4 us pass before the first keys are there and 5 behind the last.  12 warps 118.8 and 94.0 us, 10 warps 114.7 and 90.7 us, 6
// warps with two stages 132 and 100 us; tiles of 32 keys with 12 warps and two stages 134.6 and 104 us, of 128 keys with 6 warps 132
// and 93 us.  A tile's parts in a loop instead of unrolled 119 and 94 us; copies issued by one lane instead of four 114.5 and 87.4 us.
template <typename T, int D, int KEYS>
cudaError_t by_group(const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, cudaStream_t stream,
                     int* workers) {
  using F = gk::Q8Format<T, D>;
  const typename F::Maps maps = {tk, tv};
  constexpr int kBlocks = D == 64 ? 3 : 2;  // (of half as many bytes)
  if (a.g <= 4) return gk::launch<F, 1, gk::kTwinColumns, KEYS, 1, 4, kBlocks>(a, maps, num_sms, stream, workers);
  if (a.g <= 8) return gk::launch<F, 1, gk::kTwoParts, KEYS, 1, 4, kBlocks>(a, maps, num_sms, stream, workers);
  return gk::launch<F, 2, gk::kTwoParts, KEYS, 1, 4, 2>(a, maps, num_sms, stream, workers);
}

template <typename T, int D>
cudaError_t by_keys(const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, cudaStream_t stream, int* workers) {
  return a.window > 0 ? by_group<T, D, gk::kWindow>(a, tk, tv, num_sms, stream, workers)
                      : by_group<T, D, gk::kEvery>(a, tk, tv, num_sms, stream, workers);
}

}  // namespace

cudaError_t launch_decode_q8(int dtype, int D, const GatherArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms,
                             cudaStream_t stream, int* workers) {
  if (dtype == PA_F16)
    return D == 128 ? by_keys<__half, 128>(a, tk, tv, num_sms, stream, workers)
                    : by_keys<__half, 64>(a, tk, tv, num_sms, stream, workers);
  return D == 128 ? by_keys<__nv_bfloat16, 128>(a, tk, tv, num_sms, stream, workers)
                  : by_keys<__nv_bfloat16, 64>(a, tk, tv, num_sms, stream, workers);
}

}  // namespace pa
