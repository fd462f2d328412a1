// How a batch's work, numbered in int32, is cut into ranges: integers only, for kernels and for the host's tests.  Totals may
// be as large as INT32_MAX: no sum here passes that.
#pragma once

#ifdef __CUDACC__
#define PA_RANGES __host__ __device__ __forceinline__
#else
#define PA_RANGES inline
#endif

namespace pa {

// Parts of 16 keys of L >= 0 tokens; at least one.
PA_RANGES int parts16(int L) { return ((L > 1 ? L - 1 : 0) >> 4) + 1; }

// First unit of worker w (0 .. workers) where `total` units are cut evenly among `workers` (< 2^15 of them).
PA_RANGES int first_unit(int total, int workers, int w) {
  const int per = total / workers;
  return w * per + static_cast<int>(static_cast<unsigned>(w * (total - per * workers)) / workers);
}

constexpr int kMinKeys = 64;   // a decode's (s, h) is cut into pieces of this many keys or more: of half as many where its pieces
                               // can still be joined at once, of twice as many (it is left whole) where it has no more than 128
constexpr int kFlat = 24;      // up to this many pieces are joined at once

// How a decode's tiles are cut: worker w has the tiles start(w) .. start(w + 1) - 1.
struct Cut {
  int total, workers, per, rest;  // total = per * workers + rest; workers^2 < 2^31
  PA_RANGES int start(int w) const { return w * per + static_cast<int>(static_cast<unsigned>(w * rest) / workers); }
  // the worker of tile x: a division in fp32 is off by at most one
  PA_RANGES int owner(int x) const {
    int w = static_cast<int>((x + 0.5f) * (static_cast<float>(workers) / total));
    w = w < workers - 1 ? w : workers - 1;
    if (start(w) > x) --w;
    if (w + 1 < workers && start(w + 1) <= x) ++w;
    return w;
  }
};

// The cut of `total` tiles of `keys` keys, of `pairs` (sequence, head), among up to all_warps warps.
PA_RANGES Cut cut_tiles(int total, int pairs, int all_warps, int keys) {
  // A join costs as much as about 128 keys: shorter (s, h) are left whole (64 keys of 8 heads: 7.6 us, cut in two
  // 8.8).  Fewer keys a worker where the pieces can still be joined at once (512 keys of 8 heads in pieces of 32 keys
  // 9.1 us, of 64 10.7; 4096 keys 17.3 and 15.8).
  const int mean = total / pairs;
  const int tiles = mean < 1 << 20 ? mean : 1 << 20;  // of a (s, h), on average
  const int min_keys = tiles * keys <= 2 * kMinKeys ? 2 * kMinKeys : tiles * keys <= kFlat * (kMinKeys / 2) ? kMinKeys / 2 : kMinKeys;
  const int piece = min_keys > keys ? min_keys / keys : 1;
  Cut cut;
  cut.workers = total / piece > pairs ? total / piece : pairs;
  if (cut.workers > all_warps) cut.workers = all_warps;
  // no more workers than the longest range needs: fewer pieces in the same time (1 x 16000 tokens: 24 -> 18 us)
  const int longest = (total - 1) / cut.workers + 1;
  cut.workers = (total - 1) / longest + 1;
  // A multiple of the (s, h) where that leaves few warps idle: sequences of one length are then cut at their ends
  // (64 listed frames for 4 x 32 heads: 22.7 -> 19.8 us).
  if (cut.workers / pairs * pairs * 10 >= cut.workers * 9) cut.workers = cut.workers / pairs * pairs;
  cut.total = total;
  cut.per = total / cut.workers;
  cut.rest = total - cut.per * cut.workers;
  return cut;
}

}  // namespace pa
