// Checks the integer cuts of csrc/ranges.h over random and extreme totals; built with -fsanitize=undefined, so that a
// sum that passes int32 ends the program.
#include "ranges.h"

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

static void fail(const char* what, long long a, long long b, long long c) {
  std::printf("%s: %lld %lld %lld\n", what, a, b, c);
  std::exit(1);
}

static void check_cut(int total, int pairs, int warps, int keys, std::mt19937& rng) {
  const pa::Cut cut = pa::cut_tiles(total, pairs, warps, keys);
  if (cut.workers < 1 || cut.workers > warps || cut.total != total) fail("workers", total, pairs, cut.workers);
  if (cut.start(0) != 0 || cut.start(cut.workers) != total) fail("ends", total, pairs, cut.workers);
  const int64_t most = (static_cast<int64_t>(total) + cut.workers - 1) / cut.workers;
  for (int w = 0; w < cut.workers; ++w) {
    const int64_t n = static_cast<int64_t>(cut.start(w + 1)) - cut.start(w);
    if (n < 0 || n > most) fail("range", total, w, n);
    if (n > 0 && (cut.owner(cut.start(w)) != w || cut.owner(cut.start(w + 1) - 1) != w)) fail("owner", total, cut.workers, w);
  }
  for (int i = 0; i < 20; ++i) {
    const int x = static_cast<int>(rng() % static_cast<unsigned>(total)), w = cut.owner(x);
    if (w < 0 || w >= cut.workers || cut.start(w) > x || cut.start(w + 1) <= x) fail("owner of", total, cut.workers, x);
  }
}

int main() {
  std::mt19937 rng(1);
  for (int i = 0; i < 3000; ++i) {
    const int bits = static_cast<int>(rng() % 31) + 1;
    int total = static_cast<int>(rng() & ((1u << bits) - 1));
    if (i % 3 == 0) total = INT_MAX - static_cast<int>(rng() % 3000);
    if (total < 1) total = 1;
    int pairs = 1 << (rng() % 20);
    if (pairs > total) pairs = total;  // every (sequence, head) has a tile
    check_cut(total, pairs, static_cast<int>(152 * 4 * (1 + rng() % 3)), rng() % 2 ? 64 : 16, rng);
    const int workers = 1 + static_cast<int>(rng() % 32767);
    int before = 0;
    if (pa::first_unit(total, workers, workers) != total) fail("first_unit", total, workers, workers);
    for (int w = 0; w <= workers; w += 1 + static_cast<int>(rng() % 64)) {
      const int x = pa::first_unit(total, workers, w);
      if (x < before) fail("first_unit", total, workers, w);
      before = x;
    }
  }
  for (int64_t L : {0LL, 1LL, 15LL, 16LL, 17LL, 32LL, 33LL, INT_MAX - 15LL, INT_MAX - 8LL, static_cast<long long>(INT_MAX)}) {
    const int64_t want = L <= 16 ? 1 : (L + 15) / 16;
    if (pa::parts16(static_cast<int>(L)) != want) fail("parts16", L, want, pa::parts16(static_cast<int>(L)));
  }
  std::puts("ok");
  return 0;
}
