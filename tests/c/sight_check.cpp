// Checks what a window and its sinks see (Sight, csrc/ranges.h): every token that is seen lies in exactly the parts that say so, over small cases
// exhaustively and next to int32's end; built with -fsanitize=undefined, so that a sum that passes int32 ends the program.
#include "ranges.h"

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

static void fail(const char* what, long long L, long long window, long long sinks) {
  std::printf("%s: L %lld window %lld sinks %lld\n", what, L, window, sinks);
  std::exit(1);
}

static void check(int L, int window, int sinks) {
  const pa::Sight x = pa::sight_of(L, window, sinks);
  if (x.parts < 1 || x.sink_parts < 0 || x.sink_parts > x.parts) fail("parts", L, window, sinks);
  const int64_t first = static_cast<int64_t>(L) - window;
  const int64_t start = first <= 0 || sinks >= first ? 0 : first;
  if (x.start != start || x.sinks != (start ? sinks : 0)) fail("start", L, window, sinks);
  const int64_t want = (start ? (static_cast<int64_t>(sinks) + 15) / 16 : 0) + (L > 0 ? (L - (start & ~15LL) + 15) / 16 : 1);
  if (x.parts != want) fail("count", L, window, sinks);
  for (int p : {0, x.sink_parts - 1, x.sink_parts, x.parts - 1}) {
    if (p < 0) continue;
    const int64_t base = p < x.sink_parts ? 16LL * p : (start & ~15LL) + 16LL * (p - x.sink_parts);
    if (x.base(p) != base || (L > 0 && base >= L)) fail("base", L, window, sinks);
  }
  if (L > 500) return;
  for (int j = 0; j < L; ++j) {
    int seen = 0;
    for (int p = 0; p < x.parts; ++p) {
      const int base = x.base(p);
      if (j < base || j >= base + 16) continue;
      seen += p < x.sink_parts ? j < x.sinks : j >= x.start;
    }
    if (seen != (j >= L - window || j < sinks ? 1 : 0)) fail("seen", L, window, sinks);
  }
}

int main() {
  for (int L = 0; L < 70; ++L)
    for (int window = 1; window < 75; ++window)
      for (int sinks = 0; sinks < 75; ++sinks) check(L, window, sinks);
  for (int L : {0, 1, 480, INT_MAX - 20, INT_MAX - 16, INT_MAX - 1, INT_MAX})
    for (int window : {1, 15, 16, 17, 479, INT_MAX - 17, INT_MAX - 1, INT_MAX})
      for (int sinks : {0, 1, 15, 16, 17, 400, INT_MAX - 40, INT_MAX - 1, INT_MAX}) check(L, window, sinks);
  std::puts("ok");
  return 0;
}
