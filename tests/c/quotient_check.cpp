// Checks the quotients of csrc/ranges.h against the compiler's, with reciprocals off by up to two steps of fp32 either way, as the
// kernels' are; built with -fsanitize=undefined, so that a sum or product that passes int32 ends the program.
#include "ranges.h"

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

static void check(int64_t a, int b) {
  if (a < 0 || a > INT_MAX || b < 1) return;
  const int x = static_cast<int>(a), want = x / b;
  float inv = 1.f / static_cast<float>(b);
  inv = std::nextafterf(std::nextafterf(inv, 0.f), 0.f);
  for (int off = -2; off <= 2; ++off, inv = std::nextafterf(inv, 4.f)) {
    const int got = pa::quotient_by(x, b, inv);
    if (got == want) continue;
    std::printf("%d / %d, reciprocal off by %d steps: %d, not %d\n", x, b, off, got, want);
    std::exit(1);
  }
  if (pa::quotient(x, b) != want) std::printf("quotient %d / %d\n", x, b), std::exit(1);
}

static void check_around(int64_t a, int b) {
  for (int64_t d = -2; d <= 2; ++d) check(a + d, b);
}

int main() {
  std::mt19937_64 rng(1);
  auto any = [&](int64_t n) { return static_cast<int64_t>(rng() % static_cast<uint64_t>(n)); };
  auto divisors = [&](auto f) {
    for (int b = 1; b <= 5000; ++b) f(b);
    for (int i = 0; i < 31; ++i)
      for (int64_t d = -3; d <= 3; ++d)
        if (const int64_t b = (int64_t{1} << i) + d; b >= 1 && b <= INT_MAX) f(static_cast<int>(b));
    for (int d = 0; d < 2000; ++d) f(INT_MAX - d);
    for (int i = 0; i < 20000; ++i) f(static_cast<int>(1 + any(int64_t{1} << (1 + any(31))) % INT_MAX));
  };
  divisors([&](int b) {
    const int64_t most = INT_MAX / b;
    for (int64_t m : {int64_t{0}, int64_t{1}, int64_t{2}, most - 1, most, most + 1}) check_around(m * b, b);
    check_around(INT_MAX, b);
    for (int i = 0; i < 20; ++i) {
      check_around(any(most + 1) * b, b);
      check(any(int64_t{INT_MAX} + 1), b);
    }
  });
  std::puts("ok");
  return 0;
}
