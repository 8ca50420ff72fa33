// overlapping() of spans.h against every pair of spans, on random lists.
#include <cstdio>
#include <random>

#include "spans.h"

using fp8bsq::Span;

static bool pairs(const std::vector<Span> &spans) {
  for (const Span &a : spans)
    for (const Span &b : spans)
      if (&a != &b && a.end > b.begin && b.end > a.begin) return true;
  return false;
}

int main() {
  std::mt19937_64 rng(1);
  const auto below = [&](uint64_t n) { return (uintptr_t)(rng() % n); };
  int found[2] = {0, 0};
  for (int round = 0; round < 40000; ++round) {
    // few bytes, so that lists collide; now and then addresses that differ in high bits too
    const uint64_t room = 1 + below(round % 3 ? 4000 : 60), far = round % 5 ? 0 : (uint64_t)below(1 << 20) << 26;
    const int count = 1 + (int)below(round % 7 ? 12 : 150);
    const bool neighbours = below(2), repeat = below(4) == 0;
    std::vector<Span> spans;
    uintptr_t next = 4096;
    for (int i = 0; i < count; ++i) {
      const uintptr_t bytes = 1 + below(8), at = (neighbours ? next : 4096 + below(room)) + (below(2) ? far : 0);
      next += bytes + below(2);
      spans.push_back({at, at + bytes});
    }
    if (repeat) spans.push_back(spans[below(spans.size())]);
    if (below(2)) std::shuffle(spans.begin(), spans.end(), rng);
    const bool want = pairs(spans);
    ++found[want];
    if (fp8bsq::overlapping(spans) != want) {
      std::printf("round %d: %d spans, expected %d\n", round, (int)spans.size(), want);
      return 1;
    }
  }
  std::printf("%d apart, %d overlapping\n", found[0], found[1]);
  return found[0] > 1000 && found[1] > 1000 && !fp8bsq::overlapping({}) ? 0 : 1;
}
