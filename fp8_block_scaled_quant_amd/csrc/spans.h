// Whether tensors of a list share memory.  Host code.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

namespace fp8bsq {

struct Span {   // bytes [begin, end), at least one
  uintptr_t begin, end;
};

// By ascending address: two counting passes over the upper 16 bits that the
// addresses differ in, and a comparing sort only where those tie (240 spans from
// all over the memory take 2 us, by comparisons alone 9).
inline void sort_by_address(std::vector<Span> &spans) {
  const auto less = [](const Span &a, const Span &b) { return a.begin < b.begin; };
  if (std::is_sorted(spans.begin(), spans.end(), less)) return;
  uintptr_t low = UINTPTR_MAX, high = 0;
  for (const Span &s : spans) {
    low = std::min(low, s.begin);
    high = std::max(high, s.begin);
  }
  int shift = 0;
  while ((high - low) >> shift > 0xFFFF) ++shift;
  std::vector<Span> from(spans.size());
  for (int pass = 0; pass < 2; ++pass, shift += 8) {
    uint32_t at[257] = {};
    spans.swap(from);
    for (const Span &s : from) ++at[((s.begin - low) >> shift & 255) + 1];
    for (int i = 1; i < 256; ++i) at[i] += at[i - 1];
    for (const Span &s : from) spans[at[(s.begin - low) >> shift & 255]++] = s;
  }
  if (!std::is_sorted(spans.begin(), spans.end(), less)) std::sort(spans.begin(), spans.end(), less);
}

inline bool overlapping(std::vector<Span> spans) {
  sort_by_address(spans);
  for (size_t i = 1; i < spans.size(); ++i)   // none before reaches past the last one's begin
    if (spans[i].begin < spans[i - 1].end) return true;
  return false;
}

}  // namespace fp8bsq
