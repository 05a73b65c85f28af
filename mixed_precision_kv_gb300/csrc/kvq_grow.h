// How a buffer grows (no CUDA in here).
#pragma once
#include <algorithm>
#include <cstddef>

namespace kvq {

// A new buffer of at least `need` bytes in place of one of `have`: twice as large
// as that one, so that a buffer that grows step by step is seldom replaced, but
// past `most` only as far as needed; `need` alone if there is no memory for more.
// try_alloc(bytes): whether it could be had.  Returns its size, or 0.
template <class Try>
size_t grow(size_t have, size_t need, size_t most, Try&& try_alloc) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t least = up(need), want = up(std::max(need, std::min(2 * have, most)));
  if (try_alloc(want)) return want;
  return want > least && try_alloc(least) ? least : 0;
}

}  // namespace kvq
