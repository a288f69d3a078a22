// Whether two matrices share bytes of memory (host only, no CUDA).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

namespace beam {

// `rows` rows of `width` bytes, `pitch` bytes (at least `width`) from one to the next.
struct Span {
  const void* at;
  int64_t rows, width, pitch;
};

// Exact for columns of one larger matrix (the same pitch), for contiguous matrices and for single
// rows.  Of two matrices with gaps and different pitches the first rows are looked at.
inline bool overlap(Span a, Span b) {
  using Wide = __int128;  // a pitch is what the caller says
  constexpr int64_t kRows = 1 << 16;
  const auto floor_div = [](Wide n, Wide d) { return n >= 0 ? n / d : -((-n + d - 1) / d); };
  struct Run {
    Wide at, rows, width, pitch;
    Wide end() const { return at + (rows - 1) * pitch + width; }
  };
  const auto run = [](const Span& s) {
    const Wide at = static_cast<Wide>(reinterpret_cast<uintptr_t>(s.at));
    if (s.rows == 1 || s.pitch == s.width) {  // one long row
      const Wide all = static_cast<Wide>(s.rows) * s.width;
      return Run{at, 1, all, all};
    }
    return Run{at, s.rows, s.width, s.pitch};
  };
  if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  Run p = run(a), q = run(b);
  if (p.end() <= q.at || q.end() <= p.at) return false;
  // q's first row that ends behind `from`, and whether it starts before `to`
  const auto touches = [&](Wide from, Wide to) {
    const Wide r = std::max<Wide>(0, floor_div(from - q.at - q.width, q.pitch) + 1);
    return r < q.rows && q.at + r * q.pitch < to;
  };
  if (p.rows > q.rows) std::swap(p, q);
  if (p.rows > 1 && p.pitch == q.pitch) {
    // a row of q less a row of p, k apart: they meet where -q.width < d + k pitch < p.width
    const Wide d = q.at - p.at;
    const Wide k = std::max(floor_div(-q.width - d, q.pitch) + 1, -(p.rows - 1));
    return k <= q.rows - 1 && d + k * q.pitch < p.width;
  }
  for (Wide r = 0; r < std::min<Wide>(p.rows, kRows); ++r) {
    const Wide from = p.at + r * p.pitch;
    if (touches(from, from + p.width)) return true;
  }
  return false;
}

// Whether an output shares bytes with one of the other matrices.
inline bool overlaps_any(const Span& out, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (overlap(out, o)) return true;
  return false;
}

}  // namespace beam
