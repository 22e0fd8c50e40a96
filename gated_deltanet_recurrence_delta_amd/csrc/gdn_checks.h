// Host-side checks of the C entry points' buffers.  Internal header: every
// definition sits in an unnamed namespace of the including file.
#ifndef GDN_CHECKS_H
#define GDN_CHECKS_H

#include <stdint.h>

#include <initializer_list>

namespace {

inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

inline bool misaligned(std::initializer_list<const void*> ps, uintptr_t to) {
  for (const void* p : ps)
    if (misaligned(p, to)) return true;
  return false;
}

struct Range {
  const void* p;
  long long bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes;
}

// Whether an output overlaps an input or another output.
inline bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* a = outs.begin(); a != outs.end(); ++a) {
    for (const Range* b = a + 1; b != outs.end(); ++b)
      if (overlap(*a, *b)) return true;
    for (const Range& b : ins)
      if (overlap(*a, b)) return true;
  }
  return false;
}

}  // namespace

#endif  // GDN_CHECKS_H
