// Memory that a call's arguments cover, for refusing outputs laid over other
// arguments: host arithmetic in plain C++.
#pragma once
#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace wsg {

struct Span {
  const void* at;
  size_t bytes;
};

// rows x width elements of `elem` bytes, `stride` elements from row to row.
inline Span span_rows(const void* at, long long rows, long long stride, long long width, size_t elem) {
  if (!at || rows <= 0 || width <= 0) return Span{nullptr, 0};
  return Span{at, static_cast<size_t>((rows - 1) * stride + width) * elem};
}

inline bool spans_meet(const Span& x, const Span& y) {
  if (!x.at || !y.at || !x.bytes || !y.bytes) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(x.at), q = reinterpret_cast<uintptr_t>(y.at);
  return p < q ? q - p < x.bytes : p - q < y.bytes;
}

// Whether an output meets an input or another output.
inline bool outputs_meet(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (spans_meet(*o, i)) return true;
    for (const Span* p = o + 1; p != outs.end(); ++p)
      if (spans_meet(*o, *p)) return true;
  }
  return false;
}

}  // namespace wsg
