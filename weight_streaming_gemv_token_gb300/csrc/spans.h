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

// `pages` pages of `page` bytes.
inline Span span_pool(const void* at, long long pages, long long page) {
  if (!at || pages <= 0 || page <= 0) return Span{nullptr, 0};
  const long long most = 1ll << 62;
  return Span{at, static_cast<size_t>(pages > most / page ? most : pages * page)};
}

inline bool spans_meet(const Span& x, const Span& y) {
  if (!x.at || !y.at || !x.bytes || !y.bytes) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(x.at), q = reinterpret_cast<uintptr_t>(y.at);
  return p < q ? q - p < x.bytes : p - q < y.bytes;
}

// Several equal spans, `stride` bytes from one to the next: rows of a tensor, layers of a pool.
struct Spans {
  Span first;
  long long count, stride;
};

// Whether two such series meet. Between equal strides each span is looked at (columns of one
// buffer do not meet); otherwise what either covers as a whole.
inline bool series_meet(Spans x, Spans y) {
  if (!x.first.at || !y.first.at || !x.first.bytes || !y.first.bytes || x.count <= 0 || y.count <= 0) return false;
  if (x.count == 1) x.stride = y.stride;
  if (y.count == 1) y.stride = x.stride;
  if (x.stride != y.stride || x.stride <= 0) {
    auto whole = [](const Spans& s) { return Span{s.first.at, static_cast<size_t>((s.count - 1) * s.stride) + s.first.bytes}; };
    return spans_meet(whole(x), whole(y));
  }
  // y's span j begins `off + d * stride` behind x's span i, d = j - i: whether for one it lies
  // between -y's bytes and x's; the least d above the former, and not below -(count of x - 1)
  using Wide = __int128;
  const Wide s = x.stride, off = static_cast<Wide>(reinterpret_cast<uintptr_t>(y.first.at)) - static_cast<Wide>(reinterpret_cast<uintptr_t>(x.first.at));
  const Wide low = -static_cast<Wide>(y.first.bytes) - off;
  Wide d = (low >= 0 ? low / s : -((-low + s - 1) / s)) + 1;
  if (d < 1 - static_cast<Wide>(x.count)) d = 1 - static_cast<Wide>(x.count);
  return d <= static_cast<Wide>(y.count) - 1 && off + d * s < static_cast<Wide>(x.first.bytes);
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
