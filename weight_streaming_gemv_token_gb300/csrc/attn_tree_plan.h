// How a call of attn_tree_paged is cut up, and its limits on sizes: arithmetic in
// plain C++ for host and device, so that it can be tested without a GPU.
//
// The work is a line of key tiles: first those of the shared prefix, head by head and,
// within a head, row tile by row tile (of all rows of the step); then request by
// request, head by head, row tile by row tile those of the request's own keys. The
// tiles of one (request, head, row tile) are a segment, in front of which kAtExtra units
// without a tile stand for what a segment costs beside its tiles (queries, first and last
// steps; without them the CTA with a step's shortest requests ends last: 64 rows behind
// 131,072 shared tokens 148 us, with them 127). Each CTA takes an equal share
// of the W units in all, across segments; its part of a segment is a piece. Numbering
// segments j = 0, 1, .. along the line, the piece of CTA c in segment j has the number
// c + j: along the line every new piece has a new c or a new j, so no two share a number.
#pragma once
#include <cstdint>

#include "../../include/wsg.h"
#include "paging.h"

namespace wsg {

constexpr int kAtBatch = 4096, kAtKeyShift = 7, kAtKeys = 1 << kAtKeyShift;  // requests; keys a tile
constexpr int kAtExtra = 2;
constexpr long long kAtUnits = 1ll << 37;  // of all requests: what their sums hold (AtSums)

// What the cutting goes by. rows * group < 2^24, capacity <= 2^30: 32-bit arithmetic.
struct AtCut {
  int group, n_kv;
  int mshift;              // log2 of the rows (token, query head of the group) of a row tile
  int chain;               // no mask: a row sees the rows up to itself
  int capacity;            // tokens that a table row can hold
};

WSG_HD int at_row_tiles(const AtCut& c, int rows) { return (rows * c.group + (1 << c.mshift) - 1) >> c.mshift; }

// Keys that row tile t of a request of n tokens and `rows` rows looks at, and its key
// tiles (one at least: a row without keys has a result too).
WSG_HD int at_keys(const AtCut& c, int n, int rows, int t) {
  unsigned seen = static_cast<unsigned>(rows);
  if (c.chain) {
    const unsigned last = ((static_cast<unsigned>(t + 1) << c.mshift) - 1u) / static_cast<unsigned>(c.group) + 1u;
    if (last < seen) seen = last;
  }
  const unsigned keys = static_cast<unsigned>(n) + seen, cap = static_cast<unsigned>(c.capacity);
  return static_cast<int>(keys < cap ? keys : cap);
}
WSG_HD int at_tiles(const AtCut& c, int n, int rows, int t) {
  const int k = (at_keys(c, n, rows, t) + kAtKeys - 1) >> kAtKeyShift;
  return k < 1 ? 1 : k;
}
// Units of one head of a request's row tiles before t.
WSG_HD long long at_units_before(const AtCut& c, int n, int rows, int t) {
  if (!c.chain) return static_cast<long long>(t) * (at_tiles(c, n, rows, 0) + kAtExtra);
  long long sum = 0;
  for (int u = 0; u < t; ++u) sum += at_tiles(c, n, rows, u) + kAtExtra;
  return sum;
}
WSG_HD long long at_head_units(const AtCut& c, int n, int rows) { return at_units_before(c, n, rows, at_row_tiles(c, rows)); }

// x / y of non-negative numbers; the 64-bit division, some 100 instructions, only where needed.
WSG_HD long long at_div(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<unsigned>(x) / static_cast<unsigned>(y);
  return x / y;
}

// The shares of C CTAs of a line of W units: W mod C of W / C + 1 units, then the others.
struct AtShares {
  long long each, more;  // W / C, W mod C
};
WSG_HD AtShares at_shares(long long W, int C) {
  const long long q = at_div(W, C);
  return AtShares{q, W - q * C};
}
// First unit of CTA c, and the CTA that has unit p.
WSG_HD long long at_first(const AtShares& s, int c) { return s.each * c + (c < s.more ? c : s.more); }
WSG_HD int at_owner(const AtShares& s, long long p) {
  const long long big = s.more * (s.each + 1);
  return static_cast<int>(p < big ? at_div(p, s.each + 1) : s.more + at_div(p - big, s.each));
}

// Most units that requests can have at these sizes, rows in row tiles of 16 and tables full: a
// request's row tiles are its rows * group / 16 and one more.
inline long long at_most_units(const attn_tree_args* a) {
  const long long tiles = ((static_cast<long long>(a->table_stride) << page_shift(a->page_size)) + kAtKeys - 1) / kAtKeys;
  return (static_cast<long long>(a->rows) * a->n_q / 16 + static_cast<long long>(a->batch < a->rows ? a->batch : a->rows) * a->n_kv) *
         ((tiles < 1 ? 1 : tiles) + kAtExtra);
}

inline bool attn_tree_sizes_ok(const attn_tree_args* a) {
  auto type = [](int t) { return t == DEC_F32 || t == DEC_BF16; };
  return a->batch >= 0 && a->batch <= kAtBatch && a->rows >= 0 && a->n_kv >= 1 && a->n_q >= a->n_kv && a->n_q <= 65535 &&
         static_cast<long long>(a->rows) * a->n_q < 1ll << 24 && a->n_q % a->n_kv == 0 && a->n_q / a->n_kv <= 16 &&
         a->head_dim >= 8 && a->head_dim <= 128 && a->head_dim % 8 == 0 && type(a->qdtype) && type(a->kvdtype) &&
         a->prefix_len >= 0 && page_shift(a->page_size) >= 0 && a->num_pages >= 0 && a->table_stride >= 0 &&
         a->mask_words >= 0 && a->mask_words <= 1 << 20 &&
         (static_cast<long long>(a->table_stride) << page_shift(a->page_size)) + a->prefix_len <= (1ll << 30) &&
         at_most_units(a) < kAtUnits;
}

// Which kernel runs, and the workspace.
struct AtPlan {
  bool tc;            // attn_tree_tc_kernel
  int per_sm, ctas;   // CTAs an SM, in all: the shares of the line
  AtCut cut;
  int prefix_row_tiles, prefix_tiles;  // of a head; of a segment
  long long pieces;   // numbers that pieces can have
  int seams;          // records of seams: the most segments there can be, or the CTAs
  size_t o, ml, rec, line, total;  // workspace: outputs, (reference, sum), records (of rows or seams), the line's length
};

// Where a row's pieces are: its own segment's first tile is unit `line` for head 0, of
// `tiles` (0: a row without a result), `head` units on for the next head; its
// number is seg for head 0, row_tiles on for the next.
struct AtRow {
  long long line, head;
  int32_t tiles, seg, row_tiles;
  int32_t at, next, pad;  // row (token * group) within the row tile; tiles of the row tile behind it
};

// Without a prefix a row has one segment, and only segments that are cut need joining: at
// most one starts in a CTA's share and ends behind it. Its pieces have the numbers id ..
// id + pieces - 1 (0 pieces: none). Records lie by segment where there are no more of
// those than CTAs, else by CTA.
struct AtSeam {
  long long id;
  int32_t pieces, begin, m0, nrows, g, pad;
};

inline AtPlan attn_tree_plan(const attn_tree_args* a, int sms) {
  AtPlan p{};
  p.total = 256;
  if (a->batch == 0 || a->rows == 0) return p;
  const int group = a->n_q / a->n_kv;
  p.cut.group = group;
  p.cut.n_kv = a->n_kv;
  p.cut.chain = a->mask == nullptr;
  p.cut.capacity = a->table_stride << page_shift(a->page_size);
  // rows that a request brings on average; key tiles a CTA, were the tables full
  const long long most = static_cast<long long>(a->rows) * group / (a->batch < a->rows ? a->batch : a->rows);
  const long long full = (static_cast<long long>(a->batch) * p.cut.capacity + a->prefix_len) / kAtKeys * a->n_kv / sms;
  // bfloat16 throughout, a head of 64 or 128, pages of whole swizzled groups of rows: on the
  // tensor cores, but for rows that one row tile of 16 holds (all of the step's, where a
  // prefix is read once a row tile) and, with heads of 128, not too many keys. Warp-level and
  // tensor-core form: 1 token x 500 9.7 and 12.8 us, 256 x 500 104 and 173, 8 x 4,096 33 and
  // 37, 32 x 4,096 98 and 99, 16 x 16,000 174 and 172; of heads of 64, where the latter's
  // softmax takes longer than the bytes, 8 x 4,096 24 and 31, 48 x 7,000 120 and 194. (By the
  // tables' width: the lengths are on the device.)
  const bool few = most <= 16 && (a->prefix_len == 0 || static_cast<long long>(a->rows) * group <= 16);
  const bool brief = a->head_dim == 64 || full <= 48 || p.cut.capacity <= 1024;
  p.tc = a->qdtype == DEC_BF16 && a->kvdtype == DEC_BF16 && (a->head_dim == 128 || a->head_dim == 64) && a->page_size >= 8 &&
         a->table_stride > 0 && a->num_pages > 0 && static_cast<long long>(a->num_pages) * a->n_kv < 1ll << 31 &&
         (a->prefix_len == 0 || a->prefix_stride < 1ll << 31) && !(few && brief);
  // otherwise as many rows a row tile as a request brings on average, 16 to 64. In tiles of
  // 16, of 32 or 64, float32 queries: 8 x 32 rows x 4,096 tokens of bfloat16 79 and 73 us,
  // 32 x 128 rows 932 and 692; of float32, where a block's chain bounds either, 117 and 120,
  // 1,610 and 1,545.
  if (p.tc)
    p.cut.mshift = 7;
  else if (a->kvdtype == DEC_F32)
    p.cut.mshift = most <= 32 ? 4 : 6;
  else
    p.cut.mshift = most <= 16 ? 4 : most <= 32 ? 5 : 6;
  const int mt = 1 << p.cut.mshift;
  if (a->prefix_len > 0) {
    p.prefix_row_tiles = at_row_tiles(p.cut, a->rows);
    p.prefix_tiles = (a->prefix_len + kAtKeys - 1) / kAtKeys;
  }
  // the requests' row tiles: rows * group / mt whole ones at most, one more each
  const long long own = static_cast<long long>(a->rows) * group / mt + (a->batch < a->rows ? a->batch : a->rows);
  const long long segments = (own + p.prefix_row_tiles) * a->n_kv;
  // as many small CTAs an SM as there are segments for (and as rings and row groups allow):
  // 256 requests of one token x 16 tokens with one 64 us, with two 35, with four 25 (27 since a
  // block's products are added by themselves); 4 requests of 8 rows x 1,000 15, 16 and 17; 64 of
  // 32 float32 rows x 100 73 and 48.
  if (p.tc || a->kvdtype == DEC_F32)
    p.per_sm = 1;
  else if (p.cut.mshift > 4)
    p.per_sm = segments > sms ? 2 : 1;
  else
    p.per_sm = segments > sms ? 4 : 2 * segments > sms || a->prefix_len > 0 ? 2 : 1;
  p.ctas = sms * p.per_sm;
  p.pieces = p.ctas + segments;
  p.seams = segments < p.ctas ? static_cast<int>(segments) : p.ctas;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = static_cast<size_t>(p.pieces) * mt;
  p.o = 0;
  p.ml = up(rows * a->head_dim * 4);
  p.rec = p.ml + up(rows * 8);
  p.line = p.rec + up(a->prefix_len > 0 ? static_cast<size_t>(a->rows) * sizeof(AtRow) : static_cast<size_t>(p.ctas) * sizeof(AtSeam));
  p.total = p.line + 256;
  return p;
}

}  // namespace wsg
