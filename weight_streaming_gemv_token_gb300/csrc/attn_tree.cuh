// What the kernels of attn_tree_paged share: arguments, the way along the line of key
// tiles (attn_tree_plan.h), masks of drafted rows.
#pragma once
#include "attn_rows.cuh"
#include "attn_tree_plan.h"

namespace wsg {

struct AtArgs {
  AmArgs a;  // queries, prefix, pools, scale; of the rest `rows` (of the step) and `batch`
  AtCut cut;
  const int32_t* row_start;
  const uint32_t* mask;
  int words;
  int prefix_row_tiles, prefix_tiles;
  void* out;
  long long out_stride;
  int out16;  // rows of out can be written in 16-byte pieces
  float* lse;
  AtRow* rec;        // with a prefix: of every row
  AtSeam* seam;      // without: [seams], by segment (seam_segs) or by CTA
  int seams, seam_segs;
  int per_sm;        // CTAs an SM
  long long* total;  // [1]: units of the line
};

// A piece: keys k0 .. k1 - 1 of a segment against its rows.
struct AtPiece {
  bool prefix, whole;  // whole: the whole segment, whose rows have no prefix
  int s, g;
  int begin, rows, n;  // the request's first row, its rows, its tokens in pages
  int m0, nrows;       // the row tile: first row (token * group + head) and rows
  int k0, k1;
  int tiles;           // key tiles, one at least; 0: no piece, the share has ended
  long long id;
};

// The way of a CTA along the line.
struct AtWalk {
  long long pos, end, prefix;  // units; those of the prefix
  long long seg;               // number of the segment at hand
  // the request at hand (s < 0: none yet)
  int s, begin, rows, n, g, t, unit, row_tiles;  // unit: the place in the segment
  int first_s, first_begin;    // where the requests begin for this CTA
  AtShares shares;
  AtSeam seam;                 // the segment that starts in this share and is cut behind it
  int seam_seg;
  int segs;                    // of all requests
  int seg0, seg1;              // segments whose first tile lies in this share: seg0 .. seg1 - 1

  __device__ __forceinline__ static int clamp_row(const AtArgs& a, int r) { return min(max(0, r), a.a.rows); }

  // request i, whose rows start at `from` or behind
  __device__ __forceinline__ void enter(const AtArgs& a, int i, int from) {
    s = i;
    begin = max(from, clamp_row(a, a.row_start[i]));
    n = a.a.len[i];
    rows = n < 0 ? 0 : max(0, clamp_row(a, a.row_start[i + 1]) - begin);
    row_tiles = at_row_tiles(a.cut, rows);
    g = t = 0;
  }

  // The next piece.
  __device__ __forceinline__ AtPiece next(const AtArgs& a) {
    AtPiece p;
    p.tiles = 0;
    if (pos >= end) return p;
    int kt;
    if (pos < prefix) {
      const int at = static_cast<int>(seg), head = at / a.prefix_row_tiles, rt = at - head * a.prefix_row_tiles;
      kt = a.prefix_tiles;
      p.prefix = true;
      p.whole = false;  // a row has own keys too
      p.s = -1;
      p.g = head;
      p.begin = 0;
      p.rows = a.a.rows;
      p.n = 0;
      p.m0 = rt << a.cut.mshift;
      p.k1 = a.a.plen;
    } else {
      if (s < 0) {
        enter(a, first_s, first_begin);  // the first request with rows
      } else if (t >= row_tiles) {
        t = 0;
        if (++g >= a.cut.n_kv) {
          do {
            if (s + 1 >= a.a.batch) return p;  // (there is one: tiles are left)
            const int reach = max(begin, clamp_row(a, a.row_start[s + 1]));
            enter(a, s + 1, reach);
          } while (rows == 0);
        }
      }
      kt = at_tiles(a.cut, n, rows, t);
      // (the CTA with a request's first unit reports tokens beyond the tables)
      if (g == 0 && t == 0 && unit == 0 && static_cast<long long>(n) + rows > a.cut.capacity && (threadIdx.x & 31) == 0)
        atomicOr(a.a.err, ERR_BAD_PAGE);
      p.prefix = false;
      p.whole = prefix == 0;
      p.s = s;
      p.g = g;
      p.begin = begin;
      p.rows = rows;
      p.n = n;
      p.m0 = t << a.cut.mshift;
      p.k1 = at_keys(a.cut, n, rows, t);
      ++t;
    }
    const int left = kt + kAtExtra - unit, take = static_cast<int>(min(static_cast<long long>(left), end - pos));
    const int t0 = max(0, unit - kAtExtra), t1 = max(0, unit + take - kAtExtra);
    p.whole = p.whole && t0 == 0 && t1 == kt;
    p.nrows = min(1 << a.cut.mshift, p.rows * a.cut.group - p.m0);
    p.k0 = t0 << kAtKeyShift;
    p.k1 = min(p.k1, t1 << kAtKeyShift);
    p.tiles = t1 - t0;  // (0: the share ends in front of the segment's tiles)
    p.id = seg + blockIdx.x;
    if (t0 == 0 && t1 > 0 && t1 < kt) {  // (the share's last piece)
      seam_seg = static_cast<int>(seg);
      seam.id = p.id;
      seam.pieces = at_owner(shares, pos + left - 1) - static_cast<int>(blockIdx.x) + 1;
      seam.begin = p.begin;
      seam.m0 = p.m0;
      seam.nrows = p.nrows;
      seam.g = p.g;
    }
    pos += take;
    unit = 0;
    ++seg;
    if (t0 == 0 && t1 > 0) seg1 = static_cast<int>(seg);
    return p;
  }
};

// The requests' sums as one warp forms them, a run of requests a lane: units << 26 |
// segments of all requests (at most n_kv times the rows and 2^24 / 16 of those; fewer than
// 2^37 units, or the sizes are refused), of those before this lane's, and this lane's first
// request. Row starts that fall are lifted to the highest before.
struct AtSums {
  int lo, hi;          // this lane's requests
  int from, rows, len; // the first one's first row, rows, tokens
  long long size, before, all;
  int end;             // behind the requests' last row
};

// A request from its row start and the next one's, *from the highest start before: *from its
// first row; *rows; units << 26 | segments.
__device__ __forceinline__ long long at_size(const AtArgs& a, int start, int end, int len, int* from, int* rows) {
  *from = max(*from, start);
  *rows = len < 0 ? 0 : max(0, end - *from);
  if (*rows == 0) return 0;
  return (a.cut.n_kv * at_head_units(a.cut, len, *rows)) << 26 | static_cast<long long>(a.cut.n_kv * at_row_tiles(a.cut, *rows));
}

__device__ __forceinline__ AtSums at_sums(const AtArgs& a) {
  const int lane = threadIdx.x & 31, batch = a.a.batch, per = (batch + 31) >> 5;
  AtSums s;
  s.lo = min(batch, lane * per);
  s.hi = min(batch, s.lo + per);
  auto start = [&](int i) { return AtWalk::clamp_row(a, a.row_start[i]); };
  const int rs0 = start(s.lo), rs1 = start(min(batch, s.lo + 1));
  s.len = s.lo < s.hi ? a.a.len[s.lo] : -1;
  s.end = start(batch);
  bool rising = rs0 <= rs1;
  int top = s.lo < s.hi ? rs0 : 0;
#pragma unroll 2
  for (int i = s.lo + 1; i < s.hi; ++i) {
    const int x = start(i);
    rising = rising && x <= start(i + 1);
    top = max(top, x);
  }
  int before = rs0;  // the highest start before this lane's requests, or theirs
  if (!__all_sync(0xffffffffu, rising)) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, top, o);
      if (lane >= o) top = max(top, y);
    }
    s.end = max(s.end, __shfl_sync(0xffffffffu, top, 31));
    before = __shfl_up_sync(0xffffffffu, top, 1);
    if (lane == 0) before = 0;
  }
  s.from = before;
  s.rows = 0;
  s.size = s.lo < s.hi ? at_size(a, rs0, rs1, s.len, &s.from, &s.rows) : 0;
  long long sum = s.size;
  int from = s.from;
#pragma unroll 1
  for (int i = s.lo + 1; i < s.hi; ++i) {
    int r;
    sum += at_size(a, start(i), start(i + 1), a.a.len[i], &from, &r);
  }
  long long x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  s.all = __shfl_sync(0xffffffffu, x, 31);
  s.before = x - sum;
  return s;
}

// Calls f(request, first row, rows, tokens, size, sizes before) for this lane's requests.
template <typename F>
__device__ __forceinline__ void at_each(const AtArgs& a, const AtSums& s, F f) {
  if (s.lo >= s.hi) return;
  f(s.lo, s.from, s.rows, s.len, s.size, s.before);
  long long x = s.before + s.size;
  int from = s.from;
#pragma unroll 1
  for (int i = s.lo + 1; i < s.hi; ++i) {
    const int len = a.a.len[i];
    int r;
    const long long size = at_size(a, AtWalk::clamp_row(a, a.row_start[i]), AtWalk::clamp_row(a, a.row_start[i + 1]), len, &from, &r);
    f(i, from, r, len, size, x);
    x += size;
  }
}

// One warp: this CTA's place on the line. What it costs is a chain of loads, shuffles and
// divisions before the first keys can be asked for, about 2 us of a call.
__device__ __forceinline__ AtWalk at_start(const AtArgs& a) {
  const int ctas = gridDim.x, cta = blockIdx.x;
  const AtSums s = at_sums(a);
  const long long prefix_segs = static_cast<long long>(a.cut.n_kv) * a.prefix_row_tiles, prefix = prefix_segs * (a.prefix_tiles + kAtExtra);
  const long long W = prefix + (s.all >> 26);
  AtWalk w;
  w.pos = w.end = 0;
  w.shares = AtShares{1, 0};
  w.seam = AtSeam{};
  w.seam_seg = -1;
  w.segs = static_cast<int>(s.all & ((1 << 26) - 1));
  if (cta < W) {
    w.shares = at_shares(W, static_cast<int>(min(static_cast<long long>(ctas), W)));
    w.pos = at_first(w.shares, cta);
    w.end = at_first(w.shares, cta + 1);
  }
  w.s = -1;
  w.unit = w.g = w.t = w.rows = w.row_tiles = w.n = w.begin = 0;
  w.seg = 0;
  w.prefix = prefix;
  // this CTA's first unit of requests, and the request that has it
  const long long want = w.pos < w.end ? max(w.pos, prefix) - prefix : -1;
  int mine_s = -1, mine_from = 0, mine_rows = 0, mine_len = 0;
  long long mine_at = 0;
  at_each(a, s, [&](int i, int f, int r, int len, long long size, long long x) {
    if (x >> 26 <= want && want < (x >> 26) + (size >> 26)) mine_s = i, mine_from = f, mine_rows = r, mine_len = len, mine_at = x;
  });
  const unsigned who = __ballot_sync(0xffffffffu, mine_s >= 0);
  const int src = who ? __ffs(who) - 1 : 0;
  w.first_s = __shfl_sync(0xffffffffu, mine_s, src);
  w.first_begin = __shfl_sync(0xffffffffu, mine_from, src);
  if (w.pos < w.end) {
    if (w.pos < prefix) {
      w.seg = at_div(w.pos, a.prefix_tiles + kAtExtra);
      w.unit = static_cast<int>(w.pos - w.seg * (a.prefix_tiles + kAtExtra));
    } else {
      w.s = w.first_s;
      w.begin = w.first_begin;
      w.rows = __shfl_sync(0xffffffffu, mine_rows, src);
      w.n = __shfl_sync(0xffffffffu, mine_len, src);
      w.row_tiles = at_row_tiles(a.cut, w.rows);
      const long long at = __shfl_sync(0xffffffffu, mine_at, src);
      long long rest = w.pos - prefix - (at >> 26);
      if (a.cut.chain) {
        const long long head = at_head_units(a.cut, w.n, w.rows);
        w.g = static_cast<int>(at_div(rest, head));
        rest -= w.g * head;
        for (int k; rest >= (k = at_tiles(a.cut, w.n, w.rows, w.t) + kAtExtra); ++w.t) rest -= k;
      } else {
        const int k = at_tiles(a.cut, w.n, w.rows, 0) + kAtExtra, n = static_cast<int>(at_div(rest, k));
        rest -= static_cast<long long>(n) * k;
        w.g = n / w.row_tiles;
        w.t = n - w.g * w.row_tiles;
      }
      w.unit = static_cast<int>(rest);
      w.seg = prefix_segs + (at & ((1 << 26) - 1)) + static_cast<long long>(w.g) * w.row_tiles + w.t;
    }
  }
  // (the segment at hand starts here unless its first tile lies before)
  w.seg0 = static_cast<int>(w.seg) + (w.unit > kAtExtra ? 1 : 0);
  w.seg1 = w.seg0;
  return w;
}

// One warp, behind its share's last piece, without a prefix: the records that the join
// goes by.
__device__ __forceinline__ void at_seams(const AtArgs& a, const AtWalk& w) {
  const int lane = threadIdx.x & 31;
  if (!a.seam_segs) {
    if (lane == 0) a.seam[blockIdx.x] = w.seam;
    return;
  }
  // segments that start in this share, and in CTA 0 those that there are not
  for (int k = w.seg0 + lane; k < w.seg1; k += 32) a.seam[k] = k == w.seam_seg ? w.seam : AtSeam{};
  if (blockIdx.x == 0)
    for (int k = w.segs + lane; k < a.seams; k += 32) a.seam[k] = AtSeam{};
}

// One warp, with a prefix, beside the work: the rows' records, of rows r with r % gridDim.x
// == blockIdx.x (all of a request's by one lane took longer than its work for a prompt).
[[maybe_unused]] static __device__ __noinline__ void at_records(const AtArgs& a) {
  const int lane = threadIdx.x & 31;
  const AtSums s = at_sums(a);
  const long long prefix_segs = static_cast<long long>(a.cut.n_kv) * a.prefix_row_tiles, prefix = prefix_segs * (a.prefix_tiles + kAtExtra);
  if (blockIdx.x == 0 && lane == 0) *a.total = prefix + (s.all >> 26);
  at_each(a, s, [&](int i, int from, int rows, int len, long long size, long long x) {
    const int ctas = gridDim.x, place = from % ctas;  // k0: this CTA's first row of the request
    const int k0 = static_cast<int>(blockIdx.x) - place + (static_cast<int>(blockIdx.x) < place ? ctas : 0);
    if (rows == 0) {  // rows of an unused request
      const int e = max(from, AtWalk::clamp_row(a, a.row_start[i + 1]));
      for (int r = from + k0; r < e; r += ctas) a.rec[r].tiles = 0;
      return;
    }
    if (k0 >= rows) return;
    const long long head = at_head_units(a.cut, len, rows);
    const int rt = at_row_tiles(a.cut, rows);
    long long line = prefix + (x >> 26) + kAtExtra;
    int t = 0, tiles = at_tiles(a.cut, len, rows, 0);
    for (int k = k0; k < rows; k += ctas) {
      // a token's query heads may lie in two row tiles: the record is the first one's,
      // the other's follows from it
      const int at = (k * a.cut.group) >> a.cut.mshift;
      for (; t < at; ++t) line += tiles + kAtExtra, tiles = at_tiles(a.cut, len, rows, t + 1);
      AtRow r;
      r.line = line;
      r.head = head;
      r.tiles = tiles;
      r.seg = static_cast<int>(prefix_segs + (x & ((1 << 26) - 1))) + t;
      r.row_tiles = rt;
      r.at = k * a.cut.group - (t << a.cut.mshift);
      r.next = t + 1 < rt ? at_tiles(a.cut, len, rows, t + 1) : 0;
      r.pad = 0;
      a.rec[from + k] = r;
    }
  });
  if (blockIdx.x == 0) {  // rows of no request
    const int first = AtWalk::clamp_row(a, a.row_start[0]);
    for (int r = lane; r < first; r += 32) a.rec[r].tiles = 0;
    for (int r = s.end + lane; r < a.a.rows; r += 32) a.rec[r].tiles = 0;
  }
}

// Which of the 32 keys from number j0 of the drafted rows on (below 0: tokens in pages)
// row i of the request sees.
__device__ __forceinline__ uint32_t at_seen(const AtArgs& a, int begin, int i, int j0) {
  if (j0 <= -32) return 0xffffffffu;
  if (!a.mask) {
    const int k = i - j0 + 1;
    return k >= 32 ? 0xffffffffu : k > 0 ? (1u << k) - 1u : 0u;
  }
  const uint32_t* row = a.mask + static_cast<long long>(begin + i) * a.words;
  if (j0 < 0) return (a.words > 0 ? row[0] << -j0 : 0u) | ((1u << -j0) - 1u);
  const int w = j0 >> 5;
  const uint32_t lo = w < a.words ? row[w] : 0u, hi = w + 1 < a.words ? row[w + 1] : 0u;
  return __funnelshift_r(lo, hi, j0 & 31);
}

__device__ __forceinline__ bool at_odd16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }  // a bfloat16 that is not finite
// A pair of bfloat16 whose values that are not finite are 0.
__device__ __forceinline__ uint32_t at_finite2(uint32_t p) {
  if (at_odd16(p)) p &= 0xFFFF0000u;
  if (at_odd16(p >> 16)) p &= 0xFFFFu;
  return p;
}

// Elements e .. e + 3 of a row's result from its weighted sum x, reference m and sum l;
// with e = 0 its log-sum.
template <typename QT>
__device__ __forceinline__ void at_put(const AtArgs& p, int row, int head, int e, float4 x, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a NaN sum stays one
  QT* dst = static_cast<QT*>(p.out) + p.out_stride * row + static_cast<long long>(head) * p.a.d + e;
  const float r[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
  const bool vec = reinterpret_cast<uintptr_t>(dst) % (4 * sizeof(QT)) == 0;
  if constexpr (sizeof(QT) == 4) {
    if (vec) {
      *reinterpret_cast<float4*>(dst) = make_float4(r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = r[i];
    }
  } else {
    uint32_t h[2];
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(r[1]), "f"(r[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(r[3]), "f"(r[2]));
    if (vec) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)));
    }
  }
  if (p.lse && e == 0)
    p.lse[static_cast<long long>(row) * p.a.n_q + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

// by the types of queries and cache; wide: heads above 64
cudaError_t launch_tree_bf16_bf16(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_bf16_bf16_wide(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_f32_bf16(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_f32_bf16_wide(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_bf16_f32(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_bf16_f32_wide(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_f32_f32(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_f32_f32_wide(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);
dec_status launch_tree_tc(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);

}  // namespace wsg
