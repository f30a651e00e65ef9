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
  AtRow* rec;
  long long* total;  // [1]: key tiles of the line
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
  long long pos, end, prefix;  // tiles; those of the prefix
  long long seg;               // number of the segment at hand
  // the request at hand (s < 0: none yet)
  int s, begin, rows, n, g, t, tile, row_tiles;
  int first_s, first_begin;    // where the requests begin for this CTA

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
      p.prefix = false;
      p.whole = tile == 0 && prefix == 0 && kt <= end - pos;
      p.s = s;
      p.g = g;
      p.begin = begin;
      p.rows = rows;
      p.n = n;
      p.m0 = t << a.cut.mshift;
      p.k1 = at_keys(a.cut, n, rows, t);
      ++t;
    }
    const int take = static_cast<int>(min(static_cast<long long>(kt - tile), end - pos));
    p.nrows = min(1 << a.cut.mshift, p.rows * a.cut.group - p.m0);
    p.k0 = tile << kAtKeyShift;
    p.k1 = min(p.k1, (tile + take) << kAtKeyShift);
    p.tiles = take;
    p.id = seg + blockIdx.x;
    pos += take;
    tile = 0;
    ++seg;
    return p;
  }
};

// A CTA's place on the line, and the requests whose rows' records it writes (s modulo
// the CTAs; 4096 requests at most, 64 CTAs at least).
struct AtShared {
  AtWalk walk;
  int count, top;  // top: behind the requests' last row
  struct Mine {
    long long line;
    int s, begin, rows, n, seg;
  } mine[64];
};

// One warp: sums the requests' lengths, a run of them a lane, and finds this CTA's place.
__device__ __forceinline__ void at_start(const AtArgs& a, AtShared& sh) {
  const int lane = threadIdx.x & 31, batch = a.a.batch, ctas = gridDim.x, cta = blockIdx.x;
  const int per = (batch + 31) / 32, lo = min(batch, lane * per), hi = min(batch, lo + per);
  // the highest row start up to this lane's first request (starts that fall are lifted)
  int top = 0;
#pragma unroll 4
  for (int i = lo; i < hi; ++i) top = max(top, AtWalk::clamp_row(a, a.row_start[i]));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, top, o);
    if (lane >= o) top = max(top, y);
  }
  const int last = max(__shfl_sync(0xffffffffu, top, 31), AtWalk::clamp_row(a, a.row_start[batch]));
  int before = __shfl_up_sync(0xffffffffu, top, 1);
  if (lane == 0) before = 0, sh.count = 0, sh.top = last;
  __syncwarp();
  // Tiles and segments of this lane's requests, then with the sums of the lanes before
  // this CTA's place among them.
  const long long prefix_segs = static_cast<long long>(a.cut.n_kv) * a.prefix_row_tiles, prefix = prefix_segs * a.prefix_tiles;
  long long line = 0, segs = 0, want = -1;
  AtWalk w;
  w.s = -1;
  w.tile = w.g = w.t = w.rows = w.row_tiles = w.n = w.begin = 0;
  w.seg = 0;
  w.prefix = prefix;
  w.first_s = w.first_begin = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int from = before;
#pragma unroll 2
    for (int i = lo; i < hi; ++i) {
      from = max(from, AtWalk::clamp_row(a, a.row_start[i]));
      const int len = a.a.len[i], n_rows = len < 0 ? 0 : max(0, AtWalk::clamp_row(a, a.row_start[i + 1]) - from);
      const long long tl = n_rows ? a.cut.n_kv * at_head_tiles(a.cut, len, n_rows) : 0;
      if (pass) {
        if (line <= want && want < line + tl) {  // (one lane)
          sh.walk.first_s = i;
          sh.walk.first_begin = from;
          sh.walk.pos = line;
          sh.walk.seg = segs;
        }
        if (i % ctas == cta) {
          const int k = atomicAdd(&sh.count, 1);
          if (k < 64) sh.mine[k] = {prefix + line, i, from, n_rows, len, static_cast<int>(prefix_segs + segs)};
        }
      }
      line += tl;
      segs += static_cast<long long>(a.cut.n_kv) * at_row_tiles(a.cut, n_rows);
    }
    if (pass == 0) {
      long long x = line, y = segs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += u, y += v;
      }
      const long long W = prefix + __shfl_sync(0xffffffffu, x, 31);
      line = x - line;
      segs = y - segs;
      const int C = static_cast<int>(min(static_cast<long long>(ctas), W));
      w.pos = cta < C ? at_first(W, C, cta) : 0;
      w.end = cta < C ? at_first(W, C, cta + 1) : 0;
      want = w.pos < w.end ? max(w.pos, prefix) - prefix : -1;  // this CTA's first own tile
      if (cta == 0 && lane == 0) *a.total = W;
    }
  }
  __syncwarp();
  if (w.pos < w.end) {
    const long long line0 = sh.walk.pos, seg0 = sh.walk.seg;
    w.first_s = sh.walk.first_s;
    w.first_begin = sh.walk.first_begin;
    if (w.pos < prefix) {
      w.seg = at_div(w.pos, a.prefix_tiles);
      w.tile = static_cast<int>(w.pos - w.seg * a.prefix_tiles);
    } else {
      w.enter(a, w.first_s, w.first_begin);
      long long rest = w.pos - prefix - line0;
      const long long head = at_head_tiles(a.cut, w.n, w.rows);
      w.g = static_cast<int>(at_div(rest, head));
      rest -= w.g * head;
      if (a.cut.chain) {
        for (int k; rest >= (k = at_tiles(a.cut, w.n, w.rows, w.t)); ++w.t) rest -= k;
      } else {
        const int k = at_tiles(a.cut, w.n, w.rows, 0);
        w.t = static_cast<int>(at_div(rest, k));
        rest -= static_cast<long long>(w.t) * k;
      }
      w.tile = static_cast<int>(rest);
      w.seg = prefix_segs + seg0 + static_cast<long long>(w.g) * w.row_tiles + w.t;
    }
  }
  __syncwarp();
  if (lane == 0) sh.walk = w;
  __syncwarp();
}

// One warp, at any time behind at_start: the records that attn_tree_join_kernel goes by.
__device__ __forceinline__ void at_records(const AtArgs& a, const AtShared& sh) {
  const int lane = threadIdx.x & 31, count = min(64, sh.count);
  for (int k = 0; k < count; ++k) {
    const AtShared::Mine x = sh.mine[k];
    if (x.rows == 0) {  // rows of an unused request
      const int e = max(x.begin, AtWalk::clamp_row(a, a.row_start[x.s + 1]));
      for (int r = x.begin + lane; r < e; r += 32) a.rec[r].tiles = 0;
      continue;
    }
    const long long head = at_head_tiles(a.cut, x.n, x.rows);
    const int rt = at_row_tiles(a.cut, x.rows);
    if (lane == 0 && static_cast<long long>(x.n) + x.rows > a.cut.capacity) atomicOr(a.a.err, ERR_BAD_PAGE);
    for (int i = lane; i < x.rows; i += 32) {
      // a token's query heads may lie in two row tiles: the record is the first one's,
      // the other's follows from it
      const int t = (i * a.cut.group) >> a.cut.mshift;
      AtRow r;
      r.line = x.line + at_tiles_before(a.cut, x.n, x.rows, t);
      r.head = head;
      r.tiles = at_tiles(a.cut, x.n, x.rows, t);
      r.seg = x.seg + t;
      r.row_tiles = rt;
      r.at = i * a.cut.group - (t << a.cut.mshift);
      r.next = t + 1 < rt ? at_tiles(a.cut, x.n, x.rows, t + 1) : 0;
      r.pad = 0;
      a.rec[x.begin + i] = r;
    }
  }
  if (blockIdx.x == 0) {  // rows of no request
    const int first = AtWalk::clamp_row(a, a.row_start[0]);
    for (int r = lane; r < first; r += 32) a.rec[r].tiles = 0;
    for (int r = sh.top + lane; r < a.a.rows; r += 32) a.rec[r].tiles = 0;
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

cudaError_t launch_tree_bf16(const AtArgs& a, bool q_f32, const DeviceInfo& di, cudaStream_t st);
cudaError_t launch_tree_f32(const AtArgs& a, bool q_f32, const DeviceInfo& di, cudaStream_t st);
dec_status launch_tree_tc(const AtArgs& a, const DeviceInfo& di, cudaStream_t st);

}  // namespace wsg
