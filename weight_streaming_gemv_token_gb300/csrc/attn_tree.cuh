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
  float* lse;
  AtRow* rec;
  long long* total;  // [1]: key tiles of the line
};

// A piece: keys k0 .. k1 - 1 of a segment against its rows.
struct AtPiece {
  bool prefix, whole;  // whole: the whole segment
  int s, g;
  int begin, rows, n;  // the request's first row, its rows, its tokens in pages
  int m0, nrows;       // the row tile: first row (token * group + head) and rows
  int k0, k1;
  long long id;
};

struct AtShared {
  long long warp[32][2];
  int most[32];
  long long line0, seg0;        // the first request of this CTA's share: tiles and segments before it
  int s, begin;
  int count;                    // requests whose records this CTA writes
  struct {
    long long line;
    int s, begin, rows, n, seg;
  } mine[64];
};

// The way of a CTA along the line; the same in all of its threads.
struct AtWalk {
  long long pos, end, prefix;  // tiles; those of the prefix
  long long seg;               // number of the segment at hand
  int cta;
  // the request at hand
  int s, begin, rows, n, g, t, tile, row_tiles;

  __device__ __forceinline__ static int clamp_row(const AtArgs& a, int r) { return min(max(0, r), a.a.rows); }

  // Block-wide (NT threads): sums the lengths, finds this CTA's place, and writes the
  // records of the requests s with s % gridDim.x == blockIdx.x.
  template <int NT>
  __device__ __forceinline__ void start(const AtArgs& a, AtShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, batch = a.a.batch;
    const int per = (batch + NT - 1) / NT, lo = min(batch, tid * per), hi = min(batch, lo + per);
    cta = blockIdx.x;
    // the highest row start up to this thread's first request (starts that fall are lifted)
    int top = 0;
    for (int i = lo; i < hi; ++i) top = max(top, clamp_row(a, a.row_start[i]));
    int inc = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = max(inc, y);
    }
    if (lane == 31) sh.most[warp] = inc;
    if (tid == 0) sh.count = 0;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) before = 0;
    for (int w = 0; w < warp; ++w) before = max(before, sh.most[w]);
    // tiles and segments of this thread's requests
    auto size = [&](int i, int* from, int* n_rows, int* len, long long* tiles, long long* segs) {
      *from = max(*from, clamp_row(a, a.row_start[i]));
      *n_rows = max(0, clamp_row(a, a.row_start[i + 1]) - *from);
      *len = a.a.len[i];
      *tiles = *segs = 0;
      if (*len < 0) *n_rows = 0;
      if (*n_rows > 0) {
        *tiles = static_cast<long long>(a.cut.n_kv) * at_head_tiles(a.cut, *len, *n_rows);
        *segs = static_cast<long long>(a.cut.n_kv) * at_row_tiles(a.cut, *n_rows);
      }
    };
    long long sum[2] = {0, 0};
    int from = before, n_rows, len;
    for (int i = lo; i < hi; ++i) {
      long long tl, sg;
      size(i, &from, &n_rows, &len, &tl, &sg);
      sum[0] += tl, sum[1] += sg;
    }
    long long x[2] = {sum[0], sum[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const long long y = __shfl_up_sync(0xffffffffu, x[i], o);
        if (lane >= o) x[i] += y;
      }
    }
    if (lane == 31) sh.warp[warp][0] = x[0], sh.warp[warp][1] = x[1];
    __syncthreads();
    long long line = x[0] - sum[0], segs = x[1] - sum[1], own = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) line += sh.warp[w][0], segs += sh.warp[w][1];
      own += sh.warp[w][0];
    }
    prefix = static_cast<long long>(a.cut.n_kv) * a.prefix_row_tiles * a.prefix_tiles;
    const long long W = prefix + own;
    const int C = static_cast<int>(min(static_cast<long long>(gridDim.x), W));
    pos = cta < C ? at_first(W, C, cta) : 0;
    end = cta < C ? at_first(W, C, cta + 1) : 0;
    const long long prefix_segs = static_cast<long long>(a.cut.n_kv) * a.prefix_row_tiles;
    const long long want = max(pos, prefix) - prefix;  // this CTA's first own tile
    from = before;
    for (int i = lo; i < hi; ++i) {
      long long tl, sg;
      size(i, &from, &n_rows, &len, &tl, &sg);
      if (tl > 0 && line <= want && want < line + tl) sh.s = i, sh.begin = from, sh.line0 = line, sh.seg0 = segs;
      if (i % static_cast<int>(gridDim.x) == cta) {  // at most 4096 / CTAs of them
        const int k = atomicAdd(&sh.count, 1);
        if (k < 64) {
          sh.mine[k].line = prefix + line;
          sh.mine[k].s = i;
          sh.mine[k].begin = from;
          sh.mine[k].rows = n_rows;
          sh.mine[k].n = len;
          sh.mine[k].seg = static_cast<int>(prefix_segs + segs);
        }
      }
      line += tl, segs += sg;
    }
    if (tid == 0 && cta == 0) *a.total = W;
    __syncthreads();
    // ---- records, a thread a row ----
    for (int k = 0; k < min(64, sh.count); ++k) {
      const int R = sh.mine[k].rows, n_ = sh.mine[k].n, b = sh.mine[k].begin;
      const int head = R > 0 ? at_head_tiles(a.cut, n_, R) : 0, rt = at_row_tiles(a.cut, R);
      if (tid == 0 && R > 0 && static_cast<long long>(n_) + R > a.cut.capacity) atomicOr(a.a.err, ERR_BAD_PAGE);
      for (int i = tid; i < R; i += NT) {
        // a token's query heads may lie in two row tiles: the record is the first one's,
        // the other's follows from it (attn_tree_join_kernel)
        const int t = static_cast<int>(static_cast<long long>(i) * a.cut.group / a.cut.mt);
        long long l = sh.mine[k].line;
        if (a.cut.chain)
          for (int u = 0; u < t; ++u) l += at_tiles(a.cut, n_, R, u);
        else
          l += static_cast<long long>(t) * at_tiles(a.cut, n_, R, 0);
        AtRow r;
        r.line = l;
        r.head = head;
        r.tiles = at_tiles(a.cut, n_, R, t);
        r.seg = sh.mine[k].seg + t;
        r.row_tiles = rt;
        r.at = static_cast<int>(static_cast<long long>(i) * a.cut.group - static_cast<long long>(t) * a.cut.mt);
        r.next = t + 1 < rt ? at_tiles(a.cut, n_, R, t + 1) : 0;
        a.rec[b + i] = r;
      }
    }
    // rows of no request, and of unused ones
    {
      for (int k = 0; k < min(64, sh.count); ++k) {
        const int i = sh.mine[k].s;
        if (sh.mine[k].rows > 0) continue;
        const int b = sh.mine[k].begin, e = max(b, clamp_row(a, a.row_start[i + 1]));
        for (int r = b + tid; r < e; r += NT) a.rec[r].tiles = 0;
      }
      if (cta == 0) {
        const int first = clamp_row(a, a.row_start[0]);
        for (int r = tid; r < first; r += NT) a.rec[r].tiles = 0;
        int last = 0;
        for (int w = 0; w < NT / 32; ++w) last = max(last, sh.most[w]);
        last = max(last, clamp_row(a, a.row_start[batch]));
        for (int r = last + tid; r < a.a.rows; r += NT) a.rec[r].tiles = 0;
      }
    }
    // ---- this CTA's place ----
    s = -1;
    tile = 0;
    if (pos >= end) return;
    if (pos < prefix) {
      seg = pos / a.prefix_tiles;
      tile = static_cast<int>(pos - seg * a.prefix_tiles);
    } else {
      enter(a, sh.s, sh.begin);
      long long rest = pos - prefix - sh.line0;
      const int head = at_head_tiles(a.cut, n, rows);
      g = static_cast<int>(rest / head);
      rest -= static_cast<long long>(g) * head;
      t = 0;
      if (a.cut.chain) {
        for (int k; rest >= (k = at_tiles(a.cut, n, rows, t)); ++t) rest -= k;
      } else {
        const int k = at_tiles(a.cut, n, rows, 0);
        t = static_cast<int>(rest / k);
        rest -= static_cast<long long>(t) * k;
      }
      tile = static_cast<int>(rest);
      seg = prefix_segs + sh.seg0 + static_cast<long long>(g) * row_tiles + t;
    }
  }

  // request i, whose rows start at `from` or behind
  __device__ __forceinline__ void enter(const AtArgs& a, int i, int from) {
    s = i;
    begin = max(from, clamp_row(a, a.row_start[i]));
    n = a.a.len[i];
    rows = n < 0 ? 0 : max(0, clamp_row(a, a.row_start[i + 1]) - begin);
    row_tiles = at_row_tiles(a.cut, rows);
    g = t = 0;
  }

  // The next piece; false at the end of the share.
  __device__ __forceinline__ bool next(const AtArgs& a, const AtShared& sh, AtPiece* p) {
    if (pos >= end) return false;
    if (pos < prefix) {
      const int head = static_cast<int>(seg / a.prefix_row_tiles), rt = static_cast<int>(seg - static_cast<long long>(head) * a.prefix_row_tiles);
      const int take = static_cast<int>(min(static_cast<long long>(a.prefix_tiles - tile), end - pos));
      p->prefix = true;
      p->whole = false;  // a row has own keys too
      p->s = -1;
      p->g = head;
      p->begin = 0;
      p->rows = a.a.rows;
      p->n = 0;
      p->m0 = rt * a.cut.mt;
      p->nrows = static_cast<int>(min(static_cast<long long>(a.cut.mt), static_cast<long long>(a.a.rows) * a.cut.group - p->m0));
      p->k0 = tile * kAtKeys;
      p->k1 = min(a.a.plen, (tile + take) * kAtKeys);
      p->id = seg + cta;
      pos += take;
      tile = 0;
      ++seg;
      return true;
    }
    if (s < 0) {  // the first request with rows
      enter(a, sh.s, sh.begin);
    } else if (t >= row_tiles) {
      t = 0;
      if (++g >= a.cut.n_kv) {
        do {
          if (s + 1 >= a.a.batch) return false;  // (there is one: tiles are left)
          const int reach = max(begin, clamp_row(a, a.row_start[s + 1]));
          enter(a, s + 1, reach);
        } while (rows == 0);
      }
    }
    const int kt = at_tiles(a.cut, n, rows, t);
    const int take = static_cast<int>(min(static_cast<long long>(kt - tile), end - pos));
    p->prefix = false;
    p->whole = tile == 0 && take == kt && prefix == 0;
    p->s = s;
    p->g = g;
    p->begin = begin;
    p->rows = rows;
    p->n = n;
    p->m0 = t * a.cut.mt;
    p->nrows = static_cast<int>(min(static_cast<long long>(a.cut.mt), static_cast<long long>(rows) * a.cut.group - p->m0));
    p->k0 = tile * kAtKeys;
    p->k1 = min(at_keys(a.cut, n, rows, t), (tile + take) * kAtKeys);
    p->id = seg + cta;
    pos += take;
    tile = 0;
    ++seg;
    ++t;
    return true;
  }
};

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

}  // namespace wsg
