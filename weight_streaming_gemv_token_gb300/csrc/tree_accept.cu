// tree_accept_paged: the path of each drafted tree that the greedy tokens confirm, and
// the moves of its keys and values to their places in the cache ("Megakernels",
// "GPU-wide end-to-end generation": the greedy token after each row, the cache
// entries that a generation leaves).
//
// Mathematics: path_0 = 0; path_{d+1} = the lowest row c with parent path_d and drafted
// token next[path_d]. Row path_d moves from index seq_len + path_d to seq_len + d. Since
// path_d >= d and both rise, the place a move writes is never one that a later move
// reads: the moves of a 16-byte column are made in order, all loads of a batch before
// its stores, and columns are independent of each other.
//
// A CTA takes one request and some of its columns over the layers; each CTA walks the
// tree for itself (a search of its rows by one warp for each accepted row), so that
// one launch does without a wait between CTAs. Bound by memory for many layers, by the
// walk's chain of searches for few: 4.0 us for one tree of 12 rows and 2 layers, 8.5 for 32
// trees of 28 layers (26 MB read and written, 3.8 us at the copy's rate).
#include "common.h"
#include "paging.h"
#include "ptx.cuh"
#include "spans.h"

namespace wsg {
namespace {

constexpr int kTaThreads = 256, kTaPath = 256, kTaStage = 1024, kTaBatch = 8;

struct TaArgs {
  int batch, rows, path_stride, layers, n_kv, row16;  // row16: 16-byte pieces of a key
  const int32_t *row_start, *parents, *draft, *next, *len, *held;
  uint4 *k, *v;
  long long layer16;
  PagePool pool;
  const int32_t* table;
  int32_t* tokens;
  long long tokens_stride;
  int tokens_base;
  int32_t *count, *new_len, *path, *out;
  uint32_t* err;
};

// Grid: (CTAs of a request, requests).
__global__ void __launch_bounds__(kTaThreads) tree_accept_kernel(const TaArgs a) {
  __shared__ int32_t s_parent[kTaStage], s_draft[kTaStage], s_next[kTaStage], s_path[kTaPath];
  __shared__ long long s_src[kTaPath], s_dst[kTaPath];  // rows of head 0 in a pool
  __shared__ int s_count, s_moves;
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
  const bool first = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();
  const int len = a.len[b];
  const int begin = min(max(0, a.row_start[b]), a.rows), n = min(a.row_start[b + 1], a.rows) - begin;
  if (len < 0 || n <= 0) {
    if (first) {
      if (tid == 0) a.count[b] = 0, a.new_len[b] = len >= 0 ? len : a.held ? a.held[b] : -1;
      for (int d = tid; d < a.path_stride; d += kTaThreads)
        a.path[static_cast<long long>(b) * a.path_stride + d] = a.out[static_cast<long long>(b) * a.path_stride + d] = -1;
    }
    return;
  }
  // the tree in shared memory, where it fits
  const bool staged = n <= kTaStage;
  if (staged)
    for (int i = tid; i < n; i += kTaThreads) {
      s_parent[i] = a.parents ? a.parents[begin + i] : i - 1;
      s_draft[i] = a.draft[begin + i];
      s_next[i] = a.next[begin + i];
    }
  __syncthreads();
  if (tid < 32) {
    auto draft = [&](int i) { return staged ? s_draft[i] : a.draft[begin + i]; };
    auto parent = [&](int i) { return staged ? s_parent[i] : a.parents ? a.parents[begin + i] : i - 1; };
    int cur = 0, count = 0;
    while (count < a.path_stride) {
      if (lane == 0) s_path[count] = cur;
      ++count;
      const int token = staged ? s_next[cur] : a.next[begin + cur];
      int found = -1;
      if (token >= 0) {
        for (int i0 = cur + 1; i0 < n && found < 0; i0 += 32) {
          const int i = i0 + lane;
          const unsigned hit = __ballot_sync(0xffffffffu, i < n && draft(i) == token && parent(i) == cur);
          if (hit) found = i0 + __ffs(hit) - 1;
          if (!a.parents) break;  // a chain's row has one child, the next row
        }
      }
      if (found < 0) break;
      cur = found;
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  if (first) {
    if (tid == 0) a.count[b] = count, a.new_len[b] = len + count;
    for (int d = tid; d < a.path_stride; d += kTaThreads) {
      const long long at = static_cast<long long>(b) * a.path_stride + d;
      const int p = d < count ? s_path[d] : -1;
      a.path[at] = p;
      a.out[at] = p < 0 ? -1 : a.next[begin + p];
      if (p >= 0 && a.tokens) {
        const long long to = static_cast<long long>(len) + a.tokens_base + d;
        if (to < a.tokens_stride)
          a.tokens[a.tokens_stride * b + to] = a.draft[begin + p];
        else
          atomicOr(a.err, ERR_BAD_POSITION);
      }
    }
  }
  if (a.layers == 0) return;
  // ---- the moves, in order ----
  if (tid < 32) {
    const int32_t* row = a.table + static_cast<long long>(b) * a.pool.width;
    int moves = 0;
    for (int d0 = 0; d0 < count; d0 += 32) {
      const int d = d0 + lane;
      bool move = false;
      long long src = 0, dst = 0;
      if (d < count) {
        const long long from = static_cast<long long>(len) + s_path[d], to = static_cast<long long>(len) + d;
        const int sp = page_of(a.pool, row, from), dp = page_of(a.pool, row, to);
        if (sp < 0 || dp < 0) {
          if (first) atomicOr(a.err, ERR_BAD_PAGE);
        } else if (from != to) {
          move = true;
          src = pool_row(a.pool, sp, 0, from);
          dst = pool_row(a.pool, dp, 0, to);
        }
      }
      const unsigned all = __ballot_sync(0xffffffffu, move);
      if (move) {
        const int at = moves + __popc(all & ((1u << lane) - 1u));
        s_src[at] = src, s_dst[at] = dst;
      }
      moves += __popc(all);
    }
    if (lane == 0) s_moves = moves;
  }
  __syncthreads();
  const int moves = s_moves;
  if (moves == 0) return;
  const int columns = a.n_kv * a.row16;  // of a layer's keys
  const long long total = 2ll * a.layers * columns;
  for (long long i = static_cast<long long>(blockIdx.x) * kTaThreads + tid; i < total;
       i += static_cast<long long>(gridDim.x) * kTaThreads) {
    const int which = static_cast<int>(i / columns), c = static_cast<int>(i - static_cast<long long>(which) * columns);
    const int g = c / a.row16, piece = c - g * a.row16;
    uint4* pool = (which & 1 ? a.v : a.k) + a.layer16 * (which >> 1) +
                  (static_cast<long long>(g) << a.pool.shift) * a.row16 + piece;
    for (int m0 = 0; m0 < moves; m0 += kTaBatch) {
      uint4 x[kTaBatch];
#pragma unroll
      for (int m = 0; m < kTaBatch; ++m)
        if (m0 + m < moves) x[m] = pool[s_src[m0 + m] * a.row16];
#pragma unroll
      for (int m = 0; m < kTaBatch; ++m)
        if (m0 + m < moves) pool[s_dst[m0 + m] * a.row16] = x[m];
    }
  }
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" dec_status tree_accept_paged(const tree_accept_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "tree_accept_paged: NULL arguments");
  if (a->batch < 0 || a->batch > 65535 || a->rows < 0 || a->path_stride < 1 || a->path_stride > kTaPath || a->layers < 0 ||
      a->layers > 65535 || a->tokens_base < 0)
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: batch %d, rows %d, path_stride %d, layers %d, tokens_base %d",
                a->batch, a->rows, a->path_stride, a->layers, a->tokens_base);
  const int shift = page_shift(a->page_size);
  if (a->layers > 0 && (a->n_kv < 1 || a->n_kv > 16384 || a->head_dim < 8 || a->head_dim > 128 || a->head_dim % 8 ||
                        (a->kvdtype != DEC_F32 && a->kvdtype != DEC_BF16) || shift < 0 || a->num_pages < 0 ||
                        a->table_stride < 0 || a->layer_stride < 0))
    return fail(nullptr, DEC_EINVAL,
                "tree_accept_paged: n_kv %d, head_dim %d, kvdtype %d, page_size %d, num_pages %d, table_stride %d", a->n_kv,
                a->head_dim, a->kvdtype, a->page_size, a->num_pages, a->table_stride);
  if (a->batch == 0) return DEC_OK;
  if (!a->row_start || !a->seq_len || !a->count || !a->new_len || !a->path || !a->out_tokens ||
      (a->rows > 0 && (!a->draft_tokens || !a->next)) ||
      (a->layers > 0 && (!a->k_pages || !a->v_pages || (a->table_stride > 0 && !a->page_table))))
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: NULL pointer");
  const int elem = a->layers > 0 && a->kvdtype == DEC_BF16 ? 2 : 4;
  if (a->layers > 0 && (!aligned16(a->k_pages) || !aligned16(a->v_pages) || a->layer_stride * elem % 16))
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: the pools must be 16-byte aligned in every layer");
  if (!aligned_to(4, a->row_start, a->parents, a->draft_tokens, a->next, a->seq_len, a->held, a->page_table, a->tokens, a->count,
                  a->new_len, a->path, a->out_tokens))
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: a pointer is not aligned to its elements");
  if (a->tokens && a->tokens_stride < 0)
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: tokens_stride %lld", static_cast<long long>(a->tokens_stride));
  const long long layer = static_cast<long long>(a->num_pages) * a->n_kv * a->page_size * a->head_dim;
  if (a->layers > 1 && a->layer_stride < layer)
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: layers of %lld elements overlap at stride %lld", layer,
                static_cast<long long>(a->layer_stride));
  const size_t b = a->batch, r = a->rows, width = a->layers > 0 ? a->table_stride : 0;
  if (outputs_meet({{a->count, 4 * b}, {a->new_len, 4 * b}, {a->path, 4 * b * a->path_stride},
                    {a->out_tokens, 4 * b * a->path_stride},
                    {a->tokens, 4 * b * static_cast<size_t>(a->tokens ? a->tokens_stride : 0)}},
                   {{a->row_start, 4 * (b + 1)}, {a->parents, 4 * r}, {a->draft_tokens, 4 * r}, {a->next, 4 * r},
                    {a->seq_len, 4 * b}, {a->held, 4 * b}, {a->page_table, 4 * b * width}}))
    return fail(nullptr, DEC_EINVAL, "tree_accept_paged: an output overlaps another argument");
  if (a->layers > 0) {  // the pools are written too; other arguments may lie between layers
    const Span one = span_pool(a->k_pages, a->num_pages, static_cast<long long>(a->n_kv) * a->page_size * a->head_dim * elem);
    const Spans k{one, a->layers, a->layer_stride * elem}, v{{a->v_pages, one.bytes}, a->layers, a->layer_stride * elem};
    bool meet = series_meet(k, v);
    for (const Span& s : {Span{a->count, 4 * b}, {a->new_len, 4 * b}, {a->path, 4 * b * a->path_stride}, {a->out_tokens, 4 * b * a->path_stride},
                          {a->tokens, 4 * b * static_cast<size_t>(a->tokens ? a->tokens_stride : 0)}, {a->row_start, 4 * (b + 1)},
                          {a->parents, 4 * r}, {a->draft_tokens, 4 * r}, {a->next, 4 * r}, {a->seq_len, 4 * b}, {a->held, 4 * b},
                          {a->page_table, 4 * b * width}})
      meet = meet || series_meet(k, Spans{s, 1, 0}) || series_meet(v, Spans{s, 1, 0});
    if (meet) return fail(nullptr, DEC_EINVAL, "tree_accept_paged: a pool overlaps another argument");
  }
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  TaArgs k{};
  k.batch = a->batch;
  k.rows = a->rows;
  k.path_stride = a->path_stride;
  k.layers = a->layers;
  k.row_start = a->row_start;
  k.parents = a->parents;
  k.draft = a->draft_tokens;
  k.next = a->next;
  k.len = a->seq_len;
  k.held = a->held;
  k.tokens = a->tokens;
  k.tokens_stride = a->tokens_stride;
  k.tokens_base = a->tokens_base;
  k.count = a->count;
  k.new_len = a->new_len;
  k.path = a->path;
  k.out = a->out_tokens;
  k.err = di.err;
  long long ctas = 1;
  if (a->layers > 0) {
    k.n_kv = a->n_kv;
    k.row16 = a->head_dim * elem / 16;
    k.k = static_cast<uint4*>(a->k_pages);
    k.v = static_cast<uint4*>(a->v_pages);
    k.layer16 = a->layer_stride * elem / 16;
    k.pool = PagePool{a->num_pages, a->n_kv, shift, a->table_stride};
    k.table = a->page_table;
    // one column a thread, at most four CTAs an SM in all
    ctas = (2ll * a->layers * k.n_kv * k.row16 + kTaThreads - 1) / kTaThreads;
    const long long most = 4ll * di.sms / a->batch;
    if (ctas > most) ctas = most < 1 ? 1 : most;
  }
  WSG_CUDA_TRY(nullptr, launch_k(tree_accept_kernel, dim3(static_cast<unsigned>(ctas), a->batch), dim3(kTaThreads), 0,
                                 static_cast<cudaStream_t>(stream), true, k));
  return DEC_OK;
}
