// attn_tree_paged: grouped-query attention of drafted trees of several requests over a
// shared prefix, the requests' pages and the rows of their own tree ("Megakernels",
// "What runs in the DSL": grouped-query attention).
//
// The line of key tiles (attn_tree_plan.h) goes by the lengths on the device, so
// every SM has an equal share of it whatever the requests' lengths and however wide
// their tables are. A segment that lies in one CTA's share is finished there. The pieces
// of the others join exactly in attn_tree_seam_kernel, those of rows that have a prefix
// too (two segments each, whole or cut) in attn_tree_join_kernel:
//   out = sum_i o_i 2^(m_i - m) / sum_i l_i 2^(m_i - m), m = max_i m_i.
#include "attn_tree.cuh"

#include <cmath>

#include "common.h"
#include "spans.h"

namespace wsg {
namespace {

// N more partial results of a row (reference and sum q, elements y) into (m, l, x), as
// ar_merge8 does eight.
template <int N>
__device__ __forceinline__ void at_merge(const float2 (&q)[N], const float4 (&y)[N], float* m, float* l, float4* x) {
  float mn = *m;
#pragma unroll
  for (int i = 0; i < N; ++i) mn = fmaxf(mn, q[i].x);
  const float mu = mn == -INFINITY ? 0.f : mn, f = am_exp2(*m - mu);
  *l *= f;
  x->x *= f, x->y *= f, x->z *= f, x->w *= f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float e = q[i].x == -INFINITY ? 1.f : am_exp2(q[i].x - mu);
    *l = fmaf(q[i].y, e, *l);
    x->x = fmaf(y[i].x, e, x->x), x->y = fmaf(y[i].y, e, x->y), x->z = fmaf(y[i].z, e, x->z), x->w = fmaf(y[i].w, e, x->w);
  }
  *m = mn;
}

// Without a prefix: CTAs (x, .) join the rows of the cut segment with record x, a row a
// warp, lane i elements 4 i .. 4 i + 3 of a head. (All CTAs fit the GPU at once: eight
// rows of every CTA's record a CTA took 8 us for 152 records, most of them empty.)
template <typename QT>
__global__ void __launch_bounds__(256, 4) attn_tree_seam_kernel(const AtArgs p) {
  const AmArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();  // a following call's set-up may begin
  pdl_wait();
  const AtSeam s = p.seam[blockIdx.x];
  if (s.pieces == 0) return;
  const bool in = lane * 4 < a.d;
  for (int r = blockIdx.y * 8 + warp; r < s.nrows; r += 8 * gridDim.y) {
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < s.pieces; s0 += 4) {  // four pieces at a time: their loads go out together
      float2 q[4];
      float4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool have = s0 + i < s.pieces;
        const long long at = ((s.id + s0 + i) << p.cut.mshift) + r;
        q[i] = have ? a.part_ml[at] : make_float2(-INFINITY, 0.f);
        y[i] = have && in ? *reinterpret_cast<const float4*>(a.part_o + at * a.d + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      at_merge(q, y, &m, &l, &x);
    }
    const int row = s.m0 + r, token = row / a.group;
    if (in) at_put<QT>(p, s.begin + token, s.g * a.group + row - token * a.group, lane * 4, x, m, l);
  }
}

// With a prefix: one warp a (row, query head).
template <typename QT>
__global__ void __launch_bounds__(128) attn_tree_join_kernel(const AtArgs p, int ctas) {
  const AmArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();  // a following call's set-up may begin
  pdl_wait();
  for (int w = blockIdx.x * 4 + warp; w < a.rows * a.n_q; w += gridDim.x * 4) {
    const int row = w / a.n_q, head = w - row * a.n_q, g = head / a.group, h = head - g * a.group;
    AtRow rec = p.rec[row];
    const long long W = *p.total;
    if (rec.tiles == 0) continue;  // of no request, or an unused one
    const AtShares C = at_shares(W, static_cast<int>(min(static_cast<long long>(ctas), W)));
    int at = rec.at + h;
    if (at >> p.cut.mshift) {  // the row tile behind the record's
      at -= 1 << p.cut.mshift;
      rec.line += rec.tiles + kAtExtra;
      rec.tiles = rec.next;
      ++rec.seg;
    }
    const long long line = rec.line + g * rec.head;
    const int c0 = at_owner(C, line), c1 = at_owner(C, line + rec.tiles - 1);
    const long long own = rec.seg + static_cast<long long>(g) * rec.row_tiles + c0;  // number of the first piece
    const int own_n = c1 - c0 + 1;
    const int pm = row * a.group + h, rt = pm >> p.cut.mshift, pre_at = pm - (rt << p.cut.mshift);
    const long long seg = static_cast<long long>(g) * p.prefix_row_tiles + rt, from = seg * (p.prefix_tiles + kAtExtra) + kAtExtra;
    const int d0 = at_owner(C, from), pre_n = at_owner(C, from + p.prefix_tiles - 1) - d0 + 1;
    const long long pre = seg + d0;  // the prefix's pieces, as above
    const bool in = lane * 4 < a.d;
    const int parts = own_n + pre_n;
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    // eight pieces at a time: their loads go out together
    for (int s0 = 0; s0 < parts; s0 += 8) {
      float2 q[8];
      float4 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int s = s0 + i;
        const long long r = s < pre_n ? ((pre + s) << p.cut.mshift) + pre_at : ((own + s - pre_n) << p.cut.mshift) + at;
        q[i] = s < parts ? a.part_ml[r] : make_float2(-INFINITY, 0.f);
        y[i] = s < parts && in ? *reinterpret_cast<const float4*>(a.part_o + r * a.d + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      at_merge(q, y, &m, &l, &x);
    }
    if (in) at_put<QT>(p, row, head, lane * 4, x, m, l);
  }
}

// The join's kernels ask for the largest shared-memory split, which the kernels beside
// them in the stream need: an SM that changes its split first runs empty.
template <typename K>
cudaError_t at_prepare(K kern, bool* done) {
  if (*done) return cudaSuccess;
  const cudaError_t e = allow_smem_shared(kern, 0);
  *done = e == cudaSuccess;
  return e;
}

template <typename QT>
cudaError_t launch_join(const AtArgs& t, const AtPlan& p, const DeviceInfo& di, cudaStream_t s) {
  static bool done[2][64] = {};
  if (t.prefix_tiles == 0) {
    const cudaError_t e = at_prepare(attn_tree_seam_kernel<QT>, &done[0][di.device]);
    if (e != cudaSuccess) return e;
    // as many CTAs of eight rows as the GPU holds at once
    const int most = p.seams < 4 * di.sms ? 4 * di.sms / p.seams : 1, need = (1 << p.cut.mshift) / 8;
    return launch_k(attn_tree_seam_kernel<QT>, dim3(p.seams, need < most ? need : most), dim3(256), 0, s, true, t);
  }
  const cudaError_t e = at_prepare(attn_tree_join_kernel<QT>, &done[1][di.device]);
  if (e != cudaSuccess) return e;
  const long long warps = (static_cast<long long>(t.a.rows) * t.a.n_q + 3) / 4;
  return launch_k(attn_tree_join_kernel<QT>, dim3(static_cast<unsigned>(warps < 6 * di.sms ? warps : 6 * di.sms)), dim3(128), 0,
                  s, true, t, p.ctas);
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" size_t attn_tree_paged_workspace(const attn_tree_args* a) {
  if (!a || !attn_tree_sizes_ok(a)) return 0;
  DeviceInfo di;
  if (device_info(&di, nullptr) != DEC_OK) return 0;
  return attn_tree_plan(a, di.sms).total;
}

extern "C" dec_status attn_tree_paged(const attn_tree_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "attn_tree_paged: NULL arguments");
  if (!attn_tree_sizes_ok(a))
    return fail(nullptr, DEC_EINVAL,
                "attn_tree_paged: batch %d, rows %d, n_q %d, n_kv %d, head_dim %d, qdtype %d, kvdtype %d, mask_words %d, "
                "prefix_len %d, page_size %d, num_pages %d, table_stride %d",
                a->batch, a->rows, a->n_q, a->n_kv, a->head_dim, a->qdtype, a->kvdtype, a->mask_words, a->prefix_len,
                a->page_size, a->num_pages, a->table_stride);
  if (a->batch == 0 || a->rows == 0) return DEC_OK;
  const long long width = static_cast<long long>(a->n_q) * a->head_dim;
  if (!a->q || !a->out || !a->row_start || !a->seq_len || (a->prefix_len > 0 && (!a->prefix_k || !a->prefix_v)) ||
      (a->table_stride > 0 && (!a->page_table || !a->k_pages || !a->v_pages)))
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: NULL pointer");
  if (a->q_stride < 0 || (a->rows > 1 && a->out_stride < width) || (a->prefix_len > 0 && a->prefix_stride < a->prefix_len))
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: q_stride %lld, out_stride %lld, prefix_stride %lld",
                static_cast<long long>(a->q_stride), static_cast<long long>(a->out_stride),
                static_cast<long long>(a->prefix_stride));
  const bool pages = a->table_stride > 0;
  if ((a->prefix_len > 0 && (!aligned16(a->prefix_k) || !aligned16(a->prefix_v))) ||
      (pages && (!aligned16(a->k_pages) || !aligned16(a->v_pages))))
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: prefix and pools must be 16-byte aligned");
  if (!aligned_to(elem_bytes(a->qdtype), a->q, a->out) || !aligned_to(4, a->lse, a->row_start, a->mask, a->seq_len) ||
      (pages && !aligned_to(4, a->page_table)))
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: a pointer is not aligned to its elements");
  if (!a->d_workspace || reinterpret_cast<uintptr_t>(a->d_workspace) % 256)
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: workspace must be non-NULL and 256-byte aligned");
  // (a row's output is written while others, and other heads' CTAs, have yet to read their queries: only in place)
  if (a->out == a->q && a->rows > 1 && a->out_stride != a->q_stride)
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: out over q needs q's stride");
  const size_t qe = elem_bytes(a->qdtype), rows = a->rows, batch = a->batch;
  const Span q = span_rows(a->out == a->q ? nullptr : a->q, a->rows, a->q_stride, width, qe);
  const long long key = static_cast<long long>(elem_bytes(a->kvdtype)) * a->head_dim;
  auto prefix = [&](const void* p) {
    return span_rows(a->prefix_len > 0 ? p : nullptr, a->n_kv, a->prefix_stride * a->head_dim,
                     static_cast<long long>(a->prefix_len) * a->head_dim, elem_bytes(a->kvdtype));
  };
  auto pool = [&](const void* p) { return span_pool(pages ? p : nullptr, a->num_pages, key * a->n_kv * a->page_size); };
  if (outputs_meet({span_rows(a->out, a->rows, a->out_stride, width, qe), {a->lse, 4 * rows * a->n_q},
                    {a->d_workspace, a->workspace_bytes}},
                   {q, prefix(a->prefix_k), prefix(a->prefix_v), pool(a->k_pages), pool(a->v_pages), {a->row_start, 4 * (batch + 1)}, {a->mask, 4 * rows * a->mask_words}, {a->seq_len, 4 * batch},
                    {pages ? a->page_table : nullptr, 4 * batch * a->table_stride}}))
    return fail(nullptr, DEC_EINVAL, "attn_tree_paged: an output overlaps another argument");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  const AtPlan p = attn_tree_plan(a, di.sms);
  if (a->workspace_bytes < p.total)
    return fail(nullptr, DEC_ENOMEM, "attn_tree_paged: workspace has %zu bytes, %zu needed", a->workspace_bytes, p.total);
  char* w = static_cast<char*>(a->d_workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AtArgs t{};
  AmArgs& k = t.a;
  k.batch = a->batch;
  k.n_q = a->n_q;
  k.n_kv = a->n_kv;
  k.d = a->head_dim;
  k.group = a->n_q / a->n_kv;
  k.rows = a->rows;
  k.q = a->q;
  k.q_stride = a->q_stride;
  k.pk = a->prefix_k;
  k.pv = a->prefix_v;
  k.plen = a->prefix_len;
  k.pstride = a->prefix_stride;
  k.kp = a->k_pages;
  k.vp = a->v_pages;
  k.pool = PagePool{a->num_pages, a->n_kv, page_shift(a->page_size), a->table_stride};
  k.table = a->page_table;
  k.len = a->seq_len;
  k.scale_log2 = a->scale == 0.f ? 1.f : fabsf(a->scale) * 1.44269504088896340736f;
  k.q_sign = a->scale == 0.f ? 0 : a->scale < 0.f ? -1 : 1;
  k.q_even = reinterpret_cast<uintptr_t>(a->q) % 4 == 0 && a->q_stride % 2 == 0;
  k.part_o = reinterpret_cast<float*>(w + p.o);
  k.part_ml = reinterpret_cast<float2*>(w + p.ml);
  k.err = di.err;
  t.cut = p.cut;
  t.row_start = a->row_start;
  t.mask = a->mask;
  t.words = a->mask_words;
  t.prefix_row_tiles = p.prefix_row_tiles;
  t.prefix_tiles = p.prefix_tiles;
  t.out = a->out;
  t.out_stride = a->out_stride;
  t.out16 = aligned16(a->out) && (a->rows == 1 || a->out_stride * static_cast<int64_t>(qe) % 16 == 0);
  t.lse = a->lse;
  t.rec = reinterpret_cast<AtRow*>(w + p.rec);
  t.seam = reinterpret_cast<AtSeam*>(w + p.rec);
  t.seams = p.seams;
  t.seam_segs = p.pieces - p.ctas <= p.ctas;
  t.per_sm = p.per_sm;
  t.total = reinterpret_cast<long long*>(w + p.line);
  const bool qf = a->qdtype == DEC_F32;
  if (p.tc) {
    const dec_status e = launch_tree_tc(t, di, s);
    if (e != DEC_OK) return e;
  } else {
    const bool kf = a->kvdtype == DEC_F32;
    WSG_CUDA_TRY(nullptr, kf ? (qf ? launch_tree_f32_f32(t, di, s) : launch_tree_bf16_f32(t, di, s))
                             : (qf ? launch_tree_f32_bf16(t, di, s) : launch_tree_bf16_bf16(t, di, s)));
  }
  WSG_CUDA_TRY(nullptr, qf ? launch_join<float>(t, p, di, s) : launch_join<uint16_t>(t, p, di, s));
  return DEC_OK;
}
