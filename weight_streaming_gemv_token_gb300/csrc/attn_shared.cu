// attn_shared_prefix: grouped-query attention of one query token for each of
// several branches over a shared prefix and the branch's own paged tokens
// ("Megakernels", "What runs in the DSL": grouped-query attention).
//
// The rows of all branches of a key/value head (batch * group of them) form one
// matrix against the prefix, so the prefix is read once; a branch's own pages
// meet its group's rows only. Both key axes are cut into ranges so that few
// rows still fill the GPU (attn_mma.cuh), and the partial results (reference m,
// sum l, unnormalised o) of a row's ranges join exactly:
//   out = sum_i o_i 2^(m_i - m) / sum_i l_i 2^(m_i - m), m = max_i m_i.
#include <cmath>

#include "attn_mma.cuh"
#include "common.h"

namespace wsg {

cudaError_t am_launch_bf16(const AmArgs& a, bool q_f32, int mt, int items, int dev, cudaStream_t st) {
  if (q_f32)
    return mt == 2 ? am_launch_head<float, 3, 2, false>(a, items, dev, st)
                   : am_launch_head<float, 3, 1, false>(a, items, dev, st);
  return mt == 2 ? am_launch_head<uint16_t, 1, 2, false>(a, items, dev, st)
                 : am_launch_head<uint16_t, 1, 1, false>(a, items, dev, st);
}

namespace {

struct AmJoinArgs {
  int batch, n_q, d;
  int prefix_slots, own_slots, own_chunk;
  PagePool pool;
  const int32_t* len;
  const float* part_o;
  const float2* part_ml;
  void* out;
  long long out_stride;
  float* lse;
};

// One warp per (branch, query head): the partial results of its slots (those
// of the prefix, then those of the branch's own keys that hold any), in slot
// order. Lane i holds elements 4 i .. 4 i + 3 of the head.
template <typename QT>
__global__ void __launch_bounds__(128) attn_join_kernel(const AmJoinArgs a) {
  pdl_wait();
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (w >= a.batch * a.n_q) return;
  const int b = w / a.n_q;
  const int n = a.len[b];
  if (n < 0) return;
  const long long held = n < page_capacity(a.pool) ? n : page_capacity(a.pool);
  const int slots = a.prefix_slots + static_cast<int>((held + a.own_chunk - 1) / a.own_chunk);
  const long long total = static_cast<long long>(a.batch) * a.n_q;
  float m = -INFINITY, l = 0.f;
  for (int s = lane; s < slots; s += 32) m = fmaxf(m, a.part_ml[s * total + w].x);
  m = warp_max(m);
  for (int s = lane; s < slots; s += 32) {
    const float2 p = a.part_ml[s * total + w];
    l += m == -INFINITY ? p.y : p.y * am_exp2(p.x - m);
  }
  l = warp_sum(l);
  float x[4] = {};
  const bool in = lane * 4 < a.d;
#pragma unroll 4
  for (int s = 0; s < slots; ++s) {
    const float f = m == -INFINITY ? 1.f : am_exp2(a.part_ml[s * total + w].x - m);
    if (in) {
      const float4 y = *reinterpret_cast<const float4*>(a.part_o + (s * total + w) * a.d + lane * 4);
      x[0] = fmaf(y.x, f, x[0]), x[1] = fmaf(y.y, f, x[1]), x[2] = fmaf(y.z, f, x[2]), x[3] = fmaf(y.w, f, x[3]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a NaN sum stays one
  if (in) {
    QT* dst = static_cast<QT*>(a.out) + a.out_stride * b + static_cast<long long>(w % a.n_q) * a.d + lane * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(QT) == 4) {
        dst[e] = x[e] * inv;
      } else {
        uint32_t h;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(0.f), "f"(x[e] * inv));
        dst[e] = static_cast<uint16_t>(h);
      }
    }
  }
  if (a.lse && lane == 0) a.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}


bool attn_sizes_ok(const attn_shared_args* a) {
  auto type = [](int t) { return t == DEC_F32 || t == DEC_BF16; };
  return a->batch >= 0 && a->batch <= 65535 && a->n_kv >= 1 && a->n_q >= a->n_kv && a->n_q <= 65535 &&
         a->n_q % a->n_kv == 0 && a->n_q / a->n_kv <= 16 && a->head_dim >= 8 && a->head_dim <= 128 &&
         a->head_dim % 8 == 0 && type(a->qdtype) && type(a->kvdtype) && a->prefix_len >= 0 &&
         page_shift(a->page_size) >= 0 && a->num_pages >= 0 && a->table_stride >= 0 &&
         (static_cast<long long>(a->table_stride) << page_shift(a->page_size)) + a->prefix_len < (1ll << 31);
}


// How a call is cut up.
struct AsPlan {
  int mt, row_groups;
  int prefix_slots, prefix_chunk, own_slots, own_chunk;
  long long items;
  size_t o, ml, total;  // workspace offsets and size
};

AsPlan attn_plan(const attn_shared_args* a, int sms) {
  AsPlan p{};
  const bool f32 = a->kvdtype == DEC_F32;
  const int group = a->n_q / a->n_kv, rows = a->batch * group;
  const int unit = kAmWarps * (f32 ? 8 : 16);  // keys the warps of a CTA take at once
  const long long resident = 2ll * sms;        // CTAs the GPU holds
  p.mt = !f32 && rows > 16 ? 2 : 1;
  p.row_groups = (rows + 16 * p.mt - 1) / (16 * p.mt);
  // splits of an axis of `keys` keys into whole units, given that one split is `each` CTAs
  auto cut = [&](long long keys, long long each, int* slots, int* chunk) {
    const long long units = (keys + unit - 1) / unit;
    const long long want = (resident + each - 1) / each;
    const long long per = (units + want - 1) / (want < 1 ? 1 : want);
    *chunk = static_cast<int>((per < 1 ? 1 : per) * unit);
    *slots = static_cast<int>((keys + *chunk - 1) / *chunk);
  };
  cut(a->prefix_len, static_cast<long long>(a->n_kv) * p.row_groups, &p.prefix_slots, &p.prefix_chunk);
  cut(static_cast<long long>(a->table_stride) << page_shift(a->page_size),
      static_cast<long long>(a->batch) * a->n_kv, &p.own_slots, &p.own_chunk);
  p.items = static_cast<long long>(p.prefix_slots) * a->n_kv * p.row_groups +
            static_cast<long long>(p.own_slots) * a->batch * a->n_kv;
  const long long parts = static_cast<long long>(p.prefix_slots + p.own_slots) * a->batch * a->n_q;
  p.o = 0;
  p.ml = (static_cast<size_t>(parts) * a->head_dim * 4 + 255) / 256 * 256;
  p.total = (p.ml + static_cast<size_t>(parts) * 8 + 256) / 256 * 256;
  return p;
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" size_t attn_shared_prefix_workspace(const attn_shared_args* a) {
  if (!a || !attn_sizes_ok(a)) return 0;
  DeviceInfo di;
  if (device_info(&di, nullptr) != DEC_OK) return 0;
  return attn_plan(a, di.sms).total;
}

extern "C" dec_status attn_shared_prefix(const attn_shared_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: NULL arguments");
  if (!attn_sizes_ok(a))
    return fail(nullptr, DEC_EINVAL,
                "attn_shared_prefix: batch %d, n_q %d, n_kv %d, head_dim %d, qdtype %d, kvdtype %d, prefix_len %d, "
                "page_size %d, num_pages %d, table_stride %d",
                a->batch, a->n_q, a->n_kv, a->head_dim, a->qdtype, a->kvdtype, a->prefix_len, a->page_size,
                a->num_pages, a->table_stride);
  if (a->batch == 0) return DEC_OK;
  const long long width = static_cast<long long>(a->n_q) * a->head_dim;
  if (!a->q || !a->out || !a->seq_len || (a->prefix_len > 0 && (!a->prefix_k || !a->prefix_v)) ||
      (a->table_stride > 0 && (!a->page_table || !a->k_pages || !a->v_pages)))
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: NULL pointer");
  if (a->q_stride < 0 || (a->batch > 1 && a->out_stride < width) || a->prefix_stride < a->prefix_len)
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: q_stride %lld, out_stride %lld, prefix_stride %lld",
                static_cast<long long>(a->q_stride), static_cast<long long>(a->out_stride),
                static_cast<long long>(a->prefix_stride));
  if (!aligned16(a->prefix_k) || !aligned16(a->prefix_v) || !aligned16(a->k_pages) || !aligned16(a->v_pages))
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: prefix and pools must be 16-byte aligned");
  if (!a->d_workspace || reinterpret_cast<uintptr_t>(a->d_workspace) % 256)
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: workspace must be non-NULL and 256-byte aligned");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  const AsPlan p = attn_plan(a, di.sms);
  if (a->workspace_bytes < p.total)
    return fail(nullptr, DEC_ENOMEM, "attn_shared_prefix: workspace has %zu bytes, %zu needed", a->workspace_bytes,
                p.total);
  if (p.items >= 1ll << 31) return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: %lld work items", p.items);
  char* w = static_cast<char*>(a->d_workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AmArgs k{};
  k.batch = a->batch;
  k.n_q = a->n_q;
  k.n_kv = a->n_kv;
  k.d = a->head_dim;
  k.group = a->n_q / a->n_kv;
  k.rows = a->batch * k.group;
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
  k.scale_log2 = a->scale * 1.44269504088896340736f;
  k.row_groups = p.row_groups;
  k.prefix_items = p.prefix_slots * a->n_kv * p.row_groups;
  k.prefix_chunk = p.prefix_chunk;
  k.own_chunk = p.own_chunk;
  k.own_slot0 = p.prefix_slots;
  k.part_o = reinterpret_cast<float*>(w + p.o);
  k.part_ml = reinterpret_cast<float2*>(w + p.ml);
  k.err = di.err;
  const bool qf = a->qdtype == DEC_F32;
  if (p.items > 0)
    WSG_CUDA_TRY(nullptr, a->kvdtype == DEC_F32
                              ? am_launch_f32(k, qf, static_cast<int>(p.items), di.device, s)
                              : am_launch_bf16(k, qf, p.mt, static_cast<int>(p.items), di.device, s));
  AmJoinArgs j{};
  j.batch = a->batch;
  j.n_q = a->n_q;
  j.d = a->head_dim;
  j.prefix_slots = p.prefix_slots;
  j.own_slots = p.own_slots;
  j.own_chunk = p.own_chunk;
  j.pool = k.pool;
  j.len = a->seq_len;
  j.part_o = k.part_o;
  j.part_ml = k.part_ml;
  j.out = a->out;
  j.out_stride = a->out_stride;
  j.lse = a->lse;
  const dim3 grid((a->batch * a->n_q + 3) / 4);
  // a join without partial results may not overtake the stream's previous kernel
  WSG_CUDA_TRY(nullptr, qf ? launch_k(attn_join_kernel<float>, grid, dim3(128), 0, s, p.items > 0, j)
                           : launch_k(attn_join_kernel<uint16_t>, grid, dim3(128), 0, s, p.items > 0, j));
  return DEC_OK;
}
