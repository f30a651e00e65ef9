// attn_shared_prefix: grouped-query attention of one query token for each of
// several branches over a shared prefix and the branch's own paged tokens
// ("Megakernels", "What runs in the DSL": grouped-query attention).
//
// softmax over the joined keys in one pass: running maximum m, sum l of
// exp(s - m) and accumulator o, each key rescaling them when m moves; partial
// results (m, l, o) of disjoint key ranges join exactly.
//
// First kernel: a CTA per (branch, query head), its warps take the keys in
// turn, a lane holds 4 elements of the head.
#include <cmath>

#include "common.h"
#include "paging.h"
#include "ptx.cuh"

namespace wsg {
namespace {

constexpr int kAsWarps = 4;

struct AsArgs {
  int batch, n_q, n_kv, d, group;
  const void* q;
  void* out;
  float* lse;
  long long q_stride, out_stride;
  const void *pk, *pv;
  int plen;
  long long pstride;
  const void *kp, *vp;
  PagePool pool;
  const int32_t *table, *len;
  float scale;
  uint32_t* err;
};

__device__ __forceinline__ float get(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float get(const uint16_t* p, long long i) { return bf16_to_f32(p[i]); }
__device__ __forceinline__ void put(float* p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void put(uint16_t* p, long long i, float v) { p[i] = f32_to_bf16_rn(v); }

template <typename QT, typename KT>
__global__ void __launch_bounds__(32 * kAsWarps) attn_rows_kernel(const AsArgs a) {
  __shared__ float s_m[kAsWarps], s_l[kAsWarps], s_o[kAsWarps][128];
  const int b = blockIdx.x, h = blockIdx.y, g = h / a.group, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int own = a.len[b];
  if (own < 0) return;
  if (own > page_capacity(a.pool)) {
    if (threadIdx.x == 0) atomicOr(a.err, ERR_BAD_PAGE);
    own = static_cast<int>(page_capacity(a.pool));
  }
  const bool in = lane * 4 < a.d;
  float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.f;
  if (in)
    for (int e = 0; e < 4; ++e) q[e] = get(static_cast<const QT*>(a.q), a.q_stride * b + h * a.d + lane * 4 + e);
  const int total = a.plen + own;
  for (int t = warp; t < total; t += kAsWarps) {
    const KT *k, *v;
    if (t < a.plen) {
      const long long at = (a.pstride * g + t) * a.d;
      k = static_cast<const KT*>(a.pk) + at;
      v = static_cast<const KT*>(a.pv) + at;
    } else {
      const int idx = t - a.plen;
      const int page = page_of(a.pool, a.table + static_cast<long long>(b) * a.pool.width, idx);
      if (page < 0) {
        if (lane == 0) atomicOr(a.err, ERR_BAD_PAGE);
        continue;
      }
      const long long at = pool_row(a.pool, page, g, idx) * a.d;
      k = static_cast<const KT*>(a.kp) + at;
      v = static_cast<const KT*>(a.vp) + at;
    }
    float s = 0.f;
    if (in)
      for (int e = 0; e < 4; ++e) s = fmaf(q[e], get(k, lane * 4 + e), s);
    s = warp_sum(s) * a.scale;
    const float mn = fmaxf(m, s);
    const float f = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
    l = l * f + p;
    if (in)
      for (int e = 0; e < 4; ++e) o[e] = fmaf(p, get(v, lane * 4 + e), o[e] * f);
    m = mn;
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  if (in)
    for (int e = 0; e < 4; ++e) s_o[warp][lane * 4 + e] = o[e];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kAsWarps; ++w) mm = fmaxf(mm, s_m[w]);
  for (int w = 0; w < kAsWarps; ++w) ll += mm == -INFINITY ? 0.f : s_l[w] * expf(s_m[w] - mm);
  for (int e = threadIdx.x; e < a.d; e += 32 * kAsWarps) {
    float x = 0.f;
    for (int w = 0; w < kAsWarps; ++w) x += mm == -INFINITY ? 0.f : s_o[w][e] * expf(s_m[w] - mm);
    put(static_cast<QT*>(a.out), a.out_stride * b + h * a.d + e, ll > 0.f ? x / ll : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[static_cast<long long>(b) * a.n_q + h] = mm == -INFINITY ? -INFINITY : mm + logf(ll);
}

bool attn_sizes_ok(const attn_shared_args* a) {
  auto type = [](int t) { return t == DEC_F32 || t == DEC_BF16; };
  return a->batch >= 0 && a->batch <= 65535 && a->n_kv >= 1 && a->n_q >= a->n_kv && a->n_q <= 65535 &&
         a->n_q % a->n_kv == 0 && a->n_q / a->n_kv <= 16 && a->head_dim >= 8 && a->head_dim <= 128 &&
         a->head_dim % 8 == 0 && type(a->qdtype) && type(a->kvdtype) && a->prefix_len >= 0 &&
         page_shift(a->page_size) >= 0 && a->num_pages >= 0 && a->table_stride >= 0 &&
         (static_cast<long long>(a->table_stride) << page_shift(a->page_size)) + a->prefix_len < (1ll << 31);
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" size_t attn_shared_prefix_workspace(const attn_shared_args* a) {
  if (!a || !attn_sizes_ok(a)) return 0;
  DeviceInfo di;
  if (device_info(&di, nullptr) != DEC_OK) return 0;
  return 256;
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
  const size_t need = attn_shared_prefix_workspace(a);
  if (a->workspace_bytes < need)
    return fail(nullptr, DEC_ENOMEM, "attn_shared_prefix: workspace has %zu bytes, %zu needed", a->workspace_bytes, need);
  AsArgs k{};
  k.batch = a->batch;
  k.n_q = a->n_q;
  k.n_kv = a->n_kv;
  k.d = a->head_dim;
  k.group = a->n_q / a->n_kv;
  k.q = a->q;
  k.out = a->out;
  k.lse = a->lse;
  k.q_stride = a->q_stride;
  k.out_stride = a->out_stride;
  k.pk = a->prefix_k;
  k.pv = a->prefix_v;
  k.plen = a->prefix_len;
  k.pstride = a->prefix_stride;
  k.kp = a->k_pages;
  k.vp = a->v_pages;
  k.pool = PagePool{a->num_pages, a->n_kv, page_shift(a->page_size), a->table_stride};
  k.table = a->page_table;
  k.len = a->seq_len;
  k.scale = a->scale;
  k.err = di.err;
  const dim3 grid(a->batch, a->n_q), block(32 * kAsWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool qf = a->qdtype == DEC_F32, kf = a->kvdtype == DEC_F32;
  WSG_CUDA_TRY(nullptr, qf ? (kf ? launch_k(attn_rows_kernel<float, float>, grid, block, 0, s, false, k)
                                 : launch_k(attn_rows_kernel<float, uint16_t>, grid, block, 0, s, false, k))
                           : (kf ? launch_k(attn_rows_kernel<uint16_t, float>, grid, block, 0, s, false, k)
                                 : launch_k(attn_rows_kernel<uint16_t, uint16_t>, grid, block, 0, s, false, k)));
  return DEC_OK;
}
