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
#include "attn_own.cuh"
#include "attn_plan.h"
#include "attn_prefix_tc.cuh"
#include "common.h"

namespace wsg {

namespace {

struct AmJoinArgs {
  int batch, n_q, d;
  int warps;  // a row
  int prefix_slots, own_block, n_kv, group;
  long long own_seg, own_per;  // as in AmArgs
  PagePool pool;
  const int32_t* len;
  const float* part_o;
  const float2* part_ml;
  void* out;
  long long out_stride;
  float* lse;
  uint32_t* err;
};

// The partial results of one (branch, query head): its slots (those of the prefix,
// then those of the branch's own keys that hold any) are dealt to `warps` warps (1
// or 4: four rows or one row a CTA), which join in order. Lane i holds elements 4 i
// .. 4 i + 3 of the head. 256 rows of 20 slots take 2.5 us.
template <typename QT>
__global__ void __launch_bounds__(128) attn_join_kernel(const AmJoinArgs a) {
  __shared__ float s_m[4], s_l[4];
  __shared__ float4 s_x[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = a.warps == 4 ? blockIdx.x : blockIdx.x * 4 + warp;
  const int first = a.warps == 4 ? warp : 0;
  pdl_trigger();  // a following call's set-up may begin
  pdl_wait();
  if (w >= a.batch * a.n_q) return;
  const int b = w / a.n_q;
  const int n = a.len[b];
  if (n < 0) return;  // (the same for the whole CTA where it works on one row)
  const long long held = n < page_capacity(a.pool) ? n : page_capacity(a.pool);
  // (here and not by those that walk own keys: with a table of no pages there are none)
  if (n > held && w % a.n_q == 0 && (threadIdx.x & (a.warps == 4 ? 127 : 31)) == 0) atomicOr(a.err, ERR_BAD_PAGE);
  // the pieces of the line of own blocks that this row's segment lies in
  const long long blocks = (held + a.own_block - 1) / a.own_block;
  const long long seg0 = (static_cast<long long>(b) * a.n_kv + w % a.n_q / a.group) * a.own_seg;
  const int own = blocks > 0 ? static_cast<int>((seg0 + blocks - 1) / a.own_per - seg0 / a.own_per) + 1 : 0;
  const int slots = a.prefix_slots + own;
  const long long total = static_cast<long long>(a.batch) * a.n_q;
  const bool in = lane * 4 < a.d;
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  // eight slots at a time: their loads go out together
  for (int s0 = first; s0 < slots; s0 += 8 * a.warps) {
    float2 p[8];
    float4 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = s0 + i * a.warps;
      p[i] = s < slots ? a.part_ml[s * total + w] : make_float2(-INFINITY, 0.f);
      y[i] = s < slots && in ? *reinterpret_cast<const float4*>(a.part_o + (s * total + w) * a.d + lane * 4)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    ar_merge8(p, y, &m, &l, &x);
  }
  if (a.warps == 4) {
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    s_x[warp][lane] = x;
    __syncthreads();
    if (warp != 0) return;
    float mn = m;
#pragma unroll
    for (int i = 1; i < 4; ++i) mn = fmaxf(mn, s_m[i]);
    const float mu = mn == -INFINITY ? 0.f : mn;
    l = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = s_m[i] == -INFINITY ? 1.f : am_exp2(s_m[i] - mu);
      const float4 y = s_x[i][lane];
      l = fmaf(s_l[i], e, l);
      x.x = fmaf(y.x, e, x.x), x.y = fmaf(y.y, e, x.y), x.z = fmaf(y.z, e, x.z), x.w = fmaf(y.w, e, x.w);
    }
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a NaN sum stays one
  if (in) {
    QT* dst = static_cast<QT*>(a.out) + a.out_stride * b + static_cast<long long>(w % a.n_q) * a.d + lane * 4;
    const float r[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
    const bool vec = reinterpret_cast<uintptr_t>(dst) % (4 * sizeof(QT)) == 0;
    if constexpr (sizeof(QT) == 4) {
      if (vec) {
        *reinterpret_cast<float4*>(dst) = make_float4(r[0], r[1], r[2], r[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = r[e];
      }
    } else {
      uint32_t h[2];
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(r[1]), "f"(r[0]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(r[3]), "f"(r[2]));
      if (vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
  if (a.lse && lane == 0) a.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

template <int NB>
cudaError_t launch_own(const AmArgs& a, const AoArgs& o, unsigned items, int dev, cudaStream_t st) {
  constexpr size_t smem = ArGeom<128, NB, 4>::SMEM;
  static bool lifted[64] = {};
  if (!lifted[dev]) {
    const cudaError_t e = allow_smem_shared(attn_own_kernel<NB>, smem);
    if (e != cudaSuccess) return e;
    lifted[dev] = true;
  }
  return launch_k(attn_own_kernel<NB>, dim3(items), dim3(128), smem, st, true, a, o);
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
  if (!aligned_to(elem_bytes(a->qdtype), a->q, a->out) || !aligned_to(4, a->lse, a->seq_len) ||
      (a->table_stride > 0 && !aligned_to(4, a->page_table)))
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: a pointer is not aligned to its elements");
  // (a branch's output is written while others have yet to read their queries)
  if (a->out == a->q && a->batch > 1 && a->out_stride != a->q_stride)
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: out over q needs q's stride");
  if (!a->d_workspace || reinterpret_cast<uintptr_t>(a->d_workspace) % 256)
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: workspace must be non-NULL and 256-byte aligned");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  const AsPlan p = attn_plan(a, di.sms);
  if (a->workspace_bytes < p.total)
    return fail(nullptr, DEC_ENOMEM, "attn_shared_prefix: workspace has %zu bytes, %zu needed", a->workspace_bytes,
                p.total);
  if (p.prefix_items + p.own_items >= 1ll << 31 || p.own_per >= 1ll << 31)
    return fail(nullptr, DEC_EINVAL, "attn_shared_prefix: %lld work items of %lld blocks",
                p.prefix_items + p.own_items, p.own_per);
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
  k.scale_log2 = a->scale == 0.f ? 1.f : fabsf(a->scale) * 1.44269504088896340736f;
  k.q_sign = a->scale == 0.f ? 0 : a->scale < 0.f ? -1 : 1;
  k.row_groups = p.row_groups;
  k.prefix_items = p.tc ? 0 : static_cast<int>(p.prefix_items);
  k.prefix_chunk = p.prefix_chunk;
  k.own_block = p.own_block;
  k.own_seg = p.own_seg;
  k.own_per = p.own_per;
  k.q_even = reinterpret_cast<uintptr_t>(a->q) % 4 == 0 && a->q_stride % 2 == 0;
  k.own_slot0 = p.prefix_slots;
  k.part_o = reinterpret_cast<float*>(w + p.o);
  k.part_ml = reinterpret_cast<float2*>(w + p.ml);
  k.err = di.err;
  const bool qf = a->qdtype == DEC_F32;
  if (p.tc) {
    ApArgs t{};
    t.q = static_cast<const uint16_t*>(a->q);
    t.q_stride = a->q_stride;
    t.batch = a->batch;
    t.n_q = a->n_q;
    t.n_kv = a->n_kv;
    t.group = k.group;
    t.rows = k.rows;
    t.row_blocks = p.row_groups;
    t.plen = a->prefix_len;
    t.chunk = p.prefix_chunk;
    t.scale_log2 = k.scale_log2;
    t.q_sign = k.q_sign;
    t.part_o = k.part_o;
    t.part_ml = k.part_ml;
    t.err = di.err;
    alignas(64) CUtensorMap maps[2];
    for (int i = 0; i < 2; ++i) {
      const dec_status m = encode_map_3d_bf16(&maps[i], i ? a->prefix_v : a->prefix_k, a->n_kv, a->prefix_len, kApD,
                                              a->prefix_stride * kApD * 2, 64, kApKeys, nullptr);
      if (m != DEC_OK) return m;
    }
    static bool lifted[64] = {};
    if (!lifted[di.device]) {
      WSG_CUDA_TRY(nullptr, allow_smem_shared(attn_prefix_tc_kernel, kApSmem));
      lifted[di.device] = true;
    }
    WSG_CUDA_TRY(nullptr, launch_k(attn_prefix_tc_kernel, dim3(static_cast<unsigned>(p.prefix_items)), dim3(kApThreads),
                                   kApSmem, s, true, maps[0], maps[1], t));
  }
  if (p.own_joins) {
    k.first = !p.tc;
    AoArgs o{};
    o.prefix_slots = p.prefix_slots;
    o.out = a->out;
    o.out_stride = a->out_stride;
    o.lse = a->lse;
    WSG_CUDA_TRY(nullptr, k.group > 8 ? launch_own<16>(k, o, static_cast<unsigned>(p.own_items), di.device, s)
                                      : launch_own<8>(k, o, static_cast<unsigned>(p.own_items), di.device, s));
    return DEC_OK;
  }
  const int items = k.prefix_items + static_cast<int>(p.own_items);
  k.first = !p.tc;
  if (items > 0)
    WSG_CUDA_TRY(nullptr, a->kvdtype == DEC_F32 ? launch_attn_f32(k, qf, items, di.device, s)
                                                : launch_attn_bf16(k, qf, p.na, items, di.device, s));
  AmJoinArgs j{};
  j.batch = a->batch;
  j.n_q = a->n_q;
  j.d = a->head_dim;
  j.prefix_slots = p.prefix_slots;
  j.warps = p.prefix_slots + p.own_slots > 8 ? 4 : 1;
  j.own_block = p.own_block;
  j.own_seg = p.own_seg;
  j.own_per = p.own_per;
  j.n_kv = a->n_kv;
  j.group = k.group;
  j.pool = k.pool;
  j.len = a->seq_len;
  j.part_o = k.part_o;
  j.part_ml = k.part_ml;
  j.out = a->out;
  j.out_stride = a->out_stride;
  j.lse = a->lse;
  j.err = di.err;
  const int jrows = a->batch * a->n_q;
  const dim3 grid(j.warps == 4 ? jrows : (jrows + 3) / 4);
  WSG_CUDA_TRY(nullptr, qf ? launch_k(attn_join_kernel<float>, grid, dim3(128), 0, s, true, j)
                           : launch_k(attn_join_kernel<uint16_t>, grid, dim3(128), 0, s, true, j));
  return DEC_OK;
}
