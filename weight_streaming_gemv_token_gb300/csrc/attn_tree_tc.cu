// attn_tree_paged on the tensor cores: the launches of attn_tree_tc_kernel.
#include "attn_tree_tc.cuh"

namespace wsg {
namespace {

template <int D>
dec_status launch(const AtArgs& t, const CUtensorMap* maps, const DeviceInfo& di, cudaStream_t st) {
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    WSG_CUDA_TRY(nullptr, allow_smem_shared(attn_tree_tc_kernel<D>, TtGeom<D>::SMEM));
    lifted[di.device] = true;
  }
  WSG_CUDA_TRY(nullptr, launch_k(attn_tree_tc_kernel<D>, dim3(di.sms), dim3(kTtThreads), TtGeom<D>::SMEM, st, true, maps[0],
                                 maps[1], maps[2], maps[3], t));
  return DEC_OK;
}

}  // namespace

dec_status launch_tree_tc(const AtArgs& t, const DeviceInfo& di, cudaStream_t st) {
  const AmArgs& a = t.a;
  alignas(64) CUtensorMap maps[4];
  const long long page = 1ll << a.pool.shift, rows = page < kAtKeys ? page : kAtKeys;
  for (int i = 0; i < 2; ++i) {
    dec_status s = encode_map_3d_bf16(&maps[2 + i], i ? a.vp : a.kp, static_cast<long long>(a.pool.num_pages) * a.n_kv, page,
                                      a.d, page * a.d * 2, 64, static_cast<int>(rows), nullptr);
    if (s == DEC_OK && a.plen > 0)
      s = encode_map_3d_bf16(&maps[i], i ? a.pv : a.pk, a.n_kv, a.plen, a.d, a.pstride * a.d * 2, 64, kAtKeys, nullptr);
    else if (s == DEC_OK)
      maps[i] = maps[2 + i];  // never used
    if (s != DEC_OK) return s;
  }
  return a.d == 128 ? launch<128>(t, maps, di, st) : launch<64>(t, maps, di, st);
}

}  // namespace wsg
