// attn_tree_paged, float32 queries over float32 caches: the launches of attn_tree_rows_kernel.
#include "attn_tree_rows.cuh"

namespace wsg {

cudaError_t launch_tree_f32_f32(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  return a.a.d > 64 ? launch_tree_f32_f32_wide(a, di, st) : at_launch<float, 1, true>(a, di, st);
}

}  // namespace wsg
