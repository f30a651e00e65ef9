// attn_tree_paged, float32 queries over bfloat16 caches: the launches of attn_tree_rows_kernel.
#include "attn_tree_rows.cuh"

namespace wsg {

cudaError_t launch_tree_f32_bf16(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  return a.a.d > 64 ? launch_tree_f32_bf16_wide(a, di, st) : at_launch<float, 3, false>(a, di, st);
}

}  // namespace wsg
