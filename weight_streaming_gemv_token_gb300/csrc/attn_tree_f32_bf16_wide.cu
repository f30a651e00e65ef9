// attn_tree_paged, float32 queries over bfloat16 caches, heads above 64: the launches of attn_tree_rows_kernel.
#include "attn_tree_rows.cuh"

namespace wsg {

cudaError_t launch_tree_f32_bf16_wide(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  return at_launch_rows<float, 128, 3, false>(a, di, st);
}

}  // namespace wsg
