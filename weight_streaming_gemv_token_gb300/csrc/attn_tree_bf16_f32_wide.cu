// attn_tree_paged, bfloat16 queries over float32 caches, heads above 64: the launches of attn_tree_rows_kernel.
#include "attn_tree_rows.cuh"

namespace wsg {

cudaError_t launch_tree_bf16_f32_wide(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  return at_launch_rows<uint16_t, 128, 1, true>(a, di, st);
}

}  // namespace wsg
