// attn_tree_paged over bfloat16 caches: the launches of attn_tree_rows_kernel.
#include "attn_tree_rows.cuh"

namespace wsg {

cudaError_t launch_tree_bf16(const AtArgs& a, bool q_f32, const DeviceInfo& di, cudaStream_t st) {
  return q_f32 ? at_launch<float, 3, false>(a, di, st) : at_launch<uint16_t, 1, false>(a, di, st);
}

}  // namespace wsg
