// attn_shared_prefix over float32 caches: the launches of attn_mma_kernel's tf32 form.
#include "attn_mma.cuh"

namespace wsg {

cudaError_t am_launch_f32(const AmArgs& a, bool q_f32, int items, int dev, cudaStream_t st) {
  return q_f32 ? am_launch_head<float, 3, 1, true>(a, items, dev, st)
               : am_launch_head<uint16_t, 1, 1, true>(a, items, dev, st);
}

}  // namespace wsg
