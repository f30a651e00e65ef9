// attn_shared_prefix over float32 caches: the launches of attn_f32_kernel.
#include "attn_mma.cuh"

namespace wsg {

cudaError_t launch_attn_f32(const AmArgs& a, bool q_f32, int items, int dev, cudaStream_t st) {
  return q_f32 ? am_launch<float>(a, items, dev, st) : am_launch<uint16_t>(a, items, dev, st);
}

}  // namespace wsg
