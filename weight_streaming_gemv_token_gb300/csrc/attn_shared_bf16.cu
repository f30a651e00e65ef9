// attn_shared_prefix over bfloat16 caches: the launches of attn_rows_kernel.
#include "attn_rows.cuh"

namespace wsg {

cudaError_t launch_attn_bf16(const AmArgs& a, bool q_f32, int na, int items, int dev, cudaStream_t st) {
  return q_f32 ? ar_launch<float, 3>(a, na, items, dev, st) : ar_launch<uint16_t, 1>(a, na, items, dev, st);
}

}  // namespace wsg
