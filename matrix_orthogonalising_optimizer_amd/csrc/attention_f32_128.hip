// Instances of the attention kernels: fp32 heads of up to 128.
#include "attention_impl.h"

namespace dmuon {
hipError_t launch_attn_f32_128(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  return launch_attn<float, 128, 32, 32, 2, 2, 4, 1, 4, 1, false, false, 4, 4, false>(pass, a, grid, st);
}
}  // namespace dmuon
