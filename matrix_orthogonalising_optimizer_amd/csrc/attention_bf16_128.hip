// Instances of the attention kernels: bf16 heads of up to 128.
#include "attention_impl.h"

namespace dmuon {
hipError_t launch_attn_bf16_128(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  return launch_attn<bf16_t, 128, 64, 32, 2, 2, 2, 2, 4, 1, false, true, 4, 4, true>(pass, a, grid, st);
}
}  // namespace dmuon
