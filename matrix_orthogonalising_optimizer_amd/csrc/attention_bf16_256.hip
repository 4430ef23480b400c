// Instances of the attention kernels: bf16 heads of up to 256.
#include "attention_impl.h"

namespace dmuon {
hipError_t launch_attn_bf16_256(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  return launch_attn<bf16_t, 256, 32, 32, 4, 1, 4, 1, 2, 1, true, false, 4, 4, true>(pass, a, grid, st);
}
}  // namespace dmuon
