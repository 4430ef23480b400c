// Instances of the attention kernels: bf16 heads of up to 96.
#include "attention_impl.h"

namespace dmuon {
hipError_t launch_attn_bf16_96(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  return launch_attn<bf16_t, 96, 64, 32, 2, 2, 2, 2, 4, 1, false, true, 4, 4, false>(pass, a, grid, st);
}
}  // namespace dmuon
