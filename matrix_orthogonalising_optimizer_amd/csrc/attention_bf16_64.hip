// Instances of the attention kernels: bf16 heads of up to 64.
#include "attention_impl.h"

namespace dmuon {
hipError_t launch_attn_bf16_64(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  return launch_attn<bf16_t, 64, 64, 64, 4, 2, 4, 2, 4, 2, false, true, 4, 4, false>(pass, a, grid, st);
}
}  // namespace dmuon
