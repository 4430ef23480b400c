// The training operators' product kernel: bf16 operands, 128 x 128 tiles.
#include "linear_impl.h"

namespace dmuon {
hipError_t launch_linear_bf16_128(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  return launch_lin<bf16_t, bf16_t, 128>(mode, epi, a, grid, st);
}
}  // namespace dmuon
