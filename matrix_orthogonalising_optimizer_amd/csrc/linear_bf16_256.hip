// The training operators' product kernel: bf16 operands, 256 x 256 tiles.
#include "linear_impl.h"

namespace dmuon {
hipError_t launch_linear_bf16_256(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  return launch_lin<bf16_t, bf16_t, 256>(mode, epi, a, grid, st);
}
}  // namespace dmuon
