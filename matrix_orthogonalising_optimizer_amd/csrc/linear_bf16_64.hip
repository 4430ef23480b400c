// The training operators' product kernel: bf16 operands, 64 x 64 tiles.
#include "linear_impl.h"

namespace dmuon {
hipError_t launch_linear_bf16_64(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  return launch_lin<bf16_t, bf16_t, 64>(mode, epi, a, grid, st);
}
}  // namespace dmuon
