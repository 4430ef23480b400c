// The training operators' product kernel: f32 operands, 64 x 64 tiles.
#include "linear_impl.h"

namespace dmuon {
hipError_t launch_linear_f32_64(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  return launch_lin<float, float, 64>(mode, epi, a, grid, st);
}
}  // namespace dmuon
