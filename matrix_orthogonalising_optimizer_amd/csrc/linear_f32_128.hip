// The training operators' product kernel: f32 operands, 128 x 128 tiles.
#include "linear_impl.h"

namespace dmuon {
hipError_t launch_linear_f32_128(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  return launch_lin<float, float, 128>(mode, epi, a, grid, st);
}
}  // namespace dmuon
