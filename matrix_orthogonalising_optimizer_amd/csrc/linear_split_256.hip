// The training operators' product kernel: f32 operands in bf16 planes, 256 x 256 tiles.
#include "linear_impl.h"

namespace dmuon {
hipError_t launch_linear_split_256(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  return launch_lin<bf16_t, float, 256>(mode, epi, a, grid, st);
}
}  // namespace dmuon
