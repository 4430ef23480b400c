// When a 16-byte chunk of a matrix whose rows may start at any element stays
// inside the matrix (host and device).
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define DMUON_HD __host__ __device__
#else
#define DMUON_HD
#endif

namespace dmuon {

// A row-major operand of K rows, `ld` elements apart, is read in steps of `ks`
// rows.  A chunk of `vec` elements begins inside its row and may run up to
// vec - 1 elements past the row's end.  That is inside the matrix if the rows
// behind the step hold as many elements; otherwise the step's chunks have to be
// taken element by element.
DMUON_HD constexpr bool raw_step_inside(int64_t K, int64_t ld, int ks, int step, int vec) {
  return (K - (int64_t)(step + 1) * ks) * ld >= vec - 1;
}

}  // namespace dmuon
