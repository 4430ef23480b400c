// Every chunk that the product kernel reads whole from a row-major matrix with
// rows at any element: the last element read has to be one of the matrix.
// Prints the number of chunks checked, or the first one outside and exits 1.
#include <stdio.h>

#include "raw_rows.h"

int main() {
  long checked = 0;
  for (int es = 2; es <= 4; es += 2) {
    const int vec = 16 / es, ks = 128 / es;  // elements of a chunk, rows of a step
    for (int tile = 64; tile <= 128; tile *= 2)
      for (int n = 1; n <= 2 * tile + 1; n += n < 40 ? 1 : 13)
        for (int k = 0; k <= 3 * ks; ++k)
          for (int step = 0; step < k / ks; ++step)
            for (int n0 = 0; n0 < n; n0 += tile) {
              const bool edge = n0 + tile > n;
              if (edge && !dmuon::raw_step_inside(k, n, ks, step, vec)) continue;  // element by element
              for (int row = step * ks; row < (step + 1) * ks; ++row)
                for (int c = 0; c < tile / vec; ++c) {
                  const int in = c < (n - 1 - n0) / vec ? c : (n - 1 - n0) / vec;
                  const long last = (long)row * n + n0 + in * vec + vec - 1;
                  ++checked;
                  if (last >= (long)k * n) {
                    printf("%d-byte elements, %d x %d, row %d, column %d: element %ld of %ld\n", es, k, n, row,
                           n0 + in * vec, last, (long)k * n);
                    return 1;
                  }
                }
            }
  }
  printf("%ld\n", checked);
  return 0;
}
