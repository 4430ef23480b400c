// Dropout whose mask is computed where it is needed and never stored:
//   y_i = [u_i >= cut] x_i / (1 - cut / 2^16)  (+ residual_i)
// u_i is a 16-bit number of Philox 4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): counter offset + i / 8, key
// seed, word (i % 8) / 2, its lower half for even i.  Eight elements share one
// counter, so a lane's 16 bytes are one evaluation.
//
// HBM bound: with 32-bit numbers the generator's multiplications would take as
// long as the memory (four evaluations a lane's 32 bytes instead of two).  The result
// alone is rounded.  16384 x 4096 bf16 with a residual 80 us (5.0 TB/s), backward 46 us
// (5.8 TB/s, in part from the last-level cache).

#include <algorithm>

#include "heads.h"
#include "linear_impl.h"

namespace dmuon {
namespace {

__device__ __forceinline__ u32x4 philox(uint64_t counter, uint64_t key) {
  u32x4 c = {(uint32_t)counter, (uint32_t)(counter >> 32), 0u, 0u};
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c[0], b = (uint64_t)0xCD9E8D57u * c[2];
    c = u32x4{(uint32_t)(b >> 32) ^ c[1] ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c[3] ^ k1, (uint32_t)a};
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

template <int ES, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutArgs a) {
  uint64_t seed = a.seed, offset = a.offset;
  if (a.state) {
    seed = (uint64_t)a.state[0];
    offset += (uint64_t)a.state[1];
  }
  const int64_t groups = (a.n + 7) >> 3;
  cgchar *px = gload_ptr(a.x), *pr = gload_ptr(a.residual);
  gchar* py = gstore_ptr(a.y);
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
    const int left = (int)min((int64_t)8, a.n - g * 8);
    float x[8], r[8];
    if (left == 8) {
      unpack8<ES>((cgu4_any*)(px + g * 8 * ES), x);
      if constexpr (RES) unpack8<ES>((cgu4_any*)(pr + g * 8 * ES), r);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = k < left ? load_out(px, g * 8 + k, ES == 4) : 0.0f;
        if constexpr (RES) r[k] = k < left ? load_out(pr, g * 8 + k, ES == 4) : 0.0f;
      }
    }
    const u32x4 w = philox(offset + (uint64_t)g, seed);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t u = (k & 1) ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu;
      x[k] = u >= a.cut ? x[k] * a.scale : 0.0f;
      if constexpr (RES) x[k] += r[k];
    }
    if (left == 8) {
      u32x4 o[ES / 2];
      pack8<ES>(x, o);
#pragma unroll
      for (int k = 0; k < ES / 2; ++k) ((gu4_any*)(py + g * 8 * ES))[k] = o[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) store_out(py, g * 8 + k, x[k], ES == 4);
    }
  }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st) {
  if (a.n <= 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((a.n + 2047) / 2048, 8192));
  auto one = [&](auto es) {
    constexpr int ES = decltype(es)::value;
    if (a.residual) hipLaunchKernelGGL((dropout_kernel<ES, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((dropout_kernel<ES, false>), grid, dim3(256), 0, st, a);
  };
  if (a.esize == 2) one(std::integral_constant<int, 2>{});
  else one(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace dmuon
