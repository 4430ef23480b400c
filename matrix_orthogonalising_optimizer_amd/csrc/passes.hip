// Passes around the training operators' products: operand copies with padded
// rows, sums of split products with the gate's arithmetic, and the cross
// entropy's row statistics.  All are bound by HBM (or, at the small sizes,
// by their launch): every element is touched once, in 16-byte pieces where
// rows are aligned.

#include "linear_impl.h"

namespace dmuon {
namespace {

template <int ES>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return load_out(gload_ptr(p), i, ES == 4);
}
template <int ES>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  store_out(gstore_ptr(p), i, v, ES == 4);
}

// one 16-byte chunk of a destination row per thread
template <int ES>
__global__ void __launch_bounds__(256) pack_rows_kernel(const void* src, int64_t src_ld, void* dst, int64_t dst_ld,
                                                        int64_t rows, int64_t cols) {
  constexpr int V = 16 / ES;
  const int64_t per = dst_ld / V;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= rows * per) return;
  const int64_t r = c / per, k = (c - r * per) * V;
  const int64_t left = cols - k;
  const u32x4 v = load_chunk_partial<ES>(gload_ptr(src), r * src_ld + k, left < V ? (int)left : V);
  *(gu4*)(gstore_ptr(dst) + (r * dst_ld + k) * ES) = v;
}

// sum of the parts at element i
__device__ __forceinline__ float sum_at(const float* part, int64_t stride, int splits, int64_t i) {
  float s = 0.0f;
  for (int k = 0; k < splits; ++k) s += part[(int64_t)k * stride + i];
  return s;
}

template <int ES>
__global__ void __launch_bounds__(256) sum_parts_kernel(const SumArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = c / a.npad, k = c - r * a.npad;
  if (r >= a.rows) return;
  float v = 0.0f;
  if (k < a.cols) v = sum_at(a.part, a.stride, a.splits, r * a.part_ld + k) * (a.alpha ? *a.alpha : 1.0f);
  store1<ES>(a.out, r * a.ldo + k, v);
}

template <int ES, int ACT>
__global__ void __launch_bounds__(256) gate_fwd_kernel(const GateArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = c / a.npad, k = c - r * a.npad;
  if (r >= a.rows) return;
  float g = 0.0f, u = 0.0f;
  if (k < a.cols) {
    g = sum_at(a.part, a.stride, a.splits, r * a.part_ld + k);
    u = sum_at(a.part + (int64_t)a.splits * a.stride, a.stride, a.splits, r * a.part_ld + k);
  }
  store1<ES>(a.o1, r * a.ld + k, k < a.cols ? act_only<ACT>(g) * u : 0.0f);
  if (a.o2) {
    store1<ES>(a.o2, r * a.ld + k, g);
    store1<ES>(a.o3, r * a.ld + k, u);
  }
}

template <int ES, int ACT>
__global__ void __launch_bounds__(256) gate_bwd_kernel(const GateArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = c / a.npad, k = c - r * a.npad;
  if (r >= a.rows) return;
  float dg = 0.0f, du = 0.0f;
  if (k < a.cols) {
    const float dh = sum_at(a.part, a.stride, a.splits, r * a.part_ld + k);
    float f, df;
    act_both<ACT>(load1<ES>(a.g_in, r * a.ld + k), f, df);
    dg = dh * load1<ES>(a.u_in, r * a.ld + k) * df;
    du = dh * f;
  }
  store1<ES>(a.o1, r * a.ld + k, dg);
  store1<ES>(a.o2, r * a.ld + k, du);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// One workgroup per token: join the pieces' (maximum, sum) pairs into the
// token's log-sum-exp, write its loss and, for gradients, turn the stored
// exponentials e_v = exp(l_v - piece maximum) into exp(l_v - lse) - [v = y] in
// place.  The target's entry comes from its fp32 logit as expm1(l_y - lse):
// for a sure prediction 1 - p is far below the 16-bit rounding of p.  A token
// whose target is no word has loss 0 and a row of zeros.
template <int ES>
__global__ void __launch_bounds__(256) xent_rows_kernel(const XentArgs a) {
  __shared__ float red[8];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, wave = tid >> 6;
  const float2* st = a.stats + t * a.pieces;
  const int64_t y = a.targets[t];
  const bool counts = y >= 0 && y < a.vocab;
  if (!counts) {
    if (tid == 0) a.losses[t] = 0.0f;
    if (a.p) {
      char* row = (char*)a.p + t * a.ldp * ES;
      for (int64_t k = (int64_t)tid * 16; k < a.ldp * ES; k += 256 * 16)
        *(gu4*)(gstore_ptr(row) + k) = u32x4{0u, 0u, 0u, 0u};
    }
    return;
  }
  float m = -INFINITY;
  for (int i = tid; i < a.pieces; i += 256) m = fmaxf(m, st[i].x);
  m = wave_max(m);
  if ((tid & 63) == 0) red[wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float ref = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
  for (int i = tid; i < a.pieces; i += 256) {
    const float2 v = st[i];
    s += v.y * expf(v.x - ref);
  }
  s = wave_sum(s);
  if ((tid & 63) == 0) red[4 + wave] = s;
  __syncthreads();
  s = (red[4] + red[5]) + (red[6] + red[7]);
  const float lse = ref + logf(s), tl = a.target_logit[t];
  if (tid == 0) a.losses[t] = lse - tl;
  if (!a.p) return;
  const float at = expm1f(tl - lse);
  gchar* row = gstore_ptr((char*)a.p + t * a.ldp * ES);
  constexpr int V = 16 / ES;
  for (int64_t k = (int64_t)tid * V; k < a.vocab; k += 256 * V) {
    // (maximum - lse may be -inf - x: a piece without a finite logit, 0)
    const float f = expf(st[k / a.piece].x - lse);
    u32x4 v = *(gu4*)(row + k * ES);
    if constexpr (ES == 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float lo = k + 2 * q == y ? at : f * __uint_as_float(v[q] << 16);
        const float hi = k + 2 * q + 1 == y ? at : f * __uint_as_float(v[q] & 0xffff0000u);
        v[q] = pack_bf16(lo, hi);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = __float_as_uint(k + q == y ? at : f * __uint_as_float(v[q]));
    }
    *(gu4*)(row + k * ES) = v;
  }
}

__global__ void __launch_bounds__(1024) xent_count_kernel(const int64_t* targets, int64_t tokens, int64_t vocab,
                                                          float* inv_n) {
  __shared__ float red[16];
  float c = 0.0f;  // exact up to 2^24 per thread, far past any count here
  for (int64_t i = threadIdx.x; i < tokens; i += 1024) c += (targets[i] >= 0 && targets[i] < vocab) ? 1.0f : 0.0f;
  c = wave_sum(c);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    double n = 0.0;
    for (int i = 0; i < 16; ++i) n += red[i];
    *inv_n = (float)(1.0 / (n > 1.0 ? n : 1.0));
  }
}

// fixed order: bitwise the same on every run
__global__ void __launch_bounds__(1024) xent_mean_kernel(const float* losses, int64_t tokens, const float* inv_n,
                                                         float* loss) {
  __shared__ double red[1024];
  double c = 0.0;
  for (int64_t i = threadIdx.x; i < tokens; i += 1024) c += losses[i];
  red[threadIdx.x] = c;
  __syncthreads();
  for (int o = 512; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) *loss = (float)(red[0] * (double)*inv_n);
}

bool blocks_of(int64_t n, unsigned* out) {
  const int64_t b = (n + 255) / 256;
  *out = (unsigned)b;
  return b <= 0x7fffffff;
}

}  // namespace

hipError_t launch_pack_rows(const void* src, int64_t src_ld, void* dst, int64_t dst_ld, int64_t rows, int64_t cols,
                            int esize, hipStream_t st) {
  unsigned grid;
  if (!blocks_of(rows * (dst_ld / (16 / esize)), &grid)) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  if (esize == 2)
    hipLaunchKernelGGL(pack_rows_kernel<2>, dim3(grid), dim3(256), 0, st, src, src_ld, dst, dst_ld, rows, cols);
  else
    hipLaunchKernelGGL(pack_rows_kernel<4>, dim3(grid), dim3(256), 0, st, src, src_ld, dst, dst_ld, rows, cols);
  return hipGetLastError();
}

hipError_t launch_sum_parts(const SumArgs& a, hipStream_t st) {
  unsigned grid;
  if (!blocks_of(a.rows * a.npad, &grid)) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  if (a.esize == 2)
    hipLaunchKernelGGL(sum_parts_kernel<2>, dim3(grid), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(sum_parts_kernel<4>, dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_gate_fwd(const GateArgs& a, hipStream_t st) {
  unsigned grid;
  if (!blocks_of(a.rows * a.npad, &grid)) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  auto go = [&](auto act_t) {
    constexpr int ACT = decltype(act_t)::value;
    if (a.esize == 2)
      hipLaunchKernelGGL((gate_fwd_kernel<2, ACT>), dim3(grid), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((gate_fwd_kernel<4, ACT>), dim3(grid), dim3(256), 0, st, a);
  };
  if (a.act == LIN_SILU) go(std::integral_constant<int, LIN_SILU>{});
  else if (a.act == LIN_GELU) go(std::integral_constant<int, LIN_GELU>{});
  else if (a.act == LIN_GELU_TANH) go(std::integral_constant<int, LIN_GELU_TANH>{});
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_gate_bwd(const GateArgs& a, hipStream_t st) {
  unsigned grid;
  if (!blocks_of(a.rows * a.npad, &grid)) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  auto go = [&](auto act_t) {
    constexpr int ACT = decltype(act_t)::value;
    if (a.esize == 2)
      hipLaunchKernelGGL((gate_bwd_kernel<2, ACT>), dim3(grid), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((gate_bwd_kernel<4, ACT>), dim3(grid), dim3(256), 0, st, a);
  };
  if (a.act == LIN_SILU) go(std::integral_constant<int, LIN_SILU>{});
  else if (a.act == LIN_GELU) go(std::integral_constant<int, LIN_GELU>{});
  else if (a.act == LIN_GELU_TANH) go(std::integral_constant<int, LIN_GELU_TANH>{});
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_xent_rows(const XentArgs& a, hipStream_t st) {
  if (a.tokens <= 0) return hipSuccess;
  if (a.tokens > 0x7fffffff) return hipErrorInvalidValue;
  if (a.esize == 2)
    hipLaunchKernelGGL(xent_rows_kernel<2>, dim3((unsigned)a.tokens), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(xent_rows_kernel<4>, dim3((unsigned)a.tokens), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_xent_count(const int64_t* targets, int64_t tokens, int64_t vocab, float* inv_n, hipStream_t st) {
  hipLaunchKernelGGL(xent_count_kernel, dim3(1), dim3(1024), 0, st, targets, tokens, vocab, inv_n);
  return hipGetLastError();
}

hipError_t launch_xent_mean(const float* losses, int64_t tokens, const float* inv_n, float* loss, hipStream_t st) {
  hipLaunchKernelGGL(xent_mean_kernel, dim3(1), dim3(1024), 0, st, losses, tokens, inv_n, loss);
  return hipGetLastError();
}

hipError_t launch_linear(bool f32, int tile, LinMode mode, LinEpi epi, LinArgs& a, hipStream_t st) {
  if (a.nprob < 1 || a.nprob > kLinMaxProb) return hipErrorInvalidValue;
  const int nt = epi == LIN_GATE ? tile / 2 : tile;
  int64_t per_xcd = 0;
  for (int i = 0; i < a.nprob; ++i) {
    LinProb& q = a.p[i];
    if (q.M < 1 || q.N < 1 || q.K < 0 || q.splits < 1 || q.nseg < 1) return hipErrorInvalidValue;
    if (q.nseg > 1 && mode != LIN_KR) return hipErrorInvalidValue;
    if (q.splits > 1 && epi != LIN_ACC) return hipErrorInvalidValue;
    q.tiles_m = (q.M + tile - 1) / tile;
    q.tiles_n = (q.N + nt - 1) / nt;
    const int64_t n = (int64_t)q.tiles_m * q.tiles_n * q.splits;
    if (n > (1 << 28)) return hipErrorInvalidValue;
    per_xcd += (n + 7) / 8;
  }
  const int grid = (int)(per_xcd * 8);
  if (f32) {
    if (tile == 128) return launch_linear_f32_128(mode, epi, a, grid, st);
    if (tile == 64) return launch_linear_f32_64(mode, epi, a, grid, st);
  } else {
    if (tile == 256) return launch_linear_bf16_256(mode, epi, a, grid, st);
    if (tile == 128) return launch_linear_bf16_128(mode, epi, a, grid, st);
    if (tile == 64) return launch_linear_bf16_64(mode, epi, a, grid, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace dmuon
