// Passes around the training operators' products: operand copies with padded
// rows (4.6 TB/s at 35 million bf16 elements), fp32 matrices as bf16 planes,
// the rounding of an fp32 sum, and the cross entropy's rows (5.3 TB/s at
// 8192 x 50257 in bf16) and mean.  All are bound by HBM or, at the small
// sizes, by their launch: every element is touched once, in 16-byte pieces
// where rows are aligned (but for the rounded sum's stores, one element each).

#include <algorithm>

#include "linear_impl.h"

namespace dmuon {
namespace {

template <int ES>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  store_out(gstore_ptr(p), i, v, ES == 4);
}

// kPackChunks 16-byte chunks of destination rows per thread, 256 apart
constexpr int kPackChunks = 4;
template <int ES>
__global__ void __launch_bounds__(256) pack_rows_kernel(const PackArgs a, int64_t b0) {
  constexpr int V = 16 / ES;
  const int64_t blk = b0 + blockIdx.x;
  int q = 0;
  while (q + 1 < a.n && blk >= a.blk0[q + 1]) ++q;
  const int64_t cols = a.cols[q], per = a.ld[q] / V, total = a.rows[q] * per;
  cgchar* src = gload_ptr(a.src[q]);
  gchar* dst = gstore_ptr(a.dst[q]);
  const int64_t c0 = (blk - a.blk0[q]) * (256 * kPackChunks) + threadIdx.x;
  u32x4 v[kPackChunks];
#pragma unroll
  for (int i = 0; i < kPackChunks; ++i) {
    const int64_t c = c0 + i * 256;
    if (c >= total) continue;
    const int64_t r = c / per, k = (c - r * per) * V;
    if (k + V <= cols)
      v[i] = *(cgu4_any*)(src + (r * cols + k) * ES);
    else
      v[i] = load_chunk_partial<ES>(src, r * cols + k, (int)(cols - k));
  }
#pragma unroll
  for (int i = 0; i < kPackChunks; ++i) {
    const int64_t c = c0 + i * 256;
    if (c < total) *(gu4*)(dst + c * 16) = v[i];
  }
}

// Nearest bf16 to v, as fp32 (v itself cut where that is an infinity).
__device__ __forceinline__ float near_bf16(float v) {
  const float h = __uint_as_float(f32_to_bf16(v) << 16);
  return fabsf(h) == INFINITY && fabsf(v) != INFINITY ? __uint_as_float(__float_as_uint(v) & 0xffff0000u) : h;
}
// v as p[0] + p[1] + p[2], each exact in bf16; whether v is finite
__device__ __forceinline__ bool planes_of(float v, float* p) {
  const bool finite = fabsf(v) < INFINITY;
  p[0] = near_bf16(v);
  const float r = finite ? v - p[0] : 0.0f;
  p[1] = near_bf16(r);
  p[2] = r - p[1];
  return finite;
}
// eight values' planes to plane stride `plane` (elements)
__device__ __forceinline__ void store_planes(uint16_t* dst, int64_t plane, const float* v, int32_t* flag) {
  u32x4 o[3];
  bool finite = true;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a[3], b[3];
    finite &= planes_of(v[2 * k], a);
    finite &= planes_of(v[2 * k + 1], b);
#pragma unroll
    for (int q = 0; q < 3; ++q) o[q][k] = pack_bf16(a[q], b[q]);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) *(gu4*)gstore_ptr(dst + q * plane) = o[q];
  if (!finite) *flag = 1;
}

__global__ void __launch_bounds__(256) planes_kernel(const SplitArgs a, int64_t b0) {
  const int64_t blk = b0 + blockIdx.x;
  int q = 0;
  while (q + 1 < a.n && blk >= a.blk0[q + 1]) ++q;
  const int64_t rows = a.rows[q], cols = a.cols[q];
  const int64_t ld = (cols + 63) / 64 * 64, per = ld / 8, rp = (rows + 63) / 64 * 64;
  const int64_t c = (blk - a.blk0[q]) * 256 + threadIdx.x;
  if (c >= rp * per) return;
  const int64_t r = c / per, k = (c - r * per) * 8;
  float v[8];
  if (r < rows && k + 8 <= cols) {
    unpack8<4>((cgu4_any*)(gload_ptr(a.src[q]) + (r * a.src_ld[q] + k) * 4), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r < rows && k + e < cols ? a.src[q][r * a.src_ld[q] + k + e] : 0.0f;
  }
  store_planes(a.dst[q] + r * ld + k, rp * ld, v, a.flag);
}

// The fourth plane: the first one's finite values.  A workgroup per compute
// unit: nearly every call has no others, and the grid ends at once.
__global__ void __launch_bounds__(256) finite_plane_kernel(const FiniteArgs a) {
  if (*a.flag == 0) return;
  for (int q = 0; q < a.n; ++q) {
    cgu4* src = (cgu4*)gload_ptr(a.planes[q]);
    gu4* dst = (gu4*)gstore_ptr(a.planes[q] + 3 * a.plane[q]);
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < a.plane[q] / 8; c += (int64_t)gridDim.x * 256) {
      u32x4 v = src[c];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((v[k] & 0x7f800000u) == 0x7f800000u) v[k] &= 0x0000ffffu;
        if ((v[k] & 0x00007f80u) == 0x00007f80u) v[k] &= 0xffff0000u;
      }
      dst[c] = v;
    }
  }
}
__global__ void clear_flags_kernel(int32_t* flags, int n) {
  if ((int)threadIdx.x < n) flags[threadIdx.x] = 0;
}

template <int ES>
__global__ void __launch_bounds__(256) scale_round_kernel(const float* src, int64_t ld, void* out, int64_t rows,
                                                          int64_t cols, const float* alpha, int64_t b0) {
  const int64_t per = ld / 4;
  const int64_t c = (b0 + blockIdx.x) * 256 + threadIdx.x;
  const int64_t r = c / per, k = (c - r * per) * 4;
  if (r >= rows) return;
  const u32x4 v = *(cgu4*)(gload_ptr(src) + (r * ld + k) * 4);
  const float f = *alpha;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (k + e < cols) store1<ES>(out, r * cols + k + e, f * __uint_as_float(v[e]));
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
// exponentials e_v = exp(l_v - piece maximum) into exp(l_v - lse) - [v = y],
// times a power of two that keeps the sums over tokens in range, in place.
// The target's entry comes from its fp32 logit as expm1(-loss): for a sure
// prediction 1 - p is far below the 16-bit rounding of p.  A token whose target
// is no word has loss 0 and a row of zeros.
template <int ES>
__global__ void __launch_bounds__(256) xent_rows_kernel(const XentArgs a, int64_t b0) {
  __shared__ float red[8];
  const int64_t t = b0 + blockIdx.x;
  const int tid = threadIdx.x, wave = tid >> 6;
  const float2* st = a.stats + t * a.pieces;
  const int64_t y = t < a.tokens ? a.targets[t] : -1;
  // planes: pitch, and rows up to a multiple of 64 (those past the tokens, of
  // zeros, have workgroups of their own)
  const int64_t pld = (a.vocab + 63) / 64 * 64, plane = (a.tokens + 63) / 64 * 64 * pld;
  const bool counts = t < a.tokens && y >= 0 && y < a.vocab;
  if (!counts) {
    if (tid == 0 && t < a.tokens) a.losses[t] = 0.0f;
    if (ES == 4 && a.planes) {
      const float zero[8] = {};
      for (int64_t k = (int64_t)tid * 8; k < pld; k += 256 * 8) store_planes(a.planes + t * pld + k, plane, zero, a.flag);
    } else if (a.p) {
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
  // differences from the maximum: no rounding at the logits' magnitude
  const float ls = logf(s), loss = (ref - a.target_logit[t]) + ls;
  if (tid == 0) a.losses[t] = loss;
  if (!a.p) return;
  const float at = expm1f(-loss) * a.scale;
  gchar* row = gstore_ptr((char*)a.p + t * a.ldp * ES);
  if (ES == 4 && a.planes) {
    for (int64_t k = (int64_t)tid * 8; k < pld; k += 256 * 8) {
      const float f = k < a.vocab ? expf((st[k / a.piece].x - ref) - ls) * a.scale : 0.0f;
      float v[8];
      if (k + 8 <= a.vocab) {
        unpack8<4>((cgu4*)(row + k * 4), v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < a.vocab ? load_out(row, k + e, true) : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = k + e == y ? at : k + e < a.vocab ? f * v[e] : 0.0f;
      store_planes(a.planes + t * pld + k, plane, v, a.flag);
    }
    return;
  }
  constexpr int V = 16 / ES;
  for (int64_t k = (int64_t)tid * V; k < a.vocab; k += 256 * V) {
    // (a piece without a finite logit: exp(-inf), 0)
    const float f = expf((st[k / a.piece].x - ref) - ls) * a.scale;
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

// The mean over the tokens that count, by one workgroup in a fixed order:
// bitwise the same on every run.  (A last workgroup of the rows' launch could
// write it, but its acquire makes every workgroup flush its L2: 310 -> 1270 us
// at 8192 x 50257.)
__global__ void __launch_bounds__(1024) xent_mean_kernel(const int64_t* targets, const float* losses, int64_t tokens,
                                                         int64_t vocab, float scale, float* alpha, float* loss) {
  __shared__ double red[32];
  const int tid = threadIdx.x;
  double s = 0.0, n = 0.0;
#pragma unroll 4
  for (int64_t i = tid; i < tokens; i += 1024) {
    n += targets[i] >= 0 && targets[i] < vocab ? 1.0 : 0.0;
    if (losses) s += losses[i];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    n += __shfl_xor(n, o);
  }
  if ((tid & 63) == 0) {
    red[tid >> 6] = s;
    red[16 + (tid >> 6)] = n;
  }
  __syncthreads();
  if (tid != 0) return;
  s = n = 0.0;
  for (int i = 0; i < 16; ++i) {
    s += red[i];
    n += red[16 + i];
  }
  n = n > 1.0 ? n : 1.0;
  *alpha = (float)(1.0 / (n * (double)scale));
  if (losses) *loss = (float)(s / n);
}

// `blocks` workgroups of `kernel(args, first workgroup)`, in launches of fewer
// than 2^32 threads
template <class... A, class... B>
hipError_t launch_blocks(void (*kernel)(A...), int64_t blocks, hipStream_t st, const B&... args) {
  for (int64_t b0 = 0; b0 < blocks; b0 += kLinMaxGroups) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min(kLinMaxGroups, blocks - b0)), dim3(256), 0, st, args..., b0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_pack_rows(PackArgs& a, hipStream_t st) {
  a.blk0[0] = 0;
  for (int i = 0; i < a.n; ++i) {
    const int64_t chunks = a.rows[i] * (a.ld[i] / (16 / a.esize));
    a.blk0[i + 1] = a.blk0[i] + (chunks + 256 * kPackChunks - 1) / (256 * kPackChunks);
  }
  return launch_blocks(a.esize == 2 ? pack_rows_kernel<2> : pack_rows_kernel<4>, a.blk0[a.n], st, a);
}

hipError_t launch_planes(SplitArgs& a, hipStream_t st) {
  a.blk0[0] = 0;
  for (int i = 0; i < a.n; ++i) {
    const int64_t chunks = (a.rows[i] + 63) / 64 * 64 * ((a.cols[i] + 63) / 64 * 8);
    a.blk0[i + 1] = a.blk0[i] + (chunks + 255) / 256;
  }
  return launch_blocks(planes_kernel, a.blk0[a.n], st, a);
}

hipError_t launch_finite_plane(const FiniteArgs& a, hipStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < a.n; ++i) most = std::max(most, a.plane[i] / 8);
  if (most == 0) return hipSuccess;
  const unsigned grid = (unsigned)std::min<int64_t>((most + 255) / 256, kLinCu);
  hipLaunchKernelGGL(finite_plane_kernel, dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_clear_flags(int32_t* flags, int n, hipStream_t st) {
  if (n > 64) return hipErrorInvalidValue;
  hipLaunchKernelGGL(clear_flags_kernel, dim3(1), dim3(64), 0, st, flags, n);
  return hipGetLastError();
}

hipError_t launch_scale_round(const float* src, int64_t ld, void* out, int64_t rows, int64_t cols, int esize,
                              const float* alpha, hipStream_t st) {
  return launch_blocks(esize == 2 ? scale_round_kernel<2> : scale_round_kernel<4>, (rows * (ld / 4) + 255) / 256, st,
                       src, ld, out, rows, cols, alpha);
}

hipError_t launch_xent_rows(const XentArgs& a, hipStream_t st) {
  if (a.tokens <= 0) return hipSuccess;
  return launch_blocks(a.esize == 2 ? xent_rows_kernel<2> : xent_rows_kernel<4>,
                       a.planes ? (a.tokens + 63) / 64 * 64 : a.tokens, st, a);
}

hipError_t launch_xent_mean(const int64_t* targets, const float* losses, int64_t tokens, int64_t vocab, float scale,
                            float* alpha, float* loss, hipStream_t st) {
  hipLaunchKernelGGL(xent_mean_kernel, dim3(1), dim3(1024), 0, st, targets, losses, tokens, vocab, scale, alpha, loss);
  return hipGetLastError();
}

static hipError_t launch_one(LinKind kind, int tile, LinMode mode, LinEpi epi, const LinArgs& a, int grid,
                             hipStream_t st) {
  if (kind == LIN_SPLIT) {
    if (tile == 256) return launch_linear_split_256(mode, epi, a, grid, st);
  } else if (kind == LIN_F32) {
    if (tile == 128) return launch_linear_f32_128(mode, epi, a, grid, st);
    if (tile == 64) return launch_linear_f32_64(mode, epi, a, grid, st);
  } else {
    if (tile == 256) return launch_linear_bf16_256(mode, epi, a, grid, st);
    if (tile == 128) return launch_linear_bf16_128(mode, epi, a, grid, st);
    if (tile == 64) return launch_linear_bf16_64(mode, epi, a, grid, st);
  }
  return hipErrorInvalidValue;
}

// `per_xcd` workgroups for each XCD, in launches of fewer than 2^32 threads
static hipError_t launch_any(LinKind kind, int tile, LinMode mode, LinEpi epi, LinArgs& a, int64_t per_xcd,
                             hipStream_t st) {
  if (per_xcd > (1 << 27)) return hipErrorInvalidValue;
  for (int64_t s = 0; s < per_xcd; s += kLinMaxGroups / 8) {
    a.slot0 = (int32_t)s;
    const hipError_t e =
        launch_one(kind, tile, mode, epi, a, (int)(std::min(kLinMaxGroups / 8, per_xcd - s) * 8), st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_linear(LinKind kind, int tile, LinMode mode, LinEpi epi, LinArgs& a, hipStream_t st) {
  if (a.nprob < 1 || a.nprob > kLinMaxProb) return hipErrorInvalidValue;
  const int nt = epi == LIN_GATE ? tile / 2 : tile;
  int64_t per_xcd[3] = {0, 0, 0};  // workgroups per XCD, by role
  for (int i = 0; i < a.nprob; ++i) {
    LinProb& q = a.p[i];
    if (q.M < 1 || q.N < 1 || q.K < 0 || q.splits < 1 || q.nseg < 1) return hipErrorInvalidValue;
    if (q.nseg > 1 && mode != LIN_KR) return hipErrorInvalidValue;
    if (kind == LIN_SPLIT && q.K % 64) return hipErrorInvalidValue;
    q.tiles_m = (q.M + tile - 1) / tile;
    q.tiles_n = (q.N + nt - 1) / nt;
    const int64_t n = (int64_t)q.tiles_m * q.tiles_n;
    if (n * q.splits > (1 << 28)) return hipErrorInvalidValue;
    if (q.split_tiles < 0 || q.split_tiles > n || (q.split_tiles > 0 && (!q.part || q.splits < 2)))
      return hipErrorInvalidValue;
    per_xcd[LIN_WHOLE] += (n - q.split_tiles + 7) / 8;
    per_xcd[LIN_PART] += ((int64_t)q.split_tiles * q.splits + 7) / 8;
    per_xcd[LIN_JOIN] += (q.split_tiles + 7) / 8;
  }
  for (int role = LIN_WHOLE; role <= LIN_JOIN; ++role) {
    a.role = role;
    const hipError_t e = launch_any(kind, tile, mode, epi, a, per_xcd[role], st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace dmuon
