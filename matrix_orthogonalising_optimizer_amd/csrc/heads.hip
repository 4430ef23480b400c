// Norm of queries and keys per head with the position rotation, forward and
// backward, and copies of heads for the attention kernels.
//
//   r = 1 / sqrt(mean_j x_j^2 + eps),  n = x r,  y = Rot(n w)
//   g = Rot^T dy,  dw = sum over tokens and heads of g n,
//   dx = r (g w - n mean_j(g w n))
// Rot turns the pairs (i, i + R/2), or (2i, 2i + 1), of a head's first R elements by
// position times base^(-2i/R); a pair takes its position from the axis whose
// section it lies in.
//
// HBM bound: one read of x (and dy), one write.  A lane holds VEC elements of
// both sides of VEC pairs, so that the rotation stays inside a lane and the
// norm is a sum over the LPH lanes of a head.  The angles' cosines and sines
// are made once per token, in LDS, for all heads: in 64 bits up to the fraction
// of a turn (a position of 10^6 times an fp32 frequency would be off by 0.1), from there
// on in fp32.

#include <algorithm>

#include "heads.h"
#include "linear_impl.h"

namespace dmuon {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens of one step of a workgroup

// N elements from any element's address, as fp32, and back (N times ES a power of two)
template <int ES, int N>
struct Pack {
  static constexpr int W = N * ES / 4;  // words
  __device__ static void load(cgchar* p, float* v) {
    if constexpr (N * ES >= 16) {
      u32x4 w[N * ES / 16];
#pragma unroll
      for (int i = 0; i < N * ES / 16; ++i) w[i] = ((cgu4_any*)p)[i];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if constexpr (ES == 4)
          v[k] = __uint_as_float(w[k / 4][k % 4]);
        else
          v[k] = (k & 1) ? __uint_as_float(w[0][k / 2] & 0xffff0000u) : __uint_as_float(w[0][k / 2] << 16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = load_out(p, k, ES == 4);
    }
  }
  __device__ static void store(gchar* p, const float* v) {
    if constexpr (N * ES >= 16) {
#pragma unroll
      for (int i = 0; i < N * ES / 16; ++i) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (ES == 4)
            w[k] = __float_as_uint(v[4 * i + k]);
          else
            w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
        }
        ((gu4_any*)p)[i] = w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) store_out(p, k, v[k], ES == 4);
    }
  }
};

// Cosines and sines of the pairs' angles of `n` tokens from t0, in LDS.
__device__ __forceinline__ void fill_turns(const RopeArgs& a, int64_t t0, int n, float2* cs) {
  const int half = a.rot >> 1;
  for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
    const int t = i / half, p = i - t * half;
    const int64_t pos = ((const __attribute__((address_space(1))) int64_t*)a.positions)[(t0 + t) * a.axes + a.axis[p]];
    const double turns = (double)pos * a.turn[p];
    const float f = (float)(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(f, &s, &c);
    cs[i] = float2{c, s};
  }
}

// Chunk pair c of a head: its elements from `lo` and from `hi`, and whether they turn.
template <int VEC>
__device__ __forceinline__ bool rope_chunk(const RopeArgs& a, int c, int& lo, int& hi) {
  const bool turns = c * 2 * VEC < a.rot;
  if (turns && !a.interleaved) {
    lo = c * VEC;
    hi = (a.rot >> 1) + lo;
  } else {
    lo = c * 2 * VEC;
    hi = lo + VEC;
  }
  return turns;
}
// The VEC pairs of a chunk turned (by minus the angle with `back`).
template <int VEC>
__device__ __forceinline__ void rope_turn(const RopeArgs& a, const float2* cs, int c, bool back, float* x, float* y) {
  const float sign = back ? -1.0f : 1.0f;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const float2 t = cs[c * VEC + k];
    const float s = t.y * sign;
    // interleaved: x and y are one run of 2 VEC elements, pair k its elements 2k, 2k + 1
    if (VEC > 1 && a.interleaved) {
      float& u = 2 * k < VEC ? x[2 * k] : y[2 * k - VEC];
      float& v = 2 * k + 1 < VEC ? x[2 * k + 1] : y[2 * k + 1 - VEC];
      const float p = u * t.x - v * s, q = v * t.x + u * s;
      u = p;
      v = q;
    } else {
      const float p = x[k] * t.x - y[k] * s, q = y[k] * t.x + x[k] * s;
      x[k] = p;
      y[k] = q;
    }
  }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// LPH lanes per head, NC chunk pairs each.
template <int ES, int VEC, int LPH, int NC, bool BWD>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  constexpr int GROUPS = kRopeThreads / LPH;
  __shared__ float2 cs[kRopeTokens * kRopeHalf];
  const int lane = threadIdx.x % LPH, grp = threadIdx.x / LPH;
  const int half = a.rot >> 1, chunks = a.dim / (2 * VEC), heads = a.heads[0] + a.heads[1];
  const float inv = 1.0f / (float)a.dim;
  float dwl[BWD ? 2 : 1][NC * VEC], dwh[BWD ? 2 : 1][NC * VEC];
  if constexpr (BWD) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int k = 0; k < NC * VEC; ++k) dwl[s][k] = dwh[s][k] = 0.0f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * kRopeTokens; t0 < a.tokens; t0 += (int64_t)gridDim.x * kRopeTokens) {
    const int n = (int)min((int64_t)kRopeTokens, a.tokens - t0);
    __syncthreads();
    fill_turns(a, t0, n, cs);
    __syncthreads();
    // (q's heads of all tokens first: the sums of a side are one block of code)
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int hs = a.heads[side];
      for (int item = grp; item < n * hs; item += GROUPS) {
        const int t = item / hs, h = item - t * hs;
        cgchar* px = gload_ptr(a.x[side].p) + (t0 + t) * a.x[side].ts + h * a.x[side].hs;
        gchar* out = gstore_ptr(a.out[side]) + ((t0 + t) * hs + h) * (int64_t)a.dim * ES;
        float x[NC][VEC], y[NC][VEC], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = lane + i * LPH;
          int lo, hi;
          rope_chunk<VEC>(a, c, lo, hi);
          if (c < chunks) {
            Pack<ES, VEC>::load(px + lo * ES, x[i]);
            Pack<ES, VEC>::load(px + hi * ES, y[i]);
          } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[i][k] = y[i][k] = 0.0f;
          }
#pragma unroll
          for (int k = 0; k < VEC; ++k) sum = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], sum));
        }
        const bool norm = a.w[0] != nullptr;
        const float r = norm ? 1.0f / sqrtf(head_sum<LPH>(sum) * inv + a.eps) : 1.0f;
        float gx[BWD ? NC : 1][VEC], gy[BWD ? NC : 1][VEC], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = lane + i * LPH;
          int lo, hi;
          const bool turns = rope_chunk<VEC>(a, c, lo, hi);
          if (c >= chunks) continue;
          float wx[VEC], wy[VEC];
          if (norm) {
            Pack<ES, VEC>::load(gload_ptr(a.w[side]) + lo * ES, wx);
            Pack<ES, VEC>::load(gload_ptr(a.w[side]) + hi * ES, wy);
          } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) wx[k] = wy[k] = 1.0f;
          }
          if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
              x[i][k] *= r * wx[k];
              y[i][k] *= r * wy[k];
            }
            if (turns) rope_turn<VEC>(a, cs + t * half, c, false, x[i], y[i]);
            Pack<ES, VEC>::store(out + lo * ES, x[i]);
            Pack<ES, VEC>::store(out + hi * ES, y[i]);
          } else {
            cgchar* pd = gload_ptr(a.dy[side].p) + (t0 + t) * a.dy[side].ts + h * a.dy[side].hs;
            Pack<ES, VEC>::load(pd + lo * ES, gx[i]);
            Pack<ES, VEC>::load(pd + hi * ES, gy[i]);
            if (turns) rope_turn<VEC>(a, cs + t * half, c, true, gx[i], gy[i]);
            if (norm) {
#pragma unroll
              for (int k = 0; k < VEC; ++k) {
                x[i][k] *= r;
                y[i][k] *= r;
                dwl[side][i * VEC + k] = fmaf(gx[i][k], x[i][k], dwl[side][i * VEC + k]);
                dwh[side][i * VEC + k] = fmaf(gy[i][k], y[i][k], dwh[side][i * VEC + k]);
                gx[i][k] *= wx[k];
                gy[i][k] *= wy[k];
                dot = fmaf(gx[i][k], x[i][k], fmaf(gy[i][k], y[i][k], dot));
              }
            }
          }
        }
        if constexpr (BWD) {
          if (norm) dot = head_sum<LPH>(dot) * inv;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int c = lane + i * LPH;
            int lo, hi;
            rope_chunk<VEC>(a, c, lo, hi);
            if (c >= chunks) continue;
            if (norm) {
#pragma unroll
              for (int k = 0; k < VEC; ++k) {
                gx[i][k] = r * (gx[i][k] - x[i][k] * dot);
                gy[i][k] = r * (gy[i][k] - y[i][k] * dot);
              }
            }
            Pack<ES, VEC>::store(out + lo * ES, gx[i]);
            Pack<ES, VEC>::store(out + hi * ES, gy[i]);
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    if (!a.w[0]) return;
    // the groups' sums are added in order: one part per workgroup
    __shared__ float part[2][kRopeThreads / 64][2 * kRopeHalf];
    const int wave = threadIdx.x >> 6, wl = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lane + i * LPH;
        int lo, hi;
        rope_chunk<VEC>(a, c, lo, hi);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          float u = dwl[s][i * VEC + k], v = dwh[s][i * VEC + k];
#pragma unroll
          for (int o = LPH; o < 64; o <<= 1) {
            u += __shfl_xor(u, o);
            v += __shfl_xor(v, o);
          }
          if (wl < LPH && c < chunks) {
            part[s][wave][lo + k] = u;
            part[s][wave][hi + k] = v;
          }
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += kRopeThreads) {
      const int s = i >= a.dim, j = i - s * a.dim;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kRopeThreads / 64; ++w) v += part[s][w][j];
      a.part[(int64_t)blockIdx.x * 2 * a.dim + i] = v;
    }
  }
  (void)heads;
}

// dw: the parts, added in order by 16 waves and their sums in order again
template <int ES>
__global__ void __launch_bounds__(1024) rope_join_kernel(const RopeArgs a) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane, n = 2 * a.dim;
  float s = 0.0f;
  if (i < n)
    for (int p = wave; p < a.parts; p += 16) s += a.part[(int64_t)p * n + i];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < n) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += red[k][lane];
    const int side = i >= a.dim;
    store_out(gstore_ptr(a.dw[side]), i - side * a.dim, s, ES == 4);
  }
}

template <int ES, int VEC, int LPH, int NC>
void rope_inst(const RopeArgs& a, bool bwd, hipStream_t st) {
  if (bwd)
    hipLaunchKernelGGL((rope_kernel<ES, VEC, LPH, NC, true>), dim3((unsigned)a.parts), dim3(kRopeThreads), 0, st, a);
  else
    hipLaunchKernelGGL((rope_kernel<ES, VEC, LPH, NC, false>), dim3((unsigned)a.parts), dim3(kRopeThreads), 0, st, a);
}
// The widest run of elements that both sides of the pairs, and the elements that
// do not turn, are whole runs of.
template <int ES>
void rope_any(const RopeArgs& a, bool bwd, hipStream_t st) {
  if (a.dim % 16 == 0 && a.rot % 16 == 0) {
    if (a.dim <= 64) rope_inst<ES, 8, 4, 1>(a, bwd, st);
    else if (a.dim <= 128) rope_inst<ES, 8, 8, 1>(a, bwd, st);
    else rope_inst<ES, 8, 16, 1>(a, bwd, st);
  } else if (a.dim % 8 == 0 && a.rot % 8 == 0) {
    rope_inst<ES, 4, 16, 2>(a, bwd, st);
  } else {
    rope_inst<ES, 1, 16, 8>(a, bwd, st);
  }
}

template <int ES>
__global__ void __launch_bounds__(256) gather_heads_kernel(const GatherArgs a) {
  const int q = blockIdx.y;
  const int64_t per = a.dim_in, n = a.tokens[q] * a.heads[q] * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int d = (int)(i - row * per);
    const int64_t t = row / a.heads[q];
    const int h = (int)(row - t * a.heads[q]);
    const float v = d < a.dim ? load_out(gload_ptr(a.src[q]), t * a.ts[q] + h * a.hs[q] + d, ES == 4) : 0.0f;
    store_out(gstore_ptr(a.dst[q]), i, v, ES == 4);
  }
}

}  // namespace

// a workgroup per step of tokens, up to four on a compute unit
int64_t rope_parts(int64_t tokens) { return std::min<int64_t>((tokens + kRopeTokens - 1) / kRopeTokens, 1024); }

hipError_t launch_rope(const RopeArgs& a, bool bwd, hipStream_t st) {
  if (a.parts > 0) {
    if (a.esize == 2) rope_any<2>(a, bwd, st);
    else rope_any<4>(a, bwd, st);
  }
  if (bwd && a.w[0]) {
    const dim3 grid((unsigned)((2 * a.dim + 63) / 64));
    if (a.esize == 2) hipLaunchKernelGGL(rope_join_kernel<2>, grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(rope_join_kernel<4>, grid, dim3(1024), 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_gather_heads(const GatherArgs& a, hipStream_t st) {
  if (a.n == 0) return hipSuccess;
  if (a.esize == 2) hipLaunchKernelGGL(gather_heads_kernel<2>, dim3(4096, a.n), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(gather_heads_kernel<4>, dim3(4096, a.n), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace dmuon
