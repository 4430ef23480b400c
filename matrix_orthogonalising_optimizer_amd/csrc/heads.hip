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
// on in fp32.  Only the results are rounded to the caller's type.
// 16384 tokens of 32 and 8 heads of 128, bf16: forward 67 us (5.0 TB/s), backward 124 + 6 us
// (4.1 TB/s: dw's sums and more registers in the way); 4999 tokens of 12 and 12 of 80, fp32: 23 and
// 31 us, whose bytes stay in the last-level cache.

#include <algorithm>

#include "heads.h"
#include "linear_impl.h"

namespace dmuon {
namespace {

constexpr int kRopeThreads = 256;
// N elements from any element's address, as fp32, and back (N times ES a power of two)
template <int ES, int N>
struct Pack {
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

// LPH lanes per head, NC chunk pairs each.  A workgroup has heads of one side, q or k
// (both sides' sums of dw would cost the backward pass an eighth of its waves), and takes
// a.step tokens at a time; x and dy of a head are on their way together.
template <int ES, int VEC, int LPH, int NC, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, NC * VEC > 8 ? 2 : 4) rope_kernel(const RopeArgs a) {
  constexpr int GROUPS = kRopeThreads / LPH;
  __shared__ float2 cs[kRopeTokens * kRopeHalf];
  const int lane = threadIdx.x % LPH, grp = threadIdx.x / LPH;
  const int half = a.rot >> 1, chunks = a.dim / (2 * VEC);
  const int side = (int)blockIdx.x >= a.parts[0], first = (int)blockIdx.x - (side ? a.parts[0] : 0);
  const int hs = a.heads[side], step = a.step[side];
  const float inv = 1.0f / (float)a.dim;
  const bool norm = a.w[0] != nullptr;
  float dwl[NC * VEC], dwh[NC * VEC];
#pragma unroll
  for (int k = 0; k < NC * VEC; ++k) dwl[k] = dwh[k] = 0.0f;
  for (int64_t t0 = (int64_t)first * step; t0 < a.tokens; t0 += (int64_t)a.parts[side] * step) {
    const int n = (int)min((int64_t)step, a.tokens - t0);
    __syncthreads();
    fill_turns(a, t0, n, cs);
    __syncthreads();
    for (int item = grp; item < n * hs; item += GROUPS) {
      const int t = item / hs, h = item - t * hs;
      cgchar* px = gload_ptr(a.x[side].p) + (t0 + t) * a.x[side].ts + h * a.x[side].hs;
      cgchar* pd = BWD ? gload_ptr(a.dy[side].p) + (t0 + t) * a.dy[side].ts + h * a.dy[side].hs : nullptr;
      gchar* out = gstore_ptr(a.out[side]) + ((t0 + t) * hs + h) * (int64_t)a.dim * ES;
      float x[NC][VEC], y[NC][VEC], gx[BWD ? NC : 1][VEC], gy[BWD ? NC : 1][VEC], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lane + i * LPH;
        int lo, hi;
        rope_chunk<VEC>(a, c, lo, hi);
        if (c < chunks) {
          Pack<ES, VEC>::load(px + lo * ES, x[i]);
          Pack<ES, VEC>::load(px + hi * ES, y[i]);
          if constexpr (BWD) {
            Pack<ES, VEC>::load(pd + lo * ES, gx[i]);
            Pack<ES, VEC>::load(pd + hi * ES, gy[i]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            x[i][k] = y[i][k] = 0.0f;
            if constexpr (BWD) gx[i][k] = gy[i][k] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], sum));
      float r = 1.0f, up = 1.0f;
      if (norm) {
        float ms = head_sum<LPH>(sum) * inv, eps = a.eps;
        // squares past fp32's range, or all of them below it: of x times a power of two
        if (!(ms < __builtin_inff()) || ms + eps < 0x1p-90f) {
          up = ms < 1.0f ? 0x1p100f : 0x1p-70f;
          sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
              x[i][k] *= up;
              y[i][k] *= up;
              sum = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], sum));
            }
          ms = head_sum<LPH>(sum) * inv;
          eps = eps * up * up;
        }
        r = 1.0f / sqrtf(ms + eps);
      }
      float dot = 0.0f;
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
          if (turns) rope_turn<VEC>(a, cs + t * half, c, true, gx[i], gy[i]);
          if (norm) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
              x[i][k] *= r;
              y[i][k] *= r;
              dwl[i * VEC + k] = fmaf(gx[i][k], x[i][k], dwl[i * VEC + k]);
              dwh[i * VEC + k] = fmaf(gy[i][k], y[i][k], dwh[i * VEC + k]);
              gx[i][k] *= wx[k];
              gy[i][k] *= wy[k];
              dot = fmaf(gx[i][k], x[i][k], fmaf(gy[i][k], y[i][k], dot));
            }
          }
        }
      }
      if constexpr (BWD) {
        if (norm) dot = head_sum<LPH>(dot) * inv;
        r *= up;
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
  if constexpr (BWD) {
    if (!norm) return;
    // the groups' sums are added in order: one part per workgroup
    __shared__ float part[kRopeThreads / 64][2 * kRopeHalf];
    const int wave = threadIdx.x >> 6, wl = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + i * LPH;
      int lo, hi;
      rope_chunk<VEC>(a, c, lo, hi);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float u = dwl[i * VEC + k], v = dwh[i * VEC + k];
#pragma unroll
        for (int o = LPH; o < 64; o <<= 1) {
          u += __shfl_xor(u, o);
          v += __shfl_xor(v, o);
        }
        if (wl < LPH && c < chunks) {
          part[wave][lo + k] = u;
          part[wave][hi + k] = v;
        }
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.dim; j += kRopeThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kRopeThreads / 64; ++w) v += part[w][j];
      a.part[(int64_t)blockIdx.x * a.dim + j] = v;
    }
  }
}

// dw: the parts, added in order by 16 waves and their sums in order again
template <int ES>
__global__ void __launch_bounds__(1024) rope_join_kernel(const RopeArgs a) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int side = blockIdx.y, i = blockIdx.x * 64 + lane, n = a.dim;
  const int from = side ? a.parts[0] : 0;
  float s = 0.0f;
  if (i < n) {
    const float* part = a.part + (int64_t)from * n + i;
    int p = wave;
    for (; p + 15 * 16 < a.parts[side]; p += 16 * 16) {  // sixteen loads at a time
      float v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = part[(int64_t)(p + 16 * k) * n];
#pragma unroll
      for (int k = 0; k < 16; ++k) s += v[k];
    }
    for (; p < a.parts[side]; p += 16) s += part[(int64_t)p * n];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < n) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += red[k][lane];
    store_out(gstore_ptr(a.dw[side]), i, s, ES == 4);
  }
}

template <int ES, int VEC, int LPH, int NC>
void rope_inst(const RopeArgs& a, bool bwd, hipStream_t st) {
  const dim3 grid((unsigned)(a.parts[0] + a.parts[1]));
  if (bwd) hipLaunchKernelGGL((rope_kernel<ES, VEC, LPH, NC, true>), grid, dim3(kRopeThreads), 0, st, a);
  else hipLaunchKernelGGL((rope_kernel<ES, VEC, LPH, NC, false>), grid, dim3(kRopeThreads), 0, st, a);
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

// Forward: a workgroup per step of 128 heads or more (4 rounds of the widest
// groups).  Backward: as many workgroups as run at once, each of which leaves one part
// of dw, divided as the sides' heads are, and steps half as long, which come out
// more even.
void rope_cut(RopeArgs& a, bool bwd) {
  const int64_t all = a.heads[0] + a.heads[1], most = bwd ? 1024 : (int64_t)1 << 20;
  for (int s = 0; s < 2; ++s) {
    const int64_t h = a.heads[s];
    a.step[s] = 1;
    a.parts[s] = 0;
    if (h == 0) continue;
    a.step[s] = (int32_t)std::min<int64_t>(kRopeTokens, std::max<int64_t>(1, (bwd ? 64 : 128) / h));
    a.parts[s] = (int32_t)std::min((a.tokens + a.step[s] - 1) / a.step[s], std::max<int64_t>(1, most * h / all));
  }
}

hipError_t launch_rope(const RopeArgs& a, bool bwd, hipStream_t st) {
  if (a.parts[0] + a.parts[1] > 0) {
    if (a.esize == 2) rope_any<2>(a, bwd, st);
    else rope_any<4>(a, bwd, st);
  }
  if (bwd && a.w[0]) {
    const dim3 grid((unsigned)((a.dim + 63) / 64), 2);
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
