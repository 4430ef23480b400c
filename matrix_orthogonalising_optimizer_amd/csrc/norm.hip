// Layer norm, forward and backward, with the weight's and bias's gradients.
//
//   mu = mean_j x_j,  r = 1 / sqrt(mean_j (x_j - mu)^2 + eps)
//   y = (x - mu) r w + b
//   g = dy w,  xh = (x - mu) r
//   dx = r (g - mean g - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// HBM bound: one pass over x (and dy) with the row held in registers; the
// variance is the mean of squares about the mean of those registers, so a
// large common offset costs no digits.  A row belongs to 16 or 32 lanes (width
// up to 128, 256), to one wave (1024) or to one workgroup; rows wider than 16384
// are read three times.  32768 x 4096 in bf16: forward 110 us (4.9 TB/s),
// backward 184 us (4.4 TB/s) and 7 us for the parts.
// The backward pass keeps each workgroup's sums of dw and db in registers
// over all its rows and writes one part per workgroup; a second launch adds
// the parts in a fixed order (no atomics: the same bits on every run).

#include <algorithm>

#include "linear_impl.h"

namespace dmuon {
namespace {

// Sum over the `tpr` threads of a row, in every one of them.
__device__ __forceinline__ float group_sum(float v, float* red, int tpr, int tid) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    if (o < tpr) v += __shfl_xor(v, o);
  if (tpr <= 64) return v;
  const int nw = tpr >> 6;
  __syncthreads();  // the previous sum has been read
  if ((tid & 63) == 0) red[tid >> 6] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < nw; ++i) v += red[i];
  return v;
}

// EPT elements per thread of a row shared by TPR threads, in groups of 8
// consecutive elements.  Rows may start at any element: global memory takes
// unaligned 16-byte accesses, and a wave's are whole lines but for the first
// and last.  EVEN: the width is a multiple of 8; otherwise the row's last
// group is taken element by element.
template <int ES, int TPR, int EPT, bool EVEN>
struct RowMap {
  __device__ static int col(int k, int t) { return ((k >> 3) * TPR + t) * 8 + (k & 7); }
  __device__ static void load(const void* base, int64_t off, int width, int t, float* v) {
    cgchar* p = gload_ptr(base) + off * ES;
#pragma unroll
    for (int c = 0; c < EPT / 8; ++c) {
      const int j = (c * TPR + t) * 8;
      if (j + 8 <= width) {
        unpack8<ES>((cgu4_any*)(p + (int64_t)j * ES), v + 8 * c);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * c + k] = !EVEN && j + k < width ? load_out(p, j + k, ES == 4) : 0.0f;
      }
    }
  }
  __device__ static void store(void* base, int64_t off, int width, int t, const float* v) {
    gchar* p = gstore_ptr(base) + off * ES;
#pragma unroll
    for (int c = 0; c < EPT / 8; ++c) {
      const int j = (c * TPR + t) * 8;
      if (j + 8 <= width) {
        u32x4 o[ES / 2];
        pack8<ES>(v + 8 * c, o);
#pragma unroll
        for (int k = 0; k < ES / 2; ++k) ((gu4_any*)(p + (int64_t)j * ES))[k] = o[k];
      } else if (!EVEN) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (j + k < width) store_out(p, j + k, v[8 * c + k], ES == 4);
      }
    }
  }
};

template <int ES, int TPR, int EPT, bool EVEN>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) layernorm_fwd_kernel(const NormFwdArgs a) {
  using R = RowMap<ES, TPR, EPT, EVEN>;
  constexpr int BS = TPR < 256 ? 256 : TPR;
  __shared__ float red[BS / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (BS / TPR) + threadIdx.x / TPR;
  if (row >= a.rows) return;  // whole rows, and whole workgroups when TPR > 64
  const int width = (int)a.width;
  float x[EPT];
  R::load(a.x, row * width, width, t, x);
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < EPT; ++k) s += x[k];
  const float mean = group_sum(s, red, TPR, threadIdx.x) / (float)width;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < EPT; ++k) {
    x[k] = R::col(k, t) < width ? x[k] - mean : 0.0f;
    s = fmaf(x[k], x[k], s);
  }
  const float rstd = 1.0f / sqrtf(group_sum(s, red, TPR, threadIdx.x) / (float)width + a.eps);
  float w[EPT];
  R::load(a.w, 0, width, t, w);
#pragma unroll
  for (int k = 0; k < EPT; ++k) x[k] = x[k] * rstd * w[k];
  if (a.b) {
    R::load(a.b, 0, width, t, w);
#pragma unroll
    for (int k = 0; k < EPT; ++k) x[k] += w[k];
  }
  R::store(a.y, row * width, width, t, x);
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

// rows wider than the register kernels: one workgroup per row, three reads
template <int ES>
__global__ void __launch_bounds__(512) layernorm_fwd_wide_kernel(const NormFwdArgs a) {
  __shared__ float red[8];
  const int64_t row = blockIdx.x, width = a.width;
  cgchar* x = gload_ptr(a.x) + row * width * ES;
  float s = 0.0f;
  for (int64_t j = threadIdx.x; j < width; j += 512) s += load_out(x, j, ES == 4);
  const float mean = group_sum(s, red, 512, threadIdx.x) / (float)width;
  s = 0.0f;
  for (int64_t j = threadIdx.x; j < width; j += 512) {
    const float d = load_out(x, j, ES == 4) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.0f / sqrtf(group_sum(s, red, 512, threadIdx.x) / (float)width + a.eps);
  gchar* y = gstore_ptr(a.y) + row * width * ES;
  for (int64_t j = threadIdx.x; j < width; j += 512) {
    const float v = (load_out(x, j, ES == 4) - mean) * rstd * load_out(gload_ptr(a.w), j, ES == 4);
    store_out(y, j, a.b ? v + load_out(gload_ptr(a.b), j, ES == 4) : v, ES == 4);
  }
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

// Groups of 8 of x and dy as loaded (packed: half the registers of fp32 for
// 16-bit types), so that the next row's loads fit beside the sums.
template <int ES, int TPR, int EPT, bool EVEN>
struct RawRow {
  u32x4 v[EPT / 8][ES / 2];
  __device__ void load(const void* base, int64_t off, int width, int t) {
    cgchar* p = gload_ptr(base) + off * ES;
#pragma unroll
    for (int c = 0; c < EPT / 8; ++c) {
      const int j = (c * TPR + t) * 8;
#pragma unroll
      for (int h = 0; h < ES / 2; ++h) {
        if (j + 8 <= width)
          v[c][h] = *((cgu4_any*)(p + (int64_t)j * ES) + h);
        else
          v[c][h] = EVEN ? u32x4{0u, 0u, 0u, 0u} : load_chunk_partial<ES>(p, j + 4 * h, width - j - 4 * h);
      }
    }
  }
  __device__ void get(int c, float* f) const { unpack8<ES>(v[c], f); }
};

template <int ES, int TPR, int EPT, bool EVEN>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) layernorm_bwd_kernel(const NormBwdArgs a) {
  using R = RowMap<ES, TPR, EPT, EVEN>;
  using Raw = RawRow<ES, TPR, EPT, EVEN>;
  constexpr int BS = TPR < 256 ? 256 : TPR, RPB = BS / TPR;
  // the next row's loads run under this row's sums where the registers last
  // (16 values a thread of 1024 threads: spilled, 292 -> 451 us at 8192 x 16384)
  constexpr bool AHEAD = TPR * EPT <= 8192;
  __shared__ float red[BS / 64];
  __shared__ float join[RPB > 1 ? 2 * TPR * EPT : 1];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int width = (int)a.width;
  const float inv = 1.0f / (float)width;
  Raw w, x, dy;
  float dw[EPT], db[EPT];
  w.load(a.w, 0, width, t);
#pragma unroll
  for (int k = 0; k < EPT; ++k) dw[k] = db[k] = 0.0f;
  const int64_t step = (int64_t)a.parts * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + grp;
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](Raw& x_, Raw& dy_, float& mean_, float& rstd_, int64_t r) __attribute__((always_inline)) {
    x_.load(a.x, r * width, width, t);
    dy_.load(a.dy, r * width, width, t);
    mean_ = a.mean[r];
    rstd_ = a.rstd[r];
  };
  if (AHEAD && row < a.rows) load(x, dy, mean, rstd, row);
  for (; row < a.rows; row += step) {
    Raw nx, ndy;
    float nmean = 0.0f, nrstd = 0.0f;
    if constexpr (!AHEAD) {
      load(x, dy, mean, rstd, row);
    } else if (row + step < a.rows) {
      load(nx, ndy, nmean, nrstd, row + step);
    } else {
      nx = x;
      ndy = dy;
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < EPT / 8; ++c) {
      float fx[8], fd[8], fw[8];
      x.get(c, fx);
      dy.get(c, fd);
      w.get(c, fw);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // (past the row's end dy and w are zero, which leaves no trace in the
        // sums as long as what they meet is finite: mean rstd may not be, so the
        // factor rstd of mean(g xh) comes after its sum)
        const float xc = fx[k] - mean;
        dw[8 * c + k] = fmaf(fd[k], xc * rstd, dw[8 * c + k]);
        db[8 * c + k] += fd[k];
        const float g = fd[k] * fw[k];
        s1 += g;
        s2 = fmaf(g, xc, s2);
      }
    }
    s1 = group_sum(s1, red, TPR, threadIdx.x) * inv;
    s2 = group_sum(s2, red, TPR, threadIdx.x) * inv * rstd;
    gchar* p = gstore_ptr(a.dx) + row * width * ES;
#pragma unroll
    for (int c = 0; c < EPT / 8; ++c) {
      float fx[8], fd[8], fw[8];
      x.get(c, fx);
      dy.get(c, fd);
      w.get(c, fw);
#pragma unroll
      for (int k = 0; k < 8; ++k) fx[k] = rstd * (fd[k] * fw[k] - s1 - (fx[k] - mean) * rstd * s2);
      const int j = (c * TPR + t) * 8;
      if (j + 8 <= width) {
        u32x4 o[ES / 2];
        pack8<ES>(fx, o);
#pragma unroll
        for (int h = 0; h < ES / 2; ++h) ((gu4_any*)(p + (int64_t)j * ES))[h] = o[h];
      } else if (!EVEN) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (j + k < width) store_out(p, j + k, fx[k], ES == 4);
      }
    }
    if constexpr (AHEAD) {
      x = nx;
      dy = ndy;
      mean = nmean;
      rstd = nrstd;
    }
  }
  // one part per workgroup: the groups' sums are added in order
  if constexpr (RPB > 1) {
    for (int q = 1; q < RPB; ++q) {
      __syncthreads();
      if (grp == q) {
#pragma unroll
        for (int k = 0; k < EPT; ++k) {
          join[k * TPR + t] = dw[k];
          join[(EPT + k) * TPR + t] = db[k];
        }
      }
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int k = 0; k < EPT; ++k) {
          dw[k] += join[k * TPR + t];
          db[k] += join[(EPT + k) * TPR + t];
        }
      }
    }
  }
  if (grp == 0) {
    float* p = a.part + (int64_t)blockIdx.x * 2 * width;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int j = R::col(k, t);
      if (j < width) {
        p[j] = dw[k];
        p[width + j] = db[k];
      }
    }
  }
}

// wide rows: dx by one workgroup per row, then parts of the column sums
template <int ES>
__global__ void __launch_bounds__(512) layernorm_dx_wide_kernel(const NormBwdArgs a) {
  __shared__ float red[8];
  const int64_t row = blockIdx.x, width = a.width;
  cgchar* x = gload_ptr(a.x) + row * width * ES;
  cgchar* dy = gload_ptr(a.dy) + row * width * ES;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t j = threadIdx.x; j < width; j += 512) {
    const float g = load_out(dy, j, ES == 4) * load_out(gload_ptr(a.w), j, ES == 4);
    s1 += g;
    s2 = fmaf(g, (load_out(x, j, ES == 4) - mean) * rstd, s2);
  }
  s1 = group_sum(s1, red, 512, threadIdx.x) / (float)width;
  s2 = group_sum(s2, red, 512, threadIdx.x) / (float)width;
  gchar* dx = gstore_ptr(a.dx) + row * width * ES;
  for (int64_t j = threadIdx.x; j < width; j += 512) {
    const float g = load_out(dy, j, ES == 4) * load_out(gload_ptr(a.w), j, ES == 4);
    const float xh = (load_out(x, j, ES == 4) - mean) * rstd;
    store_out(dx, j, rstd * (g - s1 - xh * s2), ES == 4);
  }
}
template <int ES>
__global__ void __launch_bounds__(256) layernorm_cols_wide_kernel(const NormBwdArgs a) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x, width = a.width;
  if (j >= width) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += a.parts) {
    const float dy = load_out(gload_ptr(a.dy), row * width + j, ES == 4);
    dw = fmaf(dy, (load_out(gload_ptr(a.x), row * width + j, ES == 4) - a.mean[row]) * a.rstd[row], dw);
    db += dy;
  }
  a.part[(int64_t)blockIdx.y * 2 * width + j] = dw;
  a.part[(int64_t)blockIdx.y * 2 * width + width + j] = db;
}

// dw (and db) from the parts: 64 columns per workgroup, 16 waves taking the
// parts in turn, eight loads in flight each, their sums joined in order
constexpr int kJoinWaves = 16;
template <int ES>
__global__ void __launch_bounds__(64 * kJoinWaves) layernorm_join_kernel(const NormBwdArgs a) {
  __shared__ float red[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t width = a.width, j = (int64_t)blockIdx.x * 64 + lane;
  const float* p = a.part + (blockIdx.y == 0 ? 0 : width) + (j < width ? j : width - 1);
  float s = 0.0f;
  int i = wave;
  for (; i + 7 * kJoinWaves < a.parts; i += 8 * kJoinWaves) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p[(int64_t)(i + k * kJoinWaves) * 2 * width];
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[k];
  }
  for (; i < a.parts; i += kJoinWaves) s += p[(int64_t)i * 2 * width];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < width) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinWaves; ++k) s += red[k][lane];
    store_out(gstore_ptr(blockIdx.y == 0 ? a.dw : a.db), j, s, ES == 4);
  }
}

constexpr int64_t kNormMaxReg = 16384;  // widest row held in registers
constexpr int64_t kNormParts = 1024;

// threads per row and elements per thread for a width
void norm_shape(int64_t width, bool bwd, int* tpr, int* ept) {
  if (width <= 128) *tpr = 16, *ept = 8;
  else if (width <= 256) *tpr = 32, *ept = 8;
  else if (width <= 512) *tpr = 64, *ept = 8;
  else if (width <= 1024) *tpr = 64, *ept = 16;
  else if (width <= 2048) *tpr = 256, *ept = 8;
  else if (width <= 4096) *tpr = 256, *ept = 16;
  else if (width <= 8192) *tpr = bwd ? 1024 : 512, *ept = bwd ? 8 : 16;  // (bwd at 512: 291 us, 1024: 198 us)
  else *tpr = 1024, *ept = 16;
}

// The forward pass of any number of rows: a launch takes less than 2^32 threads.
template <class F>
void row_launches(const NormFwdArgs& a, int64_t rows_per_group, F&& one) {
  const int64_t most = kLinMaxGroups * rows_per_group;
  for (int64_t r = 0; r < a.rows; r += most) {
    NormFwdArgs b = a;
    b.x = (const char*)a.x + r * a.width * a.esize;
    b.y = (char*)a.y + r * a.width * a.esize;
    b.mean = a.mean + r;
    b.rstd = a.rstd + r;
    b.rows = std::min(most, a.rows - r);
    one(b, dim3((unsigned)((b.rows + rows_per_group - 1) / rows_per_group)));
  }
}

template <int ES, int TPR, int EPT>
void fwd_inst(const NormFwdArgs& a, hipStream_t st) {
  constexpr int BS = TPR < 256 ? 256 : TPR;
  row_launches(a, BS / TPR, [&](const NormFwdArgs& b, dim3 grid) {
    if (a.width % 8 == 0)
      hipLaunchKernelGGL((layernorm_fwd_kernel<ES, TPR, EPT, true>), grid, dim3(BS), 0, st, b);
    else
      hipLaunchKernelGGL((layernorm_fwd_kernel<ES, TPR, EPT, false>), grid, dim3(BS), 0, st, b);
  });
}
template <int ES, int TPR, int EPT>
void bwd_inst(const NormBwdArgs& a, hipStream_t st) {
  constexpr int BS = TPR < 256 ? 256 : TPR;
  if (a.width % 8 == 0)
    hipLaunchKernelGGL((layernorm_bwd_kernel<ES, TPR, EPT, true>), dim3((unsigned)a.parts), dim3(BS), 0, st, a);
  else
    hipLaunchKernelGGL((layernorm_bwd_kernel<ES, TPR, EPT, false>), dim3((unsigned)a.parts), dim3(BS), 0, st, a);
}

template <int ES>
void fwd_any(const NormFwdArgs& a, hipStream_t st) {
  if (a.width > kNormMaxReg) {
    row_launches(a, 1, [&](const NormFwdArgs& b, dim3 grid) {
      hipLaunchKernelGGL(layernorm_fwd_wide_kernel<ES>, grid, dim3(512), 0, st, b);
    });
    return;
  }
  int tpr, ept;
  norm_shape(a.width, false, &tpr, &ept);
  if (tpr == 16) fwd_inst<ES, 16, 8>(a, st);
  else if (tpr == 32) fwd_inst<ES, 32, 8>(a, st);
  else if (tpr == 64 && ept == 8) fwd_inst<ES, 64, 8>(a, st);
  else if (tpr == 64) fwd_inst<ES, 64, 16>(a, st);
  else if (tpr == 256 && ept == 8) fwd_inst<ES, 256, 8>(a, st);
  else if (tpr == 256) fwd_inst<ES, 256, 16>(a, st);
  else if (tpr == 512) fwd_inst<ES, 512, 16>(a, st);
  else fwd_inst<ES, 1024, 16>(a, st);
}

template <int ES>
void bwd_any(const NormBwdArgs& a, hipStream_t st) {
  if (a.width > kNormMaxReg) {
    hipLaunchKernelGGL(layernorm_dx_wide_kernel<ES>, dim3((unsigned)a.rows), dim3(512), 0, st, a);
    hipLaunchKernelGGL(layernorm_cols_wide_kernel<ES>, dim3((unsigned)((a.width + 255) / 256), (unsigned)a.parts),
                       dim3(256), 0, st, a);
  } else {
    int tpr, ept;
    norm_shape(a.width, true, &tpr, &ept);
    if (tpr == 16) bwd_inst<ES, 16, 8>(a, st);
    else if (tpr == 32) bwd_inst<ES, 32, 8>(a, st);
    else if (tpr == 64 && ept == 8) bwd_inst<ES, 64, 8>(a, st);
    else if (tpr == 64) bwd_inst<ES, 64, 16>(a, st);
    else if (tpr == 256 && ept == 8) bwd_inst<ES, 256, 8>(a, st);
    else if (tpr == 256) bwd_inst<ES, 256, 16>(a, st);
    else if (ept == 8) bwd_inst<ES, 1024, 8>(a, st);
    else bwd_inst<ES, 1024, 16>(a, st);
  }
  hipLaunchKernelGGL(layernorm_join_kernel<ES>, dim3((unsigned)((a.width + 63) / 64), a.db ? 2u : 1u),
                     dim3(64 * kJoinWaves), 0, st, a);
}

}  // namespace

int64_t layernorm_parts(int64_t rows, int64_t width) {
  if (rows <= 0) return 0;
  if (width > kNormMaxReg) return rows < 64 ? rows : 64;
  int tpr, ept;
  norm_shape(width, true, &tpr, &ept);
  const int64_t rpb = tpr < 256 ? 256 / tpr : 1;
  const int64_t n = (rows + rpb - 1) / rpb;  // row groups
  // a workgroup per group up to one per compute unit, then eight groups each
  // until the GPU is full
  return n <= 256 ? n : std::min(std::max<int64_t>(n / 8, 256), kNormParts);
}

hipError_t launch_layernorm_fwd(const NormFwdArgs& a, hipStream_t st) {
  if (a.rows <= 0) return hipSuccess;
  if (a.esize == 2) fwd_any<2>(a, st);
  else fwd_any<4>(a, st);
  return hipGetLastError();
}

// rows = 0 leaves no part: the join writes zeros.  (The wide kernel's workgroup
// per row is a launch of 2^32 threads at 2^23 rows, 800 GB of x, dy and dx.)
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, hipStream_t st) {
  if (a.width > kNormMaxReg && a.rows >= 1 << 23) return hipErrorInvalidValue;
  if (a.rows <= 0) {
    const dim3 grid((unsigned)((a.width + 63) / 64), a.db ? 2u : 1u);
    if (a.esize == 2) hipLaunchKernelGGL(layernorm_join_kernel<2>, grid, dim3(64 * kJoinWaves), 0, st, a);
    else hipLaunchKernelGGL(layernorm_join_kernel<4>, grid, dim3(64 * kJoinWaves), 0, st, a);
    return hipGetLastError();
  }
  if (a.esize == 2) bwd_any<2>(a, st);
  else bwd_any<4>(a, st);
  return hipGetLastError();
}

}  // namespace dmuon
