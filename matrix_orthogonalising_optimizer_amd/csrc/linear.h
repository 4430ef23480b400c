// Launch interface of the training operators' product kernel (linear_*.hip)
// and of the passes around it (passes.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dmuon {

// C[m][n] = sum_k X(m, k) Y(n, k).  "K-major" operands store k contiguously
// (X[m ld + k]), "row-major" ones m or n contiguously (X[k ld + m]).
// Operands.  LIN_SPLIT: fp32 matrices as bf16 planes (launch_planes), three of
// whose sum is the fp32 value; the product takes the six largest of the nine
// products of planes and its results are fp32.
enum LinKind : int { LIN_BF16 = 0, LIN_F32 = 1, LIN_SPLIT = 2 };

enum LinMode : int {
  LIN_KK = 0,  // X and Y K-major: activations times a weight's rows
  LIN_KR = 1,  // X K-major, Y row-major: gradients times a weight's columns
  LIN_RR = 2,  // X and Y row-major: weight gradients (k counts tokens)
};

enum LinEpi : int {
  // C in the operands' type, times *alpha when given
  LIN_OUT = 0,
  // fp32 C (workspace); `accumulate` adds to what is there
  LIN_ACC = 1,
  // LIN_KK: Y rows of two matrices, gate (y) and up (y2), N rows each:
  // h = act(g) u into c; g into c2 and u into c3 when those are given, for
  // 16-bit operands cut to their upper halves, with four bits more of each in
  // a byte of c4 (g's in the lower half)
  LIN_GATE = 2,
  // LIN_KR: C is dh; with g = aux1, u = aux2 (and aux3 as c4): dg = dh u act'(g) into c and
  // du = dh act(g) into c2 (all with row pitch ldc)
  LIN_DGATE = 3,
  // LIN_KK: C holds logits (m tokens, n words).  Per token and piece of
  // words (half a tile wide): the maximum and the sum of exponentials
  // relative to it into stats, the target's logit into target_logit, and,
  // when c is given, those exponentials into c
  LIN_XENT = 4,
};

enum LinRole : int { LIN_WHOLE = 0, LIN_PART = 1, LIN_JOIN = 2 };

enum LinAct : int { LIN_SILU = 0, LIN_GELU = 1, LIN_GELU_TANH = 2 };

// Unless LinArgs::raw, every operand row starts 16-byte aligned (pointer and
// pitch) and holds zeros from its last element up to the next 16-byte boundary
// where the pitch reaches past it.
struct LinProb {
  const void* x;
  const void* y;
  const void* x2;  // second K segment (nseg 2) of X
  const void* y2;  // second K segment of Y, or LIN_GATE's up weights
  void* c;
  void* c2;
  void* c3;
  void* c4;
  const void* aux1;
  const void* aux2;
  const void* aux3;
  int64_t ldx, ldy, ldc;  // elements
  int64_t xplane, yplane;  // LIN_SPLIT: elements from plane to plane (K a multiple of 64)
  int64_t ld4;            // row pitch of c4 / aux3, a multiple of 16
  float* part;            // workspace of the split tiles: tile * tile floats for each and each split
  int32_t M, N, K;        // K of one segment
  int32_t npad;           // columns [N, npad) of c, c2 and c3 are written as zeros, to 16 bytes at least
  int32_t nseg;           // K segments: the product is X Y + X2 Y2 for 2
  // the last `split_tiles` tiles are computed in `splits` parts of the K range
  // each by a second launch, and put together by a third that runs their
  // epilogue
  int32_t split_tiles, splits;
  int32_t tiles_m, tiles_n;
  int16_t xflag, yflag;   // LIN_SPLIT: which of LinArgs::flags says that the fourth planes are in use
};

constexpr int kLinMaxProb = 3;
constexpr int kLinCu = 256;  // compute units
// most workgroups of one launch: its threads (up to 1024 each) have to be fewer
// than 2^32
constexpr int64_t kLinMaxGroups = 1 << 21;
struct LinArgs {
  LinProb p[kLinMaxProb];
  int32_t nprob;
  int32_t act;
  int32_t accumulate;
  int32_t role;                // LinRole of the launch
  int32_t slot0;               // its first workgroup of each XCD
  int32_t raw;                 // operand rows may start at any element (tiles up to 128)
  int32_t pieces;              // LIN_XENT: pieces per token
  const int32_t* flags;        // LIN_SPLIT
  const float* alpha;          // LIN_OUT, nullable
  const int64_t* targets;      // LIN_XENT
  float2* stats;               // LIN_XENT: [token][piece]
  float* target_logit;         // LIN_XENT
};

// Set tiles_m and tiles_n of every problem for block tile `tile` (64, 128,
// 256; LIN_F32: 64, 128; LIN_SPLIT: 256) and launch: the whole tiles, then the
// parts of the split ones and their join, as far as there are any.
hipError_t launch_linear(LinKind kind, int tile, LinMode mode, LinEpi epi, LinArgs& a, hipStream_t st);
hipError_t launch_linear_split_256(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st);
hipError_t launch_linear_bf16_256(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st);
hipError_t launch_linear_bf16_128(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st);
hipError_t launch_linear_bf16_64(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st);
hipError_t launch_linear_f32_128(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st);
hipError_t launch_linear_f32_64(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st);

// ---------------------------------------------------------------- passes.hip
// Copies of contiguous rows x cols matrices with row pitch ld (a multiple of
// 16 bytes), columns [cols, ld) zero.
constexpr int kPackMax = 5;
struct PackArgs {
  const void* src[kPackMax];
  void* dst[kPackMax];
  int64_t rows[kPackMax], cols[kPackMax], ld[kPackMax];
  int64_t blk0[kPackMax + 1];  // set by the launch
  int32_t n;
  int32_t esize;
};
hipError_t launch_pack_rows(PackArgs& a, hipStream_t st);

// fp32 rows x cols matrices (pitch src_ld) as kPlanes bf16 planes of
// round_up(rows, 64) x round_up(cols, 64) with zeros past rows and cols:
// v = p0 + p1 + p2 exactly, each the nearest bf16 to what is left (an infinity
// or NaN is p0 alone).  An infinity may meet the other operand's p0 only: its
// lower planes are zeros or of either sign, which would make NaN of it where
// fp32 keeps it.  A pass that meets one sets *flag (device, 0 before the call's
// first pass), and launch_finite_plane then fills a fourth plane, p0 without its
// infinities and NaN, that the product takes p0 from when the other plane is a
// lower one (always written and read it would cost 2 to 4%).
constexpr int kPlanes = 4;
struct SplitArgs {
  const float* src[kPackMax];
  uint16_t* dst[kPackMax];     // plane stride: rows and cols rounded up
  int64_t rows[kPackMax], cols[kPackMax], src_ld[kPackMax];
  int64_t blk0[kPackMax + 1];  // set by the launch
  int32_t n;
  int32_t* flag;
};
hipError_t launch_planes(SplitArgs& a, hipStream_t st);
struct FiniteArgs {
  uint16_t* planes[kPackMax];
  int64_t plane[kPackMax];     // elements of a plane, a multiple of 8
  int32_t n;
  const int32_t* flag;
};
hipError_t launch_finite_plane(const FiniteArgs& a, hipStream_t st);
hipError_t launch_clear_flags(int32_t* flags, int n, hipStream_t st);

// out = *alpha times an fp32 matrix (workspace, pitch ld, a multiple of 4),
// rounded to esize.
hipError_t launch_scale_round(const float* src, int64_t ld, void* out, int64_t rows, int64_t cols, int esize,
                              const float* alpha, hipStream_t st);

// Cross entropy around the logits' product.
struct XentArgs {
  const int64_t* targets;
  int64_t tokens;
  int64_t vocab;
  const float2* stats;       // [token][piece]
  int32_t pieces;
  int32_t piece;             // words per piece
  const float* target_logit;
  float* losses;             // [token]
  void* p;                   // [token][ldp]: exponentials in, softmax minus one-hot out; nullable
  int64_t ldp;
  int32_t esize;
  float scale;               // power of two that p's entries are multiplied by
  uint16_t* planes;          // given: the result goes here, as launch_planes lays it out
  int32_t* flag;             // and its flag
};
hipError_t launch_xent_rows(const XentArgs& a, hipStream_t st);
// With n = max(1, number of targets in [0, vocab)): alpha[0] = 1 / (n scale)
// and, given the losses, loss[0] = their sum / n.
hipError_t launch_xent_mean(const int64_t* targets, const float* losses, int64_t tokens, int64_t vocab, float scale,
                            float* alpha, float* loss, hipStream_t st);

// ---------------------------------------------------------------- norm.hip
struct NormFwdArgs {
  const void* x;
  const void* w;
  const void* b;   // nullable
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, width;
  float eps;
  int32_t esize;
};
hipError_t launch_layernorm_fwd(const NormFwdArgs& a, hipStream_t st);
struct NormBwdArgs {
  const void* dy;
  const void* x;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dw;
  void* db;        // nullable
  float* part;     // workspace, layernorm_parts(rows, width) * 2 * width floats
  int64_t rows, width;
  int32_t parts;   // layernorm_parts(rows, width)
  int32_t esize;
};
int64_t layernorm_parts(int64_t rows, int64_t width);
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, hipStream_t st);

}  // namespace dmuon
