// Product kernel of the training operators (gated feed-forward, linear cross
// entropy) for gfx950 MFMA:  C[m][n] = sum_k X(m, k) Y(n, k).
//
// Tile BT x BT, 256 threads = 2 x 2 waves, wave tile (BT/2) x (BT/2) of
// 32 x 32 MFMA blocks.  Y is the MFMA's A operand and X its B operand, so a
// lane's accumulators are consecutive n of one m: a row reduction over n (the
// softmax's) is in-lane but for one exchange, and the tile is staged in LDS as
// rows of C with 8-byte (16-bit types) writes.
//
// The K loop is a ring of operand stages: direct global-to-LDS loads, one
// barrier per 128 bytes of K, fragment reads of the next sub-step and the
// loads of later steps issued between MFMAs.  Tiles of 256 hold five stages
// (all of LDS; a step is 1.5 us, longer than HBM's latency).  Smaller tiles'
// steps are shorter than that: a compute unit hides the latency with nine
// stages of one workgroup, or with five of several workgroups side by side
// (launch_lin_inst).  A K-major operand's stage is BT rows of 128 bytes; a
// row-major operand's stage is the K rows of a step, BT columns each, read
// transposed (ds_read_b64_tr_b16; 32-bit types need no
// transposition, an MFMA takes one value per lane).  Rows and columns past M
// and N are clamped (their results are not stored).  What is left of K after
// the last whole step runs once behind the ring, with chunks past K taken
// from a chunk of zeros: both operands are zero there, so nothing that lies
// behind a row's end, NaN included, reaches a sum.
#pragma once

#include "gemm_impl.h"
#include "linear.h"
#include "raw_rows.h"

namespace dmuon {
namespace {

__device__ u32x4 lin_zero_chunk;  // zero-initialised, never written

typedef float f32x4 __attribute__((ext_vector_type(4)));

// 1 / x to 1 ulp in one instruction (a correctly rounded quotient costs ten,
// and the epilogues are bound by their arithmetic)
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// act(g) and act'(g) in fp32.
template <int ACT>
__device__ __forceinline__ void act_both(float g, float& a, float& da) {
  if constexpr (ACT == LIN_SILU) {
    const float s = fast_rcp(1.0f + __expf(-g));
    a = g * s;
    da = s * fmaf(g, 1.0f - s, 1.0f);
  } else if constexpr (ACT == LIN_GELU) {
    // Phi(-|g|) = exp(-g^2 / 2) t P(t), t = 1 / (1 + 0.305 |g|): P of degree 7 is
    // a fit of least relative error (1e-7 up to |g| = 14.5, 4e-7 with fp32
    // arithmetic), so that small values far out keep their digits but for the
    // exponential's, g^2 2^-24.  The exponential is the derivative's too.
    const float e = __expf(-0.5f * g * g);
    const float t = fast_rcp(fmaf(0.305f, fabsf(g), 1.0f));
    float poly = fmaf(t, 0.03663886711f, -0.1527460963f);
    poly = fmaf(t, poly, 0.1853149384f);
    poly = fmaf(t, poly, -0.03762069717f);
    poly = fmaf(t, poly, 0.1208404079f);
    poly = fmaf(t, poly, 0.1034736931f);
    poly = fmaf(t, poly, 0.1224586815f);
    poly = fmaf(t, poly, 0.1216402426f);
    const float q = t * poly * e;
    const float p = g < 0.0f ? q : 1.0f - q;
    a = g * p;
    da = fmaf(g * 0.39894228040143268f, e, p);
  } else {
    // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)) and (1 - tanh^2 z) / 4, the product
    // of that and its complement, by exp(-2 |z|): no cancellation, no overflow
    const float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float z = c * fmaf(0.044715f * g, g * g, g);
    const float e = __expf(-fabsf(z)), r = fast_rcp(1.0f + e), q = e * r;
    const float p = z < 0.0f ? q : r;
    a = g * p;
    // q is 0 from |g| = 32 on, and has to stay it when g^2 is infinite
    const float h = fminf(fabsf(g), 32.0f);
    da = fmaf(g * (r * q), c * fmaf(0.134145f * h, h, 1.0f), p);
  }
}
template <int ACT>
__device__ __forceinline__ float act_only(float g) {
  float a, da;
  act_both<ACT>(g, a, da);
  return a;
}

// f(0), f(1), .. f(N - 1), the index a compile-time constant
template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// 8 consecutive elements of `ESZ` bytes from 16-byte aligned memory, as fp32.
template <int ESZ, class P>
__device__ __forceinline__ void unpack8(P p, float* v) {
  if constexpr (ESZ == 2) {
    const u32x4 w = p[0];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    const u32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = __uint_as_float(lo[k]);
      v[k + 4] = __uint_as_float(hi[k]);
    }
  }
}
// 8 fp32 values to `ESZ`-byte elements (nearest even), ESZ / 2 chunks.
template <int ESZ>
__device__ __forceinline__ void pack8(const float* v, u32x4* o) {
  if constexpr (ESZ == 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[0][k] = pack_bf16(v[2 * k], v[2 * k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[0][k] = __float_as_uint(v[k]);
      o[1][k] = __float_as_uint(v[k + 4]);
    }
  }
}

// The block's backward pass needs g and u to better than the rounding of the
// products' operands: with g and u rounded to bf16 the errors of dx, dWg and
// dWu are 1.3 times those that the rounding of dg, du and the result alone
// make.  They are saved with 12 significant bits: bf16's upper half of the
// fp32 word and the next four bits, two values' in a byte.
// To nearest even; the low 12 bits are zero.  A NaN stays one: those of sums of
// bf16 products carry nothing in the bits whose carry could run past the top.
__device__ __forceinline__ uint32_t round12(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u + 0x7ffu + ((u >> 12) & 1u)) & 0xfffff000u;
}
// f, unknown to the compiler: it would otherwise keep what an earlier pass over
// the accumulators computed from them, which spills
__device__ __forceinline__ float opaque(float f) {
  asm("" : "+v"(f));
  return f;
}
__device__ __forceinline__ uint32_t low4(uint32_t g, uint32_t u) { return ((g >> 12) & 15u) | ((u >> 8) & 0xf0u); }
// value of the upper half `hi16` (in place, bits 16 .. 31) and its four bits
__device__ __forceinline__ float join12(uint32_t hi16, uint32_t nibble) {
  return __uint_as_float((hi16 & 0xffff0000u) | (nibble << 12));
}

typedef __attribute__((address_space(1))) u32x4 gu4;
typedef const __attribute__((address_space(1))) u32x4 cgu4;
// 16 bytes at any element's address: global memory takes unaligned accesses
// (a wave's are still whole lines but for the first and last)
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef __attribute__((address_space(1))) u32x4_any gu4_any;
typedef const __attribute__((address_space(1))) u32x4_any cgu4_any;

// SAVE: LIN_GATE writes g and u too.
// ACT: the activation of the gate's epilogues (a run-time choice would put
// three of them, unrolled over the accumulators, past the instruction cache).
// ROLE: whole tiles (K loop and epilogue), parts of split tiles (K loop, the
// accumulators to workspace) or their join (the parts added, epilogue).  They
// are kernels of their own: with more than one way out of the K loop its 256
// accumulators are copied and spilled.  A part has no epilogue (of EPI only
// LIN_GATE's operand rows matter to it), a join no K loop.
// O: type of the results.  float with bf16 operands: LIN_SPLIT, whose K loop
// runs six steps for each 64 of K, one for each pair of planes kept.
// RAW: operand rows may start at any element (not LIN_RR).  The loads then pass through
// registers (direct loads to LDS want 16-byte aligned addresses), several steps
// ahead, on their way to two steps of LDS.
// D: steps that X is fetched ahead (the ring's depth).
template <class E, class O, int BT, int MODE, int EPI, int ACT, int ROLE, bool SAVE, bool RAW, int D>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, BT >= 256 ? 1 : 4)))
linear_kernel(const LinArgs g) {
  constexpr int ES = Elt<E>::kSize, OES = Elt<O>::kSize;
  constexpr bool SPLIT = ES != OES;
  constexpr int PAIRS = SPLIT ? 6 : 1;     // steps per 128 bytes of K
  constexpr int VEC = 16 / ES;
  constexpr int KS = 128 / ES;             // K per step
  constexpr int WT = BT / 2;               // wave tile side
  constexpr int MT = WT / 32;              // 32-blocks per wave tile side
  constexpr bool TY = MODE != LIN_KK;      // Y row-major
  constexpr bool TX = MODE == LIN_RR;      // X row-major
  constexpr int OB = BT * 128;             // bytes of an operand stage
  constexpr int NOB = 2 * D + 1;           // operand stages
  constexpr int LPO = BT / 32;             // load instructions per wave and stage
  constexpr int TCH = BT / VEC;            // 16-byte chunks of a row-major stage's row
  constexpr int TR = 64 / TCH;             // its rows per load instruction
  constexpr int NT_ = (EPI == LIN_GATE) ? BT / 2 : BT;  // output columns per tile
  constexpr bool OUT32 = OES == 4 || EPI == LIN_ACC || EPI == LIN_DGATE;  // staged as fp32
  constexpr int OS = OUT32 ? 4 : 2;
  constexpr int PITCH = NT_ * OS + 16;
  constexpr int STAGED = (EPI == LIN_GATE ? 2 : 1) * BT * PITCH;
  constexpr int PASSES = STAGED > NOB * OB ? 2 : 1;
  static_assert(STAGED / PASSES <= NOB * OB, "epilogue staging");
  __shared__ __attribute__((aligned(16))) char smem[NOB * OB];

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wm = wave & 1;
  const int half = lane >> 5, lcol = lane & 31;

  // XCD-aware order: workgroups go round-robin over the 8 XCDs; each XCD takes
  // a contiguous range of every problem's tiles, so that the operand panels
  // its tiles share stay in its L2
  const int xcd = blockIdx.x & 7, slot = g.slot0 + (int)(blockIdx.x >> 3);
  int pi = -1, tile = 0, sp = 0, splits = 1;
  for (int q = 0, acc_ = 0; q < g.nprob; ++q) {
    const int st = g.p[q].split_tiles, whole = g.p[q].tiles_m * g.p[q].tiles_n - st;
    const int k = ROLE == LIN_PART ? g.p[q].splits : 1;
    const int n = ROLE == LIN_WHOLE ? whole : st * k;
    const int lo = (int)(((int64_t)n * xcd) >> 3), hi = (int)(((int64_t)n * (xcd + 1)) >> 3);
    if (slot < acc_ + (hi - lo)) {
      const int rel = lo + (slot - acc_);
      pi = q;
      tile = (ROLE == LIN_WHOLE ? 0 : whole) + rel / k;
      sp = rel % k;
      splits = k;
      break;
    }
    acc_ += hi - lo;
  }
  if (pi < 0) return;
  const LinProb& P = g.p[pi];
  int ti, tj;
  full_tile_blocked(tile, P.tiles_m, P.tiles_n, ti, tj);
  ti = __builtin_amdgcn_readfirstlane(ti);
  tj = __builtin_amdgcn_readfirstlane(tj);
  const int m0 = ti * BT, n0 = tj * NT_;
  const int M = P.M, N = P.N, K = P.K;

  // whole K steps of one segment, of all segments, and of this split
  const int ns1 = K / KS, nseg = (MODE == LIN_KR) ? P.nseg : 1;
  const int nst = ns1 * nseg * PAIRS;
  const int s0 = (int)((int64_t)nst * sp / splits), s1 = (int)((int64_t)nst * (sp + 1) / splits);
  const int ns = s1 - s0;

  // Tile bases (row 0 / column 0 of the tile at k = 0) and per-lane byte
  // offsets from them of this wave's load instructions.  K-major: instruction
  // i fills rows blk * 8 .. + 7 (blk = wave LPO + i), lane l the physical chunk
  // l % 8 of row blk * 8 + l / 8.  Row-major: stage rows blk TR .. + TR - 1,
  // lane l the physical chunk l % TCH of row blk TR + l / TCH.
  const uint32_t ldyb = (uint32_t)(P.ldy * ES), ldxb = (uint32_t)(P.ldx * ES);
  const uint64_t ybase = (uint64_t)(uintptr_t)P.y + (TY ? (uint64_t)n0 * ES : (uint64_t)n0 * (uint64_t)(P.ldy * ES));
  const uint64_t ybase2 = (uint64_t)(uintptr_t)P.y2 + (TY ? (uint64_t)n0 * ES : (uint64_t)n0 * (uint64_t)(P.ldy * ES));
  const uint64_t xbase = (uint64_t)(uintptr_t)P.x + (TX ? (uint64_t)m0 * ES : (uint64_t)m0 * (uint64_t)(P.ldx * ES));
  const uint64_t xbase2 = (uint64_t)(uintptr_t)P.x2 + (TX ? (uint64_t)m0 * ES : (uint64_t)m0 * (uint64_t)(P.ldx * ES));
  // the chunk swizzle of a row-major 16-bit stage spreads the four K rows of a
  // transposing read over the banks
  auto tr_swz = [](int k) { return ES == 4 ? 0 : (BT >= 128 ? (k & 3) << 2 : (k & 3) << 1); };
  uint32_t yoff[LPO], xoff[LPO];
#pragma unroll
  for (int i = 0; i < LPO; ++i) {
    const int blk = wave * LPO + i;
    const int r = blk * 8 + (lane >> 3), ch = (lane & 7) ^ lds_swz(r);
    const int rt = blk * TR + lane / TCH, ct = (lane % TCH) ^ tr_swz(rt);
    if constexpr (TY) {
      yoff[i] = (uint32_t)rt * ldyb + (uint32_t)(min(ct, (N - 1 - n0) / VEC) * 16);
    } else {
      // gate: the wave tile's first half holds gate rows, the second the same
      // rows of the up matrix
      const int rl = (EPI == LIN_GATE) ? (r / WT) * (WT / 2) + r % (WT / 2) : r;
      yoff[i] = (uint32_t)min(rl, N - 1 - n0) * ldyb + (uint32_t)(ch * 16);
    }
    if constexpr (TX)
      xoff[i] = (uint32_t)rt * ldxb + (uint32_t)(min(ct, (M - 1 - m0) / VEC) * 16);
    else
      xoff[i] = (uint32_t)min(r, M - 1 - m0) * ldxb + (uint32_t)(ch * 16);
  }
  // planes of step pair 0 .. 5, two bits each, the small products first:
  // (x, y) = (2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0); beside a lower plane
  // an operand with infinities or NaN takes 3, which is 0 without them
  uint32_t pair_x = 2u | 0u << 2 | 1u << 4 | 1u << 6 | 0u << 8 | 0u << 10;
  uint32_t pair_y = 0u | 2u << 2 | 1u << 4 | 0u << 6 | 1u << 8 | 0u << 10;
  if constexpr (SPLIT) {
    if (g.flags[P.xflag]) pair_x |= 3u << 2 | 3u << 8;
    if (g.flags[P.yflag]) pair_y |= 3u | 3u << 6;
    pair_x = __builtin_amdgcn_readfirstlane(pair_x);
    pair_y = __builtin_amdgcn_readfirstlane(pair_y);
  }
  const uint64_t xplane = SPLIT ? (uint64_t)P.xplane * ES : 0, yplane = SPLIT ? (uint64_t)P.yplane * ES : 0;
  // base of instruction i for K step st (over all segments)
  auto y_src = [&](int st, int i) -> uint64_t {
    uint64_t b = ybase;
    if constexpr (SPLIT) {
      const int c = st / PAIRS, pr = st - c * PAIRS;
      b += (uint64_t)((pair_y >> (2 * pr)) & 3u) * yplane;
      if constexpr (EPI == LIN_GATE) b += ((wave * LPO + i) * 8) % WT >= WT / 2 ? ybase2 - ybase : 0;
      st = c;
    } else if constexpr (EPI == LIN_GATE) {
      if (((wave * LPO + i) * 8) % WT >= WT / 2) b = ybase2;
    }
    if constexpr (MODE == LIN_KR) {
      if (st >= ns1) {
        b += ybase2 - ybase;
        st -= ns1;
      }
    }
    return b + (TY ? (uint64_t)st * KS * ldyb : (uint64_t)st * 128);
  };
  auto x_src = [&](int st) -> uint64_t {
    uint64_t b = xbase;
    if constexpr (SPLIT) {
      const int c = st / PAIRS, pr = st - c * PAIRS;
      b += (uint64_t)((pair_x >> (2 * pr)) & 3u) * xplane;
      st = c;
    }
    if constexpr (MODE == LIN_KR) {
      if (st >= ns1) {
        b += xbase2 - xbase;
        st -= ns1;
      }
    }
    return b + (TX ? (uint64_t)st * KS * ldxb : (uint64_t)st * 128);
  };
  auto lds_addr = [&](int buf, int i) -> uint32_t {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)(smem + buf * OB + (wave * LPO + i) * 1024);
  };
  // stages past this split's last step re-read it into buffers nobody reads
  auto load_y = [&](int j, int buf, int i) {
    ring_load(y_src(s0 + (j < ns ? j : ns - 1), i), yoff[i], lds_addr(buf, i));
  };
  auto load_x = [&](int j, int buf, int i) {
    ring_load(x_src(s0 + (j < ns ? j : ns - 1)), xoff[i], lds_addr(buf, i));
  };

  f32x16 acc[MT][MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // ------------------------------------------------------------ fragments
  u32x4 fy[2][MT], fx[2][MT];
  constexpr int NP = MT < 2 ? MT : 2;
  uint32_t yo[TY ? MT : 4 * NP], xo[TX ? MT : 4 * NP];
  auto tr_off = [&](int row0) -> uint32_t {
    if constexpr (ES == 4) {
      return (uint32_t)((4 * half) * (4 * BT) + (row0 + lcol) * 4);
    } else {
      // lane 4 q + x of each group of 16 supplies K row k0 + q, four columns
      // from 4 x, and receives column j = its place in the group, four K rows
      const int grp = lane >> 4, lq = lane & 15;
      const int k0 = 8 * (grp >> 1) + (lq >> 2);
      const int col = row0 + 16 * (grp & 1) + 4 * (lq & 3);
      const int c = (col >> 3) ^ tr_swz(k0);
      return (uint32_t)(k0 * (2 * BT) + c * 16 + (col & 7) * 2);
    }
  };
  auto rd_t = [&](const char* p) -> u32x4 {
    if constexpr (ES == 4) {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * 4 * BT);
      return v;
    } else {
      typedef __attribute__((address_space(3))) v4i16 lds4;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)const_cast<char*>(p)));
      const u32x2 hi =
          __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)const_cast<char*>(p + 8 * BT)));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  };
  if constexpr (TY) {
#pragma unroll
    for (int r = 0; r < MT; ++r) yo[r] = tr_off(wn * WT + r * 32);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int p = 0; p < NP; ++p) yo[s * NP + p] = (uint32_t)lds_off(wn * WT + lcol + 32 * p, 2 * s + half);
  }
  if constexpr (TX) {
#pragma unroll
    for (int r = 0; r < MT; ++r) xo[r] = tr_off(wm * WT + r * 32);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int p = 0; p < NP; ++p) xo[s * NP + p] = (uint32_t)lds_off(wm * WT + lcol + 32 * p, 2 * s + half);
  }
  // fragment r of sub-step `sub` (Y's fragments first); 64 rows on (fragment
  // r + 2) the row swizzle repeats
  constexpr int TSUB = (KS / 4) * BT * ES;  // K rows of a sub-step in a row-major stage
  auto rd = [&](int set, int bufY, int bufX, int sub, int r) {
    if (r < MT) {
      const char* s = smem + bufY * OB;
      if constexpr (TY)
        fy[set][r] = rd_t(s + yo[r] + sub * TSUB);
      else
        fy[set][r] = *reinterpret_cast<const u32x4*>(s + yo[sub * NP + r % NP] + (r / NP) * (64 * 128));
    } else {
      const int q = r - MT;
      const char* s = smem + bufX * OB;
      if constexpr (TX)
        fx[set][q] = rd_t(s + xo[q] + sub * TSUB);
      else
        fx[set][q] = *reinterpret_cast<const u32x4*>(s + xo[sub * NP + q % NP] + (q / NP) * (64 * 128));
    }
  };

  // ------------------------------------------------------------ K loop
  // Step j reads Y_j and X_j from buffers (2j) % NOB and (2j + 1) % NOB, NOB =
  // 2 D + 1.  After its barrier (every wave has read all of step j) those two
  // buffers take X_{j+D} and Y_{j+D+1} ("round j").
  constexpr int LQ3 = LPO, LQ0 = (LPO + 2) / 3, LQ1 = (LPO + 1) / 3, LQ2 = LPO / 3;
  auto load_round = [&](int R, int bufY_R, int bufX_R, int q) {
    if (q < LPO)
      load_x(R + D, bufY_R, q);
    else
      load_y(R + D + 1, bufX_R, q - LPO);
  };
  auto phase = [&](auto s_t, int rY, int rX, int rsub, int R, int lY, int lX) {
    constexpr int SS = decltype(s_t)::value;
    constexpr int SET = SS & 1, NM = MT * MT, NR = 2 * MT, NI = NM < NR ? NM : NR;
    constexpr int LQ = SS == 3 ? LQ3 : SS == 0 ? LQ0 : SS == 1 ? LQ1 : LQ2;
    constexpr int lq0 = SS == 3 ? 0 : SS == 0 ? LPO : SS == 1 ? LPO + LQ0 : LPO + LQ0 + LQ1;
    constexpr int LSTEP = LQ == 0 ? NM + 1 : (NM / LQ > 0 ? NM / LQ : 1);
#pragma unroll
    for (int x = 0; x < NM; ++x) {
      Mfma<E>::run(fy[SET][x / MT], fx[SET][x % MT], acc[x / MT][x % MT]);
      if (x < NI) rd(SET ^ 1, rY, rX, rsub, x);
      if (x % LSTEP == LSTEP - 1 && x / LSTEP < LQ) load_round(R, lY, lX, lq0 + x / LSTEP);
    }
#pragma unroll
    for (int r = NI; r < NR; ++r) rd(SET ^ 1, rY, rX, rsub, r);
#pragma unroll
    for (int q = NM / LSTEP; q < LQ; ++q) load_round(R, lY, lX, lq0 + q);
    if constexpr (ES == 2) {
#pragma unroll
      for (int x = 0; x < NM; ++x) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        if (x < NI) {
          if (x < MT ? TY : TX)
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          else
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if (x % LSTEP == LSTEP - 1 && x / LSTEP < LQ)
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // global load
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if constexpr (ROLE == LIN_JOIN) {
    // Parts lie as the accumulators do (below); they are added in order
    const int first = P.tiles_m * P.tiles_n - P.split_tiles;
    cgchar* part = gload_ptr(P.part + (int64_t)(tile - first) * P.splits * (BT * BT) + tid * 4);
    for (int k = 0; k < P.splits; ++k) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x4 v = *(cgu4*)(part + (int64_t)k * (BT * BT * 4) + ((i * MT + j) * 4 + q) * 4096);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += __uint_as_float(v[e]);
          }
    }
  }
  if (ROLE != LIN_JOIN && !RAW && ns > 0) {
#pragma unroll
    for (int j = 0; j < D; ++j) {
#pragma unroll
      for (int i = 0; i < LPO; ++i) load_y(j, 2 * j, i);
#pragma unroll
      for (int i = 0; i < LPO; ++i) load_x(j, 2 * j + 1, i);
    }
    wait_vmcnt<(2 * D - 2) * LPO>();  // Y_0 and X_0 have landed
    ring_barrier();
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;
    using S3 = std::integral_constant<int, 3>;
    // round -1's X part is X_{D-1}, above; its Y part, Y_D, follows in step 0
    // into the last buffer
    int cy = 0, py = NOB - 2, px = NOB - 1;
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) rd(0, 0, 1, 0, r);
    // small tiles: a wave whose rows or columns all lie past the edge loads its
    // share, and leaves its SIMD and LDS to the others (with the shorter rest of
    // K below: fp32, 777 tokens of 1000 x 2730 both ways 487 -> 471 us)
    const bool live = BT > 64 || (m0 + wm * WT < M && n0 + wn * (NT_ / 2) < N);
    for (int j = live ? ns : 0; j < ns; ++j) {
      const int cx = cy + 1 >= NOB ? cy + 1 - NOB : cy + 1;
#pragma unroll
      for (int q = LPO; q < 2 * LPO; ++q) load_round(j - 1, py, px, q);
      wait_vmcnt<(2 * D - 3) * LPO>();
      ring_barrier();
#pragma unroll
      for (int q = 0; q < LPO; ++q) load_round(j, cy, cx, q);
      py = cy;
      px = cx;
      cy = cy + 2 >= NOB ? cy + 2 - NOB : cy + 2;
    }
    for (int j = live ? 0 : ns; j < ns; ++j) {
      const int cx = cy + 1 >= NOB ? cy + 1 - NOB : cy + 1;
      const int ny = cy + 2 >= NOB ? cy + 2 - NOB : cy + 2;  // step j + 1
      const int nx = cy + 3 >= NOB ? cy + 3 - NOB : cy + 3;
      phase(S0{}, cy, cx, 1, j - 1, py, px);
      phase(S1{}, cy, cx, 2, j - 1, py, px);
      phase(S2{}, cy, cx, 3, j - 1, py, px);
      // X_{j+1} and Y_{j+1} have landed: behind them were issued Y_{j+2} and
      // the rounds up to j - 1
      wait_vmcnt<(2 * D - 3) * LPO>();
      ring_barrier();
      phase(S3{}, ny, nx, 0, j, cy, cx);
      py = cy;
      px = cx;
      cy = ny;
    }
    wait_vmem();  // loads that ran past the end land before LDS is reused
    __syncthreads();
  }
  if constexpr (RAW && ROLE != LIN_JOIN) {
    static_assert(!TX, "rows at any element: X is K-major");
    // Step j's chunks sit in register slot j % RD from RD steps before their
    // use; at step j slot j + 1 is written to LDS beside the step being read
    // and takes the loads of step j + 1 + RD.  One barrier per step.
    constexpr int RD = BT == 64 ? 4 : 3;
    u32x4 ry[RD][LPO], rx[RD][LPO];
    // Row-major chunks at the matrix's edge reach past their row, into the next
    // ones (columns that are not stored); a step with too little of the matrix
    // behind it takes them element by element.
    const bool edge_y = TY && n0 + BT > N;
    // Y's columns of this lane's chunk of instruction i that exist (row-major)
    auto cols_of = [&](int i) {
      const int rt = (wave * LPO + i) * TR + lane / TCH, ct = (lane % TCH) ^ tr_swz(rt);
      return N - n0 - ct * VEC;
    };
    auto chunk = [&](uint64_t at, bool edge, int n) __attribute__((always_inline)) -> u32x4 {
      cgchar* p = (cgchar*)at;
      if (edge && n < VEC) return load_chunk_partial<ES>(p, 0, n);
      return *(cgu4_any*)p;
    };
    auto fetch = [&](int j, auto slot_t) __attribute__((always_inline)) {
      constexpr int slot = decltype(slot_t)::value;
      const int step = s0 + j - (MODE == LIN_KR && s0 + j >= ns1 ? ns1 : 0);
      const bool part_y = edge_y && !raw_step_inside(K, P.ldy, KS, step, VEC);
      static_for<LPO>([&](auto i_t) __attribute__((always_inline)) {
        constexpr int i = decltype(i_t)::value;
        ry[slot][i] = chunk(y_src(s0 + j, i) + yoff[i], part_y, cols_of(i));
        rx[slot][i] = *(cgu4_any*)(x_src(s0 + j) + xoff[i]);
      });
    };
    auto stash = [&](int buf, auto slot_t) __attribute__((always_inline)) {
      constexpr int slot = decltype(slot_t)::value;
      static_for<LPO>([&](auto i_t) __attribute__((always_inline)) {
        constexpr int i = decltype(i_t)::value;
        char* d = smem + (wave * LPO + i) * 1024 + lane * 16;
        *reinterpret_cast<u32x4*>(d + 2 * buf * OB) = ry[slot][i];
        *reinterpret_cast<u32x4*>(d + (2 * buf + 1) * OB) = rx[slot][i];
      });
    };
    auto compute = [&](int buf) {
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) rd(0, 2 * buf, 2 * buf + 1, 0, r);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < 3) {
#pragma unroll
          for (int r = 0; r < 2 * MT; ++r) rd((s + 1) & 1, 2 * buf, 2 * buf + 1, s + 1, r);
        }
#pragma unroll
        for (int x = 0; x < MT * MT; ++x) Mfma<E>::run(fy[s & 1][x / MT], fx[s & 1][x % MT], acc[x / MT][x % MT]);
      }
    };
    static_for<RD>([&](auto k_t) __attribute__((always_inline)) {
      if (decltype(k_t)::value < ns) fetch(decltype(k_t)::value, k_t);
    });
    if (ns > 0) {
      stash(0, std::integral_constant<int, 0>{});
      if (RD < ns) fetch(RD, std::integral_constant<int, 0>{});
    }
    ring_barrier();
    for (int j0 = 0; j0 < ns; j0 += RD) {
      static_for<RD>([&](auto u_t) __attribute__((always_inline)) {
        constexpr int next = (decltype(u_t)::value + 1) % RD;
        const int j = j0 + decltype(u_t)::value;
        if (j >= ns) return;
        if (j + 1 < ns) {
          stash((j + 1) & 1, std::integral_constant<int, next>{});
          if (j + 1 + RD < ns) fetch(j + 1 + RD, std::integral_constant<int, next>{});
        }
        compute(j & 1);
        ring_barrier();
      });
    }
    if (K % KS != 0 && sp == splits - 1) {
      const int kt = ns1 * KS;
      for (int seg = 0; seg < nseg; ++seg) {
        static_for<LPO>([&](auto i_t) __attribute__((always_inline)) {
          constexpr int i = decltype(i_t)::value;
          const int blk = wave * LPO + i;
          const int r = blk * 8 + (lane >> 3), ch = (lane & 7) ^ lds_swz(r);
          const int rt = blk * TR + lane / TCH;
          const bool up = EPI == LIN_GATE ? (blk * 8) % WT >= WT / 2 : seg == 1;
          const uint64_t ya = (up ? ybase2 : ybase) + (TY ? (uint64_t)kt * ldyb : (uint64_t)kt * ES) + yoff[i];
          const uint64_t xa = (seg == 1 ? xbase2 : xbase) + (uint64_t)kt * ES + xoff[i];
          // elements of the chunk that exist: of the row's rest of K, or of its
          // columns where the row itself does
          const int nx = K - kt - ch * VEC;
          const int ny = TY ? (kt + rt < K ? cols_of(i) : 0) : nx;
          ry[0][i] = chunk(ya, true, ny);
          rx[0][i] = chunk(xa, true, nx);
        });
        stash(0, std::integral_constant<int, 0>{});
        ring_barrier();
        compute(0);
        ring_barrier();
      }
    }
  }
  // what is left of K in each segment, once, by the last split
  if (ROLE != LIN_JOIN && !SPLIT && !RAW && K % KS != 0 && sp == splits - 1) {
    const int kt = ns1 * KS;
    for (int seg = 0; seg < nseg; ++seg) {
      const uint64_t zero = (uint64_t)(uintptr_t)&lin_zero_chunk;
#pragma unroll
      for (int i = 0; i < LPO; ++i) {
        const int blk = wave * LPO + i;
        const int r = blk * 8 + (lane >> 3), ch = (lane & 7) ^ lds_swz(r);
        const int rt = blk * TR + lane / TCH;
        const bool iny = TY ? kt + rt < K : kt + ch * VEC < K;
        const bool inx = TX ? kt + rt < K : kt + ch * VEC < K;
        const bool up = EPI == LIN_GATE ? (blk * 8) % WT >= WT / 2 : seg == 1;
        const uint64_t ya = (up ? ybase2 : ybase) + (TY ? (uint64_t)kt * ldyb : (uint64_t)kt * ES) + yoff[i];
        const uint64_t xa = (seg == 1 ? xbase2 : xbase) + (TX ? (uint64_t)kt * ldxb : (uint64_t)kt * ES) + xoff[i];
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(iny ? ya : zero),
                                         (__attribute__((address_space(3))) void*)(smem + blk * 1024), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(inx ? xa : zero),
                                         (__attribute__((address_space(3))) void*)(smem + OB + blk * 1024), 16, 0, 0);
      }
      wait_vmem();
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s * (KS / 4) >= K - kt) break;  // zeros from here on
#pragma unroll
        for (int r = 0; r < 2 * MT; ++r) rd(0, 0, 1, s, r);
#pragma unroll
        for (int x = 0; x < MT * MT; ++x) Mfma<E>::run(fy[0][x / MT], fx[0][x % MT], acc[x / MT][x % MT]);
      }
      __syncthreads();
    }
  }

  // ------------------------------------------------------------ split tiles
  // Parts are kept as the accumulators lie: 16 bytes per lane and group of
  // four, whole lines per wave.
  if constexpr (ROLE == LIN_PART) {
    const int first = P.tiles_m * P.tiles_n - P.split_tiles;
    gchar* part = gstore_ptr(P.part + ((int64_t)(tile - first) * P.splits + sp) * (BT * BT) + tid * 4);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(gu4*)(part + ((i * MT + j) * 4 + q) * 4096) =
              u32x4{__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                    __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3])};
    return;
  }

  // ------------------------------------------------------------ epilogue
  // 32 x 32 result: lane l, register r -> n = 8 (r / 4) + 4 (l / 32) + r % 4,
  // m = l % 32.  The tile (or half of its rows) is staged in LDS as rows of C
  // and written with 16-byte row-contiguous stores.
  constexpr int SR = BT / PASSES;          // staged rows per pass
  constexpr int MTP = MT / PASSES;         // m blocks per wave and pass
  constexpr int RPW = 32 * MTP;            // staged rows per wave row
  static_assert(MTP >= 1, "passes");
  auto tile_row = [&](int pass, int r) { return (r / RPW) * WT + pass * RPW + r % RPW; };
  // four consecutive n of staged row r, column c
  auto put4 = [&](char* base, int r, int c, const float* v) {
    char* dst = base + r * PITCH + c * OS;
    if constexpr (OS == 2) {
      *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
      *reinterpret_cast<u32x4*>(dst) =
          u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
  };
  auto stage_acc = [&](int pass, float f) {
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if (j / MTP != pass) continue;
      const int r = wm * RPW + (j % MTP) * 32 + lcol;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = f * acc[i][j][q * 4 + e];
          put4(smem, r, wn * WT + i * 32 + q * 8 + half * 4, v);
        }
    }
  };
  // staged rows (OS-byte elements) of pass `pass` to matrix c with pitch ldc,
  // columns [N, npad) zero
  auto emit = [&](const char* base, int pass, void* c, int64_t ldc) {
    gchar* pc = gstore_ptr(c);
    constexpr int V = 16 / OS;
    constexpr int SEGS = NT_ / V;
    // rows may start at any element; then the lines at the ends of a tile's rows
    // are written in two parts, which L2 should put together
    const bool lines = ((ldc * OS) & 15) == 0 && ((uintptr_t)pc & 15) == 0;
    for (int b = tid; b < SR * SEGS; b += 256) {
      const int r = b / SEGS, sc = b - r * SEGS;
      const int gr = m0 + tile_row(pass, r), gc = n0 + sc * V;
      if (gr >= M || gc >= P.npad) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(base + r * PITCH + sc * 16);
      gchar* p = pc + ((int64_t)gr * ldc + gc) * OS;
      if (gc + V <= N) {
        if (lines)
          __builtin_nontemporal_store(v, (gu4*)p);
        else
          *(gu4_any*)p = v;
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (gc + k >= P.npad) continue;
          const uint32_t e = gc + k < N ? chunk_elem<OS>(v, k) : 0u;
          if constexpr (OS == 2)
            ((__attribute__((address_space(1))) uint16_t*)p)[k] = (uint16_t)e;
          else
            ((__attribute__((address_space(1))) uint32_t*)p)[k] = e;
        }
      }
    }
  };

  // The barriers below order LDS only: stores stay in flight across them, and
  // the workgroup ends without waiting for its last ones.
  if constexpr (EPI == LIN_OUT) {
    const float f = g.alpha ? *g.alpha : 1.0f;
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      if (pass) ring_barrier();
      stage_acc(pass, f);
      ring_barrier();
      emit(smem, pass, P.c, P.ldc);
    }
  } else if constexpr (EPI == LIN_ACC) {
    // workspace: fp32, pitch a multiple of 4
    gchar* pc = gstore_ptr(P.c);
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      if (pass) ring_barrier();
      stage_acc(pass, 1.0f);
      ring_barrier();
      constexpr int SEGS = NT_ / 4;
      for (int b = tid; b < SR * SEGS; b += 256) {
        const int r = b / SEGS, sc = b - r * SEGS;
        const int gr = m0 + tile_row(pass, r), gc = n0 + sc * 4;
        if (gr >= M || gc >= N) continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(smem + r * PITCH + sc * 16);
        gu4* p = (gu4*)(pc + ((int64_t)gr * P.ldc + gc) * 4);
        if (g.accumulate) {
          const u32x4 o = *p;
          u32x4 w;
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(__uint_as_float(v[k]) + __uint_as_float(o[k]));
          *p = w;
        } else {
          *p = v;
        }
      }
    }
  } else if constexpr (EPI == LIN_GATE) {
    // accumulators e and e + 8 MT (e < 8 MT, flat over i and r) are gate and up
    // of one column of h: column 32 (e / 16) + 8 (e % 16 / 4) + 4 half + e % 4
    // of the wave's WT / 2
    auto col_of = [&](int e) { return wn * (WT / 2) + (e / 16) * 32 + ((e % 16) / 4) * 8 + half * 4; };
    char* sg = smem;
    char* su = smem + SR * PITCH;
    // staging of the low bits, behind h's: a byte per column
    constexpr bool LOW4 = SAVE && OES == 2;
    constexpr int PITCH4 = NT_ + 16;
    char* s4 = smem + SR * PITCH;
    static_assert(SR * PITCH + SR * PITCH4 <= NOB * OB, "staging of the low bits");
    static_assert(!LOW4 || PASSES == 1, "the low bits' rows are the tile's");
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      if (pass) ring_barrier();
      if constexpr (SAVE) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          if (j / MTP != pass) continue;
          const int r = wm * RPW + (j % MTP) * 32 + lcol;
#pragma unroll
          for (int e = 0; e < 8 * MT; e += 4) {
            float vg[4], vu[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              vg[k] = acc[(e + k) / 16][j][(e + k) % 16];
              vu[k] = acc[(e + k + 8 * MT) / 16][j][(e + k + 8 * MT) % 16];
              if constexpr (LOW4) {
                vg[k] = __uint_as_float(round12(vg[k]));
                vu[k] = __uint_as_float(round12(vu[k]));
              }
            }
            const int c = col_of(e);
            if constexpr (LOW4) {
              auto hi = [](const float* v) {
                return u32x2{(__float_as_uint(v[0]) >> 16) | (__float_as_uint(v[1]) & 0xffff0000u),
                             (__float_as_uint(v[2]) >> 16) | (__float_as_uint(v[3]) & 0xffff0000u)};
              };
              *reinterpret_cast<u32x2*>(sg + r * PITCH + c * 2) = hi(vg);
              *reinterpret_cast<u32x2*>(su + r * PITCH + c * 2) = hi(vu);
            } else {
              put4(sg, r, c, vg);
              put4(su, r, c, vu);
            }
          }
        }
        ring_barrier();
        emit(sg, pass, P.c2, P.ldc);
        emit(su, pass, P.c3, P.ldc);
        ring_barrier();
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (j / MTP != pass) continue;
        const int r = wm * RPW + (j % MTP) * 32 + lcol;
#pragma unroll
        for (int e = 0; e < 8 * MT; e += 4) {
          float v[4];
          uint32_t low = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float vg = opaque(acc[(e + k) / 16][j][(e + k) % 16]);
            const float vu = opaque(acc[(e + k + 8 * MT) / 16][j][(e + k + 8 * MT) % 16]);
            v[k] = act_only<ACT>(vg) * vu;
            if constexpr (LOW4) low |= low4(round12(vg), round12(vu)) << (8 * k);
          }
          const int c = col_of(e);
          put4(sg, r, c, v);
          if constexpr (LOW4) *reinterpret_cast<uint32_t*>(s4 + r * PITCH4 + c) = low;
        }
      }
      ring_barrier();
      emit(sg, pass, P.c, P.ldc);
    }
    if constexpr (LOW4) {
      gchar* p4 = gstore_ptr(P.c4);
      constexpr int SEGS = NT_ / 16;
      for (int b = tid; b < BT * SEGS; b += 256) {
        const int r = b / SEGS, sc = b - r * SEGS;
        const int gr = m0 + r, gc = n0 + sc * 16;
        if (gr < M && gc < N)
          __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(s4 + r * PITCH4 + sc * 16),
                                      (gu4*)(p4 + (int64_t)gr * P.ld4 + gc));
      }
    }
  } else if constexpr (EPI == LIN_DGATE) {
    // g and u are fetched a group of segments ahead: the loads of a group are
    // issued before the stores of the group before it (one counter orders
    // both), so a group's HBM latency runs under the other's arithmetic
    cgchar* pg = gload_ptr(P.aux1);
    cgchar* pu = gload_ptr(P.aux2);
    cgchar* p4 = gload_ptr(P.aux3);
    gchar* pdg = gstore_ptr(P.c);
    gchar* pdu = gstore_ptr(P.c2);
    constexpr int SEGS = NT_ / 8;
    constexpr int IT = SR * SEGS / 256;
    constexpr int GR = IT < (OES == 2 ? 8 : 4) ? IT : (OES == 2 ? 8 : 4);
    constexpr int NG = IT / GR;
    static_assert(SR * SEGS % 256 == 0 && IT % GR == 0, "segment groups");
    constexpr int CH = OES / 2;  // 16-byte chunks per segment
    const bool ragged = n0 + BT > N;
    u32x4 wg[2][GR][CH], wu[2][GR][CH];
    u32x2 w4[2][GR];
    // segment it of a pass: its row and column, whether it is stored, and
    // whether all 8 columns are (fp32 rows are padded to 4 elements only)
    auto seg = [&](int pass, int it, int& r, int& sc, int64_t& at, bool& in, bool& whole) {
      const int b = tid + it * 256;
      r = b / SEGS;
      sc = b - r * SEGS;
      const int gr = m0 + tile_row(pass, r), gc = n0 + sc * 8;
      in = gr < M && gc < P.npad;
      whole = OES == 2 || gc + 8 <= P.npad;
      at = ((int64_t)gr * P.ldc + gc) * OES;
    };
    auto fetch = [&](auto grp_t) __attribute__((always_inline)) {
      constexpr int grp = decltype(grp_t)::value, set = grp & 1;
      static_for<GR>([&](auto k_t) __attribute__((always_inline)) {
        constexpr int k = decltype(k_t)::value;
        int r, sc;
        int64_t at;
        bool in, whole;
        seg(grp / NG, (grp % NG) * GR + k, r, sc, at, in, whole);
        static_for<CH>([&](auto c_t) __attribute__((always_inline)) {
          constexpr int c = decltype(c_t)::value;
          // chunks that are not stored are read at the matrix's start
          const int64_t from = in && (c == 0 || whole) ? at + 16 * c : 0;
          wg[set][k][c] = *(cgu4*)(pg + from);
          wu[set][k][c] = *(cgu4*)(pu + from);
        });
        if constexpr (OES == 2)
          w4[set][k] = *(const __attribute__((address_space(1))) u32x2*)(
              p4 + (in ? (int64_t)(m0 + tile_row(grp / NG, r)) * P.ld4 + n0 + sc * 8 : 0));
      });
    };
    fetch(std::integral_constant<int, 0>{});
    static_for<PASSES * NG>([&](auto grp_t) __attribute__((always_inline)) {
      constexpr int grp = decltype(grp_t)::value, pass = grp / NG, set = grp & 1;
      if constexpr (grp % NG == 0) {
        if constexpr (pass > 0) ring_barrier();
        stage_acc(pass, 1.0f);
        ring_barrier();
      }
      if constexpr (grp + 1 < PASSES * NG) fetch(std::integral_constant<int, grp + 1>{});
      __builtin_amdgcn_sched_barrier(0);
      static_for<GR>([&](auto k_t) __attribute__((always_inline)) {
        constexpr int k = decltype(k_t)::value;
        int r, sc;
        int64_t at;
        bool in, whole;
        seg(pass, (grp % NG) * GR + k, r, sc, at, in, whole);
        if (!in) return;
        float dh[8], vg[8], vu[8];
        unpack8<4>(reinterpret_cast<const u32x4*>(smem + r * PITCH + sc * 32), dh);
        unpack8<OES>(wg[set][k], vg);
        unpack8<OES>(wu[set][k], vu);
        if constexpr (OES == 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t b = w4[set][k][e / 4] >> (8 * (e % 4));
            vg[e] = join12(__float_as_uint(vg[e]), b & 15u);
            vu[e] = join12(__float_as_uint(vu[e]), (b >> 4) & 15u);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float a, da;
          act_both<ACT>(vg[e], a, da);
          vg[e] = dh[e] * vu[e] * da;
          vu[e] = dh[e] * a;
        }
        if (ragged) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool on = n0 + sc * 8 + e < N;
            vg[e] = on ? vg[e] : 0.0f;
            vu[e] = on ? vu[e] : 0.0f;
          }
        }
        u32x4 og[CH], ou[CH];
        pack8<OES>(vg, og);
        pack8<OES>(vu, ou);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (c > 0 && !whole) continue;
          __builtin_nontemporal_store(og[c], (gu4*)(pdg + at) + c);
          __builtin_nontemporal_store(ou[c], (gu4*)(pdu + at) + c);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  } else {
    // cross entropy: a lane holds half of the wave's WT words of token m, the
    // lane 32 further the other half
    const int nw = n0 + wn * WT;
    const bool ragged = nw + WT > N;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int m = m0 + wm * WT + j * 32 + lcol;
      const int64_t y = m < M ? g.targets[m] : -1;
      const int yl = (int)(y - nw < 0 ? -1 : y - nw < WT ? y - nw : -1);
      float mx = -INFINITY, tl = 0.0f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int nl = i * 32 + (r / 4) * 8 + half * 4 + r % 4;
          if (ragged && nw + nl >= N) acc[i][j][r] = -INFINITY;
          tl = yl == nl ? acc[i][j][r] : tl;
          mx = fmaxf(mx, acc[i][j][r]);
          if (r == 15) __builtin_amdgcn_sched_barrier(0);  // one block's compares at a time
        }
      // the lane that holds the target's word writes its logit
      if (y >= 0 && y < N && yl >= 0 && ((yl >> 2) & 1) == half) g.target_logit[m] = tl;
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float ref = mx == -INFINITY ? 0.0f : mx;  // no word but -inf: exponentials 0, not NaN
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float d = acc[i][j][r] - ref;
          const float e = OES == 4 ? expf(d) : __expf(d);
          acc[i][j][r] = e;
          s += e;
        }
      s += __shfl_xor(s, 32);
      if (half == 0 && m < M) g.stats[(int64_t)m * g.pieces + 2 * tj + wn] = make_float2(mx, s);
    }
    if (P.c) {
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass) {
        if (pass) ring_barrier();
        stage_acc(pass, 1.0f);
        ring_barrier();
        emit(smem, pass, P.c, P.ldc);
      }
    }
  }
}

// 4 consecutive elements at any element address, and back
template <int ESZ>
__device__ __forceinline__ f32x4 load4(cgchar* p) {
  if constexpr (ESZ == 2) {
    typedef u32x2 u32x2_any __attribute__((aligned(2)));
    const u32x2 w = *(const __attribute__((address_space(1))) u32x2_any*)p;
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                 __uint_as_float(w[1] & 0xffff0000u)};
  } else {
    return __builtin_bit_cast(f32x4, (u32x4)(*(cgu4_any*)p));
  }
}
template <int ESZ>
__device__ __forceinline__ void store4(gchar* p, f32x4 v) {
  if constexpr (ESZ == 2) {
    typedef u32x2 u32x2_any __attribute__((aligned(2)));
    *(__attribute__((address_space(1))) u32x2_any*)p = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
    *(gu4_any*)p = __builtin_bit_cast(u32x4, v);
  }
}

// Join of split tiles for the epilogues that work element by element: one
// workgroup per tile and 32 x 32 block of its wave tiles (gate: pair of blocks,
// or halves of one when a wave tile is one block).  A thread sums the parts of
// four groups of four accumulators (consecutive n of one m) in order and
// stores them.  Bound by the parts' bytes, read once.  (The cross entropy's
// rows need the whole tile: its join is linear_kernel's.)
template <class E, int BT, int EPI, int ACT, bool SAVE>
__global__ void __launch_bounds__(256) join_kernel(const LinArgs g) {
  constexpr int ES = Elt<E>::kSize;
  constexpr bool GATE = EPI == LIN_GATE;
  constexpr int WT = BT / 2, MT = WT / 32, NT_ = GATE ? BT / 2 : BT;
  constexpr int NB = GATE ? (MT + 1) / 2 : MT;  // blocks along n
  constexpr int NQ = GATE && MT == 1 ? 2 : 4;   // groups of four per block
  int t = blockIdx.x / (NB * MT), pi = 0;
  const int j = blockIdx.x % MT, i = blockIdx.x / MT % NB;
  while (t >= g.p[pi].split_tiles) t -= g.p[pi++].split_tiles;
  const LinProb& P = g.p[pi];
  int ti, tj;
  full_tile_blocked(P.tiles_m * P.tiles_n - P.split_tiles + t, P.tiles_m, P.tiles_n, ti, tj);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave >> 1, wm = wave & 1, half = lane >> 5, lcol = lane & 31;
  cgchar* part = gload_ptr(P.part + (int64_t)t * P.splits * (BT * BT) + tid * 4);
  f32x4 v[NQ], u[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) v[q] = u[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int k = 0; k < P.splits; ++k, part += BT * BT * 4) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      auto at = [&](int grp) { return ((grp / 4 * MT + j) * 4 + grp % 4) * 4096; };
      v[q] += __builtin_bit_cast(f32x4, *(cgu4*)(part + at(4 * i + q)));
      if constexpr (GATE) u[q] += __builtin_bit_cast(f32x4, *(cgu4*)(part + at(4 * i + q + 2 * MT)));
    }
  }
  const int m = ti * BT + wm * WT + j * 32 + lcol;
  if (m >= P.M) return;
  const float f = EPI == LIN_OUT && g.alpha ? *g.alpha : 1.0f;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    // n of the group's first value: as in the epilogues of linear_kernel
    const int n = tj * NT_ + wn * (NT_ / 2) + i * 32 + q * 8 + half * 4;
    if (n >= P.npad) continue;
    const int64_t at = (int64_t)m * P.ldc + n;
    const bool whole = n + 4 <= P.N;
    auto put = [&](void* c, f32x4 x) {
      if (whole) {
        store4<ES>(gstore_ptr(c) + at * ES, x);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < P.npad) store_out(gstore_ptr(c), at + e, n + e < P.N ? x[e] : 0.0f, ES == 4);
      }
    };
    if constexpr (EPI == LIN_OUT) {
      put(P.c, f * v[q]);
    } else if constexpr (EPI == LIN_ACC) {
      float* c = (float*)P.c + at;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < P.N) c[e] = g.accumulate ? c[e] + v[q][e] : v[q][e];
    } else if constexpr (GATE) {
      f32x4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = act_only<ACT>(v[q][e]) * u[q][e];
      put(P.c, h);
      if constexpr (SAVE) {
        f32x4 gs = v[q], us = u[q];
        if constexpr (ES == 2) {
          uint32_t low = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a = round12(gs[e]), b = round12(us[e]);
            low |= low4(a, b) << (8 * e);
            gs[e] = __uint_as_float(a & 0xffff0000u);  // exact in bf16
            us[e] = __uint_as_float(b & 0xffff0000u);
          }
          *(__attribute__((address_space(1))) uint32_t*)(gstore_ptr(P.c4) + (int64_t)m * P.ld4 + n) = low;
        }
        put(P.c2, gs);
        put(P.c3, us);
      }
    } else {
      // g's and u's rows reach to npad, a multiple of four
      f32x4 gv = load4<ES>(gload_ptr(P.aux1) + at * ES), uv = load4<ES>(gload_ptr(P.aux2) + at * ES);
      if constexpr (ES == 2) {
        const uint32_t low =
            *(const __attribute__((address_space(1))) uint32_t*)(gload_ptr(P.aux3) + (int64_t)m * P.ld4 + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gv[e] = join12(__float_as_uint(gv[e]), (low >> (8 * e)) & 15u);
          uv[e] = join12(__float_as_uint(uv[e]), (low >> (8 * e + 4)) & 15u);
        }
      }
      f32x4 dg, du;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, da;
        act_both<ACT>(gv[e], a, da);
        dg[e] = v[q][e] * uv[e] * da;
        du[e] = v[q][e] * a;
      }
      put(P.c, dg);
      put(P.c2, du);
    }
  }
}

// The ring's depth.  A tile of 128 leaves a compute unit to one workgroup with
// nine stages and to two with five, one of 64 to two and four.  With a
// workgroup for every place the shallow ring is the faster one, since one
// workgroup's epilogue and waits run under the others' MFMAs (bf16, 128:
// 1531 x 5464 x 2056 with its gate 138 -> 112 us, 4096 x 4096 x 1024 42 -> 36;
// fp32, 64: 101 -> 96 at 777 x 2732 x 1000); with fewer the deep one is (128:
// 1531 x 2056 x 10928 in 204 tiles 132 against 117 us; 64: 512 x 1024 x 8192
// in 128 tiles 45 against 34).  fp32 tiles of 128 are bound by the MFMA and
// always shallow.
template <class E, class O, int BT, int MODE, int EPI, int ACT, int ROLE, bool SAVE>
hipError_t launch_lin_inst(const LinArgs& a, int grid, hipStream_t st) {
  constexpr bool TAKES_RAW = BT <= 128 && MODE != LIN_RR;  // (weight gradients take padded copies)
  if constexpr (ROLE != LIN_JOIN) {
    if (a.raw) {
      if constexpr (TAKES_RAW) {
        hipLaunchKernelGGL((linear_kernel<E, O, BT, MODE, EPI, ACT, ROLE, SAVE, true, 2>), dim3(grid), dim3(256), 0, st, a);
        return hipGetLastError();
      }
      return hipErrorInvalidValue;
    }
    if constexpr (BT == 64 || (BT == 128 && Elt<E>::kSize == 2)) {
      if (grid <= kLinCu * (BT == 64 ? 2 : 1)) {
        hipLaunchKernelGGL((linear_kernel<E, O, BT, MODE, EPI, ACT, ROLE, SAVE, false, 4>), dim3(grid), dim3(256), 0, st, a);
        return hipGetLastError();
      }
    }
  }
  hipLaunchKernelGGL((linear_kernel<E, O, BT, MODE, EPI, ACT, ROLE, SAVE, false, 2>), dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

// the kernels of one epilogue: a join does not depend on the mode, a part not
// on the epilogue but for the gate's
template <class E, class O, int BT, int MODE, int EPI, int ACT = 0, bool SAVE = false>
hipError_t launch_lin_role(const LinArgs& a, int grid, hipStream_t st) {
  if (a.role == LIN_WHOLE) return launch_lin_inst<E, O, BT, MODE, EPI, ACT, LIN_WHOLE, SAVE>(a, grid, st);
  if (a.role == LIN_JOIN) {
    if constexpr (EPI == LIN_XENT) {
      return launch_lin_inst<E, O, BT, LIN_KK, EPI, ACT, LIN_JOIN, SAVE>(a, grid, st);
    } else {
      constexpr int MT = BT / 64;
      int64_t tiles = 0;
      for (int i = 0; i < a.nprob; ++i) tiles += a.p[i].split_tiles;
      const int64_t n = tiles * MT * (EPI == LIN_GATE ? (MT + 1) / 2 : MT);
      if (n > 0x7fffffff) return hipErrorInvalidValue;
      hipLaunchKernelGGL((join_kernel<O, BT, EPI, ACT, SAVE>), dim3((unsigned)n), dim3(256), 0, st, a);
      return hipGetLastError();
    }
  }
  return launch_lin_inst<E, O, BT, MODE, EPI == LIN_GATE ? LIN_GATE : LIN_OUT, 0, LIN_PART, false>(a, grid, st);
}

template <class E, class O, int BT, int MODE, int EPI, bool SAVE>
hipError_t launch_lin_act(const LinArgs& a, int grid, hipStream_t st) {
  if (a.act == LIN_SILU) return launch_lin_role<E, O, BT, MODE, EPI, LIN_SILU, SAVE>(a, grid, st);
  if (a.act == LIN_GELU) return launch_lin_role<E, O, BT, MODE, EPI, LIN_GELU, SAVE>(a, grid, st);
  if (a.act == LIN_GELU_TANH) return launch_lin_role<E, O, BT, MODE, EPI, LIN_GELU_TANH, SAVE>(a, grid, st);
  return hipErrorInvalidValue;
}

template <class E, class O, int BT>
hipError_t launch_lin(LinMode mode, LinEpi epi, const LinArgs& a, int grid, hipStream_t st) {
  if (epi == LIN_OUT) {
    if (mode == LIN_KK) return launch_lin_role<E, O, BT, LIN_KK, LIN_OUT>(a, grid, st);
    if (mode == LIN_KR) return launch_lin_role<E, O, BT, LIN_KR, LIN_OUT>(a, grid, st);
    if (mode == LIN_RR) return launch_lin_role<E, O, BT, LIN_RR, LIN_OUT>(a, grid, st);
  } else if (epi == LIN_ACC && mode == LIN_RR) {
    return launch_lin_role<E, O, BT, LIN_RR, LIN_ACC>(a, grid, st);
  } else if (epi == LIN_GATE && mode == LIN_KK) {
    if (a.p[0].c2) return launch_lin_act<E, O, BT, LIN_KK, LIN_GATE, true>(a, grid, st);
    return launch_lin_act<E, O, BT, LIN_KK, LIN_GATE, false>(a, grid, st);
  } else if (epi == LIN_DGATE && mode == LIN_KR) {
    if constexpr (BT != 128 || Elt<E>::kSize == 2) return launch_lin_act<E, O, BT, LIN_KR, LIN_DGATE, false>(a, grid, st);
  } else if (epi == LIN_XENT && mode == LIN_KK) {
    return launch_lin_role<E, O, BT, LIN_KK, LIN_XENT>(a, grid, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace dmuon
