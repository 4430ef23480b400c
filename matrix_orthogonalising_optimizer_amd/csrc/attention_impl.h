// Attention over packed sequences with grouped heads, forward and backward, on
// gfx950 MFMA.
//
//   s_ij = scale q_i . k_j  for the keys j that row i sees (all of its sequence,
//          or j <= i + keys - queries when causal),
//   p = softmax over j,  y_i = sum_j p_ij v_j,  lse_i = log sum_j exp(s_ij)
//   D_i = dy_i . y_i,  ds_ij = p_ij (dy_i . v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dy_i
//
// Scores, softmax statistics and all sums are fp32.  Rounded to bf16 (of bf16 calls; a
// matrix instruction takes no wider operand at its rate): p and ds as operands
// of the second products, each off by half a step, which the sums average; y when it is stored,
// from which D is taken.  p is not divided by its sum before the product but y after it.
// fp32 calls have fp32 matrix instructions; of theirs lse is rounded, at its own size, from which the
// backward pass forms p (kFarLse).
#pragma once

#include <algorithm>

#include "attention.h"
#include "gemm_impl.h"

namespace dmuon {
namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef uint32_t u32x4_any4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFarScore = 0x1p29f;  // of a score's multiple of scale log2 e: row_factor

// f(0), f(1), .. f(N - 1), the index a compile-time constant
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

// v of this lane and of the one 32 lanes on, in both
__device__ __forceinline__ float half_max(float v) {
  const u32x2 r = __builtin_bit_cast(
      u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const u32x2 r = __builtin_bit_cast(
      u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Probabilities are exp2(s c - R), c = scale log2 e and R = m c rounded, m the row's reference score: the
// product and difference are rounded once, and what R is off by is a factor that the row's sum has too.  From
// |R| = 2^29 on that factor would leave the exponents' range (2^16 there), but two scores of such size that
// differ at all do so by 2^32 or more in their probabilities: any c that keeps it so will do, and
// with a power of two m c is exact.
__device__ __forceinline__ float row_factor(float m, float c) {
  if (!(fabsf(m * c) >= kFarScore) || m == -__builtin_inff()) return c;
  return __uint_as_float((284u - (__float_as_uint(fabsf(m)) >> 23)) << 23);  // |m| times it: 2^30 .. 2^31
}

// The factor from sums about reference m to those about mn (m grown, or the same; -infinity for none yet).
__device__ __forceinline__ float row_rescale(float m, float cm, float mn, float cn, float c) {
#pragma clang fp contract(off)  // (references are rounded products)
  const float base = mn == -__builtin_inff() ? 0.0f : mn;
  // (of far rows what was summed vanishes, unless the reference stays)
  return __builtin_amdgcn_exp2f(cm == c && cn == c ? m * c - base * c : (m - base) * c);
}

// Backward: p = exp2(s c - L), L = lse log2 e.  What the fp32 L is off by, 2^-23 of it, is a factor of
// the row's gradients; from |L| = 4096 on (2^-11) the row's reference and sum are computed anew.
// dq leaves two numbers of a row for dk and dv: L and D, or, marked by a first one between 0 and
// 2^-60, (1 + log2 of the sum) 2^-100 and the reference, or kNoSum of a row that sees no key, or
// whose every score is -infinity, and which leaves nothing in a product, whatever it meets there.  (L takes
// no such value, nor +0: as whole numbers marks are the smallest.)
constexpr float kFarLse = 4096.0f;
constexpr float kNoSum = 0x1p-70f;
__device__ __forceinline__ bool row_marked(float w) { return w > 0.0f && w < 0x1p-60f; }

// ---------------------------------------------------------------- the work
// One workgroup's tile: 128 or 256 of a sequence's query rows from `start`
// (token-major: the `group` heads that share a key head are consecutive rows of
// a token, so that a single token's heads fill a wave), or of its keys.
struct AttnTile {
  int head;            // key head
  int q0, nq, k0, nk;  // the sequence's first rows and lengths
  int64_t start;
  int part;            // of a.parts that share the tile's work
};

// Boundary i of a list of first rows, kept inside the rows that exist whatever
// the list holds.  -1 and n + 1: the ends of the tensor; what lies before the
// first and behind the last sequence is a sequence that meets nothing.
__device__ __forceinline__ int attn_edge(const int32_t* cu, int i, int n, int rows) {
  return i < 0 ? 0 : i > n ? rows : min(max(cu[i], 0), rows);
}

// Unit (tile slot, key head, part) of this workgroup.  Workgroups go round-robin over
// the 8 XCDs: each takes heads of its own, whose keys and values stay in its L2,
// as far as they divide by 8; tiles of the others are dealt to all.  Tiles of a
// causal sequence come in the order of their work, the largest first, for all of an
// XCD's heads together; of more than 62 sequences in the list's order.  Those lists are walked
// 64 at a time by every workgroup, so a call of many short sequences takes as long as
// that (attn_cut has figures).
template <bool KEYS, int PER>
__device__ __forceinline__ bool attn_tile(const AttnArgs& a, AttnTile& t) {
  // (fewer than 2^31 units)
  const uint32_t b = a.unit0 + blockIdx.x, slots = a.slots;
  const uint32_t parts = a.parts, mine = (a.kv_heads >> 3) * parts, others = (a.kv_heads & 7) * parts;
  const uint32_t own = mine * slots, j = b >> 3, xcd = b & 7;
  uint32_t at, unit;
  if (j < own) {
    at = j / mine;
    unit = j - at * mine;
    t.head = (int)(xcd * (a.kv_heads >> 3) + unit / parts);
  } else {
    const uint32_t u = (j - own) * 8 + xcd;
    if (u >= others * slots) return false;
    at = u / others;
    unit = u - at * others;
    t.head = (int)((a.kv_heads & ~7) + unit / parts);
  }
  t.part = (int)(unit % parts);
  const int64_t slot = at;
  constexpr int per = PER;
  const int64_t mult = KEYS ? 1 : a.group;
  int64_t tile = 0, tiles = 0;
  if (!a.cu_q) {
    t.nq = (int)(a.tokens_q / a.sequences);
    t.nk = (int)(a.tokens_k / a.sequences);
    tiles = ((KEYS ? t.nk : t.nq) * mult + per - 1) / per;
    if (tiles == 0) return false;
    const int64_t s = slot / tiles;
    if (s >= a.sequences) return false;
    t.q0 = (int)s * t.nq;
    t.k0 = (int)s * t.nk;
    tile = slot - s * tiles;
  } else {
    const int lane = threadIdx.x & 63, n = a.sequences;
    const int32_t *cu = KEYS ? a.cu_k : a.cu_q, *other = KEYS ? a.cu_q : a.cu_k;
    const int rows = (int)(KEYS ? a.tokens_k : a.tokens_q), rows2 = (int)(KEYS ? a.tokens_q : a.tokens_k);
    // Lane by lane the sequences from `base`: their first row and length, those of the
    // other side (none before the first and behind the last), their tiles.
    int lo1, len1, lo2, len2, c;
    auto look = [&](int base) {
      const int sq = base + lane;
      const bool real = sq >= 1 && sq <= n;
      lo1 = attn_edge(cu, sq - 1, n, rows);
      len1 = sq <= n + 1 ? max(attn_edge(cu, sq, n, rows) - lo1, 0) : 0;
      lo2 = real ? attn_edge(other, sq - 1, n, rows2) : 0;
      len2 = real ? max(attn_edge(other, sq, n, rows2) - lo2, 0) : 0;
      c = (int)((len1 * mult + per - 1) / per);
    };
    look(0);
    int seg = -1;
    if (a.causal && n + 2 <= 64) {
      // All tiles by their work: tile x of a sequence's rows (or x-th last of its keys) is
      // of level x, and the highest levels come first.  A level's first slot is the
      // number of tiles above it.
      auto above = [&](int x) {  // tiles of level x and more
        int v = max(0, c - x);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
        return __builtin_amdgcn_readfirstlane(v);
      };
      if (above(0) <= slot) return false;
      int lo = 0, hi = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) hi = max(hi, __shfl_xor(hi, o));
      hi = __builtin_amdgcn_readfirstlane(hi);
      while (hi - lo > 1) {  // above(lo) > slot >= above(hi)
        const int mid = (lo + hi) >> 1;
        if (above(mid) > slot) lo = mid;
        else hi = mid;
      }
      uint64_t has = __ballot(c > lo);
      for (int r = (int)slot - above(lo + 1); r > 0 && has; --r) has &= has - 1;
      if (!has) return false;  // (lists that are not as stated: more tiles than 32 bits count)
      seg = __builtin_ctzll(has);
      tiles = __builtin_amdgcn_readlane(c, seg);
      tile = tiles - 1 - lo;
    } else {
      int64_t before = 0;
      for (int base = 0; base <= n + 1; base += 64) {
        if (base > 0) look(base);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int up = __shfl_up(incl, o);
          if (lane >= o) incl += up;
        }
        const uint64_t hit = __ballot(before + incl > slot);
        if (hit) {
          const int f = __builtin_ctzll(hit);
          seg = f;
          tiles = __builtin_amdgcn_readlane(c, f);
          tile = slot - (before + __builtin_amdgcn_readlane(incl, f) - tiles);
          break;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
      }
    }
    if (seg < 0) return false;
    auto of = [&](int v) { return __builtin_amdgcn_readlane(v, seg); };
    const int lo = of(lo1), len = of(len1), low = of(lo2), len_low = of(len2);
    t.q0 = KEYS ? low : lo;
    t.nq = KEYS ? len_low : len;
    t.k0 = KEYS ? lo : low;
    t.nk = KEYS ? len : len_low;
  }
  if (!KEYS && a.causal) tile = tiles - 1 - tile;
  // the same in all lanes: into scalar registers
  auto uni = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  t.head = uni(t.head);
  t.part = uni(t.part);
  t.q0 = uni(t.q0);
  t.nq = uni(t.nq);
  t.k0 = uni(t.k0);
  t.nk = uni(t.nk);
  t.start = (int64_t)uni((int)tile) * per;
  return true;
}

// A block of rows that start `rem` rows into token `token` (relative to its
// sequence): local row x is token + (rem + x) / group, head (rem + x) % group.
struct RowBase {
  int token, rem;
};
__device__ __forceinline__ RowBase row_base(const AttnArgs& a, int64_t row) {
  if (a.group == 1) return {(int)row, 0};
  const uint32_t t = (uint32_t)((uint64_t)row / (uint32_t)a.group);
  return {(int)t, (int)(row - (int64_t)t * a.group)};
}
__device__ __forceinline__ void row_of(const AttnArgs& a, const RowBase& b, int x, int& token, int& g) {
  const uint32_t y = (uint32_t)(b.rem + x);
  const uint32_t t = a.group_magic ? __umulhi(y, a.group_magic) : y;
  token = b.token + (int)t;
  g = (int)(y - t * (uint32_t)a.group);
}

// ---------------------------------------------------------------- LDS tiles
// Rows of a head in blocks of 8 rows x eight 16-byte chunks, what one direct load of
// a wave fills with eight 128-byte lines.  A block holds its chunks one behind the
// other, 8 rows each, so that a fragment's address is a lane's constant and an
// immediate; rows are swapped by fours for every other pair of chunks, and
// chunks by pairs for every other block of rows.  Sixteen consecutive rows read at
// one chunk, and four consecutive rows read at four chunks (transposing reads),
// then cover the 256 bytes of the banks once (bf16: no conflicts by the counters; fp32 has no
// transposing read, and its reads of single words conflict for 60% of the reads' cycles).
template <class E, int DP>
struct Geo {
  static constexpr int ES = Elt<E>::kSize, VEC = 16 / ES;
  static constexpr int NCB = (DP / VEC + 7) / 8;  // blocks across
  static constexpr int NCH = NCB * 8;             // chunks of a row in LDS
  static constexpr int RB = NCB * 1024;           // bytes of 8 rows
  static constexpr int NS = DP / VEC / 2;         // pairs of chunks: steps of a sum over the head's elements
  static constexpr int DB = DP / 32;              // blocks of 32 elements
  static constexpr int KF = ES == 2 ? 16 : 8;     // rows that a fragment over rows holds (both halves)
  __device__ static constexpr int at(int row, int ch) {
    const int c = (ch & 7) ^ ((row >> 3) & 1), r = (row & 7) ^ (((ch >> 1) & 1) << 2);
    return (row >> 3) * RB + (ch >> 3) * 1024 + c * 128 + r * 16;
  }
};

// Direct load of a wave's share of a tile: 16 bytes a lane from `rsrc` at voff,
// to LDS from `lds` on.  Past the buffer's end it writes zeros.  As inline
// assembly for the reason of ring_load.
__device__ __forceinline__ void tile_load(const u32x4& rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
// 4 bytes a lane
__device__ __forceinline__ void word_load(const u32x4& rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
constexpr uint32_t kOutside = 0x80000000u;  // past the end of any of these buffers

__device__ __forceinline__ uint32_t lds_at(const char* p) { return (uint32_t)(uintptr_t)(lds_char*)const_cast<char*>(p); }

// A wave's share of the loads of an operand's tile: GROUPS blocks of 8 rows, every
// NW-th.  Of two operands with fewer blocks than waves each wave loads one's.
template <class G, int ROWS, int NW>
struct TileShare {
  static constexpr int BLOCKS = ROWS / 8;
  static constexpr bool SPLIT = BLOCKS < NW;
  static constexpr int GROUPS = SPLIT ? 1 : BLOCKS / NW;
  static constexpr int LOADS = SPLIT ? G::NCB : 2 * GROUPS * G::NCB;  // of a wave for two operands
  static_assert(SPLIT ? 2 * BLOCKS == NW : BLOCKS % NW == 0, "blocks of a tile");
  int row, ch, rb, wave;  // the lane's row and chunk in the first block, that block
  __device__ TileShare(int wave_, int lane) {
    wave = wave_;
    rb = wave_ % BLOCKS;
    ch = (lane >> 3) ^ (rb & 1);
    row = 8 * rb + ((lane & 7) ^ (((ch >> 1) & 1) << 2));
  }
  // whether this wave loads the first operand, or the second
  __device__ bool mine(int which) const { return !SPLIT || wave / BLOCKS == which; }
  __device__ int row_of_group(int x) const { return row + 8 * NW * x; }
  // rows of group x, `off` of the lane's row (or kOutside) and chunk
  __device__ __forceinline__ void load(const u32x4& rsrc, uint32_t off, int nch, const char* tile, int x) const {
    const uint32_t to = lds_at(tile) + (uint32_t)((rb + NW * x) * G::RB);
#pragma unroll
    for (int i = 0; i < G::NCB; ++i)
      tile_load(rsrc, ch + 8 * i < nch ? off + (uint32_t)(128 * i) : kOutside, to + (uint32_t)(1024 * i));
  }
};

__device__ __forceinline__ u32x4 rd16(const char* p) { return *reinterpret_cast<const u32x4*>(p); }

// Fragment over a head's elements, chunks 2 s + half of rows ROW0 + l % 32: the lane's
// addresses for s = 0 and 1 and ROW0 = 0, and what is added for others.
template <class G>
struct RowFrag {
  uint32_t base[2];
  __device__ explicit RowFrag(int lane) {
    base[0] = (uint32_t)G::at(lane & 31, lane >> 5);
    base[1] = (uint32_t)G::at(lane & 31, 2 + (lane >> 5));
  }
  template <int ROW0, int S>
  __device__ __forceinline__ u32x4 read(const char* tile) const {
    return rd16(tile + base[S & 1] + G::at(ROW0, 2 * (S & ~1)));
  }
};

// Fragment over rows: lane l holds element 32 db + l % 32 of rows 4 half + 0 .. 3
// (and, 16-bit types, 8 + 4 half + 0 .. 3) of the KF rows from ROW0 on: the order in
// which the accumulators of a 32 x 32 product hold its rows, so that these are the
// other operand as they are.  base: the lane's addresses in even and odd blocks of rows.
template <class G>
struct ColFrag {
  uint32_t base[2];
  __device__ explicit ColFrag(int lane) {
    const int half = lane >> 5;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if constexpr (G::ES == 2)
        base[p] = (uint32_t)(G::at(8 * p + 4 * half + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) +
                             (lane & 1) * 8);
      else
        base[p] = (uint32_t)(G::at(8 * p + 4 * half, (lane & 31) >> 2) + (lane & 3) * 4);
    }
  }
  template <int ROW0, int DBLK>
  __device__ __forceinline__ u32x4 read(const char* tile) const {
    if constexpr (G::ES == 2) {
      typedef __attribute__((address_space(3))) v4i16 lds4;
      constexpr int more = G::at(ROW0, 4 * DBLK);
      const u32x2 lo = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)const_cast<char*>(tile + base[0] + more)));
      const u32x2 hi = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)const_cast<char*>(tile + base[1] + more)));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      constexpr int more = G::at(ROW0 & ~15, 8 * DBLK);
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const uint32_t*>(tile + base[(ROW0 >> 3) & 1] + more + 16 * j);
      return v;
    }
  }
};
// The KF values of a 32 x 32 block's accumulators from row ROW0 on, as an operand.
template <class E, int ROW0>
__device__ __forceinline__ u32x4 acc_frag(const f32x16& s) {
  constexpr int r = ROW0 / 2;
  if constexpr (Elt<E>::kSize == 2)
    return u32x4{pack_bf16(s[r], s[r + 1]), pack_bf16(s[r + 2], s[r + 3]), pack_bf16(s[r + 4], s[r + 5]),
                 pack_bf16(s[r + 6], s[r + 7])};
  else
    return u32x4{__float_as_uint(s[r]), __float_as_uint(s[r + 1]), __float_as_uint(s[r + 2]),
                 __float_as_uint(s[r + 3])};
}
// row of accumulator r of a block, without the lane's 4 half
__device__ __forceinline__ constexpr int acc_row(int r) { return 8 * (r >> 2) + (r & 3); }

template <int ES>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  if constexpr (ES == 2)
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
  else
    return (w & 0x7f800000u) == 0x7f800000u;
}
// A product over rows some of which hold infinities or NaN and are not seen by a
// lane's column: 0 times them would be NaN.  The product then takes the finite
// values alone (columns that see none of the others get the same bits as if those
// were finite), and mend_unfinite adds the others where they are seen.
template <int ES>
__device__ __forceinline__ u32x4 finite_only(u32x4 f) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (ES == 2)
      f[w] &= ((f[w] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((f[w] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
    else
      f[w] = (f[w] & 0x7f800000u) == 0x7f800000u ? 0u : f[w];
  }
  return f;
}
// acc += p v over those elements v of the 32 rows at `tile` that are not finite; bit x of
// `rows`: this lane's column sees row x.  Seldom run: a row at a time.
template <class E, class G>
__device__ __forceinline__ void mend_unfinite(const char* tile, uint32_t rows, const f32x16& p, f32x16* acc, int lane) {
  constexpr int ES = G::ES;
  const int half = lane >> 5;
#pragma nounroll
  for (int x = 0; x < 32; ++x) {
    bool bad = false;
    for (int ch = lane; ch < G::NCH; ch += 64) {
      const u32x4 v = rd16(tile + G::at(x, ch));
      bad = bad || not_finite<ES>(v[0]) || not_finite<ES>(v[1]) || not_finite<ES>(v[2]) || not_finite<ES>(v[3]);
    }
    if (__ballot(bad) == 0) continue;
    const int at = 4 * (x >> 3) + (x & 3);
    float px = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) px = r == at ? p[r] : px;
    px = __shfl(px, (lane & 31) + 32 * ((x >> 2) & 1));
    const bool seen = (rows >> x) & 1u;
#pragma unroll
    for (int db = 0; db < G::DB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t w[4];
        if constexpr (ES == 2) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(tile + G::at(x, 4 * db + g) + half * 8);
          w[0] = v[0] << 16, w[1] = v[0] & 0xffff0000u, w[2] = v[1] << 16, w[3] = v[1] & 0xffff0000u;
        } else {
          const u32x4 v = rd16(tile + G::at(x, 8 * db + 2 * g + half));
          w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[db][4 * g + j] = seen && not_finite<4>(w[j]) ? fmaf(px, __uint_as_float(w[j]), acc[db][4 * g + j])
                                                           : acc[db][4 * g + j];
        __builtin_amdgcn_sched_barrier(0);  // (reads in flight would take registers from the rest of the kernel)
      }
  }
}
// the first n of 32 rows
__device__ __forceinline__ uint32_t first_rows(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Whether this thread's share of `bytes` of LDS holds an infinity or NaN.
template <int ES, int BYTES, int NT>
__device__ __forceinline__ bool scan_tile(const char* p) {
  static_assert(BYTES % (16 * NT) == 0, "chunks of a tile");
  bool bad = false;
#pragma unroll
  for (int i = 0; i < BYTES / (16 * NT); ++i) {
    const u32x4 v = rd16(p + i * (16 * NT) + threadIdx.x * 16);
    bad = bad || not_finite<ES>(v[0]) || not_finite<ES>(v[1]) || not_finite<ES>(v[2]) || not_finite<ES>(v[3]);
  }
  return bad;
}

// Fragments loaded ahead of a loop have arrived: the compiler would otherwise wait
// for them inside, on a count that the loop's own loads in flight are part of.
template <int N>
__device__ __forceinline__ void arrived(u32x4 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f[i]));
}

// 16 bytes at p, or zeros
__device__ __forceinline__ u32x4 load_if(bool ok, cgchar* p) {
  return ok ? gload16(p) : u32x4{0u, 0u, 0u, 0u};
}

// DB blocks of accumulators (element 32 db + 8 g + 4 half + j of a row a lane) times
// f to the row at p.
template <class E, int DB>
__device__ __forceinline__ void store_row(gchar* p, const f32x16* acc, float f, int half, int dim, bool vec) {
  constexpr int ES = Elt<E>::kSize;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * db + 8 * g + 4 * half;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = acc[db][4 * g + j] * f;
      if (vec) {
        if (d < dim) {
          if constexpr (ES == 2)
            *(__attribute__((address_space(1))) u32x2*)(p + d * 2) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
          else
            *(__attribute__((address_space(1))) u32x4*)(p + d * 4) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                                          __float_as_uint(v[2]), __float_as_uint(v[3])};
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (d + j < dim) store_out(p, d + j, v[j], ES == 4);
      }
    }
}

// ---------------------------------------------------------------- forward, dq
// NW waves of 32 rows each.  S^T = K Q^T: a lane's column is its row of q, so that
// the softmax's maximum and sum run inside a lane (and one exchange), the
// accumulators of S^T are the second operand of O^T = V^T P^T as they lie, and
// rescaling is a factor per lane.  Keys and values come in tiles of KT, the next one
// loaded straight to LDS while one is computed.
// BWD: dq.  dP^T = V dO^T beside S^T, dQ^T = K^T dS^T in place of O^T.
// The scores of the next tile are computed beside this one's softmax and products: a wave's own
// products cover its arithmetic, 4.9 cycles an instruction against 32 of a product.  What bounds
// it then is the matrix cores at the clock that power allows, and the arithmetic that
// is left beside them (16384 tokens, 32 heads on 8 of 128, causal, bf16: 1.91 ms, 1.15 PFLOP/s; 8192
// tokens: forward 0.52 ms, dq 0.70 ms for 3 products, 1.18 PFLOP/s).  Single tokens: HBM
// (16 tokens, 53 760 keys: 48 us, 4.6 TB/s).
// NW: waves.  R: tiles of LDS, R - 1 of which are being loaded while one is computed.
template <class E, int DP, int KT, bool BWD, int NW, int R, int OCC>
__global__ void __launch_bounds__(64 * NW, OCC) attn_rows_kernel(const AttnArgs a) {
  using G = Geo<E, DP>;
  constexpr int ES = G::ES, NS = G::NS, DB = G::DB, KB = KT / 32;
  constexpr int TILE = KT * G::NCH * 16;
  constexpr int NT = 64 * NW, ROWS = 32 * NW;
  using Share = TileShare<G, KT, NW>;
  constexpr int L = Share::LOADS;
  static_assert((R & (R - 1)) == 0, "ring");
  __shared__ __attribute__((aligned(16))) char smem[2 * R * TILE];  // K, V, K, V, ..
  __shared__ int flag;  // some tile at the mask's edge holds an infinity or NaN

  AttnTile t;
  if (!attn_tile<false, 32 * NW>(a, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, lcol = lane & 31;
  if (threadIdx.x == 0) flag = 0;

  // this lane's row
  const RowBase rb = row_base(a, t.start);
  const int64_t nrows = (int64_t)t.nq * a.group - t.start;
  int token, g;
  row_of(a, rb, wave * 32 + lcol, token, g);
  const bool live = wave * 32 + lcol < nrows;
  const int head = t.head * a.group + g;
  const int64_t qtok = live ? t.q0 + token : 0;
  const int hd = live ? head : 0;
  // the last key that a row sees: of this lane, of the wave's rows and of the tile's
  const int shift = t.nk - t.nq;
  auto limit = [&](int tok) { return a.causal ? min(t.nk - 1, tok + shift) : t.nk - 1; };
  auto row_limit = [&](int x) {
    int tk_, g_;
    row_of(a, rb, (int)min((int64_t)x, nrows - 1), tk_, g_);
    return limit(__builtin_amdgcn_readfirstlane(tk_));
  };
  const int klim = live ? limit(token) : -1;
  const int kmax_wave = wave * 32 < nrows ? row_limit(wave * 32 + 31) : -1;
  const int kmin = row_limit(0);                      // seen by every row
  const int kend = row_limit(ROWS - 1) + 1;      // seen by some row
  const int ntiles = kend > 0 ? (kend + KT - 1) / KT : 0;

  // This part's tiles: part, part + P, ..; the first `nfull` are seen whole by all rows.
  const int P = a.parts, nt = ntiles > t.part ? (ntiles - t.part + P - 1) / P : 0;
  const int nwhole = max(0, min(ntiles, (kmin + 1) / KT)), nfull = nwhole > t.part ? (nwhole - t.part + P - 1) / P : 0;
  auto tile_of = [&](int i) { return t.part + i * P; };
  auto kbuf = [&](int i) { return smem + (i & (R - 1)) * 2 * TILE; };
  auto vbuf = [&](int i) { return smem + (i & (R - 1)) * 2 * TILE + TILE; };

  // this wave's share of a tile's loads
  const Share ts(wave, lane);
  const uint32_t koff = (uint32_t)(ts.row * (int)a.k.ts + ts.ch * 16), voff = (uint32_t)(ts.row * (int)a.v.ts + ts.ch * 16);
  const char* kp = (const char*)a.k.p + (int64_t)t.k0 * a.k.ts + (int64_t)t.head * a.k.hs;
  const char* vp = (const char*)a.v.p + (int64_t)t.k0 * a.v.ts + (int64_t)t.head * a.v.hs;
  const int nch = a.dim_in / G::VEC;
  // tile i of the keys, or of the values (past the last: nothing, but counted)
  auto load_half = [&](const char* base, int64_t stride, uint32_t off, int i, char* buf) {
    const int k0 = tile_of(i) * KT, rows = i < nt ? min(t.nk - k0, KT) : 0;
    const u32x4 rsrc = buffer_of(base + (i < nt ? k0 * stride : 0), (uint32_t)(rows > 0 ? (rows - 1) * (int)stride + a.dim_in * ES : 0));
#pragma unroll
    for (int x = 0; x < Share::GROUPS; ++x) ts.load(rsrc, off + (uint32_t)(8 * NW * x * (int)stride), nch, buf, x);
  };
  auto load_k = [&](int i) {
    if (ts.mine(0)) load_half(kp, a.k.ts, koff, i, kbuf(i));
  };
  auto load_v = [&](int i) {
    if (ts.mine(1)) load_half(vp, a.v.ts, voff, i, vbuf(i));
  };
  // the forward pass takes the keys a tile before the values
  if (nt > 0) {
    if constexpr (!BWD) load_k(0);
    for (int r = 0; r < R - 1; ++r) {
      load_v(r);
      load_k(BWD ? r : r + 1);
    }
  }

  // q (and dy) as the second operand: element chunks 2 s + half of the row
  u32x4 fq[NS], fdo[BWD ? NS : 1];
  {
    cgchar* p = gload_ptr(a.q.p) + qtok * a.q.ts + hd * a.q.hs;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = (2 * s + half) * G::VEC;
      fq[s] = load_if(live && d < a.dim_in, p + d * ES);
    }
  }
  const float c = a.scale * kLog2e;
  // p = exp2(s cr - ..): row_factor.  f: of the result, 1 / the row's sum or, of dq, the scale
  float cr = c, f = a.scale, lse2 = 0.0f, delta = 0.0f;
  bool no_sum = false;  // the row has no sum
  if constexpr (BWD) {
    cgchar* p = gload_ptr(a.dy.p) + qtok * a.dy.ts + hd * a.dy.hs;
    cgchar* py = gload_ptr(a.y.p) + qtok * a.y.ts + hd * a.y.hs;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = (2 * s + half) * G::VEC;
      fdo[s] = load_if(live && d < a.dim_in, p + d * ES);
      const u32x4 yv = load_if(live && d < a.dim_in, py + d * ES);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (ES == 2) {
          delta = fmaf(__uint_as_float(fdo[s][w] << 16), __uint_as_float(yv[w] << 16), delta);
          delta = fmaf(__uint_as_float(fdo[s][w] & 0xffff0000u), __uint_as_float(yv[w] & 0xffff0000u), delta);
        } else {
          delta = fmaf(__uint_as_float(fdo[s][w]), __uint_as_float(yv[w]), delta);
        }
      }
    }
    delta = half_sum(delta);
    const float l = live ? a.lse[(int64_t)hd * a.tokens_q + qtok] : 0.0f;
    // a row that sees nothing (lse -inf): its probabilities are 0
    no_sum = l == -__builtin_inff();
    lse2 = no_sum ? __builtin_inff() : l * kLog2e;
    const bool far = fabsf(l) < __builtin_inff() && fabsf(lse2) >= kFarLse;
    float mark = no_sum ? kNoSum : fabsf(lse2) < 0x1p-60f ? -0.0f : lse2, second = delta;
    if (__any(far)) {
      // the scores of all keys that the wave's rows see, from memory: seldom run
      float m = -__builtin_inff(), cm = c, sum = 0.0f;
#pragma nounroll
      for (int k0 = 0; k0 <= kmax_wave; k0 += 32) {
        cgchar* pk = gload_ptr(kp) + (int64_t)min(k0 + lcol, t.nk - 1) * a.k.ts;
        f32x16 s;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = 0.0f;
        each<NS>([&](auto x_t) {
          const int d = (2 * decltype(x_t)::value + half) * G::VEC;
          Mfma<E>::run(load_if(d < a.dim_in, pk + d * ES), fq[decltype(x_t)::value], s);
        });
        float top = m;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = k0 + acc_row(r) + 4 * half <= klim ? s[r] : -__builtin_inff();
          top = fmaxf(top, s[r]);
        }
        top = half_max(top);
        const float ct = row_factor(top, c), ref = top == -__builtin_inff() ? 0.0f : top * ct;
        sum *= row_rescale(m, cm, top, ct, c);
        m = top;
        cm = ct;
#pragma unroll
        for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(fmaf(s[r], cm, -ref));
      }
      sum = half_sum(sum);
      if (far) {
        const float ref = m * cm;
        cr = cm;
        lse2 = ref;
        f = a.scale / sum;
        mark = ldexpf(1.0f + log2f(sum) - fmaf(m, cm, -ref), -100);
        second = m;
      }
    }
    if (live && half == 0 && t.part == 0) {
      float* st = a.stats + ((int64_t)t.head * a.tokens_q + t.q0) * a.group + t.start + wave * 32 + lcol;
      st[0] = mark;
      st[a.tokens_q * a.heads] = second;
    }
  }

  arrived(fq);
  if constexpr (BWD) arrived(fdo);

  f32x16 o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[db][r] = 0.0f;
  const float slack = 8.0f / c;  // a maximum that has grown by less leaves factors below 2^8
  float m = -__builtin_inff(), l = 0.0f;
  const RowFrag<G> rf(lane);
  const ColFrag<G> cf(lane);
  constexpr int AHEAD = NS % 4 ? 3 : 4;

  // The order of instructions is given (pin): every product is followed by the LDS reads
  // of the fragment AHEAD products on and by a share of the arithmetic that does not wait
  // for it, so that a wave's own products cover them; left to the compiler the
  // reads came one product ahead and the arithmetic in one run.
  auto pin = [] { __builtin_amdgcn_sched_barrier(0); };
  auto none = [](auto) {};
  // fragment n of the score products: pair n % NS of chunks, block n / NS of 32 rows
  auto rows_at = [&](const char* tile, auto n_t) {
    constexpr int n = decltype(n_t)::value;
    return rf.template read<32 * (n / NS), n % NS>(tile);
  };
  // fragment n of the products over a tile's rows: rows KF (n / DB) on, elements 32 (n % DB) on
  auto cols_at = [&](const char* tile, auto n_t) {
    constexpr int n = decltype(n_t)::value;
    return cf.template read<G::KF * (n / DB), n % DB>(tile);
  };
  constexpr int NR = KB * NS, NC = DB * (KT / G::KF);  // fragments
  constexpr int XB = 32 / G::KF;                       // fragments of probabilities in a block
  constexpr int NX = KB * XB;                          // .. of a tile
  u32x4 fr[AHEAD], fc[AHEAD];
  // s = the score products of block kb with fb; `beside(x)` after product x.  The
  // fragments behind the block's are `then`'s.
  auto scores = [&](const char* tile, auto kb_t, const u32x4* fb, f32x16& s, auto&& beside, auto&& then) {
    constexpr int kb = decltype(kb_t)::value;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
    each<NS>([&](auto x_t) {
      constexpr int x = decltype(x_t)::value, n = kb * NS + x;
      Mfma<E>::run(fr[n % AHEAD], fb[x], s);
      if constexpr (x + AHEAD < NS)
        fr[n % AHEAD] = rows_at(tile, std::integral_constant<int, n + AHEAD>{});
      else
        then(std::integral_constant<int, x + AHEAD - NS>{}, fr[n % AHEAD]);
      beside(x_t);
      pin();
    });
  };
  static_assert(NS % AHEAD == 0, "a block's fragments start at register 0");
  // the first fragments of block kb of `tile`
  auto open_rows = [&](const char* tile, auto kb_t) {
    each<AHEAD>([&](auto n_t) {
      constexpr int n = decltype(kb_t)::value * NS + decltype(n_t)::value;
      fr[n % AHEAD] = rows_at(tile, std::integral_constant<int, n>{});
    });
    pin();
  };
  auto open_cols = [&](const char* tile) {
    each<AHEAD>([&](auto n_t) { fc[decltype(n_t)::value] = cols_at(tile, n_t); });
    pin();
  };
  // out^T += tile^T p^T, fragment x of p from `frag(x)`, `beside(n)` after product n
  auto frag_of = [&](const f32x16* p, auto x_t) {
    constexpr int x = decltype(x_t)::value;
    return acc_frag<E, (x % XB) * G::KF>(p[x / XB]);
  };
  auto gather = [&](const char* tile, auto&& frag, auto&& beside) {
    each<NX>([&](auto x_t) {
      constexpr int x = decltype(x_t)::value;
      const u32x4 fb = frag(x_t);
      pin();
      each<DB>([&](auto db_t) {
        constexpr int n = x * DB + decltype(db_t)::value;
        Mfma<E>::run(fc[n % AHEAD], fb, o[decltype(db_t)::value]);
        if constexpr (n + AHEAD < NC) fc[n % AHEAD] = cols_at(tile, std::integral_constant<int, n + AHEAD>{});
        beside(std::integral_constant<int, n>{});
        pin();
      });
    });
  };
  // Keys of a tile that not all rows see may hold what is not finite: added
  // where it is seen, then taken out of the tile.  Every wave comes here.
  auto unfinite = [&](char* tile, int j, const f32x16* p, bool mine) {
    if (scan_tile<ES, TILE, NT>(tile)) flag = 1;
    ring_barrier();
    if (flag == 0) return;
    if (mine) {
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
        mend_unfinite<E, G>(tile + kb * (4 * G::RB), first_rows(klim + 1 - j * KT - 32 * kb), p[kb], o, lane);
      });
    }
    ring_barrier();
    for (int b = threadIdx.x * 16; b < TILE; b += 16 * NT) {
      u32x4* x = (u32x4*)(tile + b);
      *x = finite_only<ES>(*x);
    }
    ring_barrier();
  };

  const bool alive = wave * 32 < nrows;  // some row of the wave exists
  int i = 0;

  if constexpr (!BWD) {
    // Scores are computed a tile ahead: the products of tile i + 1 run beside the
    // exponentials of tile i, the products with the values beside the maximum of the
    // next scores.
    float top = -__builtin_inff();
    auto rescale = [&] {
      // (a row's reference goes by its own scores alone, whatever the wave's others do)
      const bool grown = top > m + slack;
      if (__any(grown)) {
        const float mn = grown ? top : m, cn = row_factor(mn, c), f = row_rescale(m, cr, mn, cn, c);
        m = mn;
        cr = cn;
        l *= f;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[db][r] *= f;
      }
      return m == -__builtin_inff() ? 0.0f : m * cr;
    };
    auto prob = [&](f32x16* s, int v, float mc) {
      const float p = __builtin_amdgcn_exp2f(fmaf(s[v >> 4][v & 15], cr, -mc));
      s[v >> 4][v & 15] = p;
      l += p;
    };
    // scores of tile j, masked, and their maximum, nothing beside them
    auto alone = [&](int j, const char* K, f32x16* s) {
      const int seen = klim - j * KT - 4 * half;  // of this lane's accumulator rows
      top = -__builtin_inff();
      if (j * KT > kmax_wave) {
        each<KB>([&](auto kb_t) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[decltype(kb_t)::value][r] = -__builtin_inff();
        });
        return;
      }
      open_rows(K, std::integral_constant<int, 0>{});
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
        scores(K, kb_t, fq, s[kb], none, [&](auto n_t, u32x4& f) {
          if constexpr (kb + 1 < KB) f = rows_at(K, std::integral_constant<int, (kb + 1) * NS + decltype(n_t)::value>{});
        });
      });
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[kb][r] = 32 * kb + acc_row(r) <= seen ? s[kb][r] : -__builtin_inff();
          top = fmaxf(top, s[kb][r]);
        }
      });
      top = half_max(top);
    };
    // tile i's values and tile i + 1's keys have landed, for every wave; the buffers of the last
    // tile's values and this one's keys are free
    auto begin = [&](int i_) {
      wait_vmcnt<(R - 2) * L>();
      ring_barrier();
      load_v(i_ + R - 1);
      load_k(i_ + R);
    };
    // tile i, scores in sa; those of tile i + 1, which all rows see whole, to sb
    auto whole = [&](int i_, f32x16* sa, f32x16* sb) {
      constexpr int NV = 16 * KB, EARLY = NV * 3 / 4;  // probabilities, those beside the next scores
      const char *K = kbuf(i_ + 1), *V = vbuf(i_);
      const float mc = rescale();
      open_rows(K, std::integral_constant<int, 0>{});
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
        scores(K, kb_t, fq, sb[kb],
               [&](auto x_t) {
                 constexpr int n = kb * NS + decltype(x_t)::value;
#pragma unroll
                 for (int v = EARLY * n / NR; v < EARLY * (n + 1) / NR; ++v) prob(sa, v, mc);
               },
               [&](auto n_t, u32x4& f) {
                 constexpr int n = decltype(n_t)::value;
                 if constexpr (kb + 1 < KB)
                   f = rows_at(K, std::integral_constant<int, (kb + 1) * NS + n>{});
                 else
                   fc[n] = cols_at(V, n_t);
               });
      });
      float t0 = -__builtin_inff(), t1 = t0;
      gather(V, [&](auto x_t) { return frag_of(sa, x_t); }, [&](auto n_t) {
        constexpr int n = decltype(n_t)::value, before = (NX - 1) * DB, from = NC / 2;
        if constexpr (n < before) {
#pragma unroll
          for (int v = EARLY + (NV - EARLY) * n / before; v < EARLY + (NV - EARLY) * (n + 1) / before; ++v) prob(sa, v, mc);
        }
        if constexpr (n >= from) {
#pragma unroll
          for (int v = NV / 2 * (n - from) / (NC - from); v < NV / 2 * (n + 1 - from) / (NC - from); ++v) {
            t0 = fmaxf(t0, sb[v >> 4][v & 15]);
            t1 = fmaxf(t1, sb[(v + NV / 2) >> 4][(v + NV / 2) & 15]);
          }
        }
      });
      top = half_max(fmaxf(t0, t1));
    };
    f32x16 sa[KB], sb[KB];
    if (nt > 0) {
      wait_vmcnt<(R - 1) * L>();
      ring_barrier();
      alone(tile_of(0), kbuf(0), sa);
    }
    if (alive) {
      for (; i + 2 < nfull; i += 2) {
        begin(i);
        whole(i, sa, sb);
        begin(i + 1);
        whole(i + 1, sb, sa);
      }
    } else {
      for (; i + 2 < nfull; i += 2) {
        begin(i);
        begin(i + 1);
      }
    }
    for (; i < nt; ++i) {
      begin(i);
      const int j = tile_of(i);
      const bool mine = j * KT <= kmax_wave;
      if (mine) {
        const float mc = rescale();
#pragma unroll
        for (int v = 0; v < 16 * KB; ++v) prob(sa, v, mc);
      }
      if (i >= nfull) unfinite(vbuf(i), j, sa, mine);
      if (mine) {
        open_cols(vbuf(i));
        gather(vbuf(i), [&](auto x_t) { return frag_of(sa, x_t); }, none);
      }
      if (i + 1 < nt) alone(tile_of(i + 1), kbuf(i + 1), sa);
    }
  } else {
    auto begin = [&](int i_) {
      wait_vmcnt<(R - 2) * L>();
      ring_barrier();
      load_v(i_ + R - 1);
      load_k(i_ + R - 1);
    };
    // S of a block beside ds of the last one, dP beside the exponentials, the products with the
    // keys beside the last block's ds
    auto body = [&](int i_, auto edge_t) {
      constexpr bool EDGE = decltype(edge_t)::value;
      char *K = kbuf(i_), *V = vbuf(i_);
      const int j = tile_of(i_), seen = klim - j * KT - 4 * half;  // of this lane's accumulator rows
      const bool mine = !EDGE || j * KT <= kmax_wave;
      constexpr int LAST = KB - 1;
      f32x16 s[KB], dp[KB];
      u32x4 early[LAST * XB + 1];
      auto ds = [&](auto kb_t, int r) {
        constexpr int kb = decltype(kb_t)::value;
        s[kb][r] *= dp[kb][r] - delta;
        if constexpr (EDGE) s[kb][r] = 32 * kb + acc_row(r) <= seen ? s[kb][r] : 0.0f;
      };
      constexpr bool BESIDE = KB > 1 && !EDGE;  // the last block's ds
      if (mine) {
        open_rows(K, std::integral_constant<int, 0>{});
        each<KB>([&](auto kb_t) {
          constexpr int kb = decltype(kb_t)::value;
          scores(K, kb_t, fq, s[kb],
                 [&](auto x_t) {
                   constexpr int x = decltype(x_t)::value;
                   if constexpr (kb > 0) {
#pragma unroll
                     for (int r = 16 * x / NS; r < 16 * (x + 1) / NS; ++r) ds(std::integral_constant<int, kb - 1>{}, r);
                   }
                 },
                 [&](auto n_t, u32x4& f) { f = rows_at(V, std::integral_constant<int, kb * NS + decltype(n_t)::value>{}); });
          // (ds of the last block is done: as operands it takes half the registers)
          if constexpr (kb > 0 && !EDGE) {
            each<XB>([&](auto x_t) {
              constexpr int x = (kb - 1) * XB + decltype(x_t)::value;
              early[x] = frag_of(s, std::integral_constant<int, x>{});
            });
            pin();
          }
          scores(V, kb_t, fdo, dp[kb],
                 [&](auto x_t) {
                   constexpr int x = decltype(x_t)::value;
#pragma unroll
                   for (int r = 16 * x / NS; r < 16 * (x + 1) / NS; ++r)
                     s[kb][r] = __builtin_amdgcn_exp2f(fmaf(s[kb][r], cr, -lse2));
                 },
                 [&](auto n_t, u32x4& f) {
                   constexpr int n = decltype(n_t)::value;
                   if constexpr (kb + 1 < KB)
                     f = rows_at(K, std::integral_constant<int, (kb + 1) * NS + n>{});
                   else if constexpr (!EDGE)
                     fc[n] = cols_at(K, n_t);
                 });
        });
        if constexpr (!BESIDE) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            ds(std::integral_constant<int, LAST>{}, r);
            pin();
          }
        }
      }
      if constexpr (EDGE) {
        unfinite(K, j, s, mine);
        if (!mine) return;
        open_cols(K);
      }
      auto frag = [&](auto x_t) {
        constexpr int x = decltype(x_t)::value;
        if constexpr (!EDGE && x < LAST * XB)
          return early[x];
        else
          return frag_of(s, x_t);
      };
      gather(K, frag, [&](auto n_t) {
        constexpr int n = decltype(n_t)::value, over = LAST * XB * DB;
        if constexpr (BESIDE && n < over) {
#pragma unroll
          for (int r = 16 * n / over; r < 16 * (n + 1) / over; ++r) ds(std::integral_constant<int, LAST>{}, r);
        }
      });
    };
    if (alive) {
      for (; i < nfull; ++i) {
        begin(i);
        body(i, std::false_type{});
      }
    } else {
      for (; i < nfull; ++i) begin(i);
    }
    for (; i < nt; ++i) {
      begin(i);
      body(i, std::true_type{});
    }
  }

  wait_vmem();  // (nothing lands in LDS that is no longer this workgroup's)
  if (!live) return;
  if constexpr (!BWD) {
    l = half_sum(l);
    no_sum = l == 0.0f;
    f = 1.0f / l;
    // the sum relative to m itself
    const float mc = m * cr, lm = no_sum ? 0.0f : l * __builtin_amdgcn_exp2f(-fmaf(m, cr, -mc));
    const int64_t at = (int64_t)head * a.tokens_q + qtok;
    if (half == 0) {
      if (P > 1)
        a.partial_ml[(int64_t)t.part * a.heads * a.tokens_q + at] = float2{m, lm};
      else
        a.lse[at] = no_sum ? -__builtin_inff() : fmaf(m, a.scale, logf(lm));
    }
  }
  if (no_sum) {  // (its zeros may have met infinities)
    f = 0.0f;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[db][r] = 0.0f;
  }
  const int64_t row = qtok * a.heads + head;
  if (P > 1)  // fp32, for the join
    store_row<float, DB>(gstore_ptr(a.partial) + ((int64_t)t.part * a.tokens_q * a.heads + row) * DP * 4, o, f, half, DP, true);
  else
    store_row<E, DB>(gstore_ptr(a.out) + row * ((int64_t)a.dim * ES), o, f, half, a.dim, a.vec_out);
}

// ---------------------------------------------------------------- dk, dv
// NW waves of 32 keys each, q and dy in tiles of QT rows.  S = Q K^T and
// dP = dO V^T: a lane's column is its key, the accumulators of P and dS are
// the second operands of dV^T = dO^T P and dK^T = Q^T dS.  The rows of all heads that
// share the keys are walked, so that their sum needs no second pass.
// KLDS: the keys are read from LDS at every use, as the registers do not hold them
// beside the rest.
// 32 keys a wave and two waves a SIMD: the two sums take 128 of a wave's 256 registers at
// 128 wide heads, and 64 keys of a lone wave spilled.  LDS reads and products are level (a
// fragment from LDS serves one product), which bounds it (8192 tokens, 32 heads on 8 of 128,
// causal, bf16: 1.07 ms, 1.03 PFLOP/s; the join of 3 parts 39 us, 6 TB/s).
template <class E, int DP, int QT, bool KLDS, int NW, int R, int OCC>
__global__ void __launch_bounds__(64 * NW, OCC) attn_keys_kernel(const AttnArgs a) {
  using G = Geo<E, DP>;
  constexpr int ES = G::ES, NS = G::NS, DB = G::DB, QB = QT / 32;
  constexpr int TILE = QT * G::NCH * 16, STAGE = 2 * TILE + QT * 8;
  constexpr int NT = 64 * NW, KEYS = 32 * NW;
  constexpr int KBYTES = KLDS ? KEYS * G::NCH * 16 : 0;
  using Share = TileShare<G, QT, NW>;
  __shared__ __attribute__((aligned(16))) char smem[R * STAGE + KBYTES];  // q, dy, stats; R times; keys
  __shared__ int flag;
  __shared__ bool wave_marked[NW];
  __shared__ float refs[QT];  // of a tile with marked rows: their references, 0 for others

  AttnTile t;
  if (!attn_tile<true, 32 * NW>(a, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5;
  if (threadIdx.x == 0) flag = 0;
  // this lane's number, computed anew: what the loop seldom needs is not kept in
  // registers, which it has none to spare
  auto lane_now = [] {
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));
    return l;
  };
  auto key_of = [&](int l) { return (int)t.start + wave * 32 + (l & 31); };  // in its sequence
  const char* ktile = smem + R * STAGE;
  if constexpr (KLDS) {  // (they have landed when the first tile has)
    const TileShare<G, KEYS, NW> ks(wave, lane);
    const int rows = min(t.nk - (int)t.start, KEYS) - 1;
    const u32x4 rk = buffer_of((const char*)a.k.p + (t.k0 + t.start) * a.k.ts + (int64_t)t.head * a.k.hs,
                               (uint32_t)(rows * (int)a.k.ts + a.dim_in * ES));
#pragma unroll
    for (int x = 0; x < 4; ++x)
      ks.load(rk, (uint32_t)(ks.row_of_group(x) * (int)a.k.ts + ks.ch * 16), a.dim_in / G::VEC, ktile, x);
  }
  const char* kown = ktile + wave * (4 * G::RB);

  // Rows that see a key: all, or those of tokens from key - shift on.  Tiles are counted
  // from the last row back: all workgroups of a head walk the same tiles at the
  // same time, which then are in their XCD's L2 (8192 tokens: 26% of the reads miss it; from the
  // diagonal on the workgroups are at tiles of their own), and those that not all keys see come last,
  // the first one's rows before the sequence among them.
  const int shift = t.nk - t.nq;
  const int64_t nrows = (int64_t)t.nq * a.group;
  auto first = [&](int k) -> int64_t { return a.causal ? (int64_t)max(0, k - shift) * a.group : 0; };
  const int64_t row0 = min(first((int)t.start), nrows);
  const int64_t full0 = first(min((int)t.start + KEYS, t.nk) - 1);  // from here on every key is seen
  const int ntiles = (int)((nrows - row0 + QT - 1) / QT);
  const int nfull = (int)max((int64_t)0, (nrows - full0) / QT);

  const char* qp = (const char*)a.q.p + (int64_t)t.q0 * a.q.ts + (int64_t)t.head * a.group * a.q.hs;
  const char* dp_ = (const char*)a.dy.p + (int64_t)t.q0 * a.dy.ts + (int64_t)t.head * a.group * a.dy.hs;
  const float* sp = a.stats + ((int64_t)t.head * a.tokens_q + t.q0) * a.group;
  // part p of P takes tiles p, p + P, ..
  const int P = a.parts, drop = P * QT / a.group, drop_rem = P * QT % a.group;
  RowBase next = row_base(a, max((int64_t)0, nrows - (int64_t)(t.part + 1) * QT));  // of the next tile to load
  const int nch = a.dim_in / G::VEC;
  auto load_tile = [&](int j, char* buf) {
    const int lane = lane_now();
    const Share ts(wave, lane);
    const bool some_tile = j < ntiles;  // (past the last: nothing, but counted)
    const int64_t at0 = nrows - (int64_t)(j + 1) * QT, from = max((int64_t)0, at0);
    const int skip = (int)(at0 - from);  // rows of the tile before the sequence, negative
    const RowBase rb = at0 > 0 ? next : RowBase{0, 0};
    const u32x4 rq = buffer_of(qp + (int64_t)rb.token * a.q.ts, 0x7fffffffu);
    const u32x4 rd = buffer_of(dp_ + (int64_t)rb.token * a.dy.ts, 0x7fffffffu);
#pragma unroll
    for (int x = 0; x < Share::GROUPS; ++x) {
      const int r = ts.row_of_group(x) + skip;
      int tok, g;
      row_of(a, {0, rb.rem}, r, tok, g);
      const int some = some_tile && r >= 0 ? nch : 0;
      if (ts.mine(0)) ts.load(rq, (uint32_t)(tok * (int)a.q.ts + g * (int)a.q.hs + ts.ch * 16), some, buf, x);
      if (ts.mine(1)) ts.load(rd, (uint32_t)(tok * (int)a.dy.ts + g * (int)a.dy.hs + ts.ch * 16), some, buf + TILE, x);
    }
    // the rows' statistics, zeros before the sequence: by the first two waves
    if (wave < 2) {
      const u32x4 rs = buffer_of(sp + (some_tile ? from : 0) + (wave ? a.tokens_q * a.heads : 0), some_tile ? QT * 4 : 0);
      if (lane < QT) word_load(rs, (uint32_t)(skip * 4 + lane * 4), lds_at(buf + 2 * TILE + wave * QT * 4));
    }
    next.token -= drop;
    next.rem -= drop_rem;
    if (next.rem < 0) {
      next.rem += a.group;
      --next.token;
    }
  };

  // Whether some row of this workgroup's is marked: all tiles are then walked in a form that looks
  // (a look at each tile cost 2% of the time, and its code in the other forms spills: fp32 heads of 64
  // 113 -> 123 us).  Four numbers a load; the last may be of rows before row0 or, of fewer than four
  // rows, of the D behind them.  The first rows' are waited for here: kept in registers or LDS until the
  // operands have arrived they drive others out (fp32 heads of 128: 180 -> 196 us).
  const int64_t last4 = max((int64_t)0, nrows - 4);
  auto least_of = [&](int64_t r) {
    const u32x4_any4 w = *(const __attribute__((address_space(1))) u32x4_any4*)(gload_ptr(sp) + min(r, last4) * 4);
    return min(min(w[0], w[1]), min(w[2], w[3]));
  };
  constexpr int AHEAD_ROWS = 2 * 4 * NT;
  uint32_t least = ~0u, least1 = ~0u;
  if (row0 < nrows) {  // (a call of no rows has no statistics to read)
    least = least_of(row0 + 4 * threadIdx.x);
    least1 = least_of(row0 + 4 * threadIdx.x + 4 * NT);
  }

  // (the first tiles are on their way while the operands in registers arrive)
  int i = t.part, slot = 0;
  if (i < ntiles)
    for (int r = 0; r < R - 1; ++r) load_tile(i + r * P, smem + r * STAGE);
  u32x4 fk[KLDS ? 1 : NS], fv[NS];
  {
    const int key = key_of(lane);
    const bool live = key < t.nk;
    const int64_t r = t.k0 + (live ? key : 0);
    cgchar* kp = gload_ptr(a.k.p) + r * a.k.ts + t.head * a.k.hs;
    cgchar* vp = gload_ptr(a.v.p) + r * a.v.ts + t.head * a.v.hs;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = (2 * s + half) * G::VEC;
      if constexpr (!KLDS) fk[s] = load_if(live && d < a.dim_in, kp + d * ES);
      fv[s] = load_if(live && d < a.dim_in, vp + d * ES);
    }
    if constexpr (!KLDS) arrived(fk);
    arrived(fv);
  }
  least = min(least, least1);
#pragma unroll 8
  for (int64_t r = row0 + 4 * threadIdx.x + AHEAD_ROWS; r < nrows; r += 4 * NT) least = min(least, least_of(r));
  bool some = __any(least < __float_as_uint(0x1p-60f));
  if ((threadIdx.x & 63) == 0) wave_marked[wave] = some;
  ring_barrier();
#pragma unroll
  for (int w = 0; w < NW; ++w) some = some || wave_marked[w];
  const bool some_marked = __builtin_amdgcn_readfirstlane(some);

  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[db][r] = dv[db][r] = 0.0f;
  const float c = a.scale * kLog2e;
  const RowFrag<G> rf(lane);
  const ColFrag<G> cf(lane);

  // (the order of instructions is given, as for the rows' kernel)
  auto pin = [] { __builtin_amdgcn_sched_barrier(0); };
  constexpr int XB = 32 / G::KF, NX = XB * DB, AHEAD = 2;
  // Marked rows of tile j: their first number becomes log2 of the sum, their second D.  Seldom run.
  auto unmark = [&](int j, char* buf) {
    const int x = threadIdx.x;
    if (x >= QT) return;
    float *st = reinterpret_cast<float*>(buf + 2 * TILE) + x, ref = 0.0f;
    if (st[0] == kNoSum) {
      st[0] = __builtin_inff();
    } else if (row_marked(st[0])) {
      const int64_t row = nrows - (int64_t)(j + 1) * QT + x;
      const RowBase rb = row_base(a, row);
      const int64_t tok = t.q0 + rb.token, h = (int64_t)t.head * a.group + rb.rem;
      cgchar *pd = gload_ptr(a.dy.p) + tok * a.dy.ts + h * a.dy.hs, *py = gload_ptr(a.y.p) + tok * a.y.ts + h * a.y.hs;
      ref = st[QT];
      float d = 0.0f;
      for (int e = 0; e < a.dim; ++e) d = fmaf(load_out(pd, e, ES == 4), load_out(py, e, ES == 4), d);
      st[0] = ldexpf(st[0], 100) - 1.0f;
      st[QT] = d;
    }
    refs[x] = ref;
  };
  // EDGE: some rows are not seen by all keys.  MARKS: some are marked.
  auto tile_body = [&](int j, char* buf, auto edge_t, auto marks_t) {
    constexpr bool EDGE = decltype(edge_t)::value, MARKS = decltype(marks_t)::value;
    const int64_t at0 = nrows - (int64_t)(j + 1) * QT;
    const char *Q = buf, *DO = buf + TILE;
    const float* st = reinterpret_cast<const float*>(buf + 2 * TILE);
    bool guard = false;
    uint64_t no_sum = 0;  // bit x: row x has none
    // this lane's key sees the tile's rows from `lo` on
    const int key = EDGE ? key_of(lane_now()) : 0;
    const int64_t mine = EDGE && key < t.nk ? first(key) : nrows;
    const int lo = (int)max((int64_t)0, min(mine - at0, (int64_t)QT));
    if constexpr (EDGE) {
      if (scan_tile<ES, 2 * TILE, NT>(Q)) flag = 1;
      if constexpr (MARKS) {
        no_sum = __ballot(st[lane_now() & (QT - 1)] == kNoSum);
        ring_barrier();  // every wave has seen the marks
        unmark(j, buf);
      }
      ring_barrier();
      guard = flag != 0;
    }
#pragma nounroll
    for (int qb = 0; qb < QB; ++qb) {
      const char *q32 = Q + qb * (4 * G::RB), *d32 = DO + qb * (4 * G::RB);
      const float* st32 = st + 32 * qb + 4 * half;
      // bit x: row x of the 32 is seen; `own`: of this half's accumulators
      const uint32_t rows = EDGE ? ~(first_rows(lo - 32 * qb) | (uint32_t)(no_sum >> (32 * qb))) : ~0u, own = rows >> (4 * half);
      f32x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
      u32x4 f[AHEAD], fkl[KLDS ? AHEAD : 1];
      // fragment n: of S, of dP, of dV (rows KF at a time, then elements), of dK
      auto frag = [&](auto n_t) {
        constexpr int n = decltype(n_t)::value;
        if constexpr (n < NS) return rf.template read<0, n>(q32);
        else if constexpr (n < 2 * NS) return rf.template read<0, n - NS>(d32);
        else if constexpr (n < 2 * NS + NX) return cf.template read<G::KF * ((n - 2 * NS) / DB), (n - 2 * NS) % DB>(d32);
        else return cf.template read<G::KF * ((n - 2 * NS - NX) / DB), (n - 2 * NS - NX) % DB>(q32);
      };
      auto step = [&](auto n_t, const u32x4& fb, f32x16& acc, auto&& beside) {
        constexpr int n = decltype(n_t)::value;
        Mfma<E>::run(f[n % AHEAD], fb, acc);
        if constexpr (n + AHEAD < 2 * (NS + NX)) f[n % AHEAD] = frag(std::integral_constant<int, n + AHEAD>{});
        beside();
        pin();
      };
      // lse, or D, of accumulator rows 4 g .. 4 g + 3
      float4 st4;
      auto stats = [&](int which, int g) { st4 = *reinterpret_cast<const float4*>(st32 + which * QT + 8 * g); };
      auto stat = [&](int i) { return i == 0 ? st4.x : i == 1 ? st4.y : i == 2 ? st4.z : st4.w; };
      each<AHEAD>([&](auto n_t) {
        constexpr int n = decltype(n_t)::value;
        f[n] = frag(n_t);
        if constexpr (KLDS) fkl[n] = rf.template read<0, n>(kown);
      });
      pin();
      each<NS>([&](auto x_t) {
        constexpr int x = decltype(x_t)::value;
        if constexpr (KLDS) {
          step(x_t, fkl[x % AHEAD], s, [&] {
            if constexpr (x + AHEAD < NS) fkl[x % AHEAD] = rf.template read<0, x + AHEAD>(kown);
          });
        } else {
          step(x_t, fk[x], s, [] {});
        }
      });
      if constexpr (MARKS) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {  // (s - m <= 0 is known: the sums here may be rounded in another order)
          const float ref = refs[32 * qb + 4 * half + acc_row(r)];
          s[r] = ref != 0.0f ? fminf(s[r] - ref, 0.0f) : s[r];
        }
      }
      // dP beside the probabilities
      stats(0, 0);
      each<NS>([&](auto x_t) {
        constexpr int x = decltype(x_t)::value;
        step(std::integral_constant<int, NS + x>{}, fv[x], dp, [&] {
#pragma unroll
          for (int r = 16 * x / NS; r < 16 * (x + 1) / NS; ++r) {
            s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -stat(r & 3)));
            if ((r & 3) == 3) stats(r == 15, r == 15 ? 0 : r / 4 + 1);
            if constexpr (EDGE)  // (a comparison's result would take two scalar registers for each)
              s[r] = __uint_as_float(__float_as_uint(s[r]) & (uint32_t)__builtin_amdgcn_sbfe((int)own, acc_row(r), 1));
          }
        });
      });
      auto ds = [&](int r) {
        dp[r] = s[r] * (dp[r] - stat(r & 3));
        if ((r & 3) == 3 && r < 15) stats(1, r / 4 + 1);
        if constexpr (EDGE)
          dp[r] = __uint_as_float(__float_as_uint(dp[r]) & (uint32_t)__builtin_amdgcn_sbfe((int)own, acc_row(r), 1));
      };
      if constexpr (EDGE) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          ds(r);
          pin();
        }
        if (guard) {
          // what is not finite first; the products then meet finite values only
          mend_unfinite<E, G>(d32, rows, s, dv, lane);
          mend_unfinite<E, G>(q32, rows, dp, dk, lane);
          ring_barrier();
          for (int b = threadIdx.x * 16; b < 4 * G::RB; b += 16 * NT) {
            u32x4 *x = (u32x4*)(const_cast<char*>(q32) + b), *y = (u32x4*)(const_cast<char*>(d32) + b);
            *x = finite_only<ES>(*x);
            *y = finite_only<ES>(*y);
          }
          ring_barrier();
          each<AHEAD>([&](auto n_t) {
            constexpr int n = 2 * NS + decltype(n_t)::value;
            f[n % AHEAD] = frag(std::integral_constant<int, n>{});
          });
        }
      }
      // dV beside ds, then dK
      each<XB>([&](auto x_t) {
        constexpr int x = decltype(x_t)::value;
        const u32x4 fp = acc_frag<E, x * G::KF>(s);
        pin();
        each<DB>([&](auto db_t) {
          constexpr int at = x * DB + decltype(db_t)::value;
          step(std::integral_constant<int, 2 * NS + at>{}, fp, dv[decltype(db_t)::value], [&] {
#pragma unroll
            for (int r = 16 * at / NX; r < 16 * (at + 1) / NX; ++r)
              if constexpr (!EDGE) ds(r);
          });
        });
      });
      each<XB>([&](auto x_t) {
        constexpr int x = decltype(x_t)::value;
        const u32x4 fs = acc_frag<E, x * G::KF>(dp);
        pin();
        each<DB>([&](auto db_t) {
          constexpr int at = x * DB + decltype(db_t)::value;
          step(std::integral_constant<int, 2 * NS + NX + at>{}, fs, dk[decltype(db_t)::value], [] {});
        });
      });
    }
  };


  auto begin = [&] {
    if (wave < 2)
      wait_vmcnt<(R - 2) * (Share::LOADS + 1)>();
    else
      wait_vmcnt<(R - 2) * Share::LOADS>();
    ring_barrier();
    load_tile(i + (R - 1) * P, smem + (slot ? slot - 1 : R - 1) * STAGE);
  };
  auto walk = [&](int end, auto edge_t, auto marks_t) {
    while (i < end) {
      begin();
      tile_body(i, smem + slot * STAGE, edge_t, marks_t);
      i += P;
      slot = slot + 1 < R ? slot + 1 : 0;
    }
  };
  if (some_marked) {
    walk(ntiles, std::true_type{}, std::true_type{});
  } else {
    walk(min(nfull, ntiles), std::false_type{}, std::false_type{});
    walk(ntiles, std::true_type{}, std::false_type{});
  }

  wait_vmem();  // (nothing lands in LDS that is no longer this workgroup's)
  const int key = key_of(lane_now());
  if (key >= t.nk) return;
  const int64_t row = (int64_t)(t.k0 + key) * a.kv_heads + t.head;
  if (P > 1) {  // fp32, for attn_join_kernel
    const int64_t n = a.tokens_k * a.kv_heads, at = (int64_t)t.part * 2 * n;
    store_row<float, DB>(gstore_ptr(a.partial) + (at + row) * DP * 4, dk, a.scale, half, DP, true);
    store_row<float, DB>(gstore_ptr(a.partial) + (at + n + row) * DP * 4, dv, 1.0f, half, DP, true);
  } else {
    const int64_t at = row * ((int64_t)a.dim * ES);
    store_row<E, DB>(gstore_ptr(a.dk) + at, dk, a.scale, half, a.dim, a.vec_out);
    store_row<E, DB>(gstore_ptr(a.dv) + at, dv, 1.0f, half, a.dim, a.vec_out);
  }
}

// Four consecutive elements of a result's row.
template <int ES>
__device__ __forceinline__ void store4(gchar* out, int d, int dim, bool vec, const float* v) {
  if (vec) {
    if constexpr (ES == 2)
      *(__attribute__((address_space(1))) u32x2*)(out + d * 2) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else
      *(__attribute__((address_space(1))) u32x4*)(out + d * 4) =
          u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (d + k < dim) store_out(out, d + k, v[k], ES == 4);
  }
}

// The parts of a result put together, in order: dq, or dk and dv, are their sum; y is their
// mean weighted with l exp(scale (m - M)), m and l a part's reference and sum, M the largest m.  (Their
// logarithms would lose l where the scores are large.)  U parts' loads are issued together
// (those past the last read the last again), as each alone waits for memory (16 parts
// of 32 rows of 128: 15 -> 7 us).
template <class E, int DP, AttnPass PASS, int U>
__device__ __forceinline__ void join_rows(const AttnArgs& a) {
  constexpr int ES = Elt<E>::kSize, C = DP / 4;  // four elements a thread
  const bool keys = PASS == ATTN_JOIN_KEYS;
  const int64_t n = keys ? a.tokens_k * a.kv_heads : a.tokens_q * a.heads, rows = keys ? 2 * n : n;
  const int P = a.parts;
  const float c = a.scale * kLog2e;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * C; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / C;
    const int d = (int)(i - row * C) * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, top = -__builtin_inff(), sum = 0.0f;
    const int64_t tok = row / a.heads, at = (row - tok * a.heads) * a.tokens_q + tok;  // of lse
    if constexpr (PASS == ATTN_JOIN_FWD) {
      for (int p = 0; p < P; p += U) {
        float m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) m[u] = a.partial_ml[min(p + u, P - 1) * n + at].x;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
      }
    }
    const float base = top == -__builtin_inff() ? 0.0f : top;
    for (int p = 0; p < P; p += U) {
      u32x4 x[U];
      float2 ml[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t part = min(p + u, P - 1);
        if constexpr (PASS == ATTN_JOIN_FWD) ml[u] = a.partial_ml[part * n + at];
        x[u] = gload16(gload_ptr(a.partial) + (part * rows * DP + row * DP + d) * 4);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // (a part that the row sees nothing of; one whose weight is merely too small for fp32 counts, as a
        // NaN of its values does in a call of one part)
        bool out = p + u >= P;
        float w = 1.0f;
        if constexpr (PASS == ATTN_JOIN_FWD) {
          out = out || ml[u].y == 0.0f;
          w = ml[u].y * __builtin_amdgcn_exp2f((ml[u].x - base) * c);
        }
        sum += out ? 0.0f : w;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = out ? v[k] : fmaf(w, __uint_as_float(x[u][k]), v[k]);
      }
    }
    if constexpr (PASS == ATTN_JOIN_FWD) {
      if (d == 0) a.lse[at] = sum == 0.0f ? -__builtin_inff() : fmaf(top, a.scale, logf(sum));
      const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] *= f;
    }
    if (d >= a.dim) continue;
    void* out = !keys ? a.out : row < n ? a.dk : a.dv;
    store4<ES>(gstore_ptr(out) + (keys && row >= n ? row - n : row) * a.dim * ES, d, a.dim, a.vec_out, v);
  }
}
template <class E, int DP, AttnPass PASS>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
  if (a.parts <= 2)
    join_rows<E, DP, PASS, 2>(a);
  else if (a.parts == 3)
    join_rows<E, DP, PASS, 3>(a);
  else
    join_rows<E, DP, PASS, 8>(a);
}

template <class F>
hipError_t launch_units(const AttnArgs& a, int64_t grid, int threads, F&& f) {
  const int64_t most = (int64_t)1 << 21;  // a launch's threads have to be fewer than 2^32
  for (int64_t u = 0; u < grid; u += most) {
    AttnArgs b = a;
    b.unit0 = (uint32_t)u;
    f(b, dim3((unsigned)std::min(most, grid - u)), dim3(threads));
  }
  return hipGetLastError();
}
// Of a wide call (a.wide) eight waves share a tile, with deeper rings; W: built for such.
// FR, QR, KR: rings of the forward pass, of dq, of dk and dv; FO, QO, KO: workgroups on a compute unit;
// W..: of a wide call.
template <class E, int DP, int KT, int QT, int FR, int FO, int QR, int QO, int KR, int KO, bool KLDS, bool W, int WR,
          int WKR, bool WKLDS>
hipError_t launch_attn(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
#define ATTN_LAUNCH(nw, ...)                                                                  \
  return launch_units(a, grid, 64 * nw, [&](const AttnArgs& b, dim3 g, dim3 n) {             \
    hipLaunchKernelGGL((__VA_ARGS__), g, n, 0, st, b);                                        \
  })
  if constexpr (W) {
    if (a.wide && pass == ATTN_FWD) ATTN_LAUNCH(8, attn_rows_kernel<E, DP, KT, false, 8, WR, 2>);
    if (a.wide && pass == ATTN_DQ) ATTN_LAUNCH(8, attn_rows_kernel<E, DP, KT, true, 8, WR, 2>);
    if (a.wide && pass == ATTN_DKV) ATTN_LAUNCH(8, attn_keys_kernel<E, DP, 32, WKLDS, 8, WKR, 2>);
  }
  switch (pass) {
    case ATTN_FWD: ATTN_LAUNCH(4, attn_rows_kernel<E, DP, KT, false, 4, FR, FO>);
    case ATTN_DQ: ATTN_LAUNCH(4, attn_rows_kernel<E, DP, KT, true, 4, QR, QO>);
    case ATTN_DKV: ATTN_LAUNCH(4, attn_keys_kernel<E, DP, QT, KLDS, 4, KR, KO>);
    case ATTN_JOIN_FWD: ATTN_LAUNCH(4, attn_join_kernel<E, DP, ATTN_JOIN_FWD>);
    case ATTN_JOIN_DQ: ATTN_LAUNCH(4, attn_join_kernel<E, DP, ATTN_JOIN_DQ>);
    case ATTN_JOIN_KEYS: ATTN_LAUNCH(4, attn_join_kernel<E, DP, ATTN_JOIN_KEYS>);
  }
#undef ATTN_LAUNCH
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace dmuon
