// Attention over packed sequences with grouped heads, forward and backward, on
// gfx950 MFMA.
//
//   s_ij = scale q_i . k_j  for the keys j that row i sees (all of its sequence,
//          or j <= i + keys - queries when causal),
//   p = softmax over j,  y_i = sum_j p_ij v_j,  lse_i = log sum_j exp(s_ij)
//   D_i = dy_i . y_i,  ds_ij = p_ij (dy_i . v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dy_i
#pragma once

#include "attention.h"
#include "gemm_impl.h"

namespace dmuon {
namespace {

typedef __attribute__((address_space(3))) char lds_char;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// ---------------------------------------------------------------- the work
// One workgroup's tile: rows [start, start + 128) of a sequence's query rows
// (token-major: the `group` heads that share a key head are consecutive rows of
// a token), or its keys from `start`.
struct AttnTile {
  int head;            // key head
  int q0, nq, k0, nk;  // the sequence's first rows and lengths
  int64_t start;
};

// Boundary i of a list of first rows, kept inside the rows that exist whatever
// the list holds.  -1 and n + 1: the ends of the tensor; what lies before the
// first and behind the last sequence is a sequence that meets nothing.
__device__ __forceinline__ int attn_edge(const int32_t* cu, int i, int n, int rows) {
  return i < 0 ? 0 : i > n ? rows : min(max(cu[i], 0), rows);
}

// Unit (tile slot, key head) of this workgroup.  Workgroups go round-robin over
// the 8 XCDs: each takes heads of its own, whose keys and values stay in its L2,
// as far as they divide by 8; tiles of the others are dealt to all.  Tiles of a
// causal sequence come in the order of their work, the largest first.
template <bool KEYS>
__device__ __forceinline__ bool attn_tile(const AttnArgs& a, AttnTile& t) {
  const int64_t b = a.unit0 + blockIdx.x;
  const int64_t own = (int64_t)(a.kv_heads >> 3) * a.slots, j = b >> 3;
  const int xcd = (int)(b & 7);
  int64_t slot;
  if (j < own) {
    t.head = xcd * (a.kv_heads >> 3) + (int)(j / a.slots);
    slot = j % a.slots;
  } else {
    const int64_t u = (j - own) * 8 + xcd;
    const int64_t h = u / a.slots;
    if (h >= (a.kv_heads & 7)) return false;
    t.head = (a.kv_heads & ~7) + (int)h;
    slot = u % a.slots;
  }
  const int per = KEYS ? kAttnKeys : kAttnRows;
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
    const int32_t* cu = KEYS ? a.cu_k : a.cu_q;
    const int rows = (int)(KEYS ? a.tokens_k : a.tokens_q);
    int64_t before = 0;
    int seg = -1;
    for (int base = 0; base <= n + 1; base += 64) {
      const int s = base + lane;
      int64_t c = 0;
      if (s <= n + 1) {
        const int lo = attn_edge(cu, s - 1, n, rows), hi = attn_edge(cu, s, n, rows);
        c = hi > lo ? ((hi - lo) * mult + per - 1) / per : 0;
      }
      int64_t incl = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int64_t up = __shfl_up(incl, o);
        if (lane >= o) incl += up;
      }
      const uint64_t hit = __ballot(before + incl > slot);
      if (hit) {
        const int f = __builtin_ctzll(hit);
        seg = base + f;
        tiles = __shfl(c, f);
        tile = slot - (before + __shfl(incl, f) - tiles);
        break;
      }
      before += __shfl(incl, 63);
    }
    if (seg < 0) return false;
    const bool real = seg >= 1 && seg <= n;
    const int lo = attn_edge(cu, seg - 1, n, rows), len = max(attn_edge(cu, seg, n, rows) - lo, 0);
    const int32_t* other = KEYS ? a.cu_q : a.cu_k;
    const int rows2 = (int)(KEYS ? a.tokens_q : a.tokens_k);
    const int lo2 = real ? attn_edge(other, seg - 1, n, rows2) : 0;
    const int len2 = real ? max(attn_edge(other, seg, n, rows2) - lo2, 0) : 0;
    t.q0 = KEYS ? lo2 : lo;
    t.nq = KEYS ? len2 : len;
    t.k0 = KEYS ? lo : lo2;
    t.nk = KEYS ? len : len2;
  }
  if (!KEYS && a.causal) tile = tiles - 1 - tile;
  // the same in all lanes: into scalar registers
  auto uni = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  t.head = uni(t.head);
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
// ROWS rows of a head, DP elements each, one behind the other; the 16-byte chunks of
// a row lie swizzled, so that neither 8 consecutive rows read at one chunk nor 4
// consecutive rows read at one pair of chunks (a transposing read) meet in a bank.
template <class E, int DP>
struct Geo {
  static constexpr int ES = Elt<E>::kSize, VEC = 16 / ES;
  static constexpr int NCH = DP / VEC;                                       // chunks of a row
  static constexpr int PC = NCH <= 8 ? 8 : NCH <= 16 ? 16 : NCH <= 32 ? 32 : 64;  // its pitch
  static constexpr int ROWB = PC * 16;
  static constexpr int NS = NCH / 2;   // pairs of chunks: steps of a sum over the head's elements
  static constexpr int DB = DP / 32;   // blocks of 32 elements
  static constexpr int KF = 8 * VEC / 4;  // rows that a fragment over rows holds (both halves): 16 or 8
  static constexpr int HI = PC >= 16 ? 8 : 0;
  __device__ static constexpr int swz(int r) { return ((r & 3) << 1) | ((r >> 2) & 1) | (r & HI); }
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
constexpr uint32_t kOutside = 0x80000000u;  // past the end of any of these buffers

__device__ __forceinline__ uint32_t lds_at(const char* p) { return (uint32_t)(uintptr_t)(lds_char*)const_cast<char*>(p); }

// fragment over a head's elements: pair s of chunks of row `base` is for
// (`base` from row_frag)
template <class G>
__device__ __forceinline__ uint32_t row_frag(int r, int half) {
  return (uint32_t)(r * G::ROWB + ((half ^ G::swz(r)) << 4));
}
__device__ __forceinline__ u32x4 rd16(const char* p) { return *reinterpret_cast<const u32x4*>(p); }

// Fragment over rows: lane l holds element 32 db + l % 32 of rows 4 half + 0 .. 3
// (and, 16-bit types, 8 + 4 half + 0 .. 3) of the KF rows from row 0 on: the order in
// which the accumulators of a 32 x 32 product hold its rows, so that these are the
// other operand as they are.  col_frag: the lane's address for db = 0.
template <class G>
__device__ __forceinline__ uint32_t col_frag(int lane) {
  const int half = lane >> 5;
  if constexpr (G::ES == 2) {
    const int q = (lane & 15) >> 2, r = 4 * half + q;
    const int ch = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    return (uint32_t)(r * G::ROWB + ((ch ^ G::swz(r)) << 4) + (lane & 1) * 8);
  } else {
    return (uint32_t)(4 * half * G::ROWB + ((((lane & 31) >> 2) ^ half) << 4) + (lane & 3) * 4);
  }
}
// rows from `row0` (a multiple of KF)
template <class G, int ROW0, int DBLK>
__device__ __forceinline__ u32x4 rd_cols(const char* tile, uint32_t base) {
  if constexpr (G::ES == 2) {
    typedef __attribute__((address_space(3))) v4i16 lds4;
    constexpr uint32_t x = DBLK * 64, y = (DBLK * 64) ^ (G::HI * 16);
    const char* p = tile + (base ^ x) + ROW0 * G::ROWB;
    const char* q = tile + (base ^ y) + (ROW0 + 8) * G::ROWB;
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)const_cast<char*>(p)));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)const_cast<char*>(q)));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  } else {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = (uint32_t)((8 * DBLK) ^ (j << 1) ^ (ROW0 & G::HI)) << 4;
      v[j] = *reinterpret_cast<const uint32_t*>(tile + (base ^ x) + (ROW0 + j) * G::ROWB);
    }
    return v;
  }
}
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

// A product over rows some of which hold infinities or NaN and are not seen by this
// lane's column: 0 times them would be NaN.  The finite values as ever (columns that
// see none of the others get the same bits as if those were finite); then the others,
// a row at a time, kept where the row is seen.  `seen(x)`: for row x of the fragment.
template <class E, class F>
__device__ __forceinline__ void guarded(const u32x4& fa, const u32x4& fb, f32x16& acc, int half, F&& seen) {
  constexpr bool B16 = Elt<E>::kSize == 2;
  u32x4 fin, bad;
  uint32_t any = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t m = 0;
    if constexpr (B16) {
      m = ((fa[w] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((fa[w] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
    } else {
      m = (fa[w] & 0x7f800000u) == 0x7f800000u ? 0xffffffffu : 0u;
    }
    fin[w] = fa[w] & ~m;
    bad[w] = fa[w] & m;
    any |= m;
  }
  Mfma<E>::run(fin, fb, acc);
  if (__ballot(any != 0) == 0) return;
  constexpr int KF = B16 ? 16 : 8;
  for (int x = 0; x < KF; ++x) {
    const bool mine = ((x >> 2) & 1) == half;
    const int e = (x & 3) + 4 * (x >> 3);
    u32x4 one;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (B16)
        one[w] = mine && (e >> 1) == w ? bad[w] & ((e & 1) ? 0xffff0000u : 0xffffu) : 0u;
      else
        one[w] = mine && e == w ? bad[w] : 0u;
    }
    f32x16 next = acc;
    Mfma<E>::run(one, fb, next);
    const bool s = seen(x);
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = s ? next[r] : acc[r];
  }
}

template <int ES>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  if constexpr (ES == 2)
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
  else
    return (w & 0x7f800000u) == 0x7f800000u;
}
// Whether this thread's share of `bytes` of LDS holds an infinity or NaN.
template <int ES, int BYTES>
__device__ __forceinline__ bool scan_tile(const char* p) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < BYTES / 4096; ++i) {
    const u32x4 v = rd16(p + i * 4096 + threadIdx.x * 16);
    bad = bad || not_finite<ES>(v[0]) || not_finite<ES>(v[1]) || not_finite<ES>(v[2]) || not_finite<ES>(v[3]);
  }
  return bad;
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
// Four waves of 32 rows each.  S^T = K Q^T: a lane's column is its row of q, so that
// the softmax's maximum and sum run inside a lane (and one exchange), the
// accumulators of S^T are the second operand of O^T = V^T P^T as they lie, and
// rescaling is a factor per lane.  Keys and values come in tiles of KT, the next one
// loaded straight to LDS while one is computed.
// BWD: dq.  dP^T = V dO^T beside S^T, dQ^T = K^T dS^T in place of O^T.
template <class E, int DP, int KT, bool BWD>
struct RowKernel {
  using G = Geo<E, DP>;
  static constexpr int ES = G::ES, NS = G::NS, DB = G::DB, KB = KT / 32;
  static constexpr int TILE = KT * G::ROWB;
  static constexpr int LPT = TILE / 4096;  // load instructions of a wave
  static constexpr int LDS = 4 * TILE + 16;
};

template <class E, int DP, int KT, bool BWD, int OCC>
__global__ void __launch_bounds__(256, OCC) attn_rows_kernel(const AttnArgs a) {
  using R = RowKernel<E, DP, KT, BWD>;
  using G = typename R::G;
  constexpr int ES = R::ES, NS = R::NS, DB = R::DB, KB = R::KB, TILE = R::TILE, LPT = R::LPT;
  __shared__ __attribute__((aligned(16))) char smem[4 * TILE];  // K, V, K, V
  __shared__ int flag;  // some tile at the mask's edge holds an infinity or NaN

  AttnTile t;
  if (!attn_tile<false>(a, t)) return;
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
  const int kend = row_limit(kAttnRows - 1) + 1;      // seen by some row
  const int ntiles = kend > 0 ? (kend + KT - 1) / KT : 0;

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
  float lse2 = 0.0f, delta = 0.0f;
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
    lse2 = l == -__builtin_inff() ? __builtin_inff() : l * kLog2e;
    if (live && half == 0)
      a.stats[((int64_t)t.head * a.tokens_q + t.q0) * a.group + t.start + wave * 32 + lcol] = float2{lse2, delta};
  }

  // this lane's share of a tile's loads
  uint32_t koff[LPT], voff[LPT];
#pragma unroll
  for (int i = 0; i < LPT; ++i) {
    const int at = (wave * LPT + i) * 1024 + lane * 16;
    const int r = at / G::ROWB, ch = ((at % G::ROWB) >> 4) ^ G::swz(r);
    const bool in = ch * G::VEC < a.dim_in;
    koff[i] = in ? (uint32_t)(r * (int)a.k.ts + ch * 16) : kOutside;
    voff[i] = in ? (uint32_t)(r * (int)a.v.ts + ch * 16) : kOutside;
  }
  const char* kp = (const char*)a.k.p + (int64_t)t.k0 * a.k.ts + (int64_t)t.head * a.k.hs;
  const char* vp = (const char*)a.v.p + (int64_t)t.k0 * a.v.ts + (int64_t)t.head * a.v.hs;
  auto load_tile = [&](int j, char* buf) {
    const int k0 = j * KT, rows = min(t.nk - k0, KT) - 1;
    const u32x4 rk = buffer_of(kp + (int64_t)k0 * a.k.ts, (uint32_t)(rows * (int)a.k.ts + a.dim_in * ES));
    const u32x4 rv = buffer_of(vp + (int64_t)k0 * a.v.ts, (uint32_t)(rows * (int)a.v.ts + a.dim_in * ES));
#pragma unroll
    for (int i = 0; i < LPT; ++i) tile_load(rk, koff[i], lds_at(buf + (wave * LPT + i) * 1024));
#pragma unroll
    for (int i = 0; i < LPT; ++i) tile_load(rv, voff[i], lds_at(buf + TILE + (wave * LPT + i) * 1024));
  };

  f32x16 o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[db][r] = 0.0f;
  const float c = a.scale * kLog2e;
  const float slack = 8.0f / c;  // a maximum that has grown by less leaves factors below 2^8
  float m = -__builtin_inff(), l = 0.0f;
  const uint32_t rf = row_frag<G>(lcol, half), cf = col_frag<G>(lane);

  // S^T or dP^T of 32 keys
  auto scores = [&](const char* tile, int kb, const u32x4* fb) {
    f32x16 s;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
#pragma unroll
    for (int x = 0; x < NS; ++x) Mfma<E>::run(rd16(tile + (rf ^ (uint32_t)(x * 32)) + kb * 32 * G::ROWB), fb[x], s);
    return s;
  };
  // out^T += (rows of `tile`)^T p^T for the 32 keys of block KBLK
  auto gather = [&](const char* tile, auto kb_t, const f32x16& p, bool guard, int k0) {
    constexpr int kb = decltype(kb_t)::value;
    each<32 / G::KF>([&](auto x_t) {
      constexpr int x = decltype(x_t)::value, row0 = kb * 32 + x * G::KF;
      const u32x4 fb = acc_frag<E, x * G::KF>(p);
      each<DB>([&](auto db_t) {
        constexpr int db = decltype(db_t)::value;
        const u32x4 fa = rd_cols<G, row0, db>(tile, cf);
        if (guard)
          guarded<E>(fa, fb, o[db], half, [&](int y) { return k0 + row0 + y <= klim; });
        else
          Mfma<E>::run(fa, fb, o[db]);
      });
    });
  };
  auto tile_body = [&](int j, const char* buf, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const int k0 = j * KT;
    const char *K = buf, *V = buf + TILE;
    bool guard = false;
    if constexpr (EDGE) {
      if (scan_tile<ES, TILE>(BWD ? K : V)) flag = 1;
      ring_barrier();
      guard = flag != 0;
      if (k0 > kmax_wave) return;
    }
    const int seen = klim - k0 - 4 * half;  // of this lane's accumulator rows
    if constexpr (!BWD) {
      f32x16 s[KB];
      float top = -__builtin_inff();
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
        s[kb] = scores(K, kb, fq);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if constexpr (EDGE) s[kb][r] = 32 * kb + acc_row(r) <= seen ? s[kb][r] : -__builtin_inff();
          top = fmaxf(top, s[kb][r]);
        }
      });
      top = half_max(top);
      // (a row's reference goes by its own scores alone, whatever the wave's others do)
      const bool grown = top > m + slack;
      if (__any(grown)) {
        const float mn = grown ? top : m, base = mn == -__builtin_inff() ? 0.0f : mn;
        const float f = __builtin_amdgcn_exp2f((m - base) * c);
        m = mn;
        l *= f;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[db][r] *= f;
      }
      const float mc = m == -__builtin_inff() ? 0.0f : m * c;
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[kb][r] = __builtin_amdgcn_exp2f(fmaf(s[kb][r], c, -mc));
          l += s[kb][r];
        }
        gather(V, kb_t, s[kb], guard, k0);
      });
    } else {
      each<KB>([&](auto kb_t) {
        constexpr int kb = decltype(kb_t)::value;
        f32x16 s = scores(K, kb, fq);
        const f32x16 dp = scores(V, kb, fdo);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
          if constexpr (EDGE) s[r] = 32 * kb + acc_row(r) <= seen ? s[r] : 0.0f;
        }
        gather(K, kb_t, s, guard, k0);
      });
    }
  };

  if (ntiles > 0) load_tile(0, smem);
  int j = 0;
  auto begin = [&](int j_) {
    wait_vmem();
    ring_barrier();
    if (j_ + 1 < ntiles) load_tile(j_ + 1, smem + ((j_ + 1) & 1) * 2 * TILE);
  };
  const int nfull = min(ntiles, (kmin + 1) / KT);
  for (; j < nfull; ++j) {
    begin(j);
    tile_body(j, smem + (j & 1) * 2 * TILE, std::false_type{});
  }
  for (; j < ntiles; ++j) {
    begin(j);
    tile_body(j, smem + (j & 1) * 2 * TILE, std::true_type{});
  }

  if (!live) return;
  gchar* p = gstore_ptr(a.out) + (qtok * a.heads + head) * ((int64_t)a.dim * ES);
  if constexpr (BWD) {
    store_row<E, DB>(p, o, a.scale, half, a.dim, a.vec_out);
  } else {
    l = half_sum(l);
    store_row<E, DB>(p, o, l == 0.0f ? 0.0f : 1.0f / l, half, a.dim, a.vec_out);
    if (half == 0)
      a.lse[(int64_t)head * a.tokens_q + qtok] = l == 0.0f ? -__builtin_inff() : fmaf(m, a.scale, logf(l));
  }
}

// ---------------------------------------------------------------- dk, dv
// Four waves of 32 keys each, q and dy in tiles of QT rows.  S = Q K^T and
// dP = dO V^T: a lane's column is its key, the accumulators of P and dS are
// the second operands of dV^T = dO^T P and dK^T = Q^T dS.  The rows of all heads that
// share the keys are walked, so that their sum needs no second pass.
template <class E, int DP, int QT, int OCC>
__global__ void __launch_bounds__(256, OCC) attn_keys_kernel(const AttnArgs a) {
  using G = Geo<E, DP>;
  constexpr int ES = G::ES, NS = G::NS, DB = G::DB, QB = QT / 32;
  constexpr int TILE = QT * G::ROWB, LPT = TILE / 4096, STAGE = 2 * TILE + QT * 8;
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];  // q, dy, stats; twice
  __shared__ int flag;

  AttnTile t;
  if (!attn_tile<true>(a, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, lcol = lane & 31;
  if (threadIdx.x == 0) flag = 0;

  const int key = (int)t.start + wave * 32 + lcol;  // in its sequence
  const bool live = key < t.nk;
  u32x4 fk[NS], fv[NS];
  {
    const int64_t r = t.k0 + (live ? key : 0);
    cgchar* kp = gload_ptr(a.k.p) + r * a.k.ts + t.head * a.k.hs;
    cgchar* vp = gload_ptr(a.v.p) + r * a.v.ts + t.head * a.v.hs;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = (2 * s + half) * G::VEC;
      fk[s] = load_if(live && d < a.dim_in, kp + d * ES);
      fv[s] = load_if(live && d < a.dim_in, vp + d * ES);
    }
  }

  // rows that see a key: all, or those of tokens from key - shift on
  const int shift = t.nk - t.nq;
  const int64_t nrows = (int64_t)t.nq * a.group;
  auto first = [&](int k) -> int64_t { return a.causal ? (int64_t)max(0, k - shift) * a.group : 0; };
  const int64_t row0 = min(first((int)t.start), nrows);
  const int64_t full0 = first(min((int)t.start + kAttnKeys, t.nk) - 1);  // from here on every key is seen
  const int64_t mine = live ? first(key) : nrows;
  const int ntiles = (int)((nrows - row0 + QT - 1) / QT);

  const char* qp = (const char*)a.q.p + (int64_t)t.q0 * a.q.ts + (int64_t)t.head * a.group * a.q.hs;
  const char* dp_ = (const char*)a.dy.p + (int64_t)t.q0 * a.dy.ts + (int64_t)t.head * a.group * a.dy.hs;
  const float2* sp = a.stats + ((int64_t)t.head * a.tokens_q + t.q0) * a.group;
  RowBase rb = row_base(a, row0);  // of the next tile to load
  auto load_tile = [&](int j, char* buf) {
    const int64_t at0 = row0 + (int64_t)j * QT;
    const int rows = (int)min((int64_t)QT, nrows - at0);
    const u32x4 rq = buffer_of(qp + (int64_t)rb.token * a.q.ts, 0x7fffffffu);
    const u32x4 rd = buffer_of(dp_ + (int64_t)rb.token * a.dy.ts, 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < LPT; ++i) {
      const int at = (wave * LPT + i) * 1024 + lane * 16;
      const int r = at / G::ROWB, ch = ((at % G::ROWB) >> 4) ^ G::swz(r);
      int tok, g;
      row_of(a, {0, rb.rem}, r, tok, g);
      const bool in = r < rows && ch * G::VEC < a.dim_in;
      const uint32_t oq = in ? (uint32_t)(tok * (int)a.q.ts + g * (int)a.q.hs + ch * 16) : kOutside;
      const uint32_t od = in ? (uint32_t)(tok * (int)a.dy.ts + g * (int)a.dy.hs + ch * 16) : kOutside;
      tile_load(rq, oq, lds_at(buf + (wave * LPT + i) * 1024));
      tile_load(rd, od, lds_at(buf + TILE + (wave * LPT + i) * 1024));
    }
    // the rows' statistics, past the last row zeros
    if (wave == 0) {
      const u32x4 rs = buffer_of(sp + at0, (uint32_t)rows * 8u);
      if (lane < QT / 2) tile_load(rs, lane * 16, lds_at(buf + 2 * TILE));
    }
    rb.token += QT / a.group;
    rb.rem += QT % a.group;
    if (rb.rem >= a.group) {
      rb.rem -= a.group;
      ++rb.token;
    }
  };

  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[db][r] = dv[db][r] = 0.0f;
  const float c = a.scale * kLog2e;
  const uint32_t rf = row_frag<G>(lcol, half), cf = col_frag<G>(lane);

  auto tile_body = [&](int j, const char* buf, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const int64_t at0 = row0 + (int64_t)j * QT;
    const char *Q = buf, *DO = buf + TILE;
    const float* st = reinterpret_cast<const float*>(buf + 2 * TILE);
    bool guard = false;
    // the rows of the tile that this lane's key sees: [lo, hi)
    const int lo = (int)max((int64_t)0, min(mine - at0, (int64_t)QT)), hi = (int)min(nrows - at0, (int64_t)QT);
    if constexpr (EDGE) {
      if (scan_tile<ES, 2 * TILE>(Q)) flag = 1;
      ring_barrier();
      guard = flag != 0;
    }
    each<QB>([&](auto qb_t) {
      constexpr int qb = decltype(qb_t)::value;
      f32x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
      for (int x = 0; x < NS; ++x) Mfma<E>::run(rd16(Q + (rf ^ (uint32_t)(x * 32)) + qb * 32 * G::ROWB), fk[x], s);
#pragma unroll
      for (int x = 0; x < NS; ++x) Mfma<E>::run(rd16(DO + (rf ^ (uint32_t)(x * 32)) + qb * 32 * G::ROWB), fv[x], dp);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int r0 = 32 * qb + 8 * g;
        const float4 x = *reinterpret_cast<const float4*>(st + (r0 + 4 * half) * 2);
        const float4 y = *reinterpret_cast<const float4*>(st + (r0 + 4 * half) * 2 + 4);
        const float ls[4] = {x.x, x.z, y.x, y.z}, de[4] = {x.y, x.w, y.y, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * g + i;
          s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -ls[i]));
          dp[r] = s[r] * (dp[r] - de[i]);
          if constexpr (EDGE) {
            const int row = r0 + i + 4 * half;
            const bool in = row >= lo && row < hi;
            s[r] = in ? s[r] : 0.0f;
            dp[r] = in ? dp[r] : 0.0f;
          }
        }
      }
      each<32 / G::KF>([&](auto x_t) {
        constexpr int x = decltype(x_t)::value, at = qb * 32 + x * G::KF;
        const u32x4 fp = acc_frag<E, x * G::KF>(s), fs = acc_frag<E, x * G::KF>(dp);
        auto seen = [&](int y) { return at + y >= lo && at + y < hi; };
        each<DB>([&](auto db_t) {
          constexpr int db = decltype(db_t)::value;
          const u32x4 fa = rd_cols<G, at, db>(DO, cf), fb = rd_cols<G, at, db>(Q, cf);
          if (guard) {
            guarded<E>(fa, fp, dv[db], half, seen);
            guarded<E>(fb, fs, dk[db], half, seen);
          } else {
            Mfma<E>::run(fa, fp, dv[db]);
            Mfma<E>::run(fb, fs, dk[db]);
          }
        });
      });
    });
  };

  if (ntiles > 0) load_tile(0, smem);
  for (int j = 0; j < ntiles; ++j) {
    wait_vmem();
    ring_barrier();
    char* buf = smem + (j & 1) * STAGE;
    if (j + 1 < ntiles) load_tile(j + 1, smem + ((j + 1) & 1) * STAGE);
    const int64_t at0 = row0 + (int64_t)j * QT;
    if (at0 < full0 || at0 + QT > nrows)
      tile_body(j, buf, std::true_type{});
    else
      tile_body(j, buf, std::false_type{});
  }

  if (!live) return;
  const int64_t at = ((int64_t)(t.k0 + key) * a.kv_heads + t.head) * ((int64_t)a.dim * ES);
  store_row<E, DB>(gstore_ptr(a.dk) + at, dk, a.scale, half, a.dim, a.vec_out);
  store_row<E, DB>(gstore_ptr(a.dv) + at, dv, 1.0f, half, a.dim, a.vec_out);
}

template <class E, int DP, int KT, int QT, int OF, int OQ, int OK>
hipError_t launch_attn(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  // a launch's threads have to be fewer than 2^32
  constexpr int64_t most = (int64_t)1 << 21;
  for (int64_t u = 0; u < grid; u += most) {
    AttnArgs b = a;
    b.unit0 = u;
    const dim3 n((unsigned)(grid - u < most ? grid - u : most));
    if (pass == ATTN_FWD)
      hipLaunchKernelGGL((attn_rows_kernel<E, DP, KT, false, OF>), n, dim3(256), 0, st, b);
    else if (pass == ATTN_DQ)
      hipLaunchKernelGGL((attn_rows_kernel<E, DP, KT, true, OQ>), n, dim3(256), 0, st, b);
    else
      hipLaunchKernelGGL((attn_keys_kernel<E, DP, QT, OK>), n, dim3(256), 0, st, b);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace dmuon
