// Host side of the attention block's operators: norm and rotation of heads,
// attention over packed sequences, dropout.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "arena.h"
#include "attention.h"
#include "heads.h"

namespace dmuon {
namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxRows = (int64_t)1 << 36;  // tokens times heads
constexpr int64_t kMaxStride = (int64_t)1 << 40;

int check_dtype(int dtype) {
  if (dtype != DMUON_BF16 && dtype != DMUON_F32) return fail(DMUON_EINVAL, "unknown dtype %d", dtype);
  return DMUON_OK;
}
int check_strides(const char* what, const int64_t* s) {
  for (int i = 0; i < 2; ++i)
    if (s[i] < 0 || s[i] > kMaxStride) return fail(DMUON_EINVAL, "stride %lld of %s is out of range", (long long)s[i], what);
  return DMUON_OK;
}

// ------------------------------------------------------------ attention
void attn_cut(const dmuon_attention& d, AttnArgs& a, bool keys);
int64_t attn_grid(const dmuon_attention& d, int64_t slots, int64_t parts);

int check_attention(const dmuon_attention* d, bool bwd) {
  if (!d) return fail(DMUON_EINVAL, "the attention's description is NULL");
  TRY(check_dtype(d->dtype));
  if (d->tokens_q < 0 || d->tokens_q > kMaxTokens || d->tokens_k < 0 || d->tokens_k > kMaxTokens)
    return fail(DMUON_EINVAL, "tokens %lld, %lld are out of range", (long long)d->tokens_q, (long long)d->tokens_k);
  if (d->kv_heads < 1 || d->heads < d->kv_heads || d->heads > kMaxHeads || d->heads % d->kv_heads)
    return fail(DMUON_EINVAL, "heads %lld must be a multiple of kv_heads %lld and at most %lld", (long long)d->heads,
                (long long)d->kv_heads, (long long)kMaxHeads);
  if (d->tokens_q * d->heads > kMaxRows || d->tokens_k * d->kv_heads > kMaxRows)
    return fail(DMUON_EUNSUPPORTED, "tokens times heads exceed 2^36");
  if (d->head_dim < 1) return fail(DMUON_EINVAL, "head_dim %lld must be positive", (long long)d->head_dim);
  const int64_t most = d->dtype == DMUON_BF16 ? 256 : 128;
  if (d->head_dim > most)
    return fail(DMUON_EUNSUPPORTED, "head_dim %lld is larger than %lld", (long long)d->head_dim, (long long)most);
  if (d->sequences < 1 || d->sequences > kMaxTokens)
    return fail(DMUON_EINVAL, "sequences = %lld is out of range", (long long)d->sequences);
  if (!d->cu_q != !d->cu_k) return fail(DMUON_EINVAL, "cu_q and cu_k: both or neither");
  if (!d->cu_q && (d->tokens_q % d->sequences || d->tokens_k % d->sequences))
    return fail(DMUON_EINVAL, "tokens do not divide into %lld sequences of one length", (long long)d->sequences);
  if (!(d->scale >= 0x1p-64f && d->scale <= 0x1p64f))
    return fail(DMUON_EINVAL, "scale must lie in [2^-64, 2^64]");
  TRY(check_strides("q", d->q_stride));
  TRY(check_strides("k", d->k_stride));
  TRY(check_strides("v", d->v_stride));
  if (bwd) TRY(check_strides("dy", d->dy_stride));
  for (int keys = 0; keys <= (bwd ? 1 : 0); ++keys) {
    AttnArgs a{};
    attn_cut(*d, a, keys != 0);
    if (attn_grid(*d, a.slots, a.parts) >= (int64_t)1 << 31)  // (the kernels count tiles in 32 bits)
      return fail(DMUON_EUNSUPPORTED, "%lld sequences of %lld heads are too many tiles", (long long)d->sequences,
                  (long long)d->heads);
  }
  return DMUON_OK;
}

// head width that the kernels are built for
int attn_padded(int64_t dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : 256; }

hipError_t launch_attn(const dmuon_attention& d, AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st) {
  const int p = attn_padded(d.head_dim);
  if (d.dtype == DMUON_BF16)
    return p == 64   ? launch_attn_bf16_64(pass, a, grid, st)
           : p == 96  ? launch_attn_bf16_96(pass, a, grid, st)
           : p == 128 ? launch_attn_bf16_128(pass, a, grid, st)
                      : launch_attn_bf16_256(pass, a, grid, st);
  return p == 64 ? launch_attn_f32_64(pass, a, grid, st)
         : p == 96 ? launch_attn_f32_96(pass, a, grid, st)
                   : launch_attn_f32_128(pass, a, grid, st);
}

// The operands of one call as the kernels take them: as they are, or copies of
// those whose rows are not 16-byte aligned or not whole 16-byte chunks, or so far apart
// that the loads' 32-bit offsets do not reach.
struct Heads {
  Arena& ar;
  const dmuon_attention& d;
  int es, dim_in;
  GatherArgs g{};
  double bytes = 0.0;
  Heads(Arena& arena, const dmuon_attention& desc) : ar(arena), d(desc), es(esize_of(desc.dtype)) {
    dim_in = (int)round_up(d.head_dim, 16 / es);
    g.dim = (int)d.head_dim;
    g.dim_in = dim_in;
    g.esize = es;
  }
  AttnView add(const void* p, const int64_t* stride, int64_t tokens, int64_t heads) {
    const int64_t group = d.heads / d.kv_heads;
    const bool far = (group * stride[1] + 256 * stride[0] + dim_in) * es >= (int64_t)1 << 31;
    if (!ar.unaligned && !far && dim_in == d.head_dim && stride[0] * es % 16 == 0 && stride[1] * es % 16 == 0)
      return {p, stride[0] * es, stride[1] * es};
    void* q = ar.take(tokens * heads * dim_in * es);
    g.src[g.n] = p;
    g.dst[g.n] = q;
    g.ts[g.n] = stride[0];
    g.hs[g.n] = stride[1];
    g.tokens[g.n] = tokens;
    g.heads[g.n++] = (int)heads;
    bytes += (double)tokens * heads * (g.dim + dim_in) * es;
    return {q, heads * dim_in * es, (int64_t)dim_in * es};
  }
  int make() {
    if (g.n == 0) return DMUON_OK;
    return launch(ar, "gather_heads_kernel", 0.0, bytes, [&] { return launch_gather_heads(g, ar.st); });
  }
};

struct Attn {
  const void *q, *k, *v, *y, *dy;
  void *out, *dk, *dv;
  float* lse;
};

AttnArgs attn_args(const dmuon_attention& d, const Attn& c) {
  AttnArgs a{};
  a.lse = c.lse;
  a.cu_q = d.cu_q;
  a.cu_k = d.cu_k;
  a.tokens_q = d.tokens_q;
  a.tokens_k = d.tokens_k;
  a.sequences = (int32_t)d.sequences;
  a.heads = (int32_t)d.heads;
  a.kv_heads = (int32_t)d.kv_heads;
  a.group = (int32_t)(d.heads / d.kv_heads);
  a.group_magic = a.group == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + a.group - 1) / a.group);
  a.dim = (int32_t)d.head_dim;
  a.causal = d.causal != 0;
  a.scale = d.scale;
  return a;
}
// tiles of `per` rows, `mult` rows to a token: at most one of a sequence is not
// full, nor one of the tokens before the first and behind the last sequence
int64_t attn_slots(const dmuon_attention& d, int64_t tokens, int64_t mult, int64_t per) {
  if (d.cu_q) return tokens * mult / per + d.sequences + 2;
  return d.sequences * ((tokens / d.sequences * mult + per - 1) / per);
}
// workgroups: attn_tile
int64_t attn_grid(const dmuon_attention& d, int64_t slots, int64_t parts) {
  return 8 * ((d.kv_heads >> 3) * parts * slots + ((d.kv_heads & 7) * parts * slots + 7) / 8);
}
// workgroups of a join: four elements a thread, a few turns each
int64_t attn_join_grid(const dmuon_attention& d, int64_t rows) {
  return std::max<int64_t>(1, std::min<int64_t>((rows * attn_padded(d.head_dim) / 4 + 255) / 256, 4096));
}
// How a pass is cut: tiles of 256 rows (or keys) that eight waves share, or of 128
// that four do, and the workgroups that share a tile's work.  By the sizes alone: the
// sequences' lengths are on the device, their mean stands for them.
//  - Eight waves read a tile of keys once for twice the rows, and their ring is deeper
//    (16384 tokens, 32 heads on 8, 128 wide: forward 2180 -> 1910 us); they need
//    enough tiles, and rows to fill them (64 single tokens of 32 heads on 8 against 117 000 keys: 205 us).
//  - Few rows against many keys: parts of the keys.  Where a sequence's rows are one tile its keys alone
//    set the work of a part, and three parts for each place even out unlike lengths (those
//    64 tokens: 293 us whole, 151 + 7; sixteen of 8192 to 1 keys 52 + 7 in parts for each place,
//    50 + 7 in three; sixteen of 4096 keys each 47 + 7, 54 + 7).  32 parts at most: the join
//    reads them eight at a time (one token, 60 000 keys: 81 + 6 us in 16 parts, 48 + 9 in 32, 45 + 14 in 64).
//  - A part has at least 4 tiles, 2 of a sequence of one tile of rows (500 keys: 18 us whole, 13 + 6; 8
//    sequences of 80 wide heads 29 -> 19), or 1 in fp32, whose tiles take longer (two sequences
//    of 116 and 121 rows: forward 42 -> 20 + 8 us; 364 and 155 rows: dk and dv 51 + 6 -> 27 + 7).
//    (Tiles of dk and dv are counted as 32 rows; those of bf16 heads of up to 64 in narrow calls have 64, so
//    that their parts may have half as many.)
//  - Lists of more than 62 sequences are taken in their order: 4096 tokens behind 62 sequences of 50 to 250
//    (32 heads on 8 of 128, causal) forward 237 us, dk and dv 544; before them 233 and 426.  And they are searched by
//    every workgroup: 4096 sequences of 16 tokens forward 3.1 ms, 1000 of them 0.29, 60 of them 0.015.
//  - dk and dv: the tiles of a causal sequence differ as 1 to n in their work, and
//    with about one for each place on the GPU the longest is twice the mean (8192
//    tokens: 1660 us whole, 1005 + 28 us in two parts); three for each place (two of narrow
//    tiles) even it out.
void attn_cut(const dmuon_attention& d, AttnArgs& a, bool keys) {
  const int64_t n = d.sequences, group = d.heads / d.kv_heads;
  const int64_t mine = keys ? d.tokens_k / n : d.tokens_q * group / n;       // rows (keys) of a sequence
  const int64_t other = keys ? d.tokens_q * group / n : d.tokens_k / n;      // what each walks
  auto tiles = [&](int64_t per) { return n * std::max<int64_t>(1, (mine + per - 1) / per) * d.kv_heads; };
  const bool built = d.dtype == DMUON_BF16 && d.head_dim <= 128;
  a.wide = built && mine > 128 && tiles(256) >= (keys ? 128 : 256);
  const int64_t per = a.wide ? 256 : 128, jobs = tiles(per), places = a.wide || keys ? 256 : 512;
  const bool one = !keys && mine <= per;
  const int64_t step = keys || d.dtype == DMUON_F32 || d.head_dim > 128 ? 32 : 64;  // rows (keys) of a tile walked
  const int64_t least = d.dtype == DMUON_F32 ? 1 : one ? 2 : 4;
  const int64_t want = keys ? ((a.wide ? 3 : 2) * places + jobs - 1) / jobs : (one ? 3 : 1) * places / jobs;
  a.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>(std::min(want, other / step / least), one ? 32 : 16));
  a.slots = (uint32_t)attn_slots(d, keys ? d.tokens_k : d.tokens_q, keys ? 1 : group, per);
}
// Flops of one product over the pairs of a row and a key that it sees.  The lengths of listed sequences are on
// the device: none are counted.
double attn_flops(const dmuon_attention& d) {
  if (d.cu_q) return 0.0;
  const double n = (double)(d.tokens_q / d.sequences), m = (double)(d.tokens_k / d.sequences), full = std::min(n, m);
  const double pairs = d.causal ? full * (m - full) + full * (full + 1.0) / 2.0 : n * m;
  return 2.0 * d.head_dim * d.heads * d.sequences * pairs;
}
// Bytes of a join: the parts in, the results out.
double attn_join_bytes(const dmuon_attention& d, const AttnArgs& a, int64_t rows) {
  return (double)rows * (4.0 * a.parts * attn_padded(d.head_dim) + (double)d.head_dim * esize_of(d.dtype));
}
// the results' rows are written 8 (bf16) or 16 (fp32) bytes at a time
bool attn_vec(const dmuon_attention& d, const void* a, const void* b, const void* c) {
  return d.head_dim % 4 == 0 && !misaligned(a) && !misaligned(b) && !misaligned(c);
}

// The forward pass, or dq.
int attn_rows(Arena& ar, const dmuon_attention& d, AttnArgs& a, AttnPass pass) {
  const bool fwd = pass == ATTN_FWD;
  attn_cut(d, a, false);
  const int64_t rows = d.tokens_q * d.heads, mark = ar.used;
  if (a.parts > 1) {
    a.partial = (float*)ar.take(a.parts * rows * attn_padded(d.head_dim) * 4);
    if (fwd) a.partial_ml = (float2*)ar.take(a.parts * rows * 8);
  }
  TRY(launch(ar, fwd ? "attn_rows_kernel<fwd>" : "attn_rows_kernel<dq>", (fwd ? 2.0 : 3.0) * attn_flops(d), 0.0,
             [&] { return launch_attn(d, pass, a, attn_grid(d, a.slots, a.parts), ar.st); }));
  if (a.parts > 1)
    TRY(launch(ar, "attn_join_kernel<rows>", 0.0, attn_join_bytes(d, a, rows),
               [&] { return launch_attn(d, fwd ? ATTN_JOIN_FWD : ATTN_JOIN_DQ, a, attn_join_grid(d, rows), ar.st); }));
  ar.used = mark;
  return DMUON_OK;
}

int attention_fwd(Arena& ar, const dmuon_attention& d, const Attn& c) {
  Heads h(ar, d);
  AttnArgs a = attn_args(d, c);
  a.q = h.add(c.q, d.q_stride, d.tokens_q, d.heads);
  a.k = h.add(c.k, d.k_stride, d.tokens_k, d.kv_heads);
  a.v = h.add(c.v, d.v_stride, d.tokens_k, d.kv_heads);
  a.dim_in = h.dim_in;
  TRY(h.make());
  a.out = c.out;
  a.vec_out = attn_vec(d, c.out, nullptr, nullptr);
  return attn_rows(ar, d, a, ATTN_FWD);
}

int attention_bwd(Arena& ar, const dmuon_attention& d, const Attn& c) {
  Heads h(ar, d);
  AttnArgs a = attn_args(d, c);
  a.q = h.add(c.q, d.q_stride, d.tokens_q, d.heads);
  a.k = h.add(c.k, d.k_stride, d.tokens_k, d.kv_heads);
  a.v = h.add(c.v, d.v_stride, d.tokens_k, d.kv_heads);
  a.dy = h.add(c.dy, d.dy_stride, d.tokens_q, d.heads);
  const int64_t ys[2] = {d.heads * d.head_dim, d.head_dim};
  a.y = h.add(c.y, ys, d.tokens_q, d.heads);
  a.dim_in = h.dim_in;
  TRY(h.make());
  a.stats = (float*)ar.take(d.tokens_q * d.heads * 8);
  a.out = c.out;
  a.dk = c.dk;
  a.dv = c.dv;
  a.vec_out = attn_vec(d, c.out, c.dk, c.dv);
  if (d.tokens_q > 0) TRY(attn_rows(ar, d, a, ATTN_DQ));
  if (d.tokens_k > 0) {
    const int64_t rows = 2 * d.tokens_k * d.kv_heads;
    attn_cut(d, a, true);
    if (a.parts > 1) a.partial = (float*)ar.take(a.parts * rows * attn_padded(d.head_dim) * 4);
    TRY(launch(ar, "attn_keys_kernel", 4.0 * attn_flops(d), 0.0,
               [&] { return launch_attn(d, ATTN_DKV, a, attn_grid(d, a.slots, a.parts), ar.st); }));
    if (a.parts > 1)
      TRY(launch(ar, "attn_join_kernel<keys>", 0.0, attn_join_bytes(d, a, rows),
                 [&] { return launch_attn(d, ATTN_JOIN_KEYS, a, attn_join_grid(d, rows), ar.st); }));
  }
  return DMUON_OK;
}

// ------------------------------------------------------------ norm and rotation
int check_rope(const dmuon_rope* d, bool bwd) {
  if (!d) return fail(DMUON_EINVAL, "the rotation's description is NULL");
  TRY(check_dtype(d->dtype));
  if (d->tokens < 0 || d->tokens > kMaxTokens)
    return fail(DMUON_EINVAL, "tokens = %lld is out of range", (long long)d->tokens);
  if (d->q_heads < 0 || d->q_heads > kMaxHeads || d->k_heads < 0 || d->k_heads > kMaxHeads)
    return fail(DMUON_EINVAL, "heads %lld, %lld are out of range", (long long)d->q_heads, (long long)d->k_heads);
  if (d->head_dim < 2 || d->head_dim > 2 * kRopeHalf || d->head_dim % 2)
    return fail(DMUON_EINVAL, "head_dim %lld must be even and in [2, %d]", (long long)d->head_dim, 2 * kRopeHalf);
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 2)
    return fail(DMUON_EINVAL, "rotary_dim %lld must be even and in [0, head_dim]", (long long)d->rotary_dim);
  if (d->axes < 1 || d->axes > DMUON_ROPE_AXES) return fail(DMUON_EINVAL, "axes = %d is out of range", d->axes);
  int64_t sum = 0;
  for (int i = 0; i < d->axes; ++i) {
    if (d->sections[i] < 0) return fail(DMUON_EINVAL, "a section is negative");
    sum += d->sections[i];
  }
  if (sum != d->rotary_dim / 2)
    return fail(DMUON_EINVAL, "sections add up to %lld, not to half of rotary_dim %lld", (long long)sum,
                (long long)d->rotary_dim);
  if (!(d->base > 0.0) || !std::isfinite(d->base)) return fail(DMUON_EINVAL, "base must be positive and finite");
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return fail(DMUON_EINVAL, "eps must be finite and >= 0");
  TRY(check_strides("q", d->q_stride));
  TRY(check_strides("k", d->k_stride));
  if (bwd) {
    TRY(check_strides("dq", d->dq_stride));
    TRY(check_strides("dk", d->dk_stride));
  }
  return DMUON_OK;
}

RopeArgs rope_args(const dmuon_rope& d, const void* q, const void* k, const int64_t* positions, const void* wq,
                   const void* wk, void* out_q, void* out_k, bool bwd) {
  constexpr double kTurn = 6.283185307179586476925286766559;
  RopeArgs a{};
  const int64_t es = esize_of(d.dtype);
  a.x[0] = {q, d.q_stride[0] * es, d.q_stride[1] * es};
  a.x[1] = {k, d.k_stride[0] * es, d.k_stride[1] * es};
  a.out[0] = out_q;
  a.out[1] = out_k;
  a.w[0] = wq;
  a.w[1] = wk;
  a.positions = positions;
  a.tokens = d.tokens;
  a.heads[0] = (int32_t)d.q_heads;
  a.heads[1] = (int32_t)d.k_heads;
  a.axes = d.axes;
  a.dim = (int32_t)d.head_dim;
  a.rot = (int32_t)d.rotary_dim;
  a.interleaved = d.interleaved != 0;
  a.esize = (int32_t)es;
  rope_cut(a, bwd);
  a.eps = d.eps;
  int p = 0;
  for (int x = 0; x < d.axes; ++x)
    for (int64_t i = 0; i < d.sections[x]; ++i, ++p) {
      a.axis[p] = (uint8_t)x;
      a.turn[p] = std::pow(d.base, d.per_axis ? -(double)i / (double)d.sections[x] : -2.0 * p / (double)a.rot) / kTurn;
    }
  return a;
}

int dropout(const void* x, const void* residual, void* y, int64_t n, double p, uint64_t seed, uint64_t offset,
            const int64_t* state, int dtype, void* stream, const char* name) {
  TRY(check_dtype(dtype));
  if (n < 0 || n > (int64_t)1 << 40) return fail(DMUON_EINVAL, "n = %lld is out of range", (long long)n);
  if (!(p >= 0.0 && p <= 1.0)) return fail(DMUON_EINVAL, "p must lie in [0, 1]");
  if (n == 0) return DMUON_OK;
  if (!x || !y) return fail(DMUON_EINVAL, "x/y is NULL");
  const uint32_t cut = (uint32_t)std::nearbyint(p * 65536.0);
  DropoutArgs a{x, residual, y, n, seed, offset, state, cut, cut == 65536 ? 0.0f : (float)(65536.0 / (65536.0 - cut)),
                esize_of(dtype)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return guard([&]() -> int {
    HIP_TRY(timed_launch(name, 0.0, (residual ? 3.0 : 2.0) * n * a.esize, st, [&] { return launch_dropout(a, st); }));
    return DMUON_OK;
  });
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int64_t dmuon_attention_fwd_workspace(const dmuon_attention* desc, int unaligned) {
  TRY(check_attention(desc, false));
  Arena ar;
  ar.unaligned = unaligned != 0;
  TRY(attention_fwd(ar, *desc, Attn{}));
  return ar.peak;
}

int dmuon_attention_fwd(const dmuon_attention* desc, const void* q, const void* k, const void* v, void* y, float* lse,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  TRY(check_attention(desc, false));
  if (desc->tokens_q == 0) return DMUON_OK;
  if (!q || !y || !lse) return fail(DMUON_EINVAL, "q/y/lse is NULL");
  if (desc->tokens_k > 0 && (!k || !v)) return fail(DMUON_EINVAL, "k/v is NULL");
  Attn c{};
  c.q = q, c.k = k, c.v = v, c.out = y, c.lse = lse;
  return sized(workspace, workspace_bytes, misaligned(q) || misaligned(k) || misaligned(v), stream,
                    [&](Arena& ar) { return attention_fwd(ar, *desc, c); });
}

int64_t dmuon_attention_bwd_workspace(const dmuon_attention* desc, int unaligned) {
  TRY(check_attention(desc, true));
  Arena ar;
  ar.unaligned = unaligned != 0;
  TRY(attention_bwd(ar, *desc, Attn{}));
  return ar.peak;
}

int dmuon_attention_bwd(const dmuon_attention* desc, const void* dy, const void* q, const void* k, const void* v,
                        const void* y, const float* lse, void* dq, void* dk, void* dv, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  TRY(check_attention(desc, true));
  if (desc->tokens_q > 0 && (!dy || !q || !y || !lse || !dq)) return fail(DMUON_EINVAL, "dy/q/y/lse/dq is NULL");
  if (desc->tokens_k > 0 && (!k || !v || !dk || !dv)) return fail(DMUON_EINVAL, "k/v/dk/dv is NULL");
  Attn c{};
  c.dy = dy, c.q = q, c.k = k, c.v = v, c.y = y, c.lse = const_cast<float*>(lse), c.out = dq, c.dk = dk, c.dv = dv;
  const bool un = misaligned(dy) || misaligned(q) || misaligned(k) || misaligned(v) || misaligned(y);
  return sized(workspace, workspace_bytes, un, stream,
                    [&](Arena& ar) { return attention_bwd(ar, *desc, c); });
}

int dmuon_qk_norm_rope_fwd(const dmuon_rope* desc, const void* q, const void* k, const int64_t* positions,
                           const void* q_weight, const void* k_weight, void* q_out, void* k_out, void* stream) {
  TRY(check_rope(desc, false));
  if (!q_weight != !k_weight) return fail(DMUON_EINVAL, "q_weight and k_weight: both or neither");
  if (desc->tokens == 0) return DMUON_OK;
  if (!positions) return fail(DMUON_EINVAL, "positions is NULL");
  if (desc->q_heads > 0 && (!q || !q_out)) return fail(DMUON_EINVAL, "q/q_out is NULL");
  if (desc->k_heads > 0 && (!k || !k_out)) return fail(DMUON_EINVAL, "k/k_out is NULL");
  const RopeArgs a = rope_args(*desc, q, k, positions, q_weight, k_weight, q_out, k_out, false);
  const double n = (double)a.tokens * (a.heads[0] + a.heads[1]) * a.dim * a.esize;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return guard([&]() -> int {
    HIP_TRY(timed_launch("rope_kernel<fwd>", 0.0, 2.0 * n, st, [&] { return launch_rope(a, false, st); }));
    return DMUON_OK;
  });
}

int64_t dmuon_qk_norm_rope_bwd_workspace(const dmuon_rope* desc) {
  TRY(check_rope(desc, true));
  RopeArgs a{};
  a.tokens = desc->tokens;
  a.heads[0] = (int32_t)desc->q_heads;
  a.heads[1] = (int32_t)desc->k_heads;
  rope_cut(a, true);
  return (int64_t)(a.parts[0] + a.parts[1]) * desc->head_dim * 4;
}

int dmuon_qk_norm_rope_bwd(const dmuon_rope* desc, const void* dq, const void* dk, const void* q, const void* k,
                           const int64_t* positions, const void* q_weight, const void* k_weight, void* dq_in,
                           void* dk_in, void* dq_weight, void* dk_weight, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  TRY(check_rope(desc, true));
  if (!q_weight != !k_weight) return fail(DMUON_EINVAL, "q_weight and k_weight: both or neither");
  if (q_weight && (!dq_weight || !dk_weight)) return fail(DMUON_EINVAL, "dq_weight/dk_weight is NULL");
  if (desc->tokens > 0) {
    if (!positions) return fail(DMUON_EINVAL, "positions is NULL");
    if (desc->q_heads > 0 && (!dq || !q || !dq_in)) return fail(DMUON_EINVAL, "dq/q/dq_in is NULL");
    if (desc->k_heads > 0 && (!dk || !k || !dk_in)) return fail(DMUON_EINVAL, "dk/k/dk_in is NULL");
  }
  const int64_t need = dmuon_qk_norm_rope_bwd_workspace(desc);
  if (q_weight && need > 0) {
    if (need > workspace_bytes)
      return fail(DMUON_EINVAL, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
      return fail(DMUON_EINVAL, "workspace is NULL or not 256-byte aligned");
  }
  RopeArgs a = rope_args(*desc, q, k, positions, q_weight, k_weight, dq_in, dk_in, true);
  a.dy[0] = {dq, desc->dq_stride[0] * a.esize, desc->dq_stride[1] * a.esize};
  a.dy[1] = {dk, desc->dk_stride[0] * a.esize, desc->dk_stride[1] * a.esize};
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.part = (float*)workspace;
  const double n = (double)a.tokens * (a.heads[0] + a.heads[1]) * a.dim * a.esize;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return guard([&]() -> int {
    HIP_TRY(timed_launch("rope_kernel<bwd>", 0.0, 3.0 * n, st, [&] { return launch_rope(a, true, st); }));
    return DMUON_OK;
  });
}

int dmuon_dropout_fwd(const void* x, const void* residual, void* y, int64_t n, double p, uint64_t seed, uint64_t offset,
                      const int64_t* state, int dtype, void* stream) {
  return dropout(x, residual, y, n, p, seed, offset, state, dtype, stream, "dropout_kernel<fwd>");
}

int dmuon_dropout_bwd(const void* dy, void* dx, int64_t n, double p, uint64_t seed, uint64_t offset,
                      const int64_t* state, int dtype, void* stream) {
  return dropout(dy, nullptr, dx, n, p, seed, offset, state, dtype, stream, "dropout_kernel<bwd>");
}

}  // extern "C"
