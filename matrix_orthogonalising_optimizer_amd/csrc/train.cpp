// Host side of the training operators: layer norm, the gated feed-forward
// block and the linear cross entropy.  Arguments are checked, the workspace
// is laid out and the launches are enqueued; nothing is allocated or kept.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "dmuon.h"
#include "errors.h"
#include "linear.h"
#include "timing.h"

namespace dmuon {
namespace {

#define HIP_TRY(expr)                                                              \
  do {                                                                             \
    hipError_t e_ = (expr);                                                        \
    if (e_ != hipSuccess)                                                          \
      return fail(DMUON_EHIP, "%s failed: %s", #expr, hipGetErrorString(e_));      \
  } while (0)
#define TRY(expr)                  \
  do {                             \
    const int rc_ = (expr);        \
    if (rc_ != DMUON_OK) return rc_; \
  } while (0)

constexpr int64_t kMaxWidth = (int64_t)1 << 20;
constexpr int64_t kMaxVocab = (int64_t)1 << 22;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kDefaultBlock = (int64_t)2 << 30;

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int esize_of(int dtype) { return dtype == DMUON_BF16 ? 2 : 4; }
bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// Workspace laid out front to back.  Without a base it only counts, which is
// how the *_workspace functions size a call: they run it without launches.
// Nothing in a call's layout or choices may depend on more than its sizes,
// its type and `unaligned`, so that both runs agree; a launch behind memory
// that was not counted is refused.
struct Arena {
  char* base = nullptr;
  int64_t cap = 0;
  int64_t used = 0, peak = 0;
  bool dry = true;
  bool unaligned = false;  // some pointer of the call is not 16-byte aligned
  hipStream_t st = nullptr;
  void* take(int64_t bytes) {
    void* p = base ? base + used : nullptr;
    used += round_up(bytes, 256);
    peak = std::max(peak, used);
    return p;
  }
};

template <class F>
int launch(const Arena& ar, const char* name, double flops, double bytes, F&& f) {
  if (ar.dry) return DMUON_OK;
  if (ar.peak > ar.cap) return fail(DMUON_EINVAL, "%s: workspace overrun", name);
  const hipError_t e = timed_launch(name, flops, bytes, ar.st, f);
  if (e != hipSuccess) return fail(DMUON_EHIP, "%s: %s", name, hipGetErrorString(e));
  return DMUON_OK;
}

// A matrix as the product kernels take it: rows 16-byte aligned, or the
// planes of an fp32 matrix.
struct Mat {
  const void* p;
  int64_t ld;
  int64_t plane = 0;
  int16_t flag = 0;  // planes': which of the call's flags is theirs
};
// Row pitch of the library's own matrices.  Rows are padded to 16 bytes, long
// ones to 128: a K step's 128 bytes of a row are then one line of the caches,
// not two halves (1531 x 2056 x 10928 with both operands so: 123 -> 97 us;
// 1531 x 2056 x 5464: 56 -> 43).
int64_t padded(int64_t cols, int es) { return round_up(cols, 16 / es); }
int64_t pitch(int64_t cols, int es) { return cols * es < 1024 ? padded(cols, es) : round_up(cols, 128 / es); }
bool needs_copy(const Arena& ar, int64_t cols, int es) { return (cols * es) % 16 != 0 || ar.unaligned; }

// The form in which a call's products take their operands.
struct Form {
  LinKind kind;
  bool raw;  // rows that start at any element as they are
};
// Operands of one call in that form.  LIN_BF16, LIN_F32: as they are, or,
// unless raw, copies with padded rows of those whose rows do not start 16-byte
// aligned.  LIN_SPLIT: planes.  One launch for all.
struct Operands {
  Arena& ar;
  LinKind kind;
  bool raw;
  PackArgs a{};
  SplitArgs s{};
  FiniteArgs fin{};
  double bytes = 0.0;
  const int16_t flag;  // LIN_SPLIT: which of the call's flags is these operands'
  Operands(Arena& arena, Form f, int32_t* flags, int16_t which)
      : ar(arena), kind(f.kind), raw(f.raw), flag(which) {
    a.esize = kind == LIN_BF16 ? 2 : 4;
    fin.flag = s.flag = flags ? flags + which : nullptr;
  }
  // `always`: copied also when raw (activations of few tokens, which the
  // weight gradients' product, not raw, takes too)
  Mat add(const void* p, int64_t rows, int64_t cols, int64_t src_ld = 0, bool always = false) {
    if (kind == LIN_SPLIT) {
      const int64_t ld = round_up(cols, 64), plane = round_up(rows, 64) * ld;
      // (4352 bytes behind each matrix: those of power-of-two sizes would all start
      // at the same channels of the memory; 4096 tokens of 2048 x 8192, both ways:
      // 6.18 -> 6.10 ms)
      void* q = ar.take(kPlanes * plane * 2 + 17 * 256);
      s.src[s.n] = (const float*)p;
      s.dst[s.n] = (uint16_t*)q;
      s.rows[s.n] = rows;
      s.cols[s.n] = cols;
      s.src_ld[s.n++] = src_ld ? src_ld : cols;
      fin.planes[fin.n] = (uint16_t*)q;
      fin.plane[fin.n++] = plane;
      bytes += (double)rows * cols * 4 + (double)plane * 6;
      return {q, ld, plane, flag};
    }
    if (src_ld) return {p, src_ld};  // the library's own: padded
    if ((raw && !always) || !needs_copy(ar, cols, a.esize)) return {p, cols};
    const int64_t ld = pitch(cols, a.esize);
    void* q = ar.take(rows * ld * a.esize);
    a.src[a.n] = p;
    a.dst[a.n] = q;
    a.rows[a.n] = rows;
    a.cols[a.n] = cols;
    a.ld[a.n++] = ld;
    bytes += (double)rows * (cols + ld) * a.esize;
    return {q, ld};
  }
  int make() {
    if (a.n > 0) {
      TRY(launch(ar, "pack_rows_kernel", 0.0, bytes, [&] { return launch_pack_rows(a, ar.st); }));
    } else if (s.n > 0) {
      TRY(launch(ar, "planes_kernel", 0.0, bytes, [&] { return launch_planes(s, ar.st); }));
      TRY(launch(ar, "finite_plane_kernel", 0.0, 0.0, [&] { return launch_finite_plane(fin, ar.st); }));
    }
    return DMUON_OK;
  }
};

// How a launch of `n` problems is cut: the block tile, and how many of the
// last tiles are split along K, in how many parts.
struct Cut {
  int tile = 64;
  int64_t split_tiles = 0;
  int splits = 1;
  double us = 0.0;  // modelled time
};

// What the workgroups of one launch cost, in microseconds (measured on this
// GPU, operands in HBM): `places` workgroups run on a compute unit at once;
// `busy` is the time of a tile's K step (128 bytes of K) when all places are
// taken, over their number, `lat` that of a workgroup alone, `over` what a tile
// costs outside the K loop, with the gate's epilogues `gate` and `dgate`.
struct Rate {
  int places;
  double busy, lat, over, gate, dgate;
};
Rate lin_rate(Form form, int tile, double units) {
  const bool f32 = form.kind == LIN_F32;
  if (form.kind == LIN_SPLIT) return {1, 1.55, 1.55, 16.0, 24.0, 24.0};
  // clock and caches give the others more when not all compute units run (256:
  // 1.0 us a step on 64 of them, 1.35 on 208, 1.52 on all)
  const double fill = std::min(1.0, units / kLinCu), step = 1.0 + 0.52 * fill * fill;
  if (tile == 256) return {1, step, step, 8.0, 18.0, 26.0};
  Rate r;
  if (tile == 128 && f32)
    r = {2, 1.80, 2.00, 3.5, 7.0, 0.0};
  else if (form.raw || units <= kLinCu * (tile == 64 ? 2 : 1))  // the deep ring, or as many of the raw one
    r = tile == 128 ? Rate{form.raw ? 2 : 1, 0.36 + 0.20 * fill, 0.36 + 0.20 * fill, 3.5, 5.2, 5.2}
        : f32       ? Rate{2, 0.50, 0.57, 1.2, 1.8, 1.8}
                    : Rate{2, 0.25, 0.24, 1.2, 1.8, 1.8};
  else
    r = tile == 128 ? Rate{2, 0.52, 0.52, 1.0, 2.0, 4.0}
        : f32       ? Rate{4, 0.45, 0.52, 1.0, 3.7, 2.3}
                    : Rate{4, 0.24, 0.40, 0.8, 1.2, 1.2};
  if (form.raw) r.busy *= f32 ? 1.12 : 1.7, r.lat *= f32 ? 1.2 : 1.6;
  return r;
}

// Modelled time.  fp32 products are bound by the MFMA: tiles of 128 gain 2 to
// 10% when they fill rounds (gate of 2048 x 4096 x 2048: 493 against 548 us), and
// lose with the gate's backward epilogue (112 against 79 us at 2048 x 4096 x
// 512), which has none.  At full compute units a bf16 tile of 256 costs per
// product 0.75 of one of 128 and 0.4 of one of 64, and loses when there are too
// few tiles.  The tiles that do not fill a last round on all compute units (all
// of them, when there are fewer) may be split: their parts are a second launch,
// written and read once more, and joined by a third (one token
// through 4096 x 11008: 42 us whole, 23 us in four parts).
Cut pick_cut(Form form, LinEpi epi, const LinProb* p, int n) {
  constexpr double kLaunch = 3.0, kBytesPerUs = 8.0e6;
  const LinKind kind = form.kind;
  const bool f32 = kind == LIN_F32;
  Cut best;
  for (int tile = kind == LIN_SPLIT ? 256 : 64; tile <= (f32 || form.raw ? 128 : 256); tile *= 2) {
    if (f32 && tile == 128 && epi == LIN_DGATE) break;
    const double side = epi == LIN_GATE ? tile / 2 : tile;
    double tiles = 0, steps = 0;
    for (int i = 0; i < n; ++i) {
      const double b = std::ceil(p[i].M / (double)tile) * std::ceil(p[i].N / side);
      tiles += b;
      steps += b * std::ceil(p[i].K / (f32 ? 32.0 : 64.0)) * p[i].nseg * (kind == LIN_SPLIT ? 6 : 1);
    }
    const double mean = steps / tiles;
    auto time = [&](double units, double st) {
      const Rate r = lin_rate(form, tile, units);
      const double over = epi == LIN_GATE ? r.gate : epi == LIN_DGATE ? r.dgate : r.over;
      const double cu = std::ceil(units / kLinCu), full = std::floor(cu / r.places) * r.places, rest = cu - full;
      return full * (st * r.busy + over) + (rest > 0 ? std::max(rest * (st * r.busy + over), st * r.lat + over) : 0.0);
    };
    const double t1 = kLaunch + time(tiles, mean);
    if (best.us == 0.0 || t1 < best.us) best = {tile, 0, 1, t1};
    const double full = std::floor(tiles / kLinCu) * kLinCu, rest = tiles - full;
    if (rest == 0) continue;
    for (int s = 2; s <= 64; s += s < 4 ? 1 : s / 2) {
      if (mean / s < 2.0) break;
      const double parts = rest * s;
      if (parts > 8 * kLinCu) break;
      // a gate's join moves its matrices as well, in pieces of rows
      const bool gate = epi == LIN_GATE || epi == LIN_DGATE;
      const double join = (gate ? 6.0 : 3.0) + rest * tile * tile * (gate ? 64.0 : 4.0) / kBytesPerUs;
      const double t = (full > 0 ? kLaunch + time(full, mean) : 0.0) + 2 * kLaunch + time(parts, mean / s) +
                       parts * tile * tile * 8.0 / kBytesPerUs + join;
      if (t < best.us) best = {tile, (int64_t)rest, s, t};
    }
  }
  return best;
}

// A product's sizes, for the model.
struct Shape {
  LinEpi epi;
  int64_t M, N, K;
  int nseg;
  bool aligned = false;  // never raw
};
// The form that a call's products are modelled to be fastest in.
//  - Of the call's operands `copy` elements have rows that do not start 16-byte
//    aligned.  A product can take them raw, at 1.6 times the K step of a small
//    tile, or from padded copies (2 bytes read and written per element and 5 us):
//    raw wins for few tokens (10 tokens of 3463 x 20480, both ways: 562 us with
//    copies, 410 raw), copies for many.
//  - fp32 products can run on planes: six bf16 products take 0.65 of the time
//    of one in fp32 at full compute units (4096 tokens of 2048 x 8192: 142
//    against 207 TFLOP/s), at the cost of writing `split` elements as planes in
//    `launches` passes and of having only large tiles.
Form pick_form(int dtype, const Shape* s, int n, double copy, double split, int launches) {
  const LinKind plain = dtype == DMUON_BF16 ? LIN_BF16 : LIN_F32;
  const int es = dtype == DMUON_BF16 ? 2 : 4;
  auto cost = [&](Form f) {
    double t = f.kind == LIN_SPLIT ? split * 10.0 / 4.0e6 + 6.0 * launches
                                   : (copy > 0 && !f.raw ? copy * 2.0 * es / 4.0e6 + 5.0 : 0.0);
    for (int i = 0; i < n; ++i) {
      LinProb p{};
      p.M = (int32_t)std::max<int64_t>(1, s[i].M);
      p.N = (int32_t)s[i].N;
      p.K = (int32_t)s[i].K;
      p.nseg = s[i].nseg;
      t += pick_cut({f.kind, f.raw && !s[i].aligned}, s[i].epi, &p, 1).us;
    }
    return t;
  };
  Form best{plain, false};
  double best_t = cost(best);
  auto offer = [&](Form f) {
    const double t = cost(f);
    if (t < best_t) best = f, best_t = t;
  };
  if (copy > 0) offer({plain, true});
  if (plain == LIN_F32) offer({LIN_SPLIT, false});
  return best;
}

// Two cleared flags for the planes of a call's operands and of what it computes
// from them (LIN_SPLIT).
int take_flags(Arena& ar, Form form, int32_t** flags) {
  *flags = nullptr;
  if (form.kind != LIN_SPLIT) return DMUON_OK;
  *flags = (int32_t*)ar.take(8);
  return launch(ar, "clear_flags_kernel", 0.0, 8.0, [&] { return launch_clear_flags(*flags, 2, ar.st); });
}

std::string lin_name(Form form, int tile, LinMode mode, LinEpi epi) {
  static const char* const kinds[] = {"bf16, ", "f32, ", "split, "};
  static const char* const modes[] = {"kk", "kr", "rr"};
  static const char* const epis[] = {"out", "acc", "gate", "dgate", "xent"};
  return std::string("linear_kernel<") + kinds[form.kind] + std::to_string(tile) + ", " + modes[mode] +
         ", " + epis[epi] + (form.raw ? ", raw>" : ">");
}

LinProb prob(const Mat& x, const Mat& y, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K) {
  LinProb p{};
  p.x = x.p;
  p.ldx = x.ld;
  p.xplane = x.plane;
  p.xflag = x.flag;
  p.y = y.p;
  p.ldy = y.ld;
  p.yplane = y.plane;
  p.yflag = y.flag;
  p.c = c;
  p.ldc = ldc;
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.K = (int32_t)(x.plane ? round_up(K, 64) : K);  // planes are zero from K on
  p.npad = (int32_t)N;
  p.nseg = 1;
  p.splits = 1;
  return p;
}

// Launch the problems of `a` cut as `cut` says (or as pick_cut finds best).
int run(Arena& ar, Form form, const int32_t* flags, LinMode mode, LinEpi epi, LinArgs& a, const Cut* given = nullptr) {
  const Cut cut = given ? *given : pick_cut(form, epi, a.p, a.nprob);
  const int64_t mark = ar.used;
  double flops = 0.0;
  int64_t left = cut.split_tiles;
  for (int i = a.nprob - 1; i >= 0; --i) {
    LinProb& p = a.p[i];
    const int64_t side = epi == LIN_GATE ? cut.tile / 2 : cut.tile;
    const int64_t tiles = ((p.M + cut.tile - 1) / cut.tile) * ((p.N + side - 1) / side);
    const int64_t mine = std::min(left, tiles);
    left -= mine;
    if (tiles > (1 << 26)) return fail(DMUON_EUNSUPPORTED, "a product of %d x %d is too large", p.M, p.N);
    p.split_tiles = (int32_t)mine;
    p.splits = mine > 0 ? cut.splits : 1;
    p.part = mine > 0 ? (float*)ar.take(mine * cut.splits * cut.tile * cut.tile * 4) : nullptr;
    flops += (epi == LIN_GATE ? 4.0 : 2.0) * p.M * p.N * p.K * p.nseg;
  }
  ar.used = mark;  // the next launch on the stream may use the parts' memory
  a.raw = form.raw;
  a.flags = flags;
  if (ar.dry) return DMUON_OK;
  return launch(ar, lin_name(form, cut.tile, mode, epi).c_str(), flops, 0.0,
                [&] { return launch_linear(form.kind, cut.tile, mode, epi, a, ar.st); });
}

// ---------------------------------------------------------------- gated block
struct Ffn {
  const void *dy, *x, *wg, *wu, *wd;
  void *y, *dx, *dwg, *dwu, *dwd;
  void* saved;
  int64_t T, d, f;
  int act, dtype;
};

// What the forward pass leaves: planes g, u and h of T rows with padded pitch
// and, for 16-bit types, the plane of g's and u's low bits.
int64_t low_ld(int64_t f) { return round_up(f, 16); }
int64_t saved_bytes(int64_t T, int64_t f, int es) {
  return 3 * T * pitch(f, es) * es + (es == 2 ? T * low_ld(f) : 0);
}

int ffn_fwd(Arena& ar, const Ffn& q) {
  const int es = esize_of(q.dtype);
  const int64_t fp = pitch(q.f, es);
  const Shape shapes[] = {{LIN_GATE, q.T, q.f, q.d, 1}, {LIN_OUT, q.T, q.d, q.f, 1}};
  const double df = (double)q.d * q.f;
  // elements of x, Wg, Wu (rows of d) and Wd (rows of f) that need copies
  const double copy = (needs_copy(ar, q.d, es) ? (double)q.T * q.d + 2.0 * df : 0.0) + (needs_copy(ar, q.f, es) ? df : 0.0);
  const Form form = pick_form(q.dtype, shapes, 2, copy, (double)q.T * (q.d + q.f) + 3.0 * df, 2);
  int32_t* flags;
  TRY(take_flags(ar, form, &flags));
  Operands ops(ar, form, flags, 0);
  const Mat x = ops.add(q.x, q.T, q.d), wg = ops.add(q.wg, q.f, q.d), wu = ops.add(q.wu, q.f, q.d),
            wd = ops.add(q.wd, q.d, q.f);
  TRY(ops.make());
  const int64_t plane = q.T * fp * es;
  char* sv = (char*)q.saved;
  // sized for the call without `saved`, which alone needs h here
  void* h = sv ? sv + 2 * plane : ar.take(plane);
  LinArgs a{};
  a.nprob = 1;
  a.act = q.act;
  a.p[0] = prob(x, wg, h, fp, q.T, q.f, q.d);
  a.p[0].y2 = wu.p;
  a.p[0].c2 = sv;
  a.p[0].c3 = sv ? sv + plane : nullptr;
  a.p[0].c4 = sv ? sv + 3 * plane : nullptr;
  a.p[0].ld4 = low_ld(q.f);
  a.p[0].npad = (int32_t)padded(q.f, es);
  TRY(run(ar, form, flags, LIN_KK, LIN_GATE, a));
  Operands mid(ar, form, flags, 1);
  const Mat hm = mid.add(h, q.T, q.f, fp);
  TRY(mid.make());
  LinArgs b{};
  b.nprob = 1;
  b.p[0] = prob(hm, wd, q.y, q.d, q.T, q.d, q.f);
  TRY(run(ar, form, flags, LIN_KK, LIN_OUT, b));
  return DMUON_OK;
}

int ffn_bwd(Arena& ar, const Ffn& q) {
  const int es = esize_of(q.dtype);
  const int64_t fp = pitch(q.f, es);
  const Shape shapes[] = {
      {LIN_DGATE, q.T, q.f, q.d, 1}, {LIN_OUT, q.T, q.d, q.f, 2}, {LIN_OUT, 3 * q.f, q.d, q.T, 1, true}};
  const double df = (double)q.d * q.f;
  const double copy =
      (needs_copy(ar, q.d, es) ? 2.0 * q.T * q.d + 2.0 * df : 0.0) + (needs_copy(ar, q.f, es) ? df : 0.0);
  const Form form = pick_form(q.dtype, shapes, 3, copy, (double)q.T * (2.0 * q.d + 3.0 * q.f) + 3.0 * df, 2);
  int32_t* flags;
  TRY(take_flags(ar, form, &flags));
  Operands ops(ar, form, flags, 0);
  const Mat dy = ops.add(q.dy, q.T, q.d, 0, true), x = ops.add(q.x, q.T, q.d, 0, true),
            wg = ops.add(q.wg, q.f, q.d), wu = ops.add(q.wu, q.f, q.d), wd = ops.add(q.wd, q.d, q.f);
  TRY(ops.make());
  const int64_t plane = q.T * fp * es;
  const char* sv = (const char*)q.saved;
  void* dg = ar.take(plane);
  void* du = ar.take(plane);
  Operands mid(ar, form, flags, 1);
  const Mat dgm = mid.add(dg, q.T, q.f, fp), dum = mid.add(du, q.T, q.f, fp), hm = mid.add(sv + 2 * plane, q.T, q.f, fp);
  if (q.T > 0) {
    LinArgs a{};
    a.nprob = 1;
    a.act = q.act;
    a.p[0] = prob(dy, wd, dg, fp, q.T, q.f, q.d);
    a.p[0].c2 = du;
    a.p[0].aux1 = sv;
    a.p[0].aux2 = sv + plane;
    a.p[0].aux3 = sv + 3 * plane;
    a.p[0].ld4 = low_ld(q.f);
    a.p[0].npad = (int32_t)padded(q.f, es);
    TRY(run(ar, form, flags, LIN_KR, LIN_DGATE, a));
    TRY(mid.make());
    LinArgs b{};
    b.nprob = 1;
    b.p[0] = prob(dgm, wg, q.dx, q.d, q.T, q.d, q.f);
    b.p[0].x2 = dum.p;
    b.p[0].y2 = wu.p;
    b.p[0].nseg = 2;
    TRY(run(ar, form, flags, LIN_KR, LIN_OUT, b));
  }
  // the three weight gradients share one grid (tokens = 0: zeros)
  LinArgs w{};
  w.nprob = 3;
  w.p[0] = prob(dgm, x, q.dwg, q.d, q.f, q.d, q.T);
  w.p[1] = prob(dum, x, q.dwu, q.d, q.f, q.d, q.T);
  w.p[2] = prob(dy, hm, q.dwd, q.f, q.d, q.f, q.T);
  TRY(run(ar, {form.kind, false}, flags, LIN_RR, LIN_OUT, w));
  return DMUON_OK;
}

// ---------------------------------------------------------------- cross entropy
struct Xent {
  const void *x, *w;
  const int64_t* targets;
  float *loss, *losses;
  void *dx, *dw;
  int64_t T, d, V;
  int dtype;
  int64_t max_block;
  bool grad;
};

int xent(Arena& ar, const Xent& q) {
  const int es = esize_of(q.dtype);
  const int64_t vp = pitch(q.V, es);
  // by the logits' product alone, as everything that sets the order of the loss's
  // sums: its bits do not depend on whether the gradients are asked for
  const Shape logits{LIN_XENT, q.T, q.V, q.d, 1};
  const double copy = needs_copy(ar, q.d, es) ? (double)(q.T + q.V) * q.d : 0.0;
  const Form form = pick_form(q.dtype, &logits, 1, copy, (double)(q.T + q.V) * q.d, 1);
  const bool split = form.kind == LIN_SPLIT;
  int32_t* flags;
  TRY(take_flags(ar, form, &flags));
  Operands ops(ar, form, flags, 0);
  const Mat x = ops.add(q.x, q.T, q.d, 0, q.grad), w = ops.add(q.w, q.V, q.d);
  TRY(ops.make());
  float* alpha = (float*)ar.take(4);
  float* tl = (float*)ar.take(q.T * 4);
  // tokens per block of a call with gradients: within the cap, whole 256-row tiles
  const int64_t cap = q.max_block > 0 ? q.max_block : kDefaultBlock;
  const int64_t vs = round_up(q.V, 64), row = vp * es + (split ? 2 * kPlanes * vs : 0);
  int64_t tb = q.T;
  if (q.T * row > cap) tb = std::min(q.T, std::max<int64_t>(256, cap / row / 256 * 256));
  // the tile of a block's logits sets the pieces; in the last of several, which
  // may be of another size, none is split
  LinProb shape{};
  shape.M = (int32_t)std::max<int64_t>(1, tb);
  shape.N = (int32_t)q.V;
  shape.K = (int32_t)q.d;
  shape.nseg = 1;
  Cut cut = pick_cut(form, LIN_XENT, &shape, 1);
  if (tb < q.T) cut.split_tiles = 0;
  if (!q.grad) tb = q.T;  // the loss alone keeps no exponentials: one block
  const int64_t blocks = tb > 0 ? (q.T + tb - 1) / tb : 0;
  // dl is held times 2^-ceil(log2 tokens), so that dW's sums over tokens stay
  // within twice x's largest magnitude; the products divide it out
  float scale = 1.0f;
  while (scale * (float)q.T > 1.0f) scale *= 0.5f;
  auto mean = [&](const float* losses) {
    return launch(ar, "xent_mean_kernel", 0.0, 12.0 * q.T,
                  [&] { return launch_xent_mean(q.targets, losses, q.T, q.V, scale, alpha, q.loss, ar.st); });
  };
  // the gradients' products scale by the count, so with several blocks of
  // tokens it is taken first
  if (blocks > 1) TRY(mean(nullptr));
  const int tile = cut.tile;
  const int64_t pieces = (q.V + tile - 1) / tile * 2;
  float2* stats = (float2*)ar.take(tb * pieces * 8);
  void* p = q.grad ? ar.take(tb * vp * es) : nullptr;
  const int64_t prows = round_up(tb, 64);
  void* planes = q.grad && split ? ar.take(kPlanes * prows * vs * 2) : nullptr;
  float* dw_acc = q.grad && blocks > 1 ? (float*)ar.take(q.V * round_up(q.d, 4) * 4) : nullptr;
  for (int64_t b = 0; b < blocks; ++b) {
    const int64_t t0 = b * tb, tn = std::min(tb, q.T - t0);
    const Mat xb{(const char*)x.p + t0 * x.ld * (split ? 2 : es), x.ld, x.plane, x.flag};
    LinArgs l{};
    l.nprob = 1;
    l.pieces = (int32_t)pieces;
    l.targets = q.targets + t0;
    l.stats = stats;
    l.target_logit = tl + t0;
    l.p[0] = prob(xb, w, p, vp, tn, q.V, q.d);
    l.p[0].npad = (int32_t)padded(q.V, es);
    TRY(run(ar, form, flags, LIN_KK, LIN_XENT, l, &cut));
    XentArgs r{};
    r.targets = q.targets + t0;
    r.tokens = tn;
    r.vocab = q.V;
    r.stats = stats;
    r.pieces = (int32_t)pieces;
    r.piece = tile / 2;
    r.target_logit = tl + t0;
    r.losses = q.losses + t0;
    r.p = p;
    r.ldp = vp;
    r.esize = es;
    r.planes = (uint16_t*)planes;
    r.flag = flags ? flags + 1 : nullptr;
    r.scale = scale;
    TRY(launch(ar, "xent_rows_kernel", 0.0, (p ? 2.0 * tn * vp * es : 0.0) + 8.0 * tn * pieces,
               [&] { return launch_xent_rows(r, ar.st); }));
    if (planes) {
      FiniteArgs fin{};
      fin.planes[0] = r.planes;
      fin.plane[0] = round_up(tn, 64) * vs;
      fin.n = 1;
      fin.flag = r.flag;
      TRY(launch(ar, "finite_plane_kernel", 0.0, 0.0, [&] { return launch_finite_plane(fin, ar.st); }));
    }
    if (b == blocks - 1) TRY(mean(q.losses));
    if (!q.grad) continue;
    const Mat pm = split ? Mat{planes, vs, round_up(tn, 64) * vs, 1} : Mat{p, vp};
    LinArgs dx{};
    dx.nprob = 1;
    dx.alpha = alpha;
    dx.p[0] = prob(pm, w, (char*)q.dx + t0 * q.d * es, q.d, tn, q.d, q.V);
    TRY(run(ar, form, flags, LIN_KR, LIN_OUT, dx));
    LinArgs dw{};
    dw.nprob = 1;
    if (blocks == 1) {
      dw.alpha = alpha;
      dw.p[0] = prob(pm, xb, q.dw, q.d, q.V, q.d, tn);
      TRY(run(ar, {form.kind, false}, flags, LIN_RR, LIN_OUT, dw));
    } else {
      dw.accumulate = b > 0;
      dw.p[0] = prob(pm, xb, dw_acc, round_up(q.d, 4), q.V, q.d, tn);
      TRY(run(ar, {form.kind, false}, flags, LIN_RR, LIN_ACC, dw));
    }
  }
  if (q.grad && blocks > 1) {
    TRY(launch(ar, "scale_round_kernel", 0.0, (double)q.V * q.d * (4 + es), [&] {
      return launch_scale_round(dw_acc, round_up(q.d, 4), q.dw, q.V, q.d, es, alpha, ar.st);
    }));
  }
  if (blocks == 0) TRY(mean(q.loss));  // (no token's loss is read)
  if (q.grad && blocks == 0) {
    LinArgs dw{};  // no tokens: zeros
    dw.nprob = 1;
    dw.p[0] = prob({x.p, vp}, x, q.dw, q.d, q.V, q.d, 0);
    TRY(run(ar, {split ? LIN_F32 : form.kind, false}, flags, LIN_RR, LIN_OUT, dw));
  }
  return DMUON_OK;
}

int check_sizes(int64_t tokens, int64_t d, int dtype) {
  if (dtype != DMUON_BF16 && dtype != DMUON_F32) return fail(DMUON_EINVAL, "unknown dtype %d", dtype);
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(DMUON_EINVAL, "tokens (rows) = %lld is out of range", (long long)tokens);
  if (d < 1 || d > kMaxWidth) return fail(DMUON_EINVAL, "width %lld is out of [1, 2^20]", (long long)d);
  return DMUON_OK;
}
int check_hidden(int64_t f) {
  if (f < 1 || f > kMaxWidth) return fail(DMUON_EINVAL, "hidden width %lld is out of [1, 2^20]", (long long)f);
  return DMUON_OK;
}
int check_vocab(int64_t v) {
  if (v < 1 || v > kMaxVocab) return fail(DMUON_EINVAL, "vocabulary %lld is out of [1, 2^22]", (long long)v);
  return DMUON_OK;
}
int check_act(int act) {
  if (act < DMUON_ACT_SILU || act > DMUON_ACT_GELU_TANH) return fail(DMUON_EINVAL, "unknown activation %d", act);
  return DMUON_OK;
}
// No C++ exception crosses the C boundary.
template <class F>
auto guard(F&& f) -> decltype(f()) {
  try {
    return f();
  } catch (...) {
    return fail(DMUON_ENOMEM, "host allocation failed");
  }
}
// run `f` dry, then, when the workspace holds it, for real
template <class F>
int sized(void* ws, int64_t bytes, bool unaligned, void* stream, F&& f) {
  Arena dry;
  dry.unaligned = unaligned;
  TRY(f(dry));
  if (dry.peak > bytes)
    return fail(DMUON_EINVAL, "workspace of %lld bytes, %lld needed", (long long)bytes, (long long)dry.peak);
  if (dry.peak > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)))
    return fail(DMUON_EINVAL, "workspace is NULL or not 256-byte aligned");
  Arena ar;
  ar.base = (char*)ws;
  ar.cap = bytes;
  ar.dry = false;
  ar.unaligned = unaligned;
  ar.st = static_cast<hipStream_t>(stream);
  return guard([&] { return f(ar); });
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_layernorm_fwd(const void* x, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                        int64_t rows, int64_t width, float eps, int dtype, void* stream) {
  TRY(check_sizes(rows, width, dtype));
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(DMUON_EINVAL, "eps must be finite and >= 0");
  if (!weight) return fail(DMUON_EINVAL, "weight is NULL");
  if (rows == 0) return DMUON_OK;
  if (!x || !y || !mean || !rstd) return fail(DMUON_EINVAL, "x/y/mean/rstd is NULL");
  NormFwdArgs a{x, weight, bias, y, mean, rstd, rows, width, eps, esize_of(dtype)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return guard([&]() -> int {
    HIP_TRY(timed_launch("layernorm_fwd_kernel", 0.0, 2.0 * rows * width * a.esize, st,
                         [&] { return launch_layernorm_fwd(a, st); }));
    return DMUON_OK;
  });
}

int64_t dmuon_layernorm_bwd_workspace(int64_t rows, int64_t width) {
  TRY(check_sizes(rows, width, DMUON_F32));
  return layernorm_parts(rows, width) * 2 * width * 4;
}

int dmuon_layernorm_bwd(const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
                        void* dx, void* dweight, void* dbias, int64_t rows, int64_t width, int dtype,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  TRY(check_sizes(rows, width, dtype));
  if (!weight || !dweight) return fail(DMUON_EINVAL, "weight/dweight is NULL");
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return fail(DMUON_EINVAL, "dy/x/mean/rstd/dx is NULL");
  const int64_t need = dmuon_layernorm_bwd_workspace(rows, width);
  if (need > workspace_bytes)
    return fail(DMUON_EINVAL, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return fail(DMUON_EINVAL, "workspace is NULL or not 256-byte aligned");
  NormBwdArgs a{dy, x, weight, mean, rstd, dx, dweight, dbias, (float*)workspace, rows, width,
                (int32_t)layernorm_parts(rows, width), esize_of(dtype)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return guard([&]() -> int {
    HIP_TRY(timed_launch("layernorm_bwd_kernel", 0.0, 3.0 * rows * width * a.esize, st,
                         [&] { return launch_layernorm_bwd(a, st); }));
    return DMUON_OK;
  });
}

int64_t dmuon_gated_ffn_saved(int64_t tokens, int64_t hidden, int dtype) {
  TRY(check_sizes(tokens, 1, dtype));
  TRY(check_hidden(hidden));
  return saved_bytes(tokens, hidden, esize_of(dtype));
}

int64_t dmuon_gated_ffn_fwd_workspace(int64_t tokens, int64_t d, int64_t hidden, int dtype, int unaligned) {
  TRY(check_sizes(tokens, d, dtype));
  TRY(check_hidden(hidden));
  Arena ar;
  ar.unaligned = unaligned != 0;
  Ffn q{};
  q.T = tokens, q.d = d, q.f = hidden, q.dtype = dtype;
  if (tokens > 0) TRY(ffn_fwd(ar, q));
  return ar.peak;
}

int dmuon_gated_ffn_fwd(const void* x, const void* w_gate, const void* w_up, const void* w_down, void* y,
                        void* saved, int64_t tokens, int64_t d, int64_t hidden, int act, int dtype,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  TRY(check_sizes(tokens, d, dtype));
  TRY(check_hidden(hidden));
  TRY(check_act(act));
  if (!w_gate || !w_up || !w_down) return fail(DMUON_EINVAL, "w_gate/w_up/w_down is NULL");
  if (tokens == 0) return DMUON_OK;
  if (!x || !y) return fail(DMUON_EINVAL, "x/y is NULL");
  if (saved && (reinterpret_cast<uintptr_t>(saved) & 255)) return fail(DMUON_EINVAL, "saved is not 256-byte aligned");
  Ffn q{};
  q.x = x, q.wg = w_gate, q.wu = w_up, q.wd = w_down, q.y = y, q.saved = saved;
  q.T = tokens, q.d = d, q.f = hidden, q.act = act, q.dtype = dtype;
  const bool un = misaligned(x) || misaligned(w_gate) || misaligned(w_up) || misaligned(w_down);
  return sized(workspace, workspace_bytes, un, stream,
               [&](Arena& ar) { return ffn_fwd(ar, q); });
}

int64_t dmuon_gated_ffn_bwd_workspace(int64_t tokens, int64_t d, int64_t hidden, int dtype, int unaligned) {
  TRY(check_sizes(tokens, d, dtype));
  TRY(check_hidden(hidden));
  Arena ar;
  ar.unaligned = unaligned != 0;
  Ffn q{};
  q.T = tokens, q.d = d, q.f = hidden, q.dtype = dtype;
  TRY(ffn_bwd(ar, q));
  return ar.peak;
}

int dmuon_gated_ffn_bwd(const void* dy, const void* x, const void* w_gate, const void* w_up, const void* w_down,
                        const void* saved, void* dx, void* dw_gate, void* dw_up, void* dw_down, int64_t tokens,
                        int64_t d, int64_t hidden, int act, int dtype, void* workspace, int64_t workspace_bytes,
                        void* stream) {
  TRY(check_sizes(tokens, d, dtype));
  TRY(check_hidden(hidden));
  TRY(check_act(act));
  if (!w_gate || !w_up || !w_down || !dw_gate || !dw_up || !dw_down)
    return fail(DMUON_EINVAL, "a weight or weight gradient is NULL");
  if (tokens > 0 && (!dy || !x || !saved || !dx)) return fail(DMUON_EINVAL, "dy/x/saved/dx is NULL");
  if (saved && (reinterpret_cast<uintptr_t>(saved) & 255)) return fail(DMUON_EINVAL, "saved is not 256-byte aligned");
  Ffn q{};
  q.dy = dy, q.x = x, q.wg = w_gate, q.wu = w_up, q.wd = w_down, q.saved = const_cast<void*>(saved);
  q.dx = dx, q.dwg = dw_gate, q.dwu = dw_up, q.dwd = dw_down;
  q.T = tokens, q.d = d, q.f = hidden, q.act = act, q.dtype = dtype;
  const bool un =
      misaligned(dy) || misaligned(x) || misaligned(w_gate) || misaligned(w_up) || misaligned(w_down);
  return sized(workspace, workspace_bytes, un, stream, [&](Arena& ar) { return ffn_bwd(ar, q); });
}

int64_t dmuon_linear_xent_workspace(int64_t tokens, int64_t d, int64_t vocab, int dtype, int grad,
                                    int64_t max_block, int unaligned) {
  TRY(check_sizes(tokens, d, dtype));
  TRY(check_vocab(vocab));
  Arena ar;
  ar.unaligned = unaligned != 0;
  Xent q{};
  q.T = tokens, q.d = d, q.V = vocab, q.dtype = dtype, q.max_block = max_block, q.grad = grad != 0;
  TRY(xent(ar, q));
  return ar.peak;
}

int dmuon_linear_xent(const void* x, const void* weight, const int64_t* targets, float* loss, float* losses,
                      void* dx, void* dweight, int64_t tokens, int64_t d, int64_t vocab, int dtype,
                      int64_t max_block, void* workspace, int64_t workspace_bytes, void* stream) {
  TRY(check_sizes(tokens, d, dtype));
  TRY(check_vocab(vocab));
  if (!weight || !loss) return fail(DMUON_EINVAL, "weight/loss is NULL");
  if (tokens > 0 && (!x || !targets || !losses)) return fail(DMUON_EINVAL, "x/targets/losses is NULL");
  if (!dx != !dweight && tokens > 0) return fail(DMUON_EINVAL, "dx and dweight: both or neither");
  if (max_block < 0) return fail(DMUON_EINVAL, "max_block must be >= 0");
  Xent q{};
  q.x = x, q.w = weight, q.targets = targets, q.loss = loss, q.losses = losses, q.dx = dx, q.dw = dweight;
  q.T = tokens, q.d = d, q.V = vocab, q.dtype = dtype, q.max_block = max_block, q.grad = dweight != nullptr;
  return sized(workspace, workspace_bytes, misaligned(x) || misaligned(weight), stream,
               [&](Arena& ar) { return xent(ar, q); });
}

}  // extern "C"
