// Host side of the state-space block's operators declared in include/rnn.h:
// argument validation, workspace layout and the enqueue of their kernels.
// Nothing is kept between calls.
#include <cmath>

#include "api_checks.hpp"
#include "state_block_kernels.hpp"

using namespace rnnk;

namespace {

static_assert(RNN_CONV_MAX_W == kConvMaxW, "the longest filter");
static_assert(RNN_SELECTIVE_MAX_N == kSelMaxN, "the longest state");

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// ---------------------------------------------------------------------------
// Causal convolution
// ---------------------------------------------------------------------------
int validate(const RnnCausalConvDesc* d) {
  if (!d) return RNN_E_NULL;
  if (!dtype_ok(d->dtype)) return RNN_E_UNSUPPORTED;
  if (d->T < 1 || d->B < 1 || d->C < 1 || d->W < 1) return RNN_E_SHAPE;
  if (d->W < 2 || d->W > RNN_CONV_MAX_W) return RNN_E_UNSUPPORTED;
  if (d->activation != RNN_ACT_NONE && d->activation != RNN_ACT_SILU) return RNN_E_UNSUPPORTED;
  if (d->x_t < 0 || d->x_b < 0 || d->T > kMaxGrid - 64) return RNN_E_SHAPE;
  // the forward launch, and the one that adds up the gradients of the filter
  if (conv_threads(d->T, d->B, d->C) > kMaxThreads) return RNN_E_SHAPE;
  if (8.0 * ((double)d->C + 32.0) * (d->W + 1) > kMaxThreads) return RNN_E_SHAPE;
  return RNN_OK;
}

size_t conv_workspace(const RnnCausalConvDesc* d) {
  return (size_t)conv_parts(d->T, d->B, d->C, kPlanCus) * (d->W + 1) * d->C * sizeof(float);
}

int conv_args(const RnnCausalConvDesc* d, const RnnCausalConvIO* io, CausalConvArgs* a) {
  if (!io) return RNN_E_NULL;
  const size_t e = (size_t)esize_of(d->dtype);
  RETURN_IF_BAD(need(io->x, e));
  RETURN_IF_BAD(need(io->weight, e));
  RETURN_IF_BAD(optional(io->bias, e));
  RETURN_IF_BAD(optional(io->lengths, 4));
  RETURN_IF_BAD(optional(io->state, e));
  *a = CausalConvArgs{};
  a->T = d->T; a->B = d->B; a->C = d->C; a->W = d->W; a->silu = d->activation == RNN_ACT_SILU;
  a->x = io->x; a->x_t = d->x_t; a->x_b = d->x_b;
  a->w = io->weight; a->bias = io->bias; a->lengths = io->lengths; a->state = io->state;
  const int64_t m = 16 / (int64_t)e;
  a->vec = d->C % m == 0 && d->x_t % m == 0 && d->x_b % m == 0 && aligned(io->x, 16) && aligned(io->state, 16);
  a->wvec = aligned(io->weight, 8) && aligned(io->bias, 8);
  return RNN_OK;
}

// ---------------------------------------------------------------------------
// Selective scan
// ---------------------------------------------------------------------------
int validate(const RnnSelectiveScanDesc* d) {
  if (!d) return RNN_E_NULL;
  if (!dtype_ok(d->dtype)) return RNN_E_UNSUPPORTED;
  if (d->T < 1 || d->B < 1 || d->H < 1 || d->N < 1 || d->G < 1) return RNN_E_SHAPE;
  if (d->N > RNN_SELECTIVE_MAX_N) return RNN_E_UNSUPPORTED;
  if (d->H % d->G != 0 || (d->softplus | 1) != 1 || (d->gate | 1) != 1) return RNN_E_SHAPE;
  for (int64_t s : {d->x_t, d->x_b, d->dt_t, d->dt_b, d->B_t, d->B_b, d->B_g, d->C_t, d->C_b, d->C_g})
    if (s < 0) return RNN_E_SHAPE;
  if (d->gate && (d->z_t < 0 || d->z_b < 0)) return RNN_E_SHAPE;
  if (d->T > kMaxGrid - 4096) return RNN_E_SHAPE;
  // the threads of the launches: tiles of 64 channels of a row (time is cut
  // only while they are few), the states of all rows, the numbers of dB and dC
  const double B = d->B, H = d->H, NP = sel_padded(d->N), T = d->T, G = d->G;
  const double tiles = (double)sel_group_tiles(d->H, d->G) * G;
  if ((B + 64.0) * tiles * 256.0 > kMaxThreads || B * H * NP + 256.0 > kMaxThreads) return RNN_E_SHAPE;
  if (T * B * G * 2.0 * NP + 256.0 > kMaxThreads || H * (NP + 2.0) * 4.0 + 256.0 > kMaxThreads) return RNN_E_SHAPE;
  return RNN_OK;
}

int sel_segments_of(const RnnSelectiveScanDesc* d, int* steps) {
  return sel_segments(d->T, d->B, d->H, d->N, d->G, kPlanCus, steps);
}

size_t sel_cells(const RnnSelectiveScanDesc* d) { return (size_t)d->B * d->H; }

// What the segments add to the state, and the sums of their steps.
size_t sel_map_bytes(const RnnSelectiveScanDesc* d) {
  int steps;
  const size_t segs = (size_t)sel_segments_of(d, &steps);
  return segs > 1 ? round16(segs * sel_cells(d) * sizeof(float)) : 0;
}
size_t sel_workspace(const RnnSelectiveScanDesc* d) { return sel_map_bytes(d) * (sel_padded(d->N) + 1); }

size_t sel_reserve(const RnnSelectiveScanDesc* d) {
  return (size_t)((d->T + kSelKeep - 1) / kSelKeep) * sel_cells(d) * sel_padded(d->N) * sizeof(float);
}

size_t sel_bc_bytes(const RnnSelectiveScanDesc* d) {
  return round16((size_t)sel_group_tiles(d->H, d->G) * d->T * d->B * d->G * 2 * sel_padded(d->N) * sizeof(float));
}
size_t sel_a_bytes(const RnnSelectiveScanDesc* d) {
  int steps;
  return (size_t)sel_segments_of(d, &steps) * sel_cells(d) * (sel_padded(d->N) + 2) * sizeof(float);
}
size_t sel_backward_workspace(const RnnSelectiveScanDesc* d) { return sel_workspace(d) + sel_bc_bytes(d) + sel_a_bytes(d); }

int sel_args(const RnnSelectiveScanDesc* d, const RnnSelectiveScanIO* io, void* ws, SelectiveScanArgs* a) {
  if (!io) return RNN_E_NULL;
  const size_t e = (size_t)esize_of(d->dtype);
  RETURN_IF_BAD(need(io->x, e));
  RETURN_IF_BAD(need(io->dt, e));
  if (d->gate) RETURN_IF_BAD(need(io->z, e));
  RETURN_IF_BAD(need(io->Bm, e));
  RETURN_IF_BAD(need(io->Cm, e));
  RETURN_IF_BAD(need(io->A, 4));
  RETURN_IF_BAD(optional(io->D, 4));
  RETURN_IF_BAD(optional(io->dt_bias, 4));
  RETURN_IF_BAD(optional(io->lengths, 4));
  RETURN_IF_BAD(optional(io->h0, 4));
  *a = SelectiveScanArgs{};
  a->T = d->T; a->B = d->B; a->H = d->H; a->N = d->N; a->G = d->G; a->softplus = d->softplus;
  a->x = io->x; a->x_t = d->x_t; a->x_b = d->x_b;
  a->dt = io->dt; a->dt_t = d->dt_t; a->dt_b = d->dt_b;
  if (d->gate) {
    a->z = io->z; a->z_t = d->z_t; a->z_b = d->z_b;
  }
  a->Bm = io->Bm; a->B_t = d->B_t; a->B_b = d->B_b; a->B_g = d->B_g;
  a->Cm = io->Cm; a->C_t = d->C_t; a->C_b = d->C_b; a->C_g = d->C_g;
  a->A = io->A; a->D = io->D; a->dt_bias = io->dt_bias; a->lengths = io->lengths; a->h0 = io->h0;
  a->segs = sel_segments_of(d, &a->seg_steps);
  if (a->segs > 1) {
    a->map_d = static_cast<float*>(ws);
    a->map_s = reinterpret_cast<float*>(static_cast<char*>(ws) + sel_map_bytes(d));
  }
  // whole vectors where every row of every [T, B, H] tensor and every group allows them
  const int64_t m = 16 / (int64_t)e;
  auto fits = [&](const void* p, int64_t t, int64_t b) { return aligned(p, 16) && t % m == 0 && b % m == 0; };
  a->vec = d->H / d->G % m == 0 && fits(a->x, a->x_t, a->x_b) && fits(a->dt, a->dt_t, a->dt_b) && fits(a->z, a->z_t, a->z_b);
  a->svec = d->N == sel_padded(d->N) && aligned(a->A, 16) && aligned(a->h0, 16);
  return RNN_OK;
}

int sel_forward(const RnnSelectiveScanDesc* d, const RnnSelectiveScanIO* io, void* reserve, void* ws, size_t ws_bytes,
                void* stream) {
  if (!io) return RNN_E_NULL;
  RETURN_IF_BAD(need_memory(ws, ws_bytes, sel_workspace(d)));
  SelectiveScanArgs a;
  RETURN_IF_BAD(sel_args(d, io, ws, &a));
  RETURN_IF_BAD(need(io->y, (size_t)esize_of(d->dtype)));
  RETURN_IF_BAD(optional(io->h_n, 4));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.xcds = xcds;
  a.y = io->y;
  a.h_n = io->h_n;
  if (!aligned(a.y, 16)) a.vec = 0;
  if (!aligned(a.h_n, 16)) a.svec = 0;
  a.keep = static_cast<float*>(reserve);
  return hip_status(launch_selective_scan(a, d->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// Gated feed-forward
// ---------------------------------------------------------------------------
constexpr int64_t kFeedMostWidth = 1 << 21;  // 256 rows of fp32 are 2 GiB

int validate(const RnnFeedForwardDesc* d) {
  if (!d) return RNN_E_NULL;
  if (!dtype_ok(d->dtype)) return RNN_E_UNSUPPORTED;
  if (d->activation != RNN_ACT_SILU && d->activation != RNN_ACT_GELU_TANH && d->activation != RNN_ACT_SIGMOID)
    return RNN_E_UNSUPPORTED;
  if (d->rows < 1 || d->N < 1 || d->F < 1 || d->N_out < 1 || (d->aligned | 1) != 1) return RNN_E_SHAPE;
  if (d->x_ld < d->N || d->in_ld < d->N || d->out_ld < d->F) return RNN_E_SHAPE;
  // rows, columns and steps of the products are counted in 32 bits, and so are
  // their tiles and the bytes of a tile's 256 rows
  if (d->rows > 1 << 30 || d->N > kFeedMostWidth || d->F > kFeedMostWidth / 2 || d->N_out > kFeedMostWidth) return RNN_E_SHAPE;
  auto tiles = [](double m, double n) { return (m / 128.0 + 1.0) * (n / 64.0 + 1.0) * 32.0; };
  const double r = (double)d->rows, n = d->N, f = 2.0 * d->F + 128.0, o = d->N_out;
  if (std::fmax(std::fmax(tiles(r, f), tiles(r, o)), std::fmax(tiles(f, n), std::fmax(tiles(r, n), tiles(o, f)))) > 2147483647.0)
    return RNN_E_SHAPE;
  return RNN_OK;
}

FeedSizes feed_sizes(const RnnFeedForwardDesc* d) { return FeedSizes(d->dtype == RNN_DTYPE_BF16, d->rows, d->N, d->F, d->N_out); }

// Operands that the tiled kernels cannot take as they are, and that are copied.
struct FeedCopies {
  bool x, in, out, dy;
  // those that may have to be, as far as the descriptor tells: what the workspace has room for
  FeedCopies(const RnnFeedForwardDesc* d, const FeedSizes& s) {
    x = !d->aligned || rows_off(s, d->N, d->x_ld);
    in = !d->aligned || rows_off(s, d->N, d->in_ld);
    out = !d->aligned || rows_off(s, d->F, d->out_ld);
    dy = !d->aligned || rows_off(s, d->N_out, d->N_out);
  }
  // those that have to be, each by itself
  FeedCopies(const RnnFeedForwardDesc* d, const FeedSizes& s, const RnnFeedForwardIO* io, const void* up) {
    x = !aligned(io->x, 16) || rows_off(s, d->N, d->x_ld);
    in = !aligned(io->w_in, 16) || rows_off(s, d->N, d->in_ld);
    out = !aligned(io->w_out, 16) || rows_off(s, d->F, d->out_ld);
    dy = !aligned(up, 16) || rows_off(s, d->N_out, d->N_out);
  }
  static bool rows_off(const FeedSizes& s, int64_t n, int64_t ld) { return n % s.m || ld % s.m || ld > kFeedMostWidth; }
};

// Where things lie in a workspace, one after the other.
struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += round16(n);
    return at;
  }
};

struct FeedSpace {
  size_t x, in, out, dy, h, dp, part, bytes;
};

size_t feed_part(const FeedPlan& p, size_t M, size_t N) { return p.splits > 1 ? p.splits * M * N * sizeof(float) : 0; }

// The forward (serving or training) or the backward pass.
FeedSpace feed_space(const RnnFeedForwardDesc* d, bool train, bool back) {
  const FeedSizes s = feed_sizes(d);
  const FeedCopies copy(d, s);
  const size_t e = (size_t)esize_of(d->dtype), rows = (size_t)d->rows;
  Layout l;
  FeedSpace a{};
  if (!back && s.few(train)) {  // any alignment is taken there
    if (!train) a.h = l.take(rows * s.Fp * e);
    const size_t splits = (size_t)feed_few_splits(d->rows, d->F, d->N_out, kPlanCus);
    a.part = l.take(splits > 1 ? splits * rows * d->N_out * sizeof(float) : 0);
    a.bytes = l.bytes;
    return a;
  }
  if (copy.x) a.x = l.take(rows * s.Np * e);
  if (copy.in) a.in = l.take(2 * (size_t)d->F * s.Np * e);
  if (copy.out) a.out = l.take((size_t)d->N_out * s.Fm * e);
  size_t part = 0;
  if (back) {
    if (copy.dy) a.dy = l.take(rows * s.Op * e);
    a.dp = l.take(rows * 2 * s.Fp * e);
    part = feed_part(s.plan(kFeedDx, kPlanCus), rows, d->N);
    const size_t dh = feed_part(s.plan(kFeedDh, kPlanCus), rows, s.Fp);
    if (part < dh) part = dh;
    const size_t in = feed_part(s.plan(kFeedDwIn, kPlanCus), 2 * (size_t)s.Fp, d->N);
    const size_t out = feed_part(s.plan(kFeedDwOut, kPlanCus), d->N_out, d->F);
    if (part < in) part = in;
    if (part < out) part = out;
  } else {
    if (!train) a.h = l.take(rows * s.Fp * e);
    part = feed_part(s.plan(kFeedOut, kPlanCus), rows, d->N_out);
    const size_t in = feed_part(s.plan(kFeedIn, kPlanCus), rows, 2 * (size_t)s.Fp);
    if (part < in) part = in;
  }
  a.part = l.take(part);
  a.bytes = l.bytes;
  return a;
}

// g and u, then h.
size_t feed_gu_bytes(const RnnFeedForwardDesc* d) { return (size_t)d->rows * 2 * feed_sizes(d).Fp * sizeof(float); }
size_t feed_reserve(const RnnFeedForwardDesc* d) {
  return feed_gu_bytes(d) + round16((size_t)d->rows * feed_sizes(d).Fp * esize_of(d->dtype));
}

// Operands as the kernels take them; those that they cannot take as they are
// go through one pass over all their rows.
struct FeedOperand {
  const void* p;
  int64_t ld;
};
struct FeedPacks {
  FeedPackArgs a{};
  FeedOperand add(const void* p, int64_t ld, bool pack, int64_t rows, int cols, int pitch, void* to) {
    if (!pack) return {p, ld};
    auto& t = a.t[a.count++];
    t.from = p; t.ld = ld; t.rows = rows; t.cols = cols; t.to = to; t.pitch = pitch;
    return {to, pitch};
  }
  hipError_t launch(bool bf, hipStream_t st) const { return a.count ? launch_feed_pack(a, bf, st) : hipSuccess; }
};

int feed_io(const RnnFeedForwardDesc* d, const RnnFeedForwardIO* io) {
  const size_t e = d->aligned ? 16 : (size_t)esize_of(d->dtype);
  if (!io) return RNN_E_NULL;
  RETURN_IF_BAD(need(io->x, e));
  RETURN_IF_BAD(need(io->w_in, e));
  return need(io->w_out, e);
}

#define RETURN_IF_HIP(expr)                   \
  do {                                        \
    if ((expr) != hipSuccess) return RNN_E_HIP; \
  } while (0)

int feed_forward(const RnnFeedForwardDesc* d, const RnnFeedForwardIO* io, void* reserve, void* ws, size_t ws_bytes, void* stream) {
  RETURN_IF_BAD(feed_io(d, io));
  const size_t e = (size_t)esize_of(d->dtype);
  RETURN_IF_BAD(optional(io->residual, e));
  if (io->residual && d->residual_ld < d->N_out) return RNN_E_SHAPE;
  RETURN_IF_BAD(need(io->y, e));
  const FeedSpace at = feed_space(d, reserve != nullptr, false);
  RETURN_IF_BAD(need_memory(ws, ws_bytes, at.bytes));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  const FeedSizes s = feed_sizes(d);
  const FeedCopies copy(d, s, io, nullptr);
  const bool bf = d->dtype == RNN_DTYPE_BF16;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  char* mem = static_cast<char*>(ws);
  void* h = reserve ? static_cast<char*>(reserve) + feed_gu_bytes(d) : mem + at.h;
  if (s.few(reserve != nullptr)) {
    FeedFewArgs f{};
    f.rows = (int)d->rows; f.n = d->N; f.F = d->F; f.n_out = d->N_out; f.act = d->activation;
    f.x = io->x; f.ldx = d->x_ld; f.w_in = io->w_in; f.ld_in = d->in_ld; f.w_out = io->w_out; f.ld_out = d->out_ld;
    f.residual = io->residual; f.ldr = io->residual ? d->residual_ld : 0;
    f.h = h; f.Fp = s.Fp; f.gu = static_cast<float*>(reserve); f.y = io->y;
    f.part = reinterpret_cast<float*>(mem + at.part);
    f.splits = feed_few_splits(d->rows, d->F, d->N_out, kPlanCus);
    return hip_status(launch_feed_few(f, bf, st));
  }
  FeedPacks packs;
  const FeedOperand x = packs.add(io->x, d->x_ld, copy.x, d->rows, d->N, s.Np, mem + at.x);
  const FeedOperand in = packs.add(io->w_in, d->in_ld, copy.in, 2 * (int64_t)d->F, d->N, s.Np, mem + at.in);
  const FeedOperand out = packs.add(io->w_out, d->out_ld, copy.out, d->N_out, d->F, s.Fm, mem + at.out);
  RETURN_IF_HIP(packs.launch(bf, st));
  auto* launch = bf ? launch_feed_bf16 : launch_feed_f32;
  FeedArgs a{};
  a.F = d->F; a.Fp = s.Fp; a.act = d->activation;
  a.M = (int)d->rows; a.N = s.Fp;
  a.A = x.p; a.lda = x.ld; a.KA = s.Np;
  a.B = in.p; a.ldb = in.ld; a.KB = s.Np;
  a.steps = s.steps(s.Np);
  a.out = h; a.ldo = s.Fp; a.gu = static_cast<float*>(reserve);
  FeedPlan p = s.plan(kFeedIn, kPlanCus);
  a.splits = p.splits; a.part = reinterpret_cast<float*>(mem + at.part);
  RETURN_IF_HIP(launch(kFeedIn, a, p, st));
  a.N = d->N_out;
  a.A = h; a.lda = s.Fp; a.KA = s.Fm;
  a.B = out.p; a.ldb = out.ld; a.KB = s.Fm;
  a.steps = s.steps(s.Fm);
  a.out = io->y; a.ldo = d->N_out; a.gu = nullptr;
  a.residual = io->residual; a.ldr = io->residual ? d->residual_ld : 0;
  p = s.plan(kFeedOut, kPlanCus);
  a.splits = p.splits;
  return hip_status(launch(kFeedOut, a, p, st));
}

int feed_backward(const RnnFeedForwardDesc* d, const RnnFeedForwardIO* io, const RnnFeedForwardGrads* g, const void* reserve,
                  char* mem, const FeedSpace& at, hipStream_t st) {
  const FeedSizes s = feed_sizes(d);
  const FeedCopies copy(d, s, io, g->dy);
  const bool bf = d->dtype == RNN_DTYPE_BF16;
  const int rows = (int)d->rows;
  FeedPacks packs;
  const FeedOperand x = packs.add(io->x, d->x_ld, copy.x, d->rows, d->N, s.Np, mem + at.x);
  const FeedOperand in = packs.add(io->w_in, d->in_ld, copy.in, 2 * (int64_t)d->F, d->N, s.Np, mem + at.in);
  const FeedOperand out = packs.add(io->w_out, d->out_ld, copy.out, d->N_out, d->F, s.Fm, mem + at.out);
  const FeedOperand dy = packs.add(g->dy, d->N_out, copy.dy, d->rows, d->N_out, s.Op, mem + at.dy);
  RETURN_IF_HIP(packs.launch(bf, st));
  auto* launch = bf ? launch_feed_bf16 : launch_feed_f32;
  void* dp = mem + at.dp;
  const void* h = static_cast<const char*>(reserve) + feed_gu_bytes(d);
  FeedArgs base{};
  base.F = d->F; base.Fp = s.Fp; base.act = d->activation;
  base.part = reinterpret_cast<float*>(mem + at.part);
  auto run = [&](int op, FeedArgs& a) {
    const FeedPlan p = s.plan(op, kPlanCus);
    a.splits = p.splits;
    return launch(op, a, p, st);
  };
  FeedArgs a = base;  // [dg, du]
  a.M = rows; a.N = s.Fp;
  a.A = dy.p; a.lda = dy.ld; a.KA = s.Op;
  a.B = out.p; a.ldb = out.ld; a.KB = d->N_out; a.cols_b = s.Fm;
  a.steps = s.steps(s.Op);
  a.out = dp; a.ldo = 2 * (int64_t)s.Fp;
  a.gu = const_cast<float*>(static_cast<const float*>(reserve));
  RETURN_IF_HIP(run(kFeedDh, a));
  a = base;           // dx
  a.M = rows; a.N = d->N;
  a.A = dp; a.lda = 2 * (int64_t)s.Fp; a.KA = 2 * s.Fp;
  a.B = in.p; a.ldb = in.ld; a.KB = d->F; a.cols_b = s.Np;
  a.steps = s.steps(2 * (int64_t)s.Fp);
  a.out = g->dx; a.ldo = d->N;
  RETURN_IF_HIP(run(kFeedDx, a));
  a = base;           // dw_in
  a.M = 2 * s.Fp; a.N = d->N;
  a.A = dp; a.lda = 2 * (int64_t)s.Fp; a.KA = rows; a.cols_a = 2 * s.Fp;
  a.B = x.p; a.ldb = x.ld; a.KB = rows; a.cols_b = s.Np;
  a.steps = s.steps(rows);
  a.out = g->dw_in; a.ldo = d->N; a.rows_split = s.Fp;
  RETURN_IF_HIP(run(kFeedDwIn, a));
  a = base;           // dw_out
  a.M = d->N_out; a.N = d->F;
  a.A = dy.p; a.lda = dy.ld; a.KA = rows; a.cols_a = s.Op;
  a.B = h; a.ldb = s.Fp; a.KB = rows; a.cols_b = s.Fp;
  a.steps = s.steps(rows);
  a.out = g->dw_out; a.ldo = d->F;
  return hip_status(run(kFeedDwOut, a));
}

}  // namespace

extern "C" {

int rnn_causal_conv(const RnnCausalConvDesc* desc, const RnnCausalConvIO* io, void* stream) {
  Range range("rnn_causal_conv");
  RETURN_IF_BAD(validate(desc));
  CausalConvArgs a;
  RETURN_IF_BAD(conv_args(desc, io, &a));
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(io->y, e));
  RETURN_IF_BAD(optional(io->state_n, e));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.y = io->y;
  a.state_n = io->state_n;
  if (!aligned(a.y, 16) || !aligned(a.state_n, 16)) a.vec = 0;
  return hip_status(launch_causal_conv(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int rnn_causal_conv_backward_workspace_bytes(const RnnCausalConvDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = conv_workspace(desc);
  return RNN_OK;
}

int rnn_causal_conv_backward(const RnnCausalConvDesc* desc, const RnnCausalConvIO* io, const RnnCausalConvGrads* grads,
                             void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_causal_conv_backward");
  RETURN_IF_BAD(validate(desc));
  if (!grads) return RNN_E_NULL;
  CausalConvArgs a;
  RETURN_IF_BAD(conv_args(desc, io, &a));
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(grads->dy, e));
  RETURN_IF_BAD(optional(grads->dstate_n, e));
  RETURN_IF_BAD(need(grads->dx, e));
  RETURN_IF_BAD(need(grads->dweight, 4));
  RETURN_IF_BAD(optional(grads->dbias, 4));
  RETURN_IF_BAD(optional(grads->dstate, e));
  RETURN_IF_BAD(need_memory(workspace, ws_bytes, conv_workspace(desc)));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.dy = grads->dy; a.dstate_n = grads->dstate_n;
  a.dx = grads->dx; a.dw = grads->dweight; a.db = grads->dbias; a.dstate = grads->dstate;
  a.part = static_cast<float*>(workspace);
  a.parts = conv_parts(desc->T, desc->B, desc->C, kPlanCus);
  for (const void* p : {a.dy, a.dstate_n, (const void*)a.dx, (const void*)a.dstate})
    if (!aligned(p, 16)) a.vec = 0;
  return hip_status(launch_causal_conv_backward(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int rnn_selective_scan_workspace_bytes(const RnnSelectiveScanDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = sel_workspace(desc);
  return RNN_OK;
}

int rnn_selective_scan_reserve_bytes(const RnnSelectiveScanDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = sel_reserve(desc);
  return RNN_OK;
}

int rnn_selective_scan_backward_workspace_bytes(const RnnSelectiveScanDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = sel_backward_workspace(desc);
  return RNN_OK;
}

int rnn_selective_scan(const RnnSelectiveScanDesc* desc, const RnnSelectiveScanIO* io, void* workspace, size_t ws_bytes,
                       void* stream) {
  Range range("rnn_selective_scan");
  RETURN_IF_BAD(validate(desc));
  return sel_forward(desc, io, nullptr, workspace, ws_bytes, stream);
}

int rnn_selective_scan_train(const RnnSelectiveScanDesc* desc, const RnnSelectiveScanIO* io, void* reserve,
                             size_t reserve_bytes, void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_selective_scan_train");
  RETURN_IF_BAD(validate(desc));
  if (!io) return RNN_E_NULL;
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, sel_reserve(desc)));
  return sel_forward(desc, io, reserve, workspace, ws_bytes, stream);
}

int rnn_selective_scan_backward(const RnnSelectiveScanDesc* desc, const RnnSelectiveScanIO* io,
                                const RnnSelectiveScanGrads* grads, const void* reserve, size_t reserve_bytes, void* workspace,
                                size_t ws_bytes, void* stream) {
  Range range("rnn_selective_scan_backward");
  RETURN_IF_BAD(validate(desc));
  if (!io || !grads) return RNN_E_NULL;
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, sel_reserve(desc)));
  RETURN_IF_BAD(need_memory(workspace, ws_bytes, sel_backward_workspace(desc)));
  SelectiveScanArgs a;
  RETURN_IF_BAD(sel_args(desc, io, workspace, &a));
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(grads->dy, e));
  RETURN_IF_BAD(optional(grads->dh_n, 4));
  RETURN_IF_BAD(need(grads->dx, e));
  RETURN_IF_BAD(need(grads->ddt, e));
  if (desc->gate) RETURN_IF_BAD(need(grads->dz, e));
  RETURN_IF_BAD(need(grads->dB, e));
  RETURN_IF_BAD(need(grads->dC, e));
  RETURN_IF_BAD(need(grads->dA, 4));
  RETURN_IF_BAD(optional(grads->dD, 4));
  RETURN_IF_BAD(optional(grads->ddt_bias, 4));
  RETURN_IF_BAD(optional(grads->dh0, 4));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.xcds = xcds;
  a.keep = const_cast<float*>(static_cast<const float*>(reserve));
  a.dy = grads->dy; a.dh_n = grads->dh_n;
  a.dx = grads->dx; a.ddt = grads->ddt; a.dz = desc->gate ? grads->dz : nullptr;
  a.dB = grads->dB; a.dC = grads->dC; a.dA = grads->dA; a.dD = grads->dD; a.dbias = grads->ddt_bias; a.dh0 = grads->dh0;
  a.part_bc = reinterpret_cast<float*>(static_cast<char*>(workspace) + sel_workspace(desc));
  a.part_a = reinterpret_cast<float*>(static_cast<char*>(workspace) + sel_workspace(desc) + sel_bc_bytes(desc));
  for (const void* p : {a.dy, (const void*)a.dx, (const void*)a.ddt, (const void*)a.dz})
    if (!aligned(p, 16)) a.vec = 0;
  if (!aligned(a.dh_n, 16) || !aligned(a.dh0, 16)) a.svec = 0;
  return hip_status(launch_selective_scan_backward(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int rnn_feed_forward_workspace_bytes(const RnnFeedForwardDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = feed_space(desc, false, false).bytes;
  return RNN_OK;
}

int rnn_feed_forward_train_workspace_bytes(const RnnFeedForwardDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = feed_space(desc, true, false).bytes;
  return RNN_OK;
}

int rnn_feed_forward_backward_workspace_bytes(const RnnFeedForwardDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = feed_space(desc, true, true).bytes;
  return RNN_OK;
}

int rnn_feed_forward_reserve_bytes(const RnnFeedForwardDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = feed_reserve(desc);
  return RNN_OK;
}

int rnn_feed_forward(const RnnFeedForwardDesc* desc, const RnnFeedForwardIO* io, void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_feed_forward");
  RETURN_IF_BAD(validate(desc));
  return feed_forward(desc, io, nullptr, workspace, ws_bytes, stream);
}

int rnn_feed_forward_train(const RnnFeedForwardDesc* desc, const RnnFeedForwardIO* io, void* reserve, size_t reserve_bytes,
                           void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_feed_forward_train");
  RETURN_IF_BAD(validate(desc));
  if (!io) return RNN_E_NULL;
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, feed_reserve(desc)));
  return feed_forward(desc, io, reserve, workspace, ws_bytes, stream);
}

int rnn_feed_forward_backward(const RnnFeedForwardDesc* desc, const RnnFeedForwardIO* io, const RnnFeedForwardGrads* grads,
                              const void* reserve, size_t reserve_bytes, void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_feed_forward_backward");
  RETURN_IF_BAD(validate(desc));
  if (!io || !grads) return RNN_E_NULL;
  RETURN_IF_BAD(feed_io(desc, io));
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(grads->dy, desc->aligned ? 16 : e));
  RETURN_IF_BAD(need(grads->dx, e));
  RETURN_IF_BAD(need(grads->dw_in, e));
  RETURN_IF_BAD(need(grads->dw_out, e));
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, feed_reserve(desc)));
  const FeedSpace at = feed_space(desc, true, true);
  RETURN_IF_BAD(need_memory(workspace, ws_bytes, at.bytes));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  return feed_backward(desc, io, grads, reserve, static_cast<char*>(workspace), at, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
