// Host side of the decoder block's operators declared in include/rnn.h:
// argument validation, workspace layout and the enqueue of their kernels.
// Nothing is kept between calls.
#include <cmath>

#include "api_checks.hpp"

using namespace rnnk;

namespace {

static_assert(RNN_NORM_MAX_N == kNormMaxN, "layer norm's row limit");

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
int validate(const RnnNormDesc* d) {
  if (!d) return RNN_E_NULL;
  if (!dtype_ok(d->dtype)) return RNN_E_UNSUPPORTED;
  if (d->reserved != 0 || d->N < 1 || d->rows < 1) return RNN_E_SHAPE;
  if (d->N > RNN_NORM_MAX_N) return RNN_E_UNSUPPORTED;
  if (d->rows > kMaxGrid || d->x_ld < d->N) return RNN_E_SHAPE;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return RNN_E_SHAPE;
  return RNN_OK;
}

size_t norm_workspace(const RnnNormDesc* d) {
  return (size_t)norm_backward_blocks(d->rows, d->N, kPlanCus) * 2 * (size_t)((d->N + 3) / 4 * 4) * sizeof(float);
}

// ---------------------------------------------------------------------------
// Gated scan
// ---------------------------------------------------------------------------
int scan_chunks(const RnnGatedScanDesc* d) { return (d->T + kGatedScanChunk - 1) / kGatedScanChunk; }

int validate(const RnnGatedScanDesc* d) {
  if (!d) return RNN_E_NULL;
  if (!dtype_ok(d->dtype)) return RNN_E_UNSUPPORTED;
  if (d->T < 1 || d->B < 1 || d->H < 1) return RNN_E_SHAPE;
  if (d->T > kMaxGrid - kGatedScanChunk) return RNN_E_SHAPE;
  if ((d->reverse | 1) != 1 || (d->input_gate | 1) != 1) return RNN_E_SHAPE;
  if (d->x_t < 0 || d->x_b < 0 || d->f_t < 0 || d->f_b < 0) return RNN_E_SHAPE;
  if (d->input_gate && (d->i_t < 0 || d->i_b < 0)) return RNN_E_SHAPE;
  // a workgroup per tile of channels and batch row (rounded up to XCDs); the
  // time axis is cut only while there are fewer of them than fill the device
  if (((double)d->B + 64) * gated_scan_row_threads(d->H, d->dtype == RNN_DTYPE_BF16) > kMaxThreads) return RNN_E_SHAPE;
  return RNN_OK;
}

size_t scan_state_bytes(const RnnGatedScanDesc* d) { return (size_t)scan_chunks(d) * d->B * d->H * sizeof(float); }

// One map (two numbers a channel) per segment of the time axis.
size_t scan_map_bytes(const RnnGatedScanDesc* d) {
  int each = 0;
  const size_t segs = (size_t)gated_scan_segments(d->T, d->B, d->H, d->dtype == RNN_DTYPE_BF16, kPlanCus, &each);
  return segs > 1 ? (segs * d->B * d->H * sizeof(float) + 15) / 16 * 16 : 0;
}

size_t scan_workspace(const RnnGatedScanDesc* d) { return 2 * scan_map_bytes(d); }

int scan_args(const RnnGatedScanDesc* d, const RnnGatedScanIO* io, void* ws, size_t ws_bytes, GatedScanArgs* a) {
  if (!io) return RNN_E_NULL;
  const size_t e = (size_t)esize_of(d->dtype);
  RETURN_IF_BAD(need(io->x, e));
  RETURN_IF_BAD(need(io->f, e));
  if (d->input_gate) RETURN_IF_BAD(need(io->i, e));
  RETURN_IF_BAD(optional(io->lengths, 4));
  RETURN_IF_BAD(optional(io->h0, 4));
  RETURN_IF_BAD(need_memory(ws, ws_bytes, scan_workspace(d)));
  *a = GatedScanArgs{};
  a->T = d->T; a->B = d->B; a->H = d->H; a->reverse = d->reverse;
  a->x = io->x; a->x_t = d->x_t; a->x_b = d->x_b;
  a->f = io->f; a->f_t = d->f_t; a->f_b = d->f_b;
  if (d->input_gate) {
    a->i = io->i; a->i_t = d->i_t; a->i_b = d->i_b;
  }
  a->lengths = io->lengths;
  a->h0 = io->h0;
  a->chunks = scan_chunks(d);
  a->segs = gated_scan_segments(d->T, d->B, d->H, d->dtype == RNN_DTYPE_BF16, kPlanCus, &a->seg_chunks);
  if (a->segs > 1) {
    a->map_p = static_cast<float*>(ws);
    a->map_s = reinterpret_cast<float*>(static_cast<char*>(ws) + scan_map_bytes(d));
  }
  // four channels an access when every row of every tensor allows it
  auto fits = [&](const void* p, int64_t t, int64_t b) { return aligned(p, 4 * e) && t % 4 == 0 && b % 4 == 0; };
  const bool wide = d->H % 4 == 0 && fits(a->x, a->x_t, a->x_b) && fits(a->f, a->f_t, a->f_b) && fits(a->i, a->i_t, a->i_b);
  a->width = wide ? 4 : 1;
  return RNN_OK;
}

int scan_forward(const RnnGatedScanDesc* d, const RnnGatedScanIO* io, void* reserve, void* ws, size_t ws_bytes,
                 void* stream) {
  GatedScanArgs a;
  RETURN_IF_BAD(scan_args(d, io, ws, ws_bytes, &a));
  const size_t e = (size_t)esize_of(d->dtype);
  RETURN_IF_BAD(need(io->y, e));
  RETURN_IF_BAD(optional(io->h_n, 4));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.xcds = xcds;
  a.y = io->y;
  a.h_n = io->h_n;
  if (!aligned(a.y, 4 * e)) a.width = 1;
  a.state = static_cast<float*>(reserve);
  return hip_status(launch_gated_scan(a, d->dtype == RNN_DTYPE_BF16, false, reinterpret_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// Cross attention
// ---------------------------------------------------------------------------
int64_t query_rows(const RnnAttentionDesc* d) { return (int64_t)d->Tq * (d->heads / d->kv_heads); }

AttentionPlan plan_of(const RnnAttentionDesc* d) {
  return attention_plan(d->B, d->Tq, d->Tk, d->heads, d->kv_heads, d->dtype == RNN_DTYPE_BF16, kPlanCus);
}

int validate(const RnnAttentionDesc* d) {
  if (!d) return RNN_E_NULL;
  if (!dtype_ok(d->dtype)) return RNN_E_UNSUPPORTED;
  if (d->B < 1 || d->Tq < 1 || d->Tk < 1 || d->heads < 1 || d->kv_heads < 1 || d->D < 1) return RNN_E_SHAPE;
  if (d->heads % d->kv_heads != 0 || !std::isfinite(d->scale)) return RNN_E_SHAPE;
  if (d->D > RNN_ATTENTION_MAX_D) return RNN_E_UNSUPPORTED;
  for (int64_t s : {d->q_t, d->q_b, d->q_h, d->k_t, d->k_b, d->k_h, d->v_t, d->v_b, d->v_h})
    if (s < 0) return RNN_E_SHAPE;
  const double groups = (double)d->B * d->kv_heads, rows = (double)query_rows(d);
  if (d->Tk > kMaxGrid - 1024 || rows > (double)(kMaxGrid - 1024) || groups > (double)kMaxGrid) return RNN_E_SHAPE;
  // threads of the launches: 256 per 64 query rows and per 64 keys (bf16 takes
  // as many for twice the rows); per 16 rows where there are at most 16
  const double per_group = rows <= 16 ? 256.0 : 4.0 * (rows + 64.0);
  if ((groups + 64.0) * per_group > kMaxThreads || (groups + 64.0) * 4.0 * ((double)d->Tk + 128.0) > kMaxThreads)
    return RNN_E_SHAPE;
  return RNN_OK;
}

size_t attention_stat_bytes(const RnnAttentionDesc* d) {
  return (size_t)d->B * d->kv_heads * (size_t)query_rows(d) * sizeof(float);
}

// The reserve: the log-sum-exp and, in bf16, what the rounding of o left.
size_t attention_reserve(const RnnAttentionDesc* d) {
  const size_t stat = (attention_stat_bytes(d) + 15) / 16 * 16;
  return d->dtype == RNN_DTYPE_BF16 ? stat + (size_t)d->Tq * d->B * d->heads * d->D * 2 : stat;
}

void* attention_rest(const RnnAttentionDesc* d, void* reserve) {
  if (!reserve || d->dtype != RNN_DTYPE_BF16) return nullptr;
  return static_cast<char*>(reserve) + (attention_stat_bytes(d) + 15) / 16 * 16;
}

size_t attention_workspace(const RnnAttentionDesc* d) {
  const size_t n = (size_t)plan_of(d).splits;
  return n > 1 ? n * (attention_stat_bytes(d) * ((size_t)d->D + 2) + 16) : 0;
}

int attention_args(const RnnAttentionDesc* d, const RnnAttentionIO* io, AttentionArgs* a) {
  if (!io) return RNN_E_NULL;
  const size_t e = (size_t)esize_of(d->dtype);
  RETURN_IF_BAD(need(io->q, e));
  RETURN_IF_BAD(need(io->k, e));
  RETURN_IF_BAD(need(io->v, e));
  RETURN_IF_BAD(need(io->o, e));
  RETURN_IF_BAD(optional(io->lengths, 4));
  *a = AttentionArgs{};
  a->B = d->B; a->Tq = d->Tq; a->Tk = d->Tk; a->heads = d->heads; a->kv_heads = d->kv_heads; a->D = d->D;
  a->scale = d->scale;
  a->q = io->q; a->q_t = d->q_t; a->q_b = d->q_b; a->q_h = d->q_h;
  a->k = io->k; a->k_t = d->k_t; a->k_b = d->k_b; a->k_h = d->k_h;
  a->v = io->v; a->v_t = d->v_t; a->v_b = d->v_b; a->v_h = d->v_h;
  a->lengths = io->lengths;
  a->o = io->o;
  a->splits = 1;
  const int64_t m = 16 / (int64_t)e;
  bool vec = d->D % m == 0 && aligned(a->q, 16) && aligned(a->k, 16) && aligned(a->v, 16) && aligned(a->o, 16);
  for (int64_t s : {d->q_t, d->q_b, d->q_h, d->k_t, d->k_b, d->k_h, d->v_t, d->v_b, d->v_h}) vec = vec && s % m == 0;
  a->vec = vec;
  const double span_q = (double)(d->Tq - 1) * d->q_t + (double)(d->heads - 1) * d->q_h;
  const double span_o = (double)d->Tq * d->B * d->heads * d->D;
  const double span_kv = 256.0 * (double)(d->k_t > d->v_t ? d->k_t : d->v_t);
  a->near = (std::fmax(span_q, std::fmax(span_o, span_kv)) + 128.0) * (double)e < 2147483648.0;
  return RNN_OK;
}

int attention_forward(const RnnAttentionDesc* d, const RnnAttentionIO* io, void* reserve, void* ws, size_t ws_bytes,
                      void* stream) {
  AttentionArgs a;
  RETURN_IF_BAD(attention_args(d, io, &a));
  RETURN_IF_BAD(need_memory(ws, ws_bytes, attention_workspace(d)));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  const AttentionPlan p = plan_of(d);
  a.splits = p.splits;
  a.xcds = xcds;
  if (p.splits > 1) {
    a.part_o = static_cast<float*>(ws);
    a.part_ml = a.part_o + (size_t)p.splits * (attention_stat_bytes(d) / sizeof(float)) * d->D;
  }
  a.lse = static_cast<float*>(reserve);
  a.o_rest = attention_rest(d, reserve);
  return hip_status(launch_attention(a, p, d->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int rnn_layer_norm(const RnnNormDesc* desc, const void* x, const void* residual, const void* weight, const void* bias,
                   void* y, void* sum, float* stats, void* stream) {
  Range range("rnn_layer_norm");
  RETURN_IF_BAD(validate(desc));
  if (residual && desc->residual_ld < desc->N) return RNN_E_SHAPE;
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(x, e));
  RETURN_IF_BAD(need(y, e));
  RETURN_IF_BAD(optional(residual, e));
  RETURN_IF_BAD(optional(weight, e));
  RETURN_IF_BAD(optional(bias, e));
  if (residual) RETURN_IF_BAD(need(sum, e));
  RETURN_IF_BAD(optional(stats, 4));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  NormArgs a{};
  a.rows = desc->rows; a.N = desc->N; a.eps = desc->eps;
  a.x = x; a.ldx = desc->x_ld;
  a.r = residual; a.ldr = residual ? desc->residual_ld : 0;
  a.w = weight; a.b = bias; a.y = y; a.sum = residual ? sum : nullptr; a.stats = stats;
  const int64_t m = 16 / (int64_t)e;
  a.vec = a.N % 8 == 0 && a.ldx % m == 0 && a.ldr % m == 0 && aligned(x, 16) && aligned(residual, 16) &&
          aligned(weight, 16) && aligned(bias, 16) && aligned(y, 16) && aligned(a.sum, 16);
  return hip_status(launch_layer_norm(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int rnn_layer_norm_backward_workspace_bytes(const RnnNormDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = norm_workspace(desc);
  return RNN_OK;
}

int rnn_layer_norm_backward(const RnnNormDesc* desc, const void* s, const void* weight, const float* stats, const void* dy,
                            const void* dsum, void* dx, float* dweight, float* dbias, void* workspace, size_t ws_bytes,
                            void* stream) {
  Range range("rnn_layer_norm_backward");
  RETURN_IF_BAD(validate(desc));
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(s, e));
  RETURN_IF_BAD(optional(weight, e));
  RETURN_IF_BAD(need(stats, 4));
  RETURN_IF_BAD(need(dy, e));
  RETURN_IF_BAD(optional(dsum, e));
  RETURN_IF_BAD(need(dx, e));
  if (!dweight != !dbias) return RNN_E_NULL;
  RETURN_IF_BAD(optional(dweight, 4));
  RETURN_IF_BAD(optional(dbias, 4));
  if (dweight) RETURN_IF_BAD(need_memory(workspace, ws_bytes, norm_workspace(desc)));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  NormArgs a{};
  a.rows = desc->rows; a.N = desc->N; a.eps = desc->eps;
  a.x = s; a.ldx = desc->x_ld; a.w = weight; a.stats = const_cast<float*>(stats);
  a.dy = dy; a.ds = dsum; a.dx = dx; a.dw = dweight; a.db = dbias;
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.ld_part = (desc->N + 3) / 4 * 4;
  a.blocks = norm_backward_blocks(desc->rows, desc->N, kPlanCus);
  a.vec = a.N % 8 == 0 && a.ldx % (16 / (int64_t)e) == 0 && aligned(s, 16) && aligned(weight, 16) && aligned(dy, 16) &&
          aligned(dsum, 16) && aligned(dx, 16);
  return hip_status(launch_layer_norm_backward(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int rnn_gated_scan_workspace_bytes(const RnnGatedScanDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = scan_workspace(desc);
  return RNN_OK;
}

int rnn_gated_scan_reserve_bytes(const RnnGatedScanDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = scan_state_bytes(desc);
  return RNN_OK;
}

int rnn_gated_scan(const RnnGatedScanDesc* desc, const RnnGatedScanIO* io, void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_gated_scan");
  RETURN_IF_BAD(validate(desc));
  return scan_forward(desc, io, nullptr, workspace, ws_bytes, stream);
}

int rnn_gated_scan_train(const RnnGatedScanDesc* desc, const RnnGatedScanIO* io, void* reserve, size_t reserve_bytes,
                         void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_gated_scan_train");
  RETURN_IF_BAD(validate(desc));
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, scan_state_bytes(desc)));
  return scan_forward(desc, io, reserve, workspace, ws_bytes, stream);
}

int rnn_gated_scan_backward(const RnnGatedScanDesc* desc, const RnnGatedScanIO* io, const RnnGatedScanGrads* grads,
                            const void* reserve, size_t reserve_bytes, void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_gated_scan_backward");
  RETURN_IF_BAD(validate(desc));
  if (!grads) return RNN_E_NULL;
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, scan_state_bytes(desc)));
  GatedScanArgs a;
  RETURN_IF_BAD(scan_args(desc, io, workspace, ws_bytes, &a));
  const size_t e = (size_t)esize_of(desc->dtype);
  RETURN_IF_BAD(need(grads->dy, e));
  RETURN_IF_BAD(optional(grads->dh_n, 4));
  RETURN_IF_BAD(need(grads->dx, e));
  RETURN_IF_BAD(need(grads->df, e));
  if (desc->input_gate) RETURN_IF_BAD(need(grads->di, e));
  RETURN_IF_BAD(optional(grads->dh0, 4));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.state = const_cast<float*>(static_cast<const float*>(reserve));
  a.xcds = xcds;
  a.dy = grads->dy; a.dh_n = grads->dh_n;
  a.dx = grads->dx; a.df = grads->df; a.di = desc->input_gate ? grads->di : nullptr;
  a.dh0 = grads->dh0;
  if (!aligned(a.dy, 4 * e) || !aligned(a.dx, 4 * e) || !aligned(a.df, 4 * e) || !aligned(a.di, 4 * e)) a.width = 1;
  return hip_status(launch_gated_scan(a, desc->dtype == RNN_DTYPE_BF16, true, reinterpret_cast<hipStream_t>(stream)));
}

int rnn_cross_attention_workspace_bytes(const RnnAttentionDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = attention_workspace(desc);
  return RNN_OK;
}

int rnn_cross_attention_reserve_bytes(const RnnAttentionDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = attention_reserve(desc);
  return RNN_OK;
}

int rnn_cross_attention_backward_workspace_bytes(const RnnAttentionDesc* desc, size_t* bytes) {
  RETURN_IF_BAD(validate(desc));
  if (!bytes) return RNN_E_NULL;
  *bytes = attention_stat_bytes(desc);  // delta, one value per query row
  return RNN_OK;
}

int rnn_cross_attention(const RnnAttentionDesc* desc, const RnnAttentionIO* io, void* workspace, size_t ws_bytes,
                        void* stream) {
  Range range("rnn_cross_attention");
  RETURN_IF_BAD(validate(desc));
  return attention_forward(desc, io, nullptr, workspace, ws_bytes, stream);
}

int rnn_cross_attention_train(const RnnAttentionDesc* desc, const RnnAttentionIO* io, void* reserve, size_t reserve_bytes,
                              void* workspace, size_t ws_bytes, void* stream) {
  Range range("rnn_cross_attention_train");
  RETURN_IF_BAD(validate(desc));
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, attention_reserve(desc)));
  return attention_forward(desc, io, reserve, workspace, ws_bytes, stream);
}

int rnn_cross_attention_backward(const RnnAttentionDesc* desc, const RnnAttentionIO* io, const RnnAttentionGrads* grads,
                                 const void* reserve, size_t reserve_bytes, void* workspace, size_t ws_bytes,
                                 void* stream) {
  Range range("rnn_cross_attention_backward");
  RETURN_IF_BAD(validate(desc));
  if (!grads) return RNN_E_NULL;
  AttentionArgs a;
  RETURN_IF_BAD(attention_args(desc, io, &a));
  const size_t e = (size_t)esize_of(desc->dtype);
  for (const void* p : {grads->d_o, (const void*)grads->dq, (const void*)grads->dk, (const void*)grads->dv}) {
    RETURN_IF_BAD(need(p, e));
    if (!aligned(p, 16)) a.vec = 0;
  }
  RETURN_IF_BAD(need_memory(reserve, reserve_bytes, attention_reserve(desc)));
  RETURN_IF_BAD(need_memory(workspace, ws_bytes, attention_stat_bytes(desc)));
  int xcds;
  RETURN_IF_BAD(on_device(&xcds));
  a.lse = const_cast<float*>(static_cast<const float*>(reserve));
  a.o_rest = attention_rest(desc, const_cast<void*>(reserve));
  a.delta = static_cast<float*>(workspace);
  a.xcds = xcds;
  a.cus = kPlanCus;
  a.d_o = grads->d_o; a.dq = grads->dq; a.dk = grads->dk; a.dv = grads->dv;
  return hip_status(launch_attention_backward(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
