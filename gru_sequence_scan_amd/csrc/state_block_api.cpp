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
  if (conv_threads(d->T, d->B, d->C, d->dtype == RNN_DTYPE_BF16) > kMaxThreads) return RNN_E_SHAPE;
  if (8.0 * ((double)d->C + 32.0) * (d->W + 1) > kMaxThreads) return RNN_E_SHAPE;
  return RNN_OK;
}

size_t conv_workspace(const RnnCausalConvDesc* d) {
  return (size_t)conv_parts(d->T, d->B, d->C, d->dtype == RNN_DTYPE_BF16, kPlanCus) * (d->W + 1) * d->C * sizeof(float);
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
  return sel_segments(d->T, d->B, d->H, d->G, kPlanCus, steps);
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
  a.keep = static_cast<float*>(reserve);
  return hip_status(launch_selective_scan(a, d->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
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
  a.parts = conv_parts(desc->T, desc->B, desc->C, desc->dtype == RNN_DTYPE_BF16, kPlanCus);
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
  return hip_status(launch_selective_scan_backward(a, desc->dtype == RNN_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
