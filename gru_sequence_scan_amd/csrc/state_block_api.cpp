// Host side of the state-space block's operators declared in include/rnn.h:
// argument validation, workspace layout and the enqueue of their kernels.
// Nothing is kept between calls.
#include <cmath>

#include "api_checks.hpp"
#include "state_block_kernels.hpp"

using namespace rnnk;

namespace {

static_assert(RNN_CONV_MAX_W == kConvMaxW, "the longest filter");

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

}  // extern "C"
