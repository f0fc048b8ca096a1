// Interfaces between the host code of the state-space block's operators
// (state_block_api.cpp) and their kernels. Sizes and strides are in elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_kernels.hpp"
#include "feed_forward_plan.hpp"

namespace rnnk {

// Short causal convolution (causal_conv.hip).
constexpr int kConvMaxW = 8;
struct CausalConvArgs {
  int T, B, C, W, silu;
  const void* x; int64_t x_t, x_b;
  const void* w; const void* bias;  // [C, W]; [C] or null
  const int* lengths;               // device [B] or null
  const void* state;                // [W-1, B, C] or null (zeros)
  void* y;                          // [T, B, C]
  void* state_n;                    // [W-1, B, C] or null
  // backward
  const void* dy; const void* dstate_n;
  void* dx; float* dw; float* db; void* dstate;  // db, dstate may be null
  float* part;                      // [parts, W + 1, C] partial sums of dw and db (workspace)
  int parts;
  int vec;                          // rows take 16-byte accesses
  int wvec;                         // the filters and the bias take 8-byte accesses
};
// Workgroups along time and batch of the backward pass, each with one partial sum.
int conv_parts(int T, int B, int C, int cus);
// Threads of the longest launch (backward is no longer than that).
double conv_threads(int T, int B, int C);
hipError_t launch_causal_conv(const CausalConvArgs& a, bool bf16_storage, hipStream_t stream);
hipError_t launch_causal_conv_backward(const CausalConvArgs& a, bool bf16_storage, hipStream_t stream);

// Selective scan (selective_scan.hip, selective_scan_bwd.hip).
constexpr int kSelMaxN = 64;
constexpr int kSelTile = 64;      // channels of a workgroup
constexpr int kSelKeep = 16;      // steps between two states that training keeps
struct SelectiveScanArgs {
  int T, B, H, N, G, softplus;
  const void* x; int64_t x_t, x_b;
  const void* dt; int64_t dt_t, dt_b;
  const void* z; int64_t z_t, z_b;             // null: no output gate
  const void* Bm; int64_t B_t, B_b, B_g;       // [T, B, G, N]
  const void* Cm; int64_t C_t, C_b, C_g;
  const float* A; const float* D; const float* dt_bias;  // [H, N]; [H] or null
  const int* lengths;                          // device [B] or null
  const float* h0;                             // [B, H, N] or null
  void* y; float* h_n;
  // backward
  const void* dy; const float* dh_n;
  void* dx; void* ddt; void* dz;               // dz may be null
  void* dB; void* dC;                          // [T, B, G, N]
  float* dA; float* dD; float* dbias; float* dh0;  // all but dA may be null
  float* keep;                                 // training: [ceil(T / kSelKeep), B, H, NP] state entering those steps; else null
  // the time cut into segments of seg_steps steps (workspace; segs > 1)
  int segs, seg_steps;
  float* map_s;                                // [segs, B, H, NP] what a segment adds to the state; then the state entering it
  float* map_d;                                // [segs, B, H] sum of a segment's steps
  // partial sums of the backward pass (workspace)
  float* part_bc;                              // [tiles of a group, T, B, G, 2, NP]
  float* part_a;                               // [segs, B, H, NP + 2]: dA, then dD and dbias
  int vec;                                     // rows take vector accesses
  int svec;                                    // ... and so do the states' ([.., N], N as the kernels hold it) and A's
  int xcds;
  int tiles, group_tiles;                      // of 64 channels: in all, and of a group of channels
};
// The state's length as the kernels hold it: 4, 8, 16, 32 or 64.
inline int sel_padded(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
inline int sel_group_tiles(int H, int G) { return (H / G + kSelTile - 1) / kSelTile; }
int sel_segments(int T, int B, int H, int N, int G, int cus, int* seg_steps);
hipError_t launch_selective_scan(SelectiveScanArgs a, bool bf16_storage, hipStream_t stream);
hipError_t launch_selective_scan_backward(SelectiveScanArgs a, bool bf16_storage, hipStream_t stream);

// Gated feed-forward (feed_forward.hip and its instances).
struct FeedArgs {
  int M, N;                         // the output's rows and columns, padding of F included
  const void* A; int64_t lda; int KA;  // KA: how far the operand goes along the summed dimension
  const void* B; int64_t ldb; int KB;
  int cols_a, cols_b;               // columns of an operand that lies across, in memory
  int steps;                        // of the summed dimension, 128 bytes (64 bf16, 32 fp32) each
  int F, Fp;                        // hidden size, and rounded up to whole steps
  int act;                          // RnnActivation
  // outputs
  void* out; int64_t ldo;           // kFeedIn: h; kFeedDh: [dg, du]
  const void* residual; int64_t ldr;
  float* gu;                        // [M, 2 Fp] the two projections in fp32: kFeedIn writes it (or null), kFeedDh reads it
  int rows_split;                   // output rows from here on (padded) belong after the first F; 0: one block of rows
  float* part; int splits;          // splits > 1: partial products [splits, M, N] (kFeedIn: 2 Fp for N)
};
hipError_t launch_feed_f32(int op, const FeedArgs& a, const FeedPlan& p, hipStream_t stream);
hipError_t launch_feed_bf16(int op, const FeedArgs& a, const FeedPlan& p, hipStream_t stream);
// Few rows: both projections and the activation, then the projection back.
struct FeedFewArgs {
  int rows, n, F, n_out, act;
  const void* x; int64_t ldx;
  const void* w_in; int64_t ld_in;
  const void* w_out; int64_t ld_out;
  const void* residual; int64_t ldr;
  void* h;                          // [rows, Fp] (workspace, or kept by training)
  int Fp;
  float* gu;                        // [rows, 2 Fp] the two projections in fp32, or null
  void* y;
  float* part; int splits;          // splits > 1: partial second products [splits, rows, n_out] (workspace)
};
int feed_few_splits(int64_t rows, int F, int n_out, int cus);
hipError_t launch_feed_few(const FeedFewArgs& a, bool bf16_storage, hipStream_t stream);
// Rows of up to four tensors copied to a pitch of whole 16 bytes, zeros behind
// each, in one launch.
struct FeedPackArgs {
  struct {
    const void* from; int64_t ld;
    int64_t rows; int cols;
    void* to; int pitch;
  } t[4];
  int count;
};
hipError_t launch_feed_pack(const FeedPackArgs& a, bool bf16_storage, hipStream_t stream);
// What a product's results would have become, from the sums of its partial products.
hipError_t launch_feed_join(int op, const FeedArgs& a, bool bf16_storage, hipStream_t stream);

}  // namespace rnnk
