// Interfaces between the host code of the state-space block's operators
// (state_block_api.cpp) and their kernels. Sizes and strides are in elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_kernels.hpp"

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
};
// Workgroups along time and batch of the backward pass, each with one partial sum.
int conv_parts(int T, int B, int C, bool bf16_storage, int cus);
// Threads of the longest launch (0: backward is no longer than that).
double conv_threads(int T, int B, int C, bool bf16_storage);
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
  int xcds;
  int tiles, group_tiles;                      // of 64 channels: in all, and of a group of channels
};
// The state's length as the kernels hold it: 4, 8, 16, 32 or 64.
inline int sel_padded(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
inline int sel_group_tiles(int H, int G) { return (H / G + kSelTile - 1) / kSelTile; }
int sel_segments(int T, int B, int H, int G, int cus, int* seg_steps);
hipError_t launch_selective_scan(SelectiveScanArgs a, bool bf16_storage, hipStream_t stream);
hipError_t launch_selective_scan_backward(SelectiveScanArgs a, bool bf16_storage, hipStream_t stream);

}  // namespace rnnk
