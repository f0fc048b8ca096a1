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

}  // namespace rnnk
