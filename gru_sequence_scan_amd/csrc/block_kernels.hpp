// Interfaces between the host code of the decoder block's operators
// (block_api.cpp) and their kernels. Sizes and strides are in elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"

namespace rnnk {

// Compute units and XCDs of the current device; RNN_E_DEVICE when it is not
// a gfx950.
int current_device_facts(int* cus, int* xcds);

// Gated linear recurrence (gated_scan.hip).
constexpr int kGatedScanChunk = 128;  // steps between two boundary states
struct GatedScanArgs {
  int T, B, H, reverse;
  const void* x; int64_t x_t, x_b;
  const void* f; int64_t f_t, f_b;
  const void* i; int64_t i_t, i_b;  // null: coupled gates
  const int* lengths;               // device [B] or null
  const float* h0;                  // [B, H] or null
  void* y;                          // [T, B, H]
  float* h_n;                       // [B, H] or null
  // backward
  const void* dy; const float* dh_n;
  void* dx; void* df; void* di; float* dh0;
  // chunking
  int width;                        // channels per access: 4, or 1 where rows are not aligned to it
  int chunks, segs, seg_chunks;     // of the time axis; seg_chunks chunks a segment
  float* map_p; float* map_s;       // [segs, B, H] composed maps (workspace; segs > 1)
  float* state;                     // training: [chunks, B, H] state entering a chunk; else null
  int xcds;                         // XCDs of the device
  int tiles;                        // set by launch_gated_scan
};
double gated_scan_row_threads(int H, bool bf16_storage);  // of a launch, for one batch row and segment
int gated_scan_segments(int T, int B, int H, bool bf16_storage, int cus, int* seg_chunks);
hipError_t launch_gated_scan(GatedScanArgs a, bool bf16_storage, bool backward, hipStream_t stream);

// Layer norm (layer_norm.hip).
struct NormArgs {
  int64_t rows; int N; float eps;
  int64_t row0;                     // set by launch_layer_norm: a launch's first row
  const void* x; int64_t ldx;
  const void* r; int64_t ldr;       // residual or null
  const void* w; const void* b;     // [N] or null
  void* y; void* sum;               // [rows, N]; sum only with r
  float* stats;                     // [rows, 2] mean, 1 / sqrt(var + eps); forward: may be null
  // backward (x = the tensor that was normalised)
  const void* dy; const void* ds;   // [rows, N]; ds may be null
  void* dx; float* dw; float* db;   // dw, db may be null
  float* part; int64_t ld_part;     // [blocks, 2, ld_part], ld_part = N rounded up to 4
  int blocks;
  int vec;                          // rows take 8-element accesses
};
constexpr int kNormMaxN = 16384;
// Workgroups of the backward pass, each with one row of partial sums.
int norm_backward_blocks(int64_t rows, int N, int cus);
hipError_t launch_layer_norm(const NormArgs& a, bool bf16_storage, hipStream_t stream);
hipError_t launch_layer_norm_backward(const NormArgs& a, bool bf16_storage, hipStream_t stream);

// Cross attention (attention.hip, attention_bwd.hip).
struct AttentionArgs {
  int B, Tq, Tk, heads, kv_heads, D;
  float scale;
  const void* q; int64_t q_t, q_b, q_h;
  const void* k; int64_t k_t, k_b, k_h;
  const void* v; int64_t v_t, v_b, v_h;
  const int* lengths;               // device [B] or null
  void* o;                          // [Tq, B, heads, D]
  float* lse;                       // training: [B, kv_heads, Tq * G] base-2 log-sum-exp; else null
  void* o_rest;                     // training in bf16: like o, what its rounding left; else null
  int vec;                          // rows take 16-byte accesses
  int near;                         // offsets inside a (batch row, key head) of q, do and of 256 keys fit 31 bits
  int xcds, cus;                    // of the device
  // split of the keys over workgroups (forward)
  int splits;
  float* part_o;                    // [splits, B, kv_heads, Tq * G, D]
  float* part_ml;                   // [splits, B, kv_heads, Tq * G, 2]
  // backward
  const void* d_o;
  void* dq; void* dk; void* dv;
  float* delta;                     // [B, kv_heads, Tq * G]; at large scores what the rounding of lse left
};
// How the forward pass runs: narrow (at most 16 query rows per key head, the
// waves of a workgroup divide the keys) or in tiles of query rows, and how
// many workgroups share the keys of a row.
struct AttentionPlan {
  int narrow;
  int splits;
};
AttentionPlan attention_plan(int B, int Tq, int Tk, int heads, int kv_heads, bool bf16_storage, int cus);
hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, bool bf16_storage, hipStream_t stream);
hipError_t launch_attention_backward(const AttentionArgs& a, bool bf16_storage, hipStream_t stream);

}  // namespace rnnk
