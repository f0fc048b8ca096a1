// Checks and small helpers shared by the host side of the block operators
// (block_api.cpp, state_block_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <rocprofiler-sdk-roctx/roctx.h>

#include <cstdint>

#include "../../include/rnn.h"
#include "block_kernels.hpp"

namespace rnnk {
namespace {

// A launch has at most 2^31 - 1 workgroups.
constexpr int64_t kMaxGrid = 0x7FFFFFFF;
// ... and less than 2^32 threads.
constexpr double kMaxThreads = 4294967295.0;

// A named host range (roctx) around one public call, for timeline tools.
struct Range {
  explicit Range(const char* name) { roctxRangePushA(name); }
  ~Range() { roctxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

int esize_of(int dtype) { return dtype == RNN_DTYPE_BF16 ? 2 : 4; }
bool dtype_ok(int dtype) { return dtype == RNN_DTYPE_F32 || dtype == RNN_DTYPE_BF16; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? RNN_OK : RNN_E_HIP; }

int need(const void* p, size_t a) { return !p ? RNN_E_NULL : aligned(p, a) ? RNN_OK : RNN_E_ALIGN; }
int optional(const void* p, size_t a) { return !p || aligned(p, a) ? RNN_OK : RNN_E_ALIGN; }

#define RETURN_IF_BAD(expr)           \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != RNN_OK) return rc_;    \
  } while (0)

int need_memory(const void* p, size_t have, size_t want) {
  if (want == 0) return RNN_OK;
  if (!p || have < want) return RNN_E_WORKSPACE;
  return aligned(p, 16) ? RNN_OK : RNN_E_ALIGN;
}

int on_device(int* xcds) {
  int cus = 0;
  return current_device_facts(&cus, xcds);
}

// Launches are planned for a whole MI355X, so that the size of a workspace
// does not depend on the device that is current.
constexpr int kPlanCus = 256;

}  // namespace
}  // namespace rnnk
