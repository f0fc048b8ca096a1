// Short causal convolution over time, one filter per channel, forward and
// backward.
//
//   x'_s = x_s for 0 <= s < L,  state[s + W - 1] for s < 0
//   p_t = b + sum_k w[k] x'_{t - W + 1 + k},   y_t = p_t or silu(p_t)
//   state_n[j] = x'_{L - W + 1 + j}
//
//   dp_t = dy_t (silu'(p_t) or 1) for t < L, else 0
//   dx'_s = sum_k w[k] dp_{s + W - 1 - k}  (+ dstate_n[j] at s = L - W + 1 + j)
//   dw[k] = sum_{t, b} dp_t x'_{t - W + 1 + k},   db = sum dp_t
//
// Bound by memory. A thread takes 16 bytes of channels (one channel where
// rows are not aligned) and a run of 16 steps; the W - 1 steps in front of a
// run are read again (out of the L2, where the neighbouring run's thread put
// them). Every load of a run is issued before the first is used: a step past
// the row's end reads the last one again, and what is not part of the row is
// replaced by zero. 1000 steps of 32 x 2048 channels, bf16, 4 taps, SiLU: 54
// us forward, 4.9 TB/s of the 5.1 that a large copy reaches (88 with loads
// under conditions). With x off its alignment, a channel at a time: 62 us for 47
// of aligned calls timed the same way, one after the other (backward 131 for 122).
//
// Backward computes p again from x, so the forward keeps nothing. It takes
// four channels a thread (with eight, a run's x, dy and dp leave no registers
// for a second workgroup's loads) and one exponential for SiLU and its slope:
// 124 us there, 215 without the two. 430 MB at 3.5 TB/s; vector instructions
// take three quarters of the issue slots. The sums
// over time and batch stay in a thread's registers over all runs that it
// takes, are joined by workgroup in LDS, and a second launch adds the
// workgroups' sums in a fixed order (4.8 us there).
//
// Products and sums are fp32; x, w, b, y, the state and their gradients have
// the storage type, dw and db are fp32.
#include "device_common.hpp"
#include "state_block_kernels.hpp"

namespace rnnk {
namespace {

constexpr int kConvThreads = 256;
constexpr int kRun = 16;

template <typename DT, int E>
struct alignas(sizeof(DT) * E) Vec {
  DT v[E];
};
template <typename DT>
constexpr int kWide = 16 / (int)sizeof(DT);
constexpr int kBackWide = 4;  // channels of a thread backward

template <typename DT, int E>
__device__ __forceinline__ Vec<DT, E> zero_vec() {
  Vec<DT, E> z;
#pragma unroll
  for (int e = 0; e < E; ++e) z.v[e] = (DT)0.f;
  return z;
}

// silu and its slope: s = sigma(p), silu' = s + p s (1 - s), 1 - s formed as
// sigma of the negative.
__device__ __forceinline__ float silu(float p) { return p * fsigmoid(p); }
__device__ __forceinline__ float silu_slope(float p) {
  const SigmoidPair g = fsigmoid_pair(p);
  return __builtin_fmaf(p * g.s, g.no, g.s);
}

__device__ __forceinline__ int row_length(const CausalConvArgs& a, int b) {
  const int n = a.lengths ? a.lengths[b] : a.T;
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

// x'_s for any s (past the row's end: some step of the row, which the caller
// does not use; in front of the state: zero). The load itself has no
// condition, so that many of them are on their way at once.
template <typename DT, int E>
__device__ __forceinline__ Vec<DT, E> input_at(const CausalConvArgs& a, const DT* x, const DT* state, int s, int L) {
  const int j = s + a.W - 1, last = L > 0 ? L - 1 : 0;
  const bool front = s < 0 && state;
  const DT* p = front ? state + (int64_t)(j > 0 ? j : 0) * a.B * a.C : x + (int64_t)(s < 0 ? 0 : s < last ? s : last) * a.x_t;
  const Vec<DT, E> v = *reinterpret_cast<const Vec<DT, E>*>(p);
  return (s >= 0 ? L > 0 : front && j >= 0) ? v : zero_vec<DT, E>();
}

// The taps of E channels, the oldest first; a filter shorter than KW has
// zeros in front, whose inputs are never used.
template <typename DT, int E, int KW>
__device__ __forceinline__ void load_taps(const CausalConvArgs& a, int c, float (&w)[KW][E], float (&bias)[E]) {
  if constexpr (KW <= 4 && E > 1) {
    if (a.wvec) {  // whole filters, 8 bytes an access
      constexpr int M = 8 / (int)sizeof(DT);
      Vec<DT, M> r[E * KW / M], rb[E / M];
#pragma unroll
      for (int i = 0; i < E * KW / M; ++i) r[i] = reinterpret_cast<const Vec<DT, M>*>((const DT*)a.w + (int64_t)c * KW)[i];
#pragma unroll
      for (int i = 0; i < E / M; ++i) rb[i] = reinterpret_cast<const Vec<DT, M>*>((const DT*)(a.bias ? a.bias : a.w) + c)[i];
#pragma unroll
      for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int k = 0; k < KW; ++k) w[k][e] = to_f32<DT>(r[(e * KW + k) / M].v[(e * KW + k) % M]);
        bias[e] = a.bias ? to_f32<DT>(rb[e / M].v[e % M]) : 0.f;
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int kk = k - (KW - a.W);
      w[k][e] = kk >= 0 ? to_f32<DT>(((const DT*)a.w)[(int64_t)(c + e) * a.W + kk]) : 0.f;
    }
    bias[e] = a.bias ? to_f32<DT>(((const DT*)a.bias)[c + e]) : 0.f;
  }
}

// R steps a thread: 16, or 1 where a call has few.
template <typename DT, int E, int KW, int R>
__global__ __launch_bounds__(kConvThreads) void conv_forward_kernel(CausalConvArgs a) {
  const int groups = a.C / E;
  const int64_t id = blockIdx.x * (int64_t)kConvThreads + threadIdx.x;
  const int c = (int)(id % groups) * E;
  const int64_t unit = id / groups;
  const int b = (int)(unit % a.B);
  const int64_t run = unit / a.B;
  if (run * R >= a.T) return;
  const int t0 = (int)run * R, L = row_length(a, b);
  const int64_t cell = (int64_t)b * a.C + c, y_t = (int64_t)a.B * a.C;
  const DT* x = (const DT*)a.x + b * a.x_b + c;
  const DT* state = a.state ? (const DT*)a.state + cell : nullptr;
  if (t0 == 0 && a.state_n) {
    Vec<DT, E> last[KW - 1];
#pragma unroll
    for (int j = 0; j < KW - 1; ++j) last[j] = input_at<DT, E>(a, x, state, L - a.W + 1 + j, L);
#pragma unroll
    for (int j = 0; j < KW - 1; ++j)
      if (j < a.W - 1) *reinterpret_cast<Vec<DT, E>*>((DT*)a.state_n + j * y_t + cell) = last[j];
  }
  DT* y = (DT*)a.y + cell;
  if (t0 >= L) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (t0 + r < a.T) *reinterpret_cast<Vec<DT, E>*>(y + (t0 + r) * y_t) = zero_vec<DT, E>();
    return;
  }
  Vec<DT, E> in[R + KW - 1];
  if (t0 >= KW - 1) {
#pragma unroll
    for (int r = 0; r < R + KW - 1; ++r) {
      const int s = t0 - KW + 1 + r;
      in[r] = *reinterpret_cast<const Vec<DT, E>*>(x + (int64_t)(s < L ? s : L - 1) * a.x_t);
    }
  } else {
#pragma unroll
    for (int r = 0; r < R + KW - 1; ++r) in[r] = input_at<DT, E>(a, x, state, t0 - KW + 1 + r, L);
  }
  float w[KW][E], bias[E];
  load_taps<DT, E, KW>(a, c, w, bias);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = t0 + r;
    Vec<DT, E> out;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float p = bias[e];
#pragma unroll
      for (int k = 0; k < KW; ++k)
        if (KW <= 4 || k >= KW - a.W) p = __builtin_fmaf(w[k][e], to_f32<DT>(in[r + k].v[e]), p);
      out.v[e] = from_f32<DT>(t < L ? (a.silu ? silu(p) : p) : 0.f);
    }
    if (t < a.T) *reinterpret_cast<Vec<DT, E>*>(y + t * y_t) = out;
  }
}

// Lanes across the channels: a whole wave where there are enough, else the
// lanes that are left take other runs.
__host__ __device__ inline int channel_lanes(int groups) {
  int n = 1;
  while (n < 64 && n < groups) n *= 2;
  return n;
}

// One run of the backward pass: steps [t0, t0 + kRun) of row b.
template <typename DT, int E, int KW>
__device__ __forceinline__ void backward_run(const CausalConvArgs& a, int c, int b, int t0, const float (&w)[KW][E],
                                             const float (&bias)[E], float (&dw)[KW][E], float (&db)[E]) {
  const int L = row_length(a, b);
  const int64_t cell = (int64_t)b * a.C + c, d_t = (int64_t)a.B * a.C;
  const DT* x = (const DT*)a.x + b * a.x_b + c;
  const DT* state = a.state ? (const DT*)a.state + cell : nullptr;
  const DT* dy = (const DT*)a.dy + cell;
  DT* dx = (DT*)a.dx + cell;
  const DT* dstate_n = a.dstate_n ? (const DT*)a.dstate_n + cell : nullptr;
  constexpr int kAll = kRun + KW - 1;  // steps whose dp this run needs
  if (t0 >= L && t0 > 0) {
#pragma unroll
    for (int r = 0; r < kRun; ++r)
      if (t0 + r < a.T) *reinterpret_cast<Vec<DT, E>*>(dx + (t0 + r) * d_t) = zero_vec<DT, E>();
    return;
  }
  Vec<DT, E> in[kAll + KW - 1], up[kAll];
  if (L == 0) {
#pragma unroll
    for (int r = 0; r < kAll + KW - 1; ++r) in[r] = zero_vec<DT, E>();
#pragma unroll
    for (int r = 0; r < kAll; ++r) up[r] = zero_vec<DT, E>();
  } else {
    if (t0 >= KW - 1) {
#pragma unroll
      for (int r = 0; r < kAll + KW - 1; ++r) {
        const int s = t0 - KW + 1 + r;
        in[r] = *reinterpret_cast<const Vec<DT, E>*>(x + (int64_t)(s < L ? s : L - 1) * a.x_t);
      }
    } else {
#pragma unroll
      for (int r = 0; r < kAll + KW - 1; ++r) in[r] = input_at<DT, E>(a, x, state, t0 - KW + 1 + r, L);
    }
#pragma unroll
    for (int r = 0; r < kAll; ++r) {
      const int t = t0 + r;
      up[r] = *reinterpret_cast<const Vec<DT, E>*>(dy + (t < L ? t : L - 1) * d_t);
    }
  }
  float dp[KW][E];  // dp_{t}, dp_{t-1}, ... by (t mod KW)
#pragma unroll
  for (int k = 0; k < KW; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) dp[k][e] = 0.f;
#pragma unroll
  for (int r = 0; r < kAll; ++r) {
    const int t = t0 + r;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float g = to_f32<DT>(up[r].v[e]);
      if (a.silu) {
        float p = bias[e];
#pragma unroll
        for (int k = 0; k < KW; ++k)
          if (KW <= 4 || k >= KW - a.W) p = __builtin_fmaf(w[k][e], to_f32<DT>(in[r + k].v[e]), p);
        g *= silu_slope(p);
      }
      g = t < L ? g : 0.f;
      dp[r % KW][e] = g;
      if (r < kRun && t < L) {
        db[e] += g;
#pragma unroll
        for (int k = 0; k < KW; ++k) dw[k][e] = __builtin_fmaf(g, to_f32<DT>(in[r + k].v[e]), dw[k][e]);
      }
    }
    // the input at s = t - KW + 1 is complete
    const int s = t - KW + 1;
    const bool head = s < 0 && t0 == 0 && s > -a.W;
    if (r < KW - 1 && !head) continue;  // of the run in front
    float d[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      d[e] = 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k)
        if (KW <= 4 || k >= KW - a.W) d[e] = __builtin_fmaf(w[k][e], dp[(r + KW - k) % KW][e], d[e]);
    }
    const int j = s - (L - a.W + 1);
    if (dstate_n && j >= 0 && s < L) {
      const Vec<DT, E> more = *reinterpret_cast<const Vec<DT, E>*>(dstate_n + j * d_t);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] += to_f32<DT>(more.v[e]);
    }
    Vec<DT, E> out;
#pragma unroll
    for (int e = 0; e < E; ++e) out.v[e] = from_f32<DT>(s < L ? d[e] : 0.f);
    if (s >= 0) {
      if (s < a.T) *reinterpret_cast<Vec<DT, E>*>(dx + s * d_t) = out;
    } else if (a.dstate) {
      *reinterpret_cast<Vec<DT, E>*>((DT*)a.dstate + (s + a.W - 1) * d_t + cell) = out;
    }
  }
}

template <typename DT, int E, int KW>
__global__ __launch_bounds__(kConvThreads, KW <= 4 ? 2 : 1) void conv_backward_kernel(CausalConvArgs a) {
  __shared__ float lds[kConvThreads * E];
  const int groups = a.C / E, lanes = channel_lanes(groups), slots = kConvThreads / lanes;
  const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes;
  const int group = blockIdx.x * lanes + lane;
  const bool live = group < groups;
  const int c = live ? group * E : 0;
  const int64_t runs = (a.T + kRun - 1) / kRun, units = runs * a.B;
  float w[KW][E], bias[E], dw[KW][E], db[E];
  load_taps<DT, E, KW>(a, c, w, bias);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k) dw[k][e] = 0.f;
  }
  if (live) {
    for (int64_t unit = (int64_t)blockIdx.y * slots + slot; unit < units; unit += (int64_t)a.parts * slots)
      backward_run<DT, E, KW>(a, c, (int)(unit % a.B), (int)(unit / a.B) * kRun, w, bias, dw, db);
  }
  // the slots' sums, one filter tap at a time
#pragma unroll
  for (int k = 0; k <= KW; ++k) {
    if (KW > 4 && k < KW - a.W) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) lds[threadIdx.x * E + e] = k < KW ? dw[k < KW ? k : 0][e] : db[e];
    __syncthreads();
    const int kk = k < KW ? k - (KW - a.W) : a.W;
    for (int i = threadIdx.x; i < lanes * E; i += kConvThreads) {
      float sum = 0.f;
      for (int n = 0; n < slots; ++n) sum += lds[n * lanes * E + i];
      const int ch = blockIdx.x * lanes * E + i;
      if (ch < a.C) a.part[((int64_t)blockIdx.y * (a.W + 1) + kk) * a.C + ch] = sum;
    }
    __syncthreads();
  }
}

// dw and db from the workgroups' sums: 32 channels a workgroup, eight threads
// a channel, whose sums are joined in order.
__global__ __launch_bounds__(256) void conv_reduce_kernel(CausalConvArgs a) {
  __shared__ float lds[256];
  const int k = blockIdx.y, i = threadIdx.x & 31, part0 = threadIdx.x >> 5;
  const int ch = blockIdx.x * 32 + i;
  float sum = 0.f;
  if (ch < a.C) {
#pragma unroll 8
    for (int p = part0; p < a.parts; p += 8) sum += a.part[((int64_t)p * (a.W + 1) + k) * a.C + ch];
  }
  lds[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x >= 32 || ch >= a.C) return;
  for (int p = 1; p < 8; ++p) sum += lds[p * 32 + i];
  if (k < a.W)
    a.dw[(int64_t)ch * a.W + k] = sum;
  else if (a.db)
    a.db[ch] = sum;
}

template <typename DT, int E, int KW>
hipError_t forward(const CausalConvArgs& a, hipStream_t st) {
  const int64_t lanes = (int64_t)(a.C / E) * a.B;
  if (a.T <= 8) {
    launch_kernel(conv_forward_kernel<DT, E, KW, 1>, dim3((unsigned)((lanes * a.T + kConvThreads - 1) / kConvThreads)),
                  dim3(kConvThreads), 0, st, a);
  } else {
    const int64_t n = lanes * ((a.T + kRun - 1) / kRun);
    launch_kernel(conv_forward_kernel<DT, E, KW, kRun>, dim3((unsigned)((n + kConvThreads - 1) / kConvThreads)),
                  dim3(kConvThreads), 0, st, a);
  }
  return hipGetLastError();
}

template <typename DT, int E, int KW>
hipError_t backward(const CausalConvArgs& a, hipStream_t st) {
  const int groups = a.C / E, lanes = channel_lanes(groups);
  launch_kernel(conv_backward_kernel<DT, E, KW>, dim3((unsigned)((groups + lanes - 1) / lanes), (unsigned)a.parts),
                dim3(kConvThreads), 0, st, a);
  launch_kernel(conv_reduce_kernel, dim3((unsigned)((a.C + 31) / 32), (unsigned)(a.W + 1)), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <typename DT, int E, bool BACK>
hipError_t run(const CausalConvArgs& a, hipStream_t st) {
  if constexpr (BACK) {
    switch (a.W) {
      case 2: return backward<DT, E, 2>(a, st);
      case 3: return backward<DT, E, 3>(a, st);
      case 4: return backward<DT, E, 4>(a, st);
      default: return backward<DT, E, 8>(a, st);
    }
  } else {
    switch (a.W) {
      case 2: return forward<DT, E, 2>(a, st);
      case 3: return forward<DT, E, 3>(a, st);
      case 4: return forward<DT, E, 4>(a, st);
      default: return forward<DT, E, 8>(a, st);
    }
  }
}

template <typename DT>
hipError_t run_width(const CausalConvArgs& a, bool back, hipStream_t st) {
  if (back) return a.vec ? run<DT, kBackWide, true>(a, st) : run<DT, 1, true>(a, st);
  return a.vec ? run<DT, kWide<DT>, false>(a, st) : run<DT, 1, false>(a, st);
}

}  // namespace

// About four workgroups a compute unit over all channel tiles, fewer where
// the runs do not fill them.
int conv_parts(int T, int B, int C, int cus) {
  const int E = kBackWide, groups = (C + E - 1) / E, lanes = channel_lanes(groups);
  const int64_t tiles = (groups + lanes - 1) / lanes, slots = kConvThreads / lanes;
  const int64_t units = (int64_t)((T + kRun - 1) / kRun) * B;
  int64_t parts = 4 * (int64_t)cus / tiles;
  if (parts > (units + slots - 1) / slots) parts = (units + slots - 1) / slots;
  return (int)(parts < 1 ? 1 : parts);
}

double conv_threads(int T, int B, int C) {
  const double runs = T <= 8 ? T : (T + kRun - 1) / kRun;
  return runs * B * (double)C + kConvThreads;
}

hipError_t launch_causal_conv(const CausalConvArgs& a, bool bf, hipStream_t st) {
  return bf ? run_width<bf16>(a, false, st) : run_width<float>(a, false, st);
}

hipError_t launch_causal_conv_backward(const CausalConvArgs& a, bool bf, hipStream_t st) {
  return bf ? run_width<bf16>(a, true, st) : run_width<float>(a, true, st);
}

}  // namespace rnnk
