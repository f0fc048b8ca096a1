// Layer norm over the last dimension, forward and backward, with the
// residual add in front of it.
//
//   s = x + r (stored in the storage type),  mu = mean(s),
//   v = mean((s - mu)^2),  rstd = 1 / sqrt(v + eps),
//   y = (s - mu) rstd w + b
// Backward, with n = (s - mu) rstd and gw = dy w:
//   dx = rstd (gw - mean(gw) - n mean(gw n)) (+ ds),
//   dw = sum over rows of dy n,  db = sum over rows of dy
//
// A team of threads keeps one whole row in registers, so each tensor is read
// once and the variance is taken about the row's own mean (two passes over
// registers; no difference of large sums). Sums are fp32 and reduced in a
// fixed order, so the results are deterministic.
//
// Bound by memory. 32000 x 1024 bf16 with a residual: forward 45.6 us (its
// 262 MB at 5.7 TB/s), backward 47.4 us (5.5 TB/s) and 5.4 us for the
// reduction; with loads only as a row is reached the backward took 82.
#include "block_kernels.hpp"
#include "device_common.hpp"

namespace rnnk {
namespace {

constexpr int kE = 8;  // elements per thread and chunk
constexpr int threads_of(int team) { return team < 256 ? 256 : team; }

// A row is spread over TEAM threads (a part of a wave, a wave, or the whole
// workgroup) in V chunks of kE elements a thread. With 16-byte accesses a
// thread's elements are neighbours; without, neighbouring threads take
// neighbouring elements.
template <int TEAM, bool VEC>
__device__ __forceinline__ int col_of(int v, int e, int lane) {
  return VEC ? (v * TEAM + lane) * kE + e : (v * kE + e) * TEAM + lane;
}

template <typename DT, int TEAM, int V, bool VEC>
__device__ __forceinline__ void load_row(const DT* p, int N, int lane, float (*out)[kE]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (VEC) {
      struct alignas(16) Raw { DT v[kE]; };
      const int c = col_of<TEAM, true>(v, 0, lane);
      if (c < N) {
        const Raw r = *reinterpret_cast<const Raw*>(p + c);
#pragma unroll
        for (int e = 0; e < kE; ++e) out[v][e] = to_f32<DT>(r.v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) out[v][e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int c = col_of<TEAM, false>(v, e, lane);
        out[v][e] = c < N ? to_f32<DT>(p[c]) : 0.f;
      }
    }
  }
}

template <typename DT, int TEAM, int V, bool VEC>
__device__ __forceinline__ void store_row(DT* p, int N, int lane, const float (*in)[kE]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (VEC) {
      struct alignas(16) Raw { DT v[kE]; };
      const int c = col_of<TEAM, true>(v, 0, lane);
      if (c < N) {
        Raw r;
#pragma unroll
        for (int e = 0; e < kE; ++e) r.v[e] = from_f32<DT>(in[v][e]);
        *reinterpret_cast<Raw*>(p + c) = r;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int c = col_of<TEAM, false>(v, e, lane);
        if (c < N) p[c] = from_f32<DT>(in[v][e]);
      }
    }
  }
}

// Sum over the team, the same value in every thread.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* lds) {
  constexpr int kWidth = TEAM < 64 ? TEAM : 64;
#pragma unroll
  for (int m = kWidth / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if (TEAM > 64) {
    constexpr int kWaves = TEAM / 64;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += lds[i];
  }
  return v;
}

template <typename DT, int TEAM, int V, bool VEC, bool RES>
__global__ __launch_bounds__(threads_of(TEAM)) void norm_forward_kernel(NormArgs a) {
  constexpr int kThreads = threads_of(TEAM);
  __shared__ float lds[kThreads / 64];
  const int lane = threadIdx.x % TEAM;
  const int64_t row = a.row0 + blockIdx.x * (int64_t)(kThreads / TEAM) + threadIdx.x / TEAM;
  if (row >= a.rows) return;  // whole teams
  float s[V][kE];
  load_row<DT, TEAM, V, VEC>((const DT*)a.x + row * a.ldx, a.N, lane, s);
  if (RES) {
    float r[V][kE];
    load_row<DT, TEAM, V, VEC>((const DT*)a.r + row * a.ldr, a.N, lane, r);
    // the sum is normalised as it is stored, so that the backward pass reads
    // the very values that were normalised
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kE; ++e) s[v][e] = to_f32<DT>(from_f32<DT>(s[v][e] + r[v][e]));
    store_row<DT, TEAM, V, VEC>((DT*)a.sum + row * a.N, a.N, lane, s);
  }
  float t = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < kE; ++e) t += s[v][e];
  const float mu = team_sum<TEAM>(t, lds) / (float)a.N;
  t = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      s[v][e] = col_of<TEAM, VEC>(v, e, lane) < a.N ? s[v][e] - mu : 0.f;
      t = __builtin_fmaf(s[v][e], s[v][e], t);
    }
  const float rstd = 1.0f / __builtin_sqrtf(team_sum<TEAM>(t, lds) / (float)a.N + a.eps);
  if (a.stats && lane == 0) {
    a.stats[2 * row] = mu;
    a.stats[2 * row + 1] = rstd;
  }
  float w[V][kE];
  if (a.w) {
    load_row<DT, TEAM, V, VEC>((const DT*)a.w, a.N, lane, w);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kE; ++e) s[v][e] *= rstd * w[v][e];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kE; ++e) s[v][e] *= rstd;
  }
  if (a.b) {
    load_row<DT, TEAM, V, VEC>((const DT*)a.b, a.N, lane, w);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kE; ++e) s[v][e] += w[v][e];
  }
  store_row<DT, TEAM, V, VEC>((DT*)a.y + row * a.N, a.N, lane, s);
}

// A row as it lies in memory, so that the next row's loads can be in flight
// while one is worked on. Columns past the row repeat its last ones (no load
// is conditional) and count as zero when they are taken out.
template <typename DT, int TEAM, int V, bool VEC>
struct RawRow {
  struct alignas(VEC ? 16 : sizeof(DT)) Piece { DT v[kE]; };
  Piece p[V];
  __device__ __forceinline__ void load(const DT* row, int N, int lane) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (VEC) {
        const int c = col_of<TEAM, true>(v, 0, lane);
        p[v] = *reinterpret_cast<const Piece*>(row + (c < N ? c : N - kE));
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int c = col_of<TEAM, false>(v, e, lane);
          p[v].v[e] = row[c < N ? c : N - 1];
        }
      }
    }
  }
  __device__ __forceinline__ float get(int v, int e, int N, int lane) const {
    return col_of<TEAM, VEC>(v, VEC ? 0 : e, lane) < N ? to_f32<DT>(p[v].v[e]) : 0.f;
  }
};

// Rows are dealt to the teams in turn; a thread sums dw and db of its own
// columns in registers over its rows, and the workgroup's teams join them in
// LDS into one row of partial sums. DS: a gradient of the sum is added.
template <typename DT, int TEAM, int V, bool VEC, bool DS>
__global__ __launch_bounds__(threads_of(TEAM)) void norm_backward_kernel(NormArgs a) {
  constexpr int kThreads = threads_of(TEAM), kTeams = kThreads / TEAM;
  __shared__ float lds[kThreads / 64];
  __shared__ float join[kTeams > 1 ? kThreads * kE : 1];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  float w[V][kE], dw[V][kE], db[V][kE];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < kE; ++e) w[v][e] = 1.f, dw[v][e] = 0.f, db[v][e] = 0.f;
  if (a.w) load_row<DT, TEAM, V, VEC>((const DT*)a.w, a.N, lane, w);
  const float inv = 1.0f / (float)a.N;
  // the next row's loads in flight, where there are registers for them
  constexpr bool kAhead = V <= 2;
  RawRow<DT, TEAM, V, VEC> rx, rdy, rds;
  float mu = 0.f, rstd = 0.f;
  auto load = [&](int64_t row) {
    rx.load((const DT*)a.x + row * a.ldx, a.N, lane);
    rdy.load((const DT*)a.dy + row * a.N, a.N, lane);
    if (DS && kAhead) rds.load((const DT*)a.ds + row * a.N, a.N, lane);
    mu = a.stats[2 * row];
    rstd = a.stats[2 * row + 1];
  };
  const int64_t hop = (int64_t)gridDim.x * kTeams;
  int64_t row = blockIdx.x * (int64_t)kTeams + team;
  if (kAhead && row < a.rows) load(row);
  for (; row < a.rows; row += hop) {
    if (!kAhead) load(row);
    float n[V][kE], g[V][kE], s[DS && kAhead ? V : 1][kE];
    float s1 = 0.f, s2 = 0.f;
    const float scale = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        // past the row g is zero, and n times it
        n[v][e] = (rx.get(v, e, a.N, lane) - mu) * rstd;
        g[v][e] = rdy.get(v, e, a.N, lane);
        if (DS && kAhead) s[DS && kAhead ? v : 0][e] = to_f32<DT>(rds.p[v].v[e]);
        db[v][e] += g[v][e];
        dw[v][e] = __builtin_fmaf(g[v][e], n[v][e], dw[v][e]);
        g[v][e] *= w[v][e];
        s1 += g[v][e];
        s2 = __builtin_fmaf(g[v][e], n[v][e], s2);
      }
    if (kAhead && row + hop < a.rows) load(row + hop);
    if (DS && !kAhead) rds.load((const DT*)a.ds + row * a.N, a.N, lane);
    s1 = team_sum<TEAM>(s1, lds) * inv;
    s2 = team_sum<TEAM>(s2, lds) * inv;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        g[v][e] = scale * (g[v][e] - s1 - n[v][e] * s2);
        if (DS) g[v][e] += kAhead ? s[DS && kAhead ? v : 0][e] : to_f32<DT>(rds.p[v].v[e]);
      }
    store_row<DT, TEAM, V, VEC>((DT*)a.dx + row * a.N, a.N, lane, g);
  }
  if (!a.part) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* dst = a.part + ((int64_t)blockIdx.x * 2 + which) * a.ld_part;
      if (kTeams > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kE; ++e)
          join[team * (TEAM * kE) + lane * kE + e] = which ? db[v][e] : dw[v][e];
        __syncthreads();
        for (int k = threadIdx.x; k < TEAM * kE; k += kThreads) {
          float t = 0.f;
#pragma unroll
          for (int q = 0; q < kTeams; ++q) t += join[q * (TEAM * kE) + k];
          const int c = col_of<TEAM, VEC>(v, k % kE, k / kE);
          if (c < a.N) dst[c] = t;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int c = col_of<TEAM, VEC>(v, e, lane);
          if (c < a.N) dst[c] = which ? db[v][e] : dw[v][e];
        }
      }
    }
  }
}

// dw and db from the workgroups' partial sums: a workgroup takes 64 columns
// of one of the two, 16 threads across (four columns each) by 64 along the
// partial rows, whose sums then meet in LDS.
constexpr int kReduceThreads = 1024;
__global__ __launch_bounds__(kReduceThreads) void norm_reduce_kernel(const float* __restrict__ part, int blocks, int N,
                                                                     int64_t ld, float* __restrict__ dw,
                                                                     float* __restrict__ db) {
  __shared__ f32x4 lds[kReduceThreads];
  const int which = blockIdx.y, c = blockIdx.x * 64 + (threadIdx.x & 15) * 4, along = threadIdx.x >> 4;
  f32x4 t = {0.f, 0.f, 0.f, 0.f};
  if (c < N) {
#pragma unroll 16
    for (int k = along; k < blocks; k += 64) t += *reinterpret_cast<const f32x4*>(part + ((int64_t)k * 2 + which) * ld + c);
  }
  lds[threadIdx.x] = t;
  __syncthreads();
#pragma unroll
  for (int half = 32; half > 0; half >>= 1) {
    if (along < half) lds[threadIdx.x] = t = t + lds[threadIdx.x + half * 16];
    __syncthreads();
  }
  float* out = which ? db : dw;
  if (along == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < N) out[c + j] = t[j];
  }
}

template <typename DT, int TEAM, int V, bool VEC>
void run_forward(NormArgs a, hipStream_t st) {
  constexpr int kThreads = threads_of(TEAM), kTeams = kThreads / TEAM;
  // a launch has less than 2^32 threads
  constexpr int64_t kMost = (1ll << 31) / kThreads;
  for (int64_t left = (a.rows + kTeams - 1) / kTeams; left > 0; left -= kMost, a.row0 += kMost * kTeams) {
    const dim3 grid((unsigned)(left < kMost ? left : kMost)), block(kThreads);
    if (a.r)
      launch_kernel(norm_forward_kernel<DT, TEAM, V, VEC, true>, grid, block, 0, st, a);
    else
      launch_kernel(norm_forward_kernel<DT, TEAM, V, VEC, false>, grid, block, 0, st, a);
  }
}

template <typename DT, int TEAM, int V, bool VEC>
void run_backward(const NormArgs& a, hipStream_t st) {
  launch_kernel(a.ds ? norm_backward_kernel<DT, TEAM, V, VEC, true> : norm_backward_kernel<DT, TEAM, V, VEC, false>,
                dim3((unsigned)a.blocks), dim3(threads_of(TEAM)), 0, st, a);
}

// The team of a row: as few threads as hold it in 8 or 16 elements each (the
// backward pass keeps about ten registers an element). 16 threads up to 128
// elements, a wave up to 1024, then a workgroup of 256 or 512. Past 8192
// elements a thread holds 32, and the backward pass spills: up to 26 registers
// with 16-byte accesses (16384: 3.2 to 3.7 TB/s, 8192: 3.4 to 4.3) and 195 to
// 303 without (16377: 0.5 to 1.2 TB/s).
template <typename DT, bool VEC, bool BACK>
void pick(const NormArgs& a, hipStream_t st) {
#define NORM_RUN(TEAM, V) return BACK ? run_backward<DT, TEAM, V, VEC>(a, st) : run_forward<DT, TEAM, V, VEC>(a, st)
  const int N = a.N;
  if (N <= 128) NORM_RUN(16, 1);
  if (N <= 512) NORM_RUN(64, 1);
  if (N <= 1024) NORM_RUN(64, 2);
  if (N <= 2048) NORM_RUN(256, 1);
  if (N <= 4096) NORM_RUN(256, 2);
  if (N <= 8192) NORM_RUN(512, 2);
  NORM_RUN(512, 4);
#undef NORM_RUN
}

}  // namespace

int norm_backward_blocks(int64_t rows, int N, int cus) {
  // about 1024 threads a compute unit
  const int teams = N <= 128 ? 16 : N <= 1024 ? 4 : 1, each = N <= 4096 ? 4 : N <= 8192 ? 2 : 1;
  const int64_t need = (rows + teams - 1) / teams, most = (int64_t)each * cus;
  return (int)(need < most ? need : most);
}

hipError_t launch_layer_norm(const NormArgs& a, bool bf, hipStream_t st) {
  if (bf)
    a.vec ? pick<bf16, true, false>(a, st) : pick<bf16, false, false>(a, st);
  else
    a.vec ? pick<float, true, false>(a, st) : pick<float, false, false>(a, st);
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const NormArgs& a, bool bf, hipStream_t st) {
  if (bf)
    a.vec ? pick<bf16, true, true>(a, st) : pick<bf16, false, true>(a, st);
  else
    a.vec ? pick<float, true, true>(a, st) : pick<float, false, true>(a, st);
  if (a.part)
    launch_kernel(norm_reduce_kernel, dim3((a.N + 63) / 64, 2), dim3(kReduceThreads), 0, st, (const float*)a.part, a.blocks,
                  a.N, a.ld_part, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace rnnk
