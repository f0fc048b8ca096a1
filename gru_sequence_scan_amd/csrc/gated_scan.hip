// Gated linear recurrence over time, forward and backward.
//
//   a_t = sigma(f_t)
//   u_t = (1 - a_t) x_t              (coupled gates), or
//   u_t = sigma(i_t) x_t             (a gate of its own for the input)
//   h_t = a_t h_{t-1} + u_t
//
// per channel of [T, B, H]. A step is the affine map h -> a h + u, and maps
// compose: (A, U) after (A', U') is (A A', A U' + U). So time is cut into
// chunks that are composed independently (kernel 1), the states at the chunk
// boundaries follow from the few composed maps (kernel 2), and every chunk
// is then run from its own boundary state (kernel 3).
//
// Backward, with g_t the gradient of h_t and c the part of it that comes
// from later steps:
//   g_t = dy_t + c_{t+1},  c_t = a_t g_t,  c_{L+1} = dh_n,  dh_0 = c_1
//   coupled: df = g (h_{t-1} - x) a (1 - a), dx = g (1 - a)
//   gate:    df = g h_{t-1} a (1 - a), di = g x s (1 - s), dx = g s
// c runs the same chunked way from the far end. h_{t-1} is computed again in
// fp32 from the boundary states that the training forward kept, so y (rounded
// to the storage type) is not read.
//
// All states, products and sums are fp32; only x, f, i, dy and the outputs
// y, dx, df, di have the storage type.
#include "block_kernels.hpp"
#include "device_common.hpp"

namespace rnnk {
namespace {

constexpr int kLanes = 64;    // channels of a workgroup's tile
constexpr int kThreads = 256;

// A thread takes E neighbouring channels (one access) of kSteps consecutive
// steps; the chunk is kChunk steps for every E, so that the boundary states
// do not depend on how the rows happen to be aligned.
template <int E>
struct Tile {
  static constexpr int kGroups = kLanes / E;          // threads across the channels
  static constexpr int kSlots = kThreads / kGroups;   // threads along time
  static constexpr int kSteps = 32 / E;
  static_assert(kSlots * kSteps == kGatedScanChunk, "chunk length");
};

// a = sigma(f) and 1 - a = sigma(-f), each with its own relative accuracy:
// exp of -|f| cannot overflow and neither value is formed by a difference.
__device__ __forceinline__ void gates_of(float f, float* a, float* keep) {
  const float e = fexp(-__builtin_fabsf(f));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float er = e * r;
  *a = f >= 0.f ? r : er;
  *keep = f >= 0.f ? er : r;
}

template <typename DT, int E>
__device__ __forceinline__ void load_vec(const DT* p, float* out) {
  struct alignas(sizeof(DT) * E) Raw { DT v[E]; };
  const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = to_f32<DT>(r.v[e]);
}

template <typename DT, int E>
__device__ __forceinline__ void store_vec(DT* p, const float* in) {
  struct alignas(sizeof(DT) * E) Raw { DT v[E]; };
  Raw r;
#pragma unroll
  for (int e = 0; e < E; ++e) r.v[e] = from_f32<DT>(in[e]);
  *reinterpret_cast<Raw*>(p) = r;
}

// Where a workgroup works: channel tile, batch row, chunk of steps.
struct Place {
  int b, c, L;       // batch row, chunk, the row's length
  int h;             // this thread's first channel
  int slot, s0;      // this thread's place along time and its first step
  bool live;         // the thread has channels
};

template <int E>
__device__ __forceinline__ Place place_of(const GatedScanArgs& a) {
  Place p;
  unsigned id = blockIdx.x;
  const int ct = id % a.tiles;
  id /= a.tiles;
  p.b = id % a.B;
  p.c = id / a.B;
  const int L = a.lengths ? a.lengths[p.b] : a.T;
  p.L = L < 0 ? 0 : (L > a.T ? a.T : L);
  const int grp = threadIdx.x % Tile<E>::kGroups;
  p.slot = threadIdx.x / Tile<E>::kGroups;
  p.h = ct * kLanes + grp * E;
  p.live = p.h < a.H;
  p.s0 = p.c * kGatedScanChunk + p.slot * Tile<E>::kSteps;
  return p;
}

__device__ __forceinline__ int time_of(const GatedScanArgs& a, const Place& p, int s) {
  return a.reverse && s < p.L ? p.L - 1 - s : s;
}

// The gate values a, 1 - a (or sigma(i)) and the input x of this thread's
// steps; a step past the row's end is the identity map (a = 1, u = 0).
template <typename DT, int E, bool GATE>
__device__ __forceinline__ void load_step(const GatedScanArgs& g, const Place& p, int s, float* a, float* keep, float* w,
                                          float* x) {
  if (p.live && s < p.L) {
    const int t = time_of(g, p, s);
    float f[E];
    load_vec<DT, E>((const DT*)g.f + t * g.f_t + p.b * g.f_b + p.h, f);
    load_vec<DT, E>((const DT*)g.x + t * g.x_t + p.b * g.x_b + p.h, x);
    if (GATE) {
      float i[E];
      load_vec<DT, E>((const DT*)g.i + t * g.i_t + p.b * g.i_b + p.h, i);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float no;
        gates_of(i[e], &w[e], &no);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      gates_of(f[e], &a[e], &keep[e]);
      if (!GATE) w[e] = keep[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      a[e] = 1.f;
      keep[e] = 0.f;
      w[e] = 0.f;
      x[e] = 0.f;
    }
  }
}

// Exclusive composition of the threads' maps along time. In: each thread's
// own map (P, S). Out: lds_p / lds_s [slot][channel] hold the composition of
// the slots before (forward) or after (REV) it; tot the whole chunk's map.
template <int E, bool REV>
__device__ __forceinline__ void compose_slots(float* lds_p, float* lds_s, const float* P, const float* S, int slot, int ch,
                                              float* tot_p, float* tot_s) {
  constexpr int kSlots = Tile<E>::kSlots;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lds_p[slot * kLanes + ch + e] = P[e];
    lds_s[slot * kLanes + ch + e] = S[e];
  }
  __syncthreads();
  if (threadIdx.x < kLanes) {
    float cp = 1.f, cs = 0.f;
#pragma unroll 4
    for (int n = 0; n < kSlots; ++n) {
      const int k = (REV ? kSlots - 1 - n : n) * kLanes + threadIdx.x;
      const float p = lds_p[k], s = lds_s[k];
      lds_p[k] = cp;
      lds_s[k] = cs;
      cs = p * cs + s;
      cp = p * cp;
    }
    *tot_p = cp;
    *tot_s = cs;
  }
  __syncthreads();
}

// Kernel 1: the composed map of every chunk. Forward: h -> P h + S.
// Backward (BACK): c -> P c + S from the chunk's end to its beginning.
template <typename DT, int E, bool GATE, bool BACK>
__global__ __launch_bounds__(kThreads) void scan_compose_kernel(GatedScanArgs g) {
  constexpr int kSteps = Tile<E>::kSteps;
  __shared__ float lds_p[Tile<E>::kSlots * kLanes], lds_s[Tile<E>::kSlots * kLanes];
  const Place p = place_of<E>(g);
  float P[E], S[E];
#pragma unroll
  for (int e = 0; e < E; ++e) P[e] = 1.f, S[e] = 0.f;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int s = p.s0 + (BACK ? kSteps - 1 - k : k);
    float a[E], keep[E], w[E], x[E];
    if (BACK) {
      if (p.live && s < p.L) {
        const int t = time_of(g, p, s);
        float f[E], dy[E];
        load_vec<DT, E>((const DT*)g.f + t * g.f_t + p.b * g.f_b + p.h, f);
        load_vec<DT, E>((const DT*)g.dy + ((int64_t)t * g.B + p.b) * g.H + p.h, dy);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          gates_of(f[e], &a[e], &keep[e]);
          S[e] = a[e] * (S[e] + dy[e]);
          P[e] *= a[e];
        }
      }
    } else {
      load_step<DT, E, GATE>(g, p, s, a, keep, w, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        S[e] = a[e] * S[e] + w[e] * x[e];
        P[e] *= a[e];
      }
    }
  }
  float tp, ts;
  compose_slots<E, BACK>(lds_p, lds_s, P, S, p.slot, (threadIdx.x % Tile<E>::kGroups) * E, &tp, &ts);
  const int h = (blockIdx.x % g.tiles) * kLanes + threadIdx.x;
  if (threadIdx.x < kLanes && h < g.H) {
    const int64_t o = ((int64_t)p.c * g.B + p.b) * g.H + h;
    g.map_p[o] = tp;
    g.map_s[o] = ts;
  }
}

// Kernel 2: the states at the chunk boundaries, one thread per channel.
// Forward: state[c] enters chunk c, h_n leaves the last one. Backward:
// state[c] enters chunk c from its end; dh_0 leaves the first one.
__global__ __launch_bounds__(kThreads) void scan_carry_kernel(const float* __restrict__ map_p, const float* __restrict__ map_s,
                                                              const float* __restrict__ first, float* __restrict__ state,
                                                              float* __restrict__ last, int chunks, int64_t n, int back) {
  const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (i >= n) return;
  float h = first ? first[i] : 0.f;
#pragma unroll 8
  for (int k = 0; k < chunks; ++k) {
    const int64_t o = (back ? chunks - 1 - k : k) * n + i;
    const float p = map_p[o], s = map_s[o];
    state[o] = h;
    h = p * h + s;
  }
  if (last) last[i] = h;
}

// Kernel 3, forward: runs every chunk from the state that enters it.
template <typename DT, int E, bool GATE>
__global__ __launch_bounds__(kThreads) void scan_forward_kernel(GatedScanArgs g) {
  constexpr int kSteps = Tile<E>::kSteps;
  __shared__ float lds_p[Tile<E>::kSlots * kLanes], lds_s[Tile<E>::kSlots * kLanes];
  const Place p = place_of<E>(g);
  const int ch = (threadIdx.x % Tile<E>::kGroups) * E;
  float a[kSteps][E], u[kSteps][E], P[E], S[E];
#pragma unroll
  for (int e = 0; e < E; ++e) P[e] = 1.f, S[e] = 0.f;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    float keep[E], w[E], x[E];
    load_step<DT, E, GATE>(g, p, p.s0 + k, a[k], keep, w, x);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      u[k][e] = w[e] * x[e];
      S[e] = a[k][e] * S[e] + u[k][e];
      P[e] *= a[k][e];
    }
  }
  float tp, ts;
  compose_slots<E, false>(lds_p, lds_s, P, S, p.slot, ch, &tp, &ts);
  float h[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    h[e] = 0.f;
    if (p.live) {
      const int64_t o = (int64_t)p.b * g.H + p.h + e;
      if (g.chunks > 1)
        h[e] = g.state[(int64_t)p.c * g.B * g.H + o];
      else if (g.h0)
        h[e] = g.h0[o];
      if (g.chunks == 1 && g.keep_state && p.slot == 0) g.state[o] = h[e];
    }
    h[e] = lds_p[p.slot * kLanes + ch + e] * h[e] + lds_s[p.slot * kLanes + ch + e];
  }
  if (!p.live) return;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int s = p.s0 + k;
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h[e] = a[k][e] * h[e] + u[k][e];
      y[e] = s < p.L ? h[e] : 0.f;
    }
    if (s < g.T) store_vec<DT, E>((DT*)g.y + ((int64_t)time_of(g, p, s) * g.B + p.b) * g.H + p.h, y);
  }
  // with more than one chunk kernel 2 has written h_n
  if (g.chunks == 1 && g.h_n && p.slot == Tile<E>::kSlots - 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) g.h_n[(int64_t)p.b * g.H + p.h + e] = h[e];
  }
}

// Kernel 3, backward.
template <typename DT, int E, bool GATE>
__global__ __launch_bounds__(kThreads) void scan_backward_kernel(GatedScanArgs g) {
  constexpr int kSteps = Tile<E>::kSteps;
  __shared__ float lds_p[Tile<E>::kSlots * kLanes], lds_s[Tile<E>::kSlots * kLanes];
  const Place p = place_of<E>(g);
  const int ch = (threadIdx.x % Tile<E>::kGroups) * E;
  const int at = p.slot * kLanes + ch;
  float a[kSteps][E], keep[kSteps][E], w[kSteps][E], x[kSteps][E], hp[kSteps][E];
  float P[E], S[E];
  float tp, ts;
  // h_{t-1} of every step
#pragma unroll
  for (int e = 0; e < E; ++e) P[e] = 1.f, S[e] = 0.f;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    load_step<DT, E, GATE>(g, p, p.s0 + k, a[k], keep[k], w[k], x[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      S[e] = a[k][e] * S[e] + w[k][e] * x[k][e];
      P[e] *= a[k][e];
    }
  }
  compose_slots<E, false>(lds_p, lds_s, P, S, p.slot, ch, &tp, &ts);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float h = p.live ? g.state[((int64_t)p.c * g.B + p.b) * g.H + p.h + e] : 0.f;
    h = lds_p[at + e] * h + lds_s[at + e];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      hp[k][e] = h;
      h = a[k][e] * h + w[k][e] * x[k][e];
    }
  }
  __syncthreads();
  // c of every step, from the chunk's end
  float dy[kSteps][E];
#pragma unroll
  for (int e = 0; e < E; ++e) S[e] = 0.f;
#pragma unroll
  for (int k = kSteps - 1; k >= 0; --k) {
    const int s = p.s0 + k;
    if (p.live && s < p.L) {
      load_vec<DT, E>((const DT*)g.dy + ((int64_t)time_of(g, p, s) * g.B + p.b) * g.H + p.h, dy[k]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) dy[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) S[e] = a[k][e] * (S[e] + dy[k][e]);
  }
  compose_slots<E, true>(lds_p, lds_s, P, S, p.slot, ch, &tp, &ts);
  if (!p.live) return;
  float c[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t o = (int64_t)p.b * g.H + p.h + e;
    if (g.chunks > 1)
      c[e] = g.back_state[(int64_t)p.c * g.B * g.H + o];
    else
      c[e] = g.dh_n ? g.dh_n[o] : 0.f;
    c[e] = lds_p[at + e] * c[e] + lds_s[at + e];
  }
#pragma unroll
  for (int k = kSteps - 1; k >= 0; --k) {
    const int s = p.s0 + k;
    float dx[E], df[E], di[E];
    const bool on = s < p.L;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float gt = dy[k][e] + c[e];
      c[e] = on ? a[k][e] * gt : c[e];
      const float ga = gt * a[k][e] * keep[k][e];
      dx[e] = on ? gt * w[k][e] : 0.f;
      df[e] = on ? ga * (GATE ? hp[k][e] : hp[k][e] - x[k][e]) : 0.f;
      di[e] = GATE && on ? gt * x[k][e] * w[k][e] * (1.0f - w[k][e]) : 0.f;
    }
    if (s < g.T) {
      const int64_t o = ((int64_t)time_of(g, p, s) * g.B + p.b) * g.H + p.h;
      store_vec<DT, E>((DT*)g.dx + o, dx);
      store_vec<DT, E>((DT*)g.df + o, df);
      if (GATE) store_vec<DT, E>((DT*)g.di + o, di);
    }
  }
  if (g.chunks == 1 && g.dh0 && p.slot == 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) g.dh0[(int64_t)p.b * g.H + p.h + e] = c[e];
  }
}

template <typename DT, int E, bool GATE>
hipError_t run(const GatedScanArgs& a, bool back, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.tiles * a.B * a.chunks)), block(kThreads);
  const int64_t n = (int64_t)a.B * a.H;
  const dim3 cgrid((unsigned)((n + kThreads - 1) / kThreads));
  if (back) {
    if (a.chunks > 1) {
      launch_kernel(scan_compose_kernel<DT, E, GATE, true>, grid, block, 0, st, a);
      launch_kernel(scan_carry_kernel, cgrid, block, 0, st, (const float*)a.map_p, (const float*)a.map_s, a.dh_n,
                    a.back_state, a.dh0, a.chunks, n, 1);
    }
    launch_kernel(scan_backward_kernel<DT, E, GATE>, grid, block, 0, st, a);
  } else {
    if (a.chunks > 1) {
      launch_kernel(scan_compose_kernel<DT, E, GATE, false>, grid, block, 0, st, a);
      launch_kernel(scan_carry_kernel, cgrid, block, 0, st, (const float*)a.map_p, (const float*)a.map_s, a.h0, a.state,
                    a.h_n, a.chunks, n, 0);
    }
    launch_kernel(scan_forward_kernel<DT, E, GATE>, grid, block, 0, st, a);
  }
  return hipGetLastError();
}

template <typename DT, int E>
hipError_t run_gate(const GatedScanArgs& a, bool back, hipStream_t st) {
  return a.i ? run<DT, E, true>(a, back, st) : run<DT, E, false>(a, back, st);
}

}  // namespace

hipError_t launch_gated_scan(GatedScanArgs a, bool bf, bool back, hipStream_t st) {
  a.tiles = (a.H + kLanes - 1) / kLanes;
  if (a.width == 1) return bf ? run_gate<bf16, 1>(a, back, st) : run_gate<float, 1>(a, back, st);
  return bf ? run_gate<bf16, 4>(a, back, st) : run_gate<float, 4>(a, back, st);
}

}  // namespace rnnk
