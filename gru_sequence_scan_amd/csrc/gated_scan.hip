// Gated linear recurrence over time, forward and backward.
//
//   a_t = sigma(f_t)
//   u_t = (1 - a_t) x_t              (coupled gates), or
//   u_t = sigma(i_t) x_t             (a gate of its own for the input)
//   h_t = a_t h_{t-1} + u_t
//
// per channel of [T, B, H]. A step is the affine map h -> a h + u, and maps
// compose: (A, U) after (A', U') is (A A', A U' + U).
//
// A workgroup owns 128 bytes of channels of one batch row and walks their
// time in chunks of 128 steps. A thread holds 4 channels x 4 steps of a chunk
// (one channel x 16 steps where rows are not aligned) in registers: it
// composes its own steps, a thread per channel runs the entering state
// through the threads' maps in LDS, and every thread then runs its steps from the state that enters
// them. So each tensor is read once, while the next chunk's loads are in
// flight. Where that gives too few workgroups (few channels, long time) the
// time axis is cut into segments as well: a first launch composes each
// segment's map, a second runs the state through the segments, and the walk
// starts from there; the inputs are read twice then.
//
// Backward, with g_t the gradient of h_t and c the part of it that comes
// from later steps:
//   g_t = dy_t + c_{t+1},  c_t = a_t g_t,  c_{L+1} = dh_n,  dh_0 = c_1
//   coupled: df = g (h_{t-1} - x) a (1 - a), dx = g (1 - a)
//   gate:    df = g h_{t-1} a (1 - a), di = g x s (1 - s), dx = g s
// c runs the same way from the far end. h_{t-1} is computed again in fp32
// from the state at every chunk's beginning, which the training forward kept
// (1 / 64 of a bf16 tensor), so y (rounded to the storage type) is not read.
// Every 1 - s is formed as sigma of the negative, not by a difference.
//
// All states, products and sums are fp32; only x, f, i, dy and the outputs
// y, dx, df, di have the storage type.
//
// Bound by memory. T = 1000, B = 32, H = 1024, bf16, forward: 46 us (its 197
// MB at 4.3 TB/s); a launch per step of the method over all chunks (compose,
// carry, run) took 80. T = 16384, B = 2, H = 1000, bf16: forward 36 (compose)
// + 5 + 39 us, backward 29 + 5 + 69 us. T = 500, B = 64 ragged, H = 512, fp32
// with an input gate: forward 57 us (3.0 TB/s: the longest rows' chunks follow
// each other on few compute units, and a row's tiles on one XCD), backward 71
// us (4.8 TB/s).
#include "block_kernels.hpp"
#include "device_common.hpp"

namespace rnnk {
namespace {

// A workgroup's tile is 128 bytes of channels wide. A thread takes E
// neighbouring channels (one access) of kSteps consecutive steps; the chunk is
// the same for every E, so that the kept states do not depend on how the rows
// happen to be aligned.
template <typename DT>
constexpr int kScanLanes = 128 / (int)sizeof(DT);
template <typename DT>
constexpr int kScanThreads = kScanLanes<DT> * 8;
template <typename DT, int E>
struct Tile {
  static constexpr int kLanes = kScanLanes<DT>, kThreads = kScanThreads<DT>;
  static constexpr int kGroups = kLanes / E;          // threads across the channels
  static constexpr int kSlots = kThreads / kGroups;   // threads along time
  static constexpr int kSteps = 16 / E;
  static_assert(kSlots * kSteps == kGatedScanChunk, "chunk length");
};

// a = sigma(f) and 1 - a = sigma(-f), each with its own relative accuracy:
// exp of -|f| cannot overflow and neither value is formed by a difference. The
// exponent is a rounded product, so the smaller one carries about |f| / 2 units
// in its last place (5e-6 at |f| = 80).
__device__ __forceinline__ void gates_of(float f, float* a, float* keep) {
  const float e = fexp(-__builtin_fabsf(f));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float er = e * r;
  *a = f >= 0.f ? r : er;
  *keep = f >= 0.f ? er : r;
}
__device__ __forceinline__ float sigma(float f) {
  float a, keep;
  gates_of(f, &a, &keep);
  return a;
}

template <typename DT, int E>
struct alignas(sizeof(DT) * E) Raw {
  DT v[E];
};

template <typename DT, int E>
__device__ __forceinline__ void store_vec(DT* p, const float* in) {
  Raw<DT, E> r;
#pragma unroll
  for (int e = 0; e < E; ++e) r.v[e] = from_f32<DT>(in[e]);
  *reinterpret_cast<Raw<DT, E>*>(p) = r;
}

// Where a thread works: batch row, segment of chunks, channels, place in time.
template <typename DT, int E>
struct Place {
  int b, L;          // batch row and its length
  int c0, c1;        // the segment's chunks
  int seg, ct;       // segment, channel tile
  int h, ch;         // first channel, in the tensor and in the tile
  int slot;
  bool live;         // the thread has channels
  __device__ __forceinline__ explicit Place(const GatedScanArgs& a) {
    // Workgroup ids are dealt to the XCDs in turn. The tiles of one (row,
    // segment) go to one XCD one after the other, where they share its L2:
    // rows of H channels that are not a multiple of 128 bytes have cache lines
    // that belong to two tiles.
    const unsigned slot = blockIdx.x / a.xcds, unit = slot / a.tiles * a.xcds + blockIdx.x % a.xcds;
    ct = slot % a.tiles;
    b = unit % a.B;
    seg = unit / a.B;
    c0 = seg * a.seg_chunks;
    c1 = c0 + a.seg_chunks < a.chunks ? c0 + a.seg_chunks : a.chunks;
    const int n = a.lengths ? a.lengths[b] : a.T;
    L = n < 0 ? 0 : (n > a.T ? a.T : n);
    ch = threadIdx.x % Tile<DT, E>::kGroups * E;
    this->slot = threadIdx.x / Tile<DT, E>::kGroups;
    h = ct * Tile<DT, E>::kLanes + ch;
    live = h < a.H;
  }
  __device__ __forceinline__ int step0(int chunk) const { return chunk * kGatedScanChunk + slot * Tile<DT, E>::kSteps; }
  // the time of step s < L
  __device__ __forceinline__ int time(const GatedScanArgs& a, int s) const { return a.reverse ? L - 1 - s : s; }
};

// A thread's steps of one chunk as they lie in memory. Loads are never
// conditional (a condition per step would make each wait for the one before
// it): a step past the row's end reads the last one again, and a thread past
// the last channel the first ones; neither is used.
template <typename DT, int E, bool GATE, bool DY>
struct Steps {
  static constexpr int K = Tile<DT, E>::kSteps;
  Raw<DT, E> f[K], x[K], i[GATE ? K : 1], dy[DY ? K : 1];
  __device__ __forceinline__ void load(const GatedScanArgs& g, const Place<DT, E>& p, int chunk) {
    const int s0 = p.step0(chunk), h = p.live ? p.h : 0;
    const DT* pf = (const DT*)g.f + p.b * g.f_b + h;
    const DT* px = (const DT*)g.x + p.b * g.x_b + h;
    const DT* pi = GATE ? (const DT*)g.i + p.b * g.i_b + h : nullptr;
    const DT* pd = DY ? (const DT*)g.dy + (int64_t)p.b * g.H + h : nullptr;
    const int64_t d_t = (int64_t)g.B * g.H;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int s = s0 + k < p.L ? s0 + k : p.L - 1;
      const int64_t t = p.time(g, s);
      f[k] = *reinterpret_cast<const Raw<DT, E>*>(pf + t * g.f_t);
      x[k] = *reinterpret_cast<const Raw<DT, E>*>(px + t * g.x_t);
      if (GATE) i[k] = *reinterpret_cast<const Raw<DT, E>*>(pi + t * g.i_t);
      if (DY) dy[k] = *reinterpret_cast<const Raw<DT, E>*>(pd + t * d_t);
    }
  }
};

// Runs a state through the threads' maps, in the order of their steps (or
// against it): in P, S of every slot, out the state that enters it (in S's
// place). One thread per channel carries the state: of the first wave, or of
// the second for the other direction.
template <typename DT, int E, bool AGAINST>
__device__ __forceinline__ float run_slots(const float* P, float* S, float state, int c) {
  constexpr int kSlots = Tile<DT, E>::kSlots, kLanes = Tile<DT, E>::kLanes;
#pragma unroll 8
  for (int n = 0; n < kSlots; ++n) {
    const int k = (AGAINST ? kSlots - 1 - n : n) * kLanes + c;
    const float p = P[k], s = S[k];
    S[k] = state;
    state = __builtin_fmaf(p, state, s);
  }
  return state;
}

// The composed map of a segment: h -> P h + S, or (BACK) c -> P c + S from
// the segment's end to its beginning, walked like the main pass.
template <typename DT, int E, bool GATE, bool BACK>
__global__ __launch_bounds__(kScanThreads<DT>) void scan_compose_kernel(GatedScanArgs g) {
  constexpr int K = Tile<DT, E>::kSteps, kSlots = Tile<DT, E>::kSlots, kLanes = Tile<DT, E>::kLanes;
  __shared__ float lds_p[2][kSlots * kLanes], lds_s[2][kSlots * kLanes];
  const Place<DT, E> p(g);
  if (p.seg >= g.segs) return;
  const int at = p.slot * kLanes + p.ch;
  if (BACK) {  // the map c -> a (c + dy) has dy in x's place
    g.x = g.dy;
    g.x_t = (int64_t)g.B * g.H;
    g.x_b = g.H;
  }
  const int c1 = p.c1 * kGatedScanChunk < p.L ? p.c1 : (p.L + kGatedScanChunk - 1) / kGatedScanChunk;  // chunks with steps
  const int n = c1 - p.c0;
  float tp = 1.f, ts = 0.f;
  Steps<DT, E, GATE && !BACK, false> in;
  if (n > 0) in.load(g, p, BACK ? c1 - 1 : p.c0);
  for (int q = 0; q < n; ++q) {
    const int chunk = BACK ? c1 - 1 - q : p.c0 + q, s0 = p.step0(chunk);
    float P[E], S[E];
#pragma unroll
    for (int e = 0; e < E; ++e) P[e] = 1.f, S[e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < K; ++kk) {
      const int k = BACK ? K - 1 - kk : kk;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float a, keep;
        gates_of(to_f32<DT>(in.f[k].v[e]), &a, &keep);
        const float x = to_f32<DT>(in.x[k].v[e]);
        float s;
        if (BACK)
          s = a * (S[e] + x);
        else
          s = __builtin_fmaf(a, S[e], (GATE && !BACK ? sigma(to_f32<DT>(in.i[GATE && !BACK ? k : 0].v[e])) : keep) * x);
        const bool on = s0 + k < p.L;
        S[e] = on ? s : S[e];
        P[e] = on ? P[e] * a : P[e];
      }
    }
    if (q + 1 < n) in.load(g, p, BACK ? chunk - 1 : chunk + 1);
    float *lp = lds_p[q & 1], *ls = lds_s[q & 1];
#pragma unroll
    for (int e = 0; e < E; ++e) lp[at + e] = P[e], ls[at + e] = S[e];
    lds_barrier();
    if (threadIdx.x < kLanes) {
#pragma unroll 8
      for (int m = 0; m < kSlots; ++m) {
        const int k = (BACK ? kSlots - 1 - m : m) * kLanes + threadIdx.x;
        ts = __builtin_fmaf(lp[k], ts, ls[k]);
        tp *= lp[k];
      }
    }
  }
  const int hc = p.ct * kLanes + (int)threadIdx.x;
  if (threadIdx.x < kLanes && hc < g.H) {
    const int64_t o = ((int64_t)p.seg * g.B + p.b) * g.H + hc;
    g.map_p[o] = tp;
    g.map_s[o] = ts;
  }
}

// The states that enter the segments, one thread per channel: in the place
// of their maps' S. Forward from h_0, backward from dh_n and the last
// segment.
__global__ __launch_bounds__(256) void scan_carry_kernel(const float* __restrict__ map_p, float* __restrict__ map_s,
                                                         const float* __restrict__ first, int segs, int64_t n, int back) {
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= n) return;
  float h = first ? first[i] : 0.f;
  constexpr int kBatch = 16;
  for (int k0 = 0; k0 < segs; k0 += kBatch) {
    float p[kBatch], s[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int c = k0 + k < segs ? k0 + k : segs - 1;
      const int64_t o = (back ? segs - 1 - c : c) * n + i;
      p[k] = map_p[o];
      s[k] = map_s[o];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k < segs) {
        map_s[(back ? segs - 1 - (k0 + k) : k0 + k) * n + i] = h;
        h = __builtin_fmaf(p[k], h, s[k]);
      }
  }
}

template <typename DT, int E, bool GATE>
__global__ __launch_bounds__(kScanThreads<DT>) void scan_forward_kernel(GatedScanArgs g) {
  constexpr int K = Tile<DT, E>::kSteps, kSlots = Tile<DT, E>::kSlots, kLanes = Tile<DT, E>::kLanes;
  // two sets, taken in turn: a chunk's states are read while the next one's
  // maps are written, with one barrier between each pair of phases
  __shared__ float lds_p[2][kSlots * kLanes], lds_s[2][kSlots * kLanes];
  const Place<DT, E> p(g);
  if (p.seg >= g.segs) return;
  const int at = p.slot * kLanes + p.ch;
  const int c = threadIdx.x & (kLanes - 1);
  const int64_t cell = (int64_t)p.b * g.H + (p.h - p.ch) + c;  // of the channel whose state this thread carries
  const bool carries = threadIdx.x < kLanes && p.h - p.ch + c < g.H;
  float state = 0.f;
  if (carries) {
    if (g.segs > 1)
      state = g.map_s[(int64_t)p.seg * g.B * g.H + cell];
    else if (g.h0)
      state = g.h0[cell];
  }
  Steps<DT, E, GATE, false> in;
  if (p.c0 * kGatedScanChunk < p.L) in.load(g, p, p.c0);
  for (int chunk = p.c0; chunk < p.c1; ++chunk) {
    const int s0 = p.step0(chunk);
    if (carries && g.state) g.state[(int64_t)chunk * g.B * g.H + cell] = state;
    if (chunk * kGatedScanChunk >= p.L) {  // nothing but zeros from here on
      if (p.live) {
        const float z[E] = {};
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (s0 + k < g.T) store_vec<DT, E>((DT*)g.y + ((int64_t)(s0 + k) * g.B + p.b) * g.H + p.h, z);
      }
      continue;
    }
    float a[K][E], u[K][E], P[E], S[E];
#pragma unroll
    for (int e = 0; e < E; ++e) P[e] = 1.f, S[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float av, keep;
        gates_of(to_f32<DT>(in.f[k].v[e]), &av, &keep);
        const float uv = (GATE ? sigma(to_f32<DT>(in.i[GATE ? k : 0].v[e])) : keep) * to_f32<DT>(in.x[k].v[e]);
        const bool on = s0 + k < p.L;
        a[k][e] = on ? av : 1.f;
        u[k][e] = on ? uv : 0.f;
        S[e] = __builtin_fmaf(a[k][e], S[e], u[k][e]);
        P[e] *= a[k][e];
      }
    if (chunk + 1 < p.c1 && (chunk + 1) * kGatedScanChunk < p.L) in.load(g, p, chunk + 1);
    float* lp = lds_p[chunk & 1];
    float* ls = lds_s[chunk & 1];
#pragma unroll
    for (int e = 0; e < E; ++e) lp[at + e] = P[e], ls[at + e] = S[e];
    lds_barrier();
    if (threadIdx.x < kLanes) state = run_slots<DT, E, false>(lp, ls, state, c);
    lds_barrier();
    if (p.live) {
      float h[E];
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = ls[at + e];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int s = s0 + k;
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          h[e] = __builtin_fmaf(a[k][e], h[e], u[k][e]);
          y[e] = s < p.L ? h[e] : 0.f;
        }
        if (s < g.T)
          store_vec<DT, E>((DT*)g.y + ((int64_t)(s < p.L ? p.time(g, s) : s) * g.B + p.b) * g.H + p.h, y);
      }
    }
  }
  if (carries && g.h_n && p.seg == g.segs - 1) g.h_n[cell] = state;
}

template <typename DT, int E, bool GATE>
__global__ __launch_bounds__(kScanThreads<DT>) void scan_backward_kernel(GatedScanArgs g) {
  constexpr int K = Tile<DT, E>::kSteps, kSlots = Tile<DT, E>::kSlots, kLanes = Tile<DT, E>::kLanes;
  __shared__ float lds_p[2][kSlots * kLanes], lds_s[2][kSlots * kLanes], lds_c[2][kSlots * kLanes];
  const Place<DT, E> p(g);
  if (p.seg >= g.segs) return;
  const int at = p.slot * kLanes + p.ch;
  const int c = threadIdx.x & (kLanes - 1), wave = (threadIdx.x & 63) < kLanes ? threadIdx.x >> 6 : -1;
  const int64_t cell = (int64_t)p.b * g.H + (p.h - p.ch) + c;
  const bool channel = p.h - p.ch + c < g.H;
  // the first wave runs h forward through a chunk, the second c backward
  float carry = 0.f;
  if (wave == 1 && channel) {
    if (g.segs > 1)
      carry = g.map_s[(int64_t)p.seg * g.B * g.H + cell];
    else if (g.dh_n)
      carry = g.dh_n[cell];
  }
  const int64_t d_t = (int64_t)g.B * g.H;
  Steps<DT, E, GATE, true> in;
  int chunk = p.c1 - 1;
  // chunks past the row's end
  for (; chunk >= p.c0 && chunk * kGatedScanChunk >= p.L; --chunk) {
    if (p.live) {
      const float z[E] = {};
      const int s0 = p.step0(chunk);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (s0 + k < g.T) {
          const int64_t o = (s0 + k) * d_t + (int64_t)p.b * g.H + p.h;
          store_vec<DT, E>((DT*)g.dx + o, z);
          store_vec<DT, E>((DT*)g.df + o, z);
          if (GATE) store_vec<DT, E>((DT*)g.di + o, z);
        }
    }
  }
  float entering = 0.f;
  if (chunk >= p.c0) {
    in.load(g, p, chunk);
    if (wave == 0 && channel) entering = g.state[chunk * d_t + cell];
  }
  for (; chunk >= p.c0; --chunk) {
    const int s0 = p.step0(chunk);
    // with a gate: slope a (1 - a) in keep's place, u = s x in x's and u (1 - s)
    // in v; each factor 1 - s has its own accuracy (see gates_of)
    float a[K][E], keep[K][E], w[GATE ? K : 1][E], x[K][E], v[GATE ? K : 1][E], dy[K][E], P[E], S[E], C[E];
#pragma unroll
    for (int e = 0; e < E; ++e) P[e] = 1.f, S[e] = 0.f, C[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float av, kv;
        gates_of(to_f32<DT>(in.f[k].v[e]), &av, &kv);
        const bool on = s0 + k < p.L;
        a[k][e] = on ? av : 1.f;
        keep[k][e] = on ? (GATE ? av * kv : kv) : 0.f;
        x[k][e] = on ? to_f32<DT>(in.x[k].v[e]) : 0.f;
        dy[k][e] = on ? to_f32<DT>(in.dy[k].v[e]) : 0.f;
        if (GATE) {
          float open, shut;
          gates_of(to_f32<DT>(in.i[GATE ? k : 0].v[e]), &open, &shut);
          w[k][e] = on ? open : 0.f;
          x[k][e] *= w[k][e];
          v[k][e] = x[k][e] * shut;
        }
        S[e] = __builtin_fmaf(a[k][e], S[e], GATE ? x[k][e] : keep[k][e] * x[k][e]);
        P[e] *= a[k][e];
      }
#pragma unroll
    for (int k = K - 1; k >= 0; --k)
#pragma unroll
      for (int e = 0; e < E; ++e) C[e] = a[k][e] * (C[e] + dy[k][e]);
    float next = 0.f;
    if (chunk > p.c0) {
      in.load(g, p, chunk - 1);
      if (wave == 0 && channel) next = g.state[(chunk - 1) * d_t + cell];
    }
    float *lp = lds_p[chunk & 1], *ls = lds_s[chunk & 1], *lc = lds_c[chunk & 1];
#pragma unroll
    for (int e = 0; e < E; ++e) lp[at + e] = P[e], ls[at + e] = S[e], lc[at + e] = C[e];
    lds_barrier();
    if (wave == 0) run_slots<DT, E, false>(lp, ls, entering, c);
    if (wave == 1) carry = run_slots<DT, E, true>(lp, lc, carry, c);
    entering = next;
    lds_barrier();
    if (p.live) {
      float hp[K][E], h[E], cc[E];
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = ls[at + e], cc[e] = lc[at + e];
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          hp[k][e] = h[e];
          h[e] = __builtin_fmaf(a[k][e], h[e], GATE ? x[k][e] : keep[k][e] * x[k][e]);
        }
#pragma unroll
      for (int k = K - 1; k >= 0; --k) {
        const int s = s0 + k;
        float dx[E], df[E], di[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float gt = dy[k][e] + cc[e];
          cc[e] = a[k][e] * gt;
          // past the row's end a = 1 carries c on, and keep = 0 (w = v = 0) ends the rest
          if (GATE) {
            dx[e] = gt * w[GATE ? k : 0][e];
            df[e] = gt * keep[k][e] * hp[k][e];
            di[e] = gt * v[GATE ? k : 0][e];
          } else {
            dx[e] = gt * keep[k][e];
            df[e] = gt * a[k][e] * keep[k][e] * (hp[k][e] - x[k][e]);
          }
          if (s >= p.L) dx[e] = df[e] = 0.f;
          if (GATE && s >= p.L) di[e] = 0.f;
        }
        if (s < g.T) {
          const int64_t o = (s < p.L ? p.time(g, s) : s) * d_t + (int64_t)p.b * g.H + p.h;
          store_vec<DT, E>((DT*)g.dx + o, dx);
          store_vec<DT, E>((DT*)g.df + o, df);
          if (GATE) store_vec<DT, E>((DT*)g.di + o, di);
        }
      }
    }
  }
  if (wave == 1 && channel && g.dh0 && p.seg == 0) g.dh0[cell] = carry;
}

// A few steps (one, where a model answers token by token): a thread runs E
// channels through all of them, nothing is shared.
constexpr int kShort = 8;
template <typename DT, int E, bool GATE>
__global__ __launch_bounds__(256) void scan_short_kernel(GatedScanArgs g) {
  const int64_t per = (g.H + E - 1) / E, id = blockIdx.x * (int64_t)256 + threadIdx.x;
  const int b = (int)(id / per), h = (int)(id % per) * E;
  if (b >= g.B) return;
  const int n = g.lengths ? g.lengths[b] : g.T, L = n < 0 ? 0 : (n > g.T ? g.T : n);
  const int64_t cell = (int64_t)b * g.H + h, y_t = (int64_t)g.B * g.H;
  float state[E];
#pragma unroll
  for (int e = 0; e < E; ++e) state[e] = g.h0 ? g.h0[cell + e] : 0.f;
  if (g.state) {
#pragma unroll
    for (int e = 0; e < E; ++e) g.state[cell + e] = state[e];
  }
  for (int s = 0; s < g.T; ++s) {
    const int64_t t = g.reverse && s < L ? L - 1 - s : s;
    float y[E] = {};
    if (s < L) {
      const Raw<DT, E> f = *reinterpret_cast<const Raw<DT, E>*>((const DT*)g.f + t * g.f_t + b * g.f_b + h);
      const Raw<DT, E> x = *reinterpret_cast<const Raw<DT, E>*>((const DT*)g.x + t * g.x_t + b * g.x_b + h);
      Raw<DT, E> i;
      if (GATE) i = *reinterpret_cast<const Raw<DT, E>*>((const DT*)g.i + t * g.i_t + b * g.i_b + h);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float a, keep;
        gates_of(to_f32<DT>(f.v[e]), &a, &keep);
        state[e] = y[e] = __builtin_fmaf(a, state[e], (GATE ? sigma(to_f32<DT>(i.v[e])) : keep) * to_f32<DT>(x.v[e]));
      }
    }
    store_vec<DT, E>((DT*)g.y + t * y_t + cell, y);
  }
  if (g.h_n) {
#pragma unroll
    for (int e = 0; e < E; ++e) g.h_n[cell + e] = state[e];
  }
}

template <typename DT, int E, bool GATE>
hipError_t run(const GatedScanArgs& a, bool back, hipStream_t st) {
  if (!back && a.T <= kShort) {
    const int64_t n = (int64_t)a.B * ((a.H + E - 1) / E);
    launch_kernel(scan_short_kernel<DT, E, GATE>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const int64_t units = (int64_t)a.B * a.segs;
  const dim3 grid((unsigned)((units + a.xcds - 1) / a.xcds * a.xcds * a.tiles)), block(Tile<DT, E>::kThreads);
  if (a.segs > 1) {
    if (back)
      launch_kernel(scan_compose_kernel<DT, E, GATE, true>, grid, block, 0, st, a);
    else
      launch_kernel(scan_compose_kernel<DT, E, GATE, false>, grid, block, 0, st, a);
    const int64_t n = (int64_t)a.B * a.H;
    launch_kernel(scan_carry_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, (const float*)a.map_p, a.map_s,
                  back ? a.dh_n : a.h0, a.segs, n, (int)back);
  }
  if (back)
    launch_kernel(scan_backward_kernel<DT, E, GATE>, grid, block, 0, st, a);
  else
    launch_kernel(scan_forward_kernel<DT, E, GATE>, grid, block, 0, st, a);
  return hipGetLastError();
}

template <typename DT, int E>
hipError_t run_gate(const GatedScanArgs& a, bool back, hipStream_t st) {
  return a.i ? run<DT, E, true>(a, back, st) : run<DT, E, false>(a, back, st);
}

}  // namespace

double gated_scan_row_threads(int H, bool bf) {
  const int lanes = bf ? kScanLanes<bf16> : kScanLanes<float>, threads = bf ? kScanThreads<bf16> : kScanThreads<float>;
  return (double)(((int64_t)H + lanes - 1) / lanes) * threads;
}

// Segments so that the walks fill the compute units' threads about once, each
// over two chunks at least; only while the tiles are fewer than half the
// compute units and the time has eight chunks: cutting it costs two launches
// and a second read of the inputs. Measured (us forward + backward, cut /
// whole): bf16, T = 4096, 96 tiles 161 / 171, 128 tiles 173 / 188, 160 tiles
// 215 / 196, 256 tiles 351 / 226; T = 2048, 128 tiles 98 / 91; T = 1024, 32
// tiles 34 / 47, T = 512 33 / 26. fp32, T = 4096, 96 tiles 113 / 137, 128
// tiles 156 / 154, 160 tiles 237 / 169; T = 1024, 32 tiles 31 / 38, T = 512
// 31 / 22.
int gated_scan_segments(int T, int B, int H, bool bf, int cus, int* seg_chunks) {
  const int lanes = bf ? kScanLanes<bf16> : kScanLanes<float>, threads = bf ? kScanThreads<bf16> : kScanThreads<float>;
  const int64_t tiles = (int64_t)B * ((H + lanes - 1) / lanes);
  const int chunks = (T + kGatedScanChunk - 1) / kGatedScanChunk;
  int64_t want = 1;
  if (2 * tiles < cus && chunks >= 8) want = (1024 / threads) * (int64_t)cus / tiles;
  if (want > chunks / 2) want = chunks / 2;
  if (want < 1) want = 1;
  *seg_chunks = (int)((chunks + want - 1) / want);
  return (chunks + *seg_chunks - 1) / *seg_chunks;
}

hipError_t launch_gated_scan(GatedScanArgs a, bool bf, bool back, hipStream_t st) {
  const int lanes = bf ? kScanLanes<bf16> : kScanLanes<float>;
  a.tiles = (a.H + lanes - 1) / lanes;
  if ((int64_t)a.B * a.segs < a.xcds) a.xcds = 1;  // fewer (row, segment)s than XCDs: spread their tiles instead
  if (a.width == 1) return bf ? run_gate<bf16, 1>(a, back, st) : run_gate<float, 1>(a, back, st);
  return bf ? run_gate<bf16, 4>(a, back, st) : run_gate<float, 4>(a, back, st);
}

}  // namespace rnnk
