// Selective scan: a linear recurrence with a state of N numbers per channel
// and a step length of its own at every time.
//
//   d_t = softplus(dt_t + bias)  (or dt_t + bias)
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t x_t B_t[n]
//   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
//
// per channel of [T, B, H]; B and C are shared by a group's channels.
//
// Bound by the issue of vector instructions: a state's step is an exponential
// (3.5 ns of a SIMD for 64 lanes) and four products or sums (1.75 ns each,
// however many waves there are): 10.1 ns together in a loop of nothing else,
// while a channel's step moves 8 bytes in bf16. With what is formed once a
// channel and step (step length, gate), handed round and summed, a wave issues
// 33 instructions a step for its 256 states. So the states stay in registers
// for the whole time, four lanes a channel; the time is walked in tiles of 32
// steps, staged through LDS with the next tile's loads in flight, and the
// scalars of a step are formed by one lane in four, 16 steps at once. T 1000,
// 32 x 1024 x 16, bf16, with gate: 167 us, of which its instructions take 130;
// the states' own exponentials and products alone need 81.
//
// Where that gives few workgroups the time is cut into segments: a first
// launch finds what each adds to the state and the sum of its steps (its
// decay is exp(A sum d)), a second runs the state through the segments, and
// the walk starts from there.
//
// All states, products and sums are fp32; x, dt, z, B, C and y have the
// storage type.
#include "selective_scan_common.hpp"

namespace rnnk {
namespace {

constexpr int kSteps = 32;
constexpr int kPart = kSelKeep;  // steps that the code is written out for

template <typename DT, int J, bool VEC, bool COMPOSE>
__global__ __launch_bounds__(kSelThreads) __attribute__((amdgpu_waves_per_eu(sel_waves(J), sel_waves(J)))) void sel_forward_kernel(SelectiveScanArgs a) {
  constexpr int NP = 4 * J;
  using Tile = SelTile<DT, kSteps, VEC>;
  __shared__ __attribute__((aligned(16))) DT lds_x[kSteps * Tile::kLd], lds_d[kSteps * Tile::kLd];
  // y takes x's place: a thread reads the slots of a tile of y that it then fills with the next x
  __shared__ __attribute__((aligned(16))) DT lds_z[COMPOSE ? 1 : kSteps * Tile::kLd];
  __shared__ __attribute__((aligned(16))) float lds_b[kSteps * NP], lds_c[COMPOSE ? 1 : kSteps * NP];
  const SelPlace p(a);
  if (p.seg >= a.segs) return;
  const int lane = threadIdx.x & 63, q = lane & 3, ch = (threadIdx.x >> 6) * 16 + (lane >> 2);
  const bool live = ch < p.live;
  const int hc = p.c0 + (live ? ch : 0);
  const int64_t cell = (int64_t)p.b * a.H + hc, cells = (int64_t)a.B * a.H;
  float A2[J], h[J];
  load_row<J>(a.A + (int64_t)hc * a.N, q * J, a.N, a.svec, A2);
#pragma unroll
  for (int j = 0; j < J; ++j) A2[j] *= kLog2e;
  if (COMPOSE) {
#pragma unroll
    for (int j = 0; j < J; ++j) h[j] = 0.f;
  } else if (a.segs > 1) {
    read_states<J>(a.map_s + (p.seg * cells + cell) * NP + q * J, h);
  } else {
    load_row<J>(a.h0 ? a.h0 + cell * a.N : nullptr, q * J, a.N, a.svec, h);
  }
  const float bias = a.dt_bias ? a.dt_bias[hc] : 0.f, D = a.D ? a.D[hc] : 0.f;
  const DT* x = (const DT*)a.x + p.b * a.x_b;
  const DT* dt = (const DT*)a.dt + p.b * a.dt_b;
  const DT* z = a.z ? (const DT*)a.z + p.b * a.z_b : nullptr;
  const DT* Bm = (const DT*)a.Bm + p.b * a.B_b + p.group * a.B_g;
  const DT* Cm = (const DT*)a.Cm + p.b * a.C_b + p.group * a.C_g;
  DT* y = (DT*)a.y + (int64_t)p.b * a.H;
  const int64_t y_t = cells;
  const int end = p.t1 < p.L ? p.t1 : p.L;  // steps there are
  float sum_d = 0.f;
  Tile tx, td, tz;
  SelRows<DT, kSteps, NP> tb, tc;
  auto load = [&](int t) {
    tx.load(x, a.x_t, t, p.L - 1, p.c0, p.live);
    td.load(dt, a.dt_t, t, p.L - 1, p.c0, p.live);
    tb.load(Bm, a.B_t, t, p.L - 1, a.N);
    if (!COMPOSE) {
      if (z) tz.load(z, a.z_t, t, p.L - 1, p.c0, p.live);
      tc.load(Cm, a.C_t, t, p.L - 1, a.N);
    }
  };
  if (p.t0 < end) load(p.t0);
  int t = p.t0;
  for (; t < end; t += kSteps) {
    tx.put(lds_x);
    td.put(lds_d);
    tb.put(lds_b, t, p.L, a.N);
    if (!COMPOSE) {
      if (z) tz.put(lds_z);
      tc.put(lds_c, t, p.L, a.N);
    }
    lds_barrier();
    if (t + kSteps < end) load(t + kSteps);
#pragma unroll 1
    for (int half = 0; half < kSteps / kPart; ++half) {
      const int from = half * kPart;
      if (!COMPOSE && a.keep && live && t + from < end)
        write_states<J>(a.keep + ((t + from) / kSelKeep * cells + cell) * NP + q * J, h);
      // B and C of the steps ahead
      float bv[kAhead + 1][J], cv[kAhead + 1][J];
      auto rows = [&](int s) {
        read_states<J>(lds_b + (from + s) * NP + q * J, bv[s % (kAhead + 1)]);
        if (!COMPOSE) read_states<J>(lds_c + (from + s) * NP + q * J, cv[s % (kAhead + 1)]);
      };
#pragma unroll
      for (int s = 0; s < kAhead; ++s) rows(s);
      // what a lane forms for its own steps, 4 g + q
      float d[kPart / 4], dx[kPart / 4], own[kPart / 4], gate[kPart / 4];
#pragma unroll
      for (int g = 0; g < kPart / 4; ++g) {
        const int at = (from + 4 * g + q) * Tile::kLd + ch;
        const bool on = t + from + 4 * g + q < p.L;  // a step past the row's end has no length
        d[g] = to_f32<DT>(lds_d[at]) + bias;
        dx[g] = on ? to_f32<DT>(lds_x[at]) : 0.f;
      }
      if (a.softplus) {
#pragma unroll
        for (int g = 0; g < kPart / 4; ++g) d[g] = step_length(d[g], 1);
      }
      if (!COMPOSE && z) {
#pragma unroll
        for (int g = 0; g < kPart / 4; ++g) {
          const float zv = to_f32<DT>(lds_z[(from + 4 * g + q) * Tile::kLd + ch]);
          gate[g] = zv * fsigmoid(zv);
        }
      } else {
#pragma unroll
        for (int g = 0; g < kPart / 4; ++g) gate[g] = 1.f;
      }
#pragma unroll
      for (int g = 0; g < kPart / 4; ++g) {
        if (!(t + from + 4 * g + q < p.L)) d[g] = 0.f;
        own[g] = D * dx[g];
        dx[g] *= d[g];
        if (COMPOSE) sum_d += d[g];
      }
#pragma unroll
      for (int g = 0; g < kPart / 4; ++g) {
        float acc[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float ds = quad_from(d[g], s), dxs = quad_from(dx[g], s);
          const int at = 4 * g + s, i = at % (kAhead + 1);
          if (at + kAhead < kPart) rows(at + kAhead);
          __builtin_amdgcn_sched_barrier(kSelKeepReads);
          acc[s] = 0.f;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(ds * A2[j]), h[j], dxs * bv[i][j]);
            if (!COMPOSE) acc[s] = __builtin_fmaf(h[j], cv[i][j], acc[s]);
          }
        }
        if (!COMPOSE) lds_x[(from + 4 * g + q) * Tile::kLd + ch] = from_f32<DT>((quad_scatter(acc, q) + own[g]) * gate[g]);
      }
    }
    lds_barrier();
    if (!COMPOSE) Tile::store(lds_x, y, y_t, t, p.t1, p.L, p.c0, p.live);
  }
  if (COMPOSE) {
    if (live) write_states<J>(a.map_s + (p.seg * cells + cell) * NP + q * J, h);
    sum_d = quad_sum(sum_d);
    if (live && q == 0) a.map_d[p.seg * cells + cell] = sum_d;
    return;
  }
  // steps past the row's end
  for (; t < p.t1; t += kSteps) Tile::store(lds_x, y, y_t, t, p.t1, p.L, p.c0, p.live);
  if (a.h_n && live && p.seg == a.segs - 1) store_row<J>(a.h_n + cell * a.N, q * J, a.N, a.svec, h);
}

// 2^e h + s for e > 126: a state after a segment. A growing channel's factor
// (A > 0, or negative steps) can be larger than any fp32 number over a segment's
// steps, where the walk step by step stays finite: at zero, for one. It goes in
// three parts then. 381 is the largest exponent that is used: 2^381 takes the
// smallest number past the largest.
__device__ __forceinline__ float sel_past(float e, float h, float s) {
  const float f = __builtin_amdgcn_exp2f(__builtin_fminf(e, 381.0f) * (1.0f / 3.0f));
  return __builtin_fmaf(f, f * (f * h), s);
}

// The states that enter the segments, one thread per state: in the place of
// what the segments add. Forward from h_0, backward from dh_n and the last
// segment.
__global__ __launch_bounds__(256) void sel_carry_kernel(SelectiveScanArgs a, const float* __restrict__ first, int NP, int back) {
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x, cells = (int64_t)a.B * a.H;
  if (i >= cells * NP) return;
  const int n = (int)(i % NP);
  const int64_t cell = i / NP;
  const bool on = n < a.N;
  const float A2 = on ? a.A[cell % a.H * a.N + n] * kLog2e : 0.f;
  float h = on && first ? first[cell * a.N + n] : 0.f;
  float* map_s = a.map_s + i;
  const float* map_d = a.map_d + cell;
  constexpr int kBatch = 16;
  for (int k0 = 0; k0 < a.segs; k0 += kBatch) {
    float s[kBatch], d[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int c = k0 + k < a.segs ? k0 + k : a.segs - 1;
      const int64_t o = (back ? a.segs - 1 - c : c) * cells;
      s[k] = map_s[o * NP];
      d[k] = map_d[o];
    }
    bool far = false;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) far |= A2 * d[k] > 126.0f;
    auto walk = [&](auto past) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < a.segs) {
          map_s[(back ? a.segs - 1 - (k0 + k) : k0 + k) * cells * NP] = h;
          h = past(A2 * d[k], s[k]);
        }
    };
    if (!far)
      walk([&](float e, float add) { return __builtin_fmaf(__builtin_amdgcn_exp2f(e), h, add); });
    else
      walk([&](float e, float add) { return e > 126.0f ? sel_past(e, h, add) : __builtin_fmaf(__builtin_amdgcn_exp2f(e), h, add); });
  }
}

// A few steps (one, where a model answers token by token): the same lanes
// without the tiles. Bound by the states' way in and out.
constexpr int kShort = 8;
template <typename DT, int J>
__global__ __launch_bounds__(kSelThreads) void sel_short_kernel(SelectiveScanArgs a) {
  constexpr int NP = 4 * J;
  const int64_t id = blockIdx.x * (int64_t)kSelThreads + threadIdx.x, cells = (int64_t)a.B * a.H;
  const int q = threadIdx.x & 3;
  const bool live = (id >> 2) < cells;
  const int64_t cell = live ? id >> 2 : 0;
  const int b = (int)(cell / a.H), hc = (int)(cell % a.H), group = hc / (a.H / a.G);
  const int len = a.lengths ? a.lengths[b] : a.T, L = len < 0 ? 0 : (len > a.T ? a.T : len);
  float A2[J], h[J];
  load_row<J>(a.A + (int64_t)hc * a.N, q * J, a.N, a.svec, A2);
#pragma unroll
  for (int j = 0; j < J; ++j) A2[j] *= kLog2e;
  load_row<J>(a.h0 ? a.h0 + cell * a.N : nullptr, q * J, a.N, a.svec, h);
  if (a.keep && live) write_states<J>(a.keep + cell * NP + q * J, h);
  const float bias = a.dt_bias ? a.dt_bias[hc] : 0.f, D = a.D ? a.D[hc] : 0.f;
  // the next step's inputs are on their way while one is worked on; past the
  // row's end they are some step of it
  struct {
    DT x, dt, z, b[J], c[J];
  } in, next;
  auto load = [&](auto& to, int t) {
    t = t < L ? t : L > 0 ? L - 1 : 0;
    to.x = ((const DT*)a.x)[t * a.x_t + b * a.x_b + hc];
    to.dt = ((const DT*)a.dt)[t * a.dt_t + b * a.dt_b + hc];
    if (a.z) to.z = ((const DT*)a.z)[t * a.z_t + b * a.z_b + hc];
    const DT* Bm = (const DT*)a.Bm + t * a.B_t + b * a.B_b + group * a.B_g;
    const DT* Cm = (const DT*)a.Cm + t * a.C_t + b * a.C_b + group * a.C_g;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = q * J + j < a.N ? q * J + j : a.N - 1;
      to.b[j] = Bm[n];
      to.c[j] = Cm[n];
    }
  };
  load(in, 0);
  for (int t = 0; t < a.T; ++t) {
    if (t + 1 < a.T) load(next, t + 1);
    float v = 0.f;
    if (t < L) {
      const float xv = to_f32<DT>(in.x);
      const float d = step_length(to_f32<DT>(in.dt) + bias, a.softplus);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool on = q * J + j < a.N;
        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A2[j]), h[j], on ? d * xv * to_f32<DT>(in.b[j]) : 0.f);
        v = __builtin_fmaf(h[j], on ? to_f32<DT>(in.c[j]) : 0.f, v);
      }
      v = __builtin_fmaf(D, xv, quad_sum(v));
      if (a.z) {
        const float zv = to_f32<DT>(in.z);
        v *= zv * fsigmoid(zv);
      }
    }
    if (live && q == 0) ((DT*)a.y)[t * cells + cell] = from_f32<DT>(v);
    in = next;
  }
  if (a.h_n && live) store_row<J>(a.h_n + cell * a.N, q * J, a.N, a.svec, h);
}

template <typename DT, int J, bool VEC>
hipError_t run(const SelectiveScanArgs& a, hipStream_t st) {
  if (a.segs > 1) {
    launch_kernel(sel_forward_kernel<DT, J, VEC, true>, sel_grid(a), dim3(kSelThreads), 0, st, a);
    const hipError_t e = launch_sel_carry(a, a.h0, 4 * J, false, st);
    if (e != hipSuccess) return e;
  }
  launch_kernel(sel_forward_kernel<DT, J, VEC, false>, sel_grid(a), dim3(kSelThreads), 0, st, a);
  return hipGetLastError();
}

template <typename DT, int J>
hipError_t run_width(const SelectiveScanArgs& a, hipStream_t st) {
  if (a.T <= kShort) {
    const int64_t n = (int64_t)a.B * a.H * 4;
    launch_kernel(sel_short_kernel<DT, J>, dim3((unsigned)((n + kSelThreads - 1) / kSelThreads)), dim3(kSelThreads), 0, st, a);
    return hipGetLastError();
  }
  return a.vec ? run<DT, J, true>(a, st) : run<DT, J, false>(a, st);
}

template <typename DT>
hipError_t run_states(const SelectiveScanArgs& a, hipStream_t st) {
  switch (sel_padded(a.N)) {
    case 4: return run_width<DT, 1>(a, st);
    case 8: return run_width<DT, 2>(a, st);
    case 16: return run_width<DT, 4>(a, st);
    case 32: return run_width<DT, 8>(a, st);
    default: return run_width<DT, 16>(a, st);
  }
}

}  // namespace

hipError_t launch_sel_carry(const SelectiveScanArgs& a, const float* first, int NP, bool back, hipStream_t st) {
  const int64_t n = (int64_t)a.B * a.H * NP;
  launch_kernel(sel_carry_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a, first, NP, (int)back);
  return hipGetLastError();
}

// The time is cut where that is expected to be faster: into segments of whole
// 64 steps, up to as many workgroups a compute unit as fit. A step of the walk
// takes 119 ns (N = 16) with one workgroup a compute unit, 190 with two and
// 350 with four (more waves fill each other's waits); in the launch that
// composes a segment 88, 137 and 255; the two launches more cost about 12 us
// and 0.1 a segment. T = 2048, 4 x 1024 channels: 226 us in one piece, 46 + 34 +
// 5 in 16 segments; T = 16384, 1 x 64 channels: 12 + 10 + 28 us in 256 segments,
// 18 + 14 + 15 in 128. The backward pass takes the same cut, which gains it as
// much (all of a pass in bf16 with gate, forward + backward, us):
//   T, rows x channels x N    one piece     4         8         16        64        as cut
//   2048, 4 x 1024 x 16       217 + 597   107 + 209  84 + 164  77 + 160  76 + 159  83 + 171
//   16384, 2 x 1000 x 16     1706 + 4689  746 + 1531 382 + 786 291 + 602 251 + 567 278 + 577
//   4096, 8 x 512 x 16        426 + 1179  197 + 398 153 + 311 140 + 301 134 + 302 140 + 300
//   4096, 2 x 1024 x 64      1076 + 4297  494 + 1320 259 + 687 208 + 675 215 + 708 208 + 676
//   500 ragged, 64 x 512 x 16  75 + 205   105 + 223 104 + 220 (8 pieces are all)    74 + 203
int sel_segments(int T, int B, int H, int N, int G, int cus, int* seg_steps) {
  const double tiles = (double)B * sel_group_tiles(H, G) * G, scale = 0.5 + sel_padded(N) / 32.0;
  const int chunks = (T + 63) / 64;
  int best = 1;
  double least = T * (tiles <= cus ? 0.12 : 0.12 + 0.075 * (tiles / cus - 1.0)) * scale;
  for (int want = 2; want <= chunks && want * tiles <= (double)sel_waves(sel_padded(N) / 4) * cus; ++want) {
    const int each = (chunks + want - 1) / want;
    if ((chunks + each - 1) / each != want) continue;
    const double load = want * tiles / cus;
    const double step = load <= 1.0 ? 0.21 : 0.21 + 0.13 * (load - 1.0);
    const double us = each * 64 * step * scale + 12.0 + 0.1 * want;
    if (us < least) {
      least = us;
      best = want;
    }
  }
  *seg_steps = best == 1 ? chunks * 64 : (chunks + best - 1) / best * 64;
  return best;
}

hipError_t launch_selective_scan(SelectiveScanArgs a, bool bf, hipStream_t st) {
  sel_tiles(a);
  return bf ? run_states<bf16>(a, st) : run_states<float>(a, st);
}

}  // namespace rnnk
