// Selective scan, backward pass.
//
// With a_t = exp(d_t A), v_t = dy_t silu(z_t), g_t the gradient of h_t and c
// the part of it that comes from later steps:
//   g_t = v_t C_t + c_{t+1},  c_t = a_t g_t,  c_{L+1} = dh_n,  dh_0 = c_1
//   w = g a h_{t-1}
//   dA = sum_t w d,  dC_t = sum_channels v h_t,  dB_t = sum_channels g d x
//   dd = sum_n w A + x sum_n g B,  ddt = dd sigma(dt + bias),  dbias = sum ddt
//   dx = d sum_n g B + D v,  dD = sum v x
//   dz = dy (sum_n C h + D x) silu'(z)
//
// The time is walked backwards in tiles of 16 steps. The training forward
// kept the state at every tile's beginning; a tile's states and decays are
// computed again from there and stay in registers. With more than four states
// a lane they would not fit: those walk a tile four steps at a time, and the
// states at the four steps' beginnings, found first, wait in LDS (1024 x 16 x
// 2048 channels, N = 32, bf16: 1207 us with eight steps at a time and all of
// it written out, 1028 so; 1024 x 8 x 2048, N = 64: 1372 and 1171). With four
// states a lane that costs more than the second workgroup a SIMD it allows
// gives (T 16384, 2 x 1000 x 16: 508 us with 16 steps, where it takes 468 now,
// 556 with eight, 598 with four). So nothing is divided by a decay, which may be zero, and y is
// not read.
//
// dB and dC are sums over the channels: a wave adds its 16 by lane
// permutations (16 sums at a time, one operation a value in place of four),
// the four waves of a workgroup meet in LDS, the tiles of a group of channels
// in memory, and a second launch adds those in a fixed order. dA, dD and dbias
// stay in registers over a workgroup's time and are added over rows and
// segments by a third.
//
// Bound by the issue of vector instructions, like the forward: 100 a step for
// the 256 states of a wave, 4.5 of them exponentials. T 16384, 2 x 1000 x 16,
// bf16, with gate: 468 us, of which its instructions take 375 (forward 165 and
// 133); 500 ragged steps of 64 x 512 x 16, fp32, without: 180 us (forward 74).
#include "selective_scan_common.hpp"

namespace rnnk {
namespace {

constexpr int kSteps = kSelKeep;  // 16

// What segment adds to c on the way to its beginning, and the sum of its
// steps.
template <typename DT, int J, bool VEC>
__global__ __launch_bounds__(kSelThreads) __attribute__((amdgpu_waves_per_eu(sel_waves(J), sel_waves(J)))) void sel_compose_back_kernel(SelectiveScanArgs a) {
  constexpr int NP = 4 * J, kTile = 32;
  using Tile = SelTile<DT, kTile, VEC>;
  __shared__ __attribute__((aligned(16))) DT lds_d[kTile * Tile::kLd], lds_v[kTile * Tile::kLd], lds_z[kTile * Tile::kLd];
  __shared__ __attribute__((aligned(16))) float lds_c[kTile * NP];
  const SelPlace p(a);
  if (p.seg >= a.segs) return;
  const int lane = threadIdx.x & 63, q = lane & 3, ch = (threadIdx.x >> 6) * 16 + (lane >> 2);
  const bool live = ch < p.live;
  const int hc = p.c0 + (live ? ch : 0);
  const int64_t cell = (int64_t)p.b * a.H + hc, cells = (int64_t)a.B * a.H;
  float A2[J], c[J];
  load_row<J>(a.A + (int64_t)hc * a.N, q * J, a.N, a.svec, A2);
#pragma unroll
  for (int j = 0; j < J; ++j) A2[j] *= kLog2e, c[j] = 0.f;
  const float bias = a.dt_bias ? a.dt_bias[hc] : 0.f;
  const DT* dt = (const DT*)a.dt + p.b * a.dt_b;
  const DT* z = a.z ? (const DT*)a.z + p.b * a.z_b : nullptr;
  const DT* dy = (const DT*)a.dy + (int64_t)p.b * a.H;
  const DT* Cm = (const DT*)a.Cm + p.b * a.C_b + p.group * a.C_g;
  const int end = p.t1 < p.L ? p.t1 : p.L;
  float sum_d = 0.f;
  Tile td, tv, tz;
  SelRows<DT, kTile, NP> tc;
  auto load = [&](int t) {
    td.load(dt, a.dt_t, t, p.L - 1, p.c0, p.live);
    tv.load(dy, cells, t, p.L - 1, p.c0, p.live);
    if (z) tz.load(z, a.z_t, t, p.L - 1, p.c0, p.live);
    tc.load(Cm, a.C_t, t, p.L - 1, a.N);
  };
  int t = p.t0 + (end - p.t0 - 1) / kTile * kTile;
  if (p.t0 < end) load(t);
  for (; t >= p.t0 && p.t0 < end; t -= kTile) {
    td.put(lds_d);
    tv.put(lds_v);
    if (z) tz.put(lds_z);
    tc.put(lds_c, t, p.L, a.N);
    lds_barrier();
    if (t > p.t0) load(t - kTile);
#pragma unroll 1
    for (int from = kTile - kSteps; from >= 0; from -= kSteps) {
      float cv[kAhead + 1][J];  // C of the steps ahead
      auto rows = [&](int s) { read_states<J>(lds_c + (from + s) * NP + q * J, cv[s % (kAhead + 1)]); };
#pragma unroll
      for (int s = 0; s < kAhead; ++s) rows(kSteps - 1 - s);
      // a lane's own steps, 4 g + q
      float d[kSteps / 4], v[kSteps / 4];
#pragma unroll
      for (int g = 0; g < kSteps / 4; ++g) {
        const int at = (from + 4 * g + q) * Tile::kLd + ch;
        d[g] = to_f32<DT>(lds_d[at]) + bias;
        v[g] = to_f32<DT>(lds_v[at]);
      }
      if (a.softplus) {
#pragma unroll
        for (int g = 0; g < kSteps / 4; ++g) d[g] = step_length(d[g], 1);
      }
      if (z) {
#pragma unroll
        for (int g = 0; g < kSteps / 4; ++g) {
          const float zv = to_f32<DT>(lds_z[(from + 4 * g + q) * Tile::kLd + ch]);
          v[g] *= zv * fsigmoid(zv);
        }
      }
#pragma unroll
      for (int g = 0; g < kSteps / 4; ++g) {
        const bool on = t + from + 4 * g + q < p.L;
        d[g] = on ? d[g] : 0.f;
        v[g] = on ? v[g] : 0.f;
        sum_d += d[g];
      }
#pragma unroll
      for (int s = kSteps - 1; s >= 0; --s) {
        if (s >= kAhead) rows(s - kAhead);
        __builtin_amdgcn_sched_barrier(kSelKeepReads);
        const float ds = quad_from(d[s / 4], s % 4), vs = quad_from(v[s / 4], s % 4);
#pragma unroll
        for (int j = 0; j < J; ++j) c[j] = __builtin_amdgcn_exp2f(ds * A2[j]) * __builtin_fmaf(vs, cv[s % (kAhead + 1)][j], c[j]);
      }
    }
    lds_barrier();
  }
  if (live) write_states<J>(a.map_s + (p.seg * cells + cell) * NP + q * J, c);
  sum_d = quad_sum(sum_d);
  if (live && q == 0) a.map_d[p.seg * cells + cell] = sum_d;
}

// Group g of a part's steps.
template <int PARTS>
__device__ __forceinline__ float of_part(const float (&v)[4], int part, int g) {
  float r = v[g];
#pragma unroll
  for (int i = 1; i < PARTS; ++i) r = part == i ? v[i * (4 / PARTS) + g] : r;
  return r;
}

template <typename DT, int J, bool VEC>
__global__ __launch_bounds__(kSelThreads, J <= 4 ? 2 : 1) void sel_backward_kernel(SelectiveScanArgs a) {
  constexpr int NP = 4 * J;
  constexpr int kPart = J <= 4 ? kSteps : 4;  // steps whose states are in registers at once
  constexpr int kParts = kSteps / kPart;
  using Tile = SelTile<DT, kSteps, VEC>;
  constexpr int kArea = kSteps * Tile::kLd;
  // x, dt, z and dy, whose places dx, ddt and dz take
  __shared__ __attribute__((aligned(16))) DT lds_x[kArea], lds_d[kArea], lds_z[kArea], lds_v[kArea];
  __shared__ __attribute__((aligned(16))) float lds_b[kSteps * NP], lds_c[kSteps * NP];
  __shared__ __attribute__((aligned(16))) float lds_sum[4][kSteps * 2 * NP];  // each wave's dB and dC
  // a lane's states at the beginnings of its parts after the first
  __shared__ __attribute__((aligned(16))) float lds_h[kParts > 1 ? (kParts - 1) * kSelThreads * J : 1];
  const SelPlace p(a);
  if (p.seg >= a.segs) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane & 3, ch = wave * 16 + (lane >> 2);
  const bool live = ch < p.live;
  const int hc = p.c0 + (live ? ch : 0);
  const int64_t cell = (int64_t)p.b * a.H + hc, cells = (int64_t)a.B * a.H;
  float A2[J], c[J], dA[J];
  load_row<J>(a.A + (int64_t)hc * a.N, q * J, a.N, a.svec, A2);
  if (a.segs > 1)
    read_states<J>(a.map_s + (p.seg * cells + cell) * NP + q * J, c);
  else
    load_row<J>(a.dh_n ? a.dh_n + cell * a.N : nullptr, q * J, a.N, a.svec, c);
#pragma unroll
  for (int j = 0; j < J; ++j) A2[j] *= kLog2e, dA[j] = 0.f;
  const float bias = a.dt_bias ? a.dt_bias[hc] : 0.f, D = a.D ? a.D[hc] : 0.f;
  float sum_D = 0.f, sum_bias = 0.f;
  const DT* x = (const DT*)a.x + p.b * a.x_b;
  const DT* dt = (const DT*)a.dt + p.b * a.dt_b;
  const DT* z = a.z ? (const DT*)a.z + p.b * a.z_b : nullptr;
  const DT* dy = (const DT*)a.dy + (int64_t)p.b * a.H;
  const DT* Bm = (const DT*)a.Bm + p.b * a.B_b + p.group * a.B_g;
  const DT* Cm = (const DT*)a.Cm + p.b * a.C_b + p.group * a.C_g;
  DT *dx = (DT*)a.dx + (int64_t)p.b * a.H, *ddt = (DT*)a.ddt + (int64_t)p.b * a.H;
  DT* dz = z ? (DT*)a.dz + (int64_t)p.b * a.H : nullptr;
  float* sums = a.part_bc + (((int64_t)p.gt * a.T * a.B + p.b) * a.G + p.group) * 2 * NP;
  const int64_t sums_t = (int64_t)a.B * a.G * 2 * NP;

  Tile tx, td, tz, tv;
  SelRows<DT, kSteps, NP> tb, tc;
  float kept[J];
  auto load = [&](int t) {
    tx.load(x, a.x_t, t, p.L - 1, p.c0, p.live);
    td.load(dt, a.dt_t, t, p.L - 1, p.c0, p.live);
    if (z) tz.load(z, a.z_t, t, p.L - 1, p.c0, p.live);
    tv.load(dy, cells, t, p.L - 1, p.c0, p.live);
    tb.load(Bm, a.B_t, t, p.L - 1, a.N);
    tc.load(Cm, a.C_t, t, p.L - 1, a.N);
    read_states<J>(a.keep + (t / kSelKeep * cells + cell) * NP + q * J, kept);
  };
  int t = p.t0 + (p.t1 - p.t0 - 1) / kSteps * kSteps;
  for (; t >= p.t0 && t >= p.L; t -= kSteps) {  // tiles past the row's end
    Tile::store(lds_x, dx, cells, t, p.t1, p.L, p.c0, p.live);
    Tile::store(lds_x, ddt, cells, t, p.t1, p.L, p.c0, p.live);
    if (z) Tile::store(lds_x, dz, cells, t, p.t1, p.L, p.c0, p.live);
  }
  if (t >= p.t0) load(t);
  for (; t >= p.t0; t -= kSteps) {
    tx.put(lds_x);
    td.put(lds_d);
    if (z) tz.put(lds_z);
    tv.put(lds_v);
    tb.put(lds_b, t, p.L, a.N);
    tc.put(lds_c, t, p.L, a.N);
    float start[J];
#pragma unroll
    for (int j = 0; j < J; ++j) start[j] = kept[j];
    lds_barrier();
    if (t > p.t0) load(t - kSteps);

    // a lane's own steps: 4 g + q
    float d[4], xd[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = (4 * g + q) * Tile::kLd + ch;
      d[g] = to_f32<DT>(lds_d[at]) + bias;
      xd[g] = to_f32<DT>(lds_x[at]);
    }
    if (a.softplus) {
#pragma unroll
      for (int g = 0; g < 4; ++g) d[g] = step_length(d[g], 1);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const bool on = live && t + 4 * g + q < p.L;
      d[g] = on ? d[g] : 0.f;
      xd[g] = on ? d[g] * xd[g] : 0.f;
    }
    float first[J];
#pragma unroll
    for (int j = 0; j < J; ++j) first[j] = start[j];
#pragma unroll 1
    for (int part = 0; part < kParts - 1; ++part) {
#pragma unroll
      for (int s = 0; s < kPart; ++s) {
        const float ds = quad_from(of_part<kParts>(d, part, s / 4), s % 4), xs = quad_from(of_part<kParts>(xd, part, s / 4), s % 4);
        float bv[J];
        read_states<J>(lds_b + (part * kPart + s) * NP + q * J, bv);
#pragma unroll
        for (int j = 0; j < J; ++j) first[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(ds * A2[j]), first[j], xs * bv[j]);
      }
      write_states<J>(lds_h + (part * kSelThreads + threadIdx.x) * J, first);
    }
#pragma unroll 1
    for (int part = kParts - 1; part >= 0; --part) {
      float da[kPart][J], hs[kPart + 1][J], dp[kPart / 4], xp[kPart / 4];
#pragma unroll
      for (int g = 0; g < kPart / 4; ++g) dp[g] = of_part<kParts>(d, part, g), xp[g] = of_part<kParts>(xd, part, g);
#pragma unroll
      for (int j = 0; j < J; ++j) hs[0][j] = first[j];
      if (part > 1) {
        read_states<J>(lds_h + ((part - 2) * kSelThreads + threadIdx.x) * J, first);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) first[j] = start[j];
      }
#pragma unroll
      for (int s = 0; s < kPart; ++s) {
        const float ds = quad_from(dp[s / 4], s % 4), xs = quad_from(xp[s / 4], s % 4);
        float bv[J];
        read_states<J>(lds_b + (part * kPart + s) * NP + q * J, bv);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          da[s][j] = __builtin_amdgcn_exp2f(ds * A2[j]);
          hs[s + 1][j] = __builtin_fmaf(da[s][j], hs[s][j], xs * bv[j]);
        }
      }
#pragma unroll
      for (int g = kPart / 4 - 1; g >= 0; --g) {
        const int gg = part * (kPart / 4) + g;
        const int at = (4 * gg + q) * Tile::kLd + ch;
        const bool on = live && t + 4 * gg + q < p.L;
        float v = to_f32<DT>(lds_v[at]), xv = to_f32<DT>(lds_x[at]);
        v = on ? v : 0.f;
        xv = on ? xv : 0.f;
        if (z) {
          // y once more, for the gate's gradient
          float acc[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            float cv[J];
            read_states<J>(lds_c + (4 * gg + s) * NP + q * J, cv);
            acc[s] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) acc[s] = __builtin_fmaf(hs[4 * g + s + 1][j], cv[j], acc[s]);
          }
          const float yv = __builtin_fmaf(D, xv, quad_scatter(acc, q));
          const float zv = to_f32<DT>(lds_z[at]);
          const SigmoidPair sg = fsigmoid_pair(zv);
          lds_z[at] = from_f32<DT>(on ? v * yv * __builtin_fmaf(zv * sg.s, sg.no, sg.s) : 0.f);
          v = on ? v * (zv * sg.s) : 0.f;
        }
        sum_D = __builtin_fmaf(v, xv, sum_D);
        float sum_w[4], sum_g[4];
        constexpr int kPerBatch = J <= 8 ? 8 / J : 1;  // steps whose 2 J sums over the channels make 16
        float val[J <= 8 ? 16 : 32];
#pragma unroll
        for (int s = 3; s >= 0; --s) {
          const float ds = quad_from(dp[g], s), xs = quad_from(xp[g], s), vs = quad_from(v, s);
          float bv[J], cv[J];
          read_states<J>(lds_b + (4 * gg + s) * NP + q * J, bv);
          read_states<J>(lds_c + (4 * gg + s) * NP + q * J, cv);
          sum_w[s] = sum_g[s] = 0.f;
          const int at0 = J <= 8 ? s % kPerBatch * 2 * J : 0;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const float gt = __builtin_fmaf(vs, cv[j], c[j]);
            c[j] = da[4 * g + s][j] * gt;
            const float w = c[j] * hs[4 * g + s][j];
            sum_g[s] = __builtin_fmaf(gt, bv[j], sum_g[s]);
            sum_w[s] = __builtin_fmaf(w, A2[j], sum_w[s]);
            dA[j] = __builtin_fmaf(w, ds, dA[j]);
            val[at0 + j] = gt * xs;
            val[at0 + J + j] = vs * hs[4 * g + s + 1][j];
          }
          // 16 sums over the wave's channels, one a lane
          const int st = 4 * gg + s, cc = lane >> 2;
          if constexpr (J == 16) {
            float lo[16], hi[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) lo[j] = val[j], hi[j] = val[16 + j];
            lds_sum[wave][st * 2 * NP + q * J + cc] = channel_scatter(lo, lane);
            lds_sum[wave][st * 2 * NP + NP + q * J + cc] = channel_scatter(hi, lane);
          } else if constexpr (J >= 2) {
            if (s % kPerBatch == 0) {
              const float sum = channel_scatter(val, lane);
              const int n = cc % J, which = cc / J % 2, ahead = cc / (2 * J);
              lds_sum[wave][(st + ahead) * 2 * NP + which * NP + q * J + n] = sum;
            }
          } else {  // eight values of four steps
            if (s == 0) {
#pragma unroll
              for (int i = 8; i < 16; ++i) val[i] = 0.f;
              const float sum = channel_scatter(val, lane);
              if (cc < 8) lds_sum[wave][(st + cc / 2) * 2 * NP + cc % 2 * NP + q] = sum;
            }
          }
        }
        const float gb = quad_scatter(sum_g, q);
        const float dd = __builtin_fmaf(quad_scatter(sum_w, q), kLn2, xv * gb);
        const float raw = to_f32<DT>(lds_d[at]) + bias;
        const float up = on ? (a.softplus ? dd * fsigmoid(raw) : dd) : 0.f;
        sum_bias += up;
        lds_d[at] = from_f32<DT>(up);
        lds_x[at] = from_f32<DT>(__builtin_fmaf(dp[g], gb, D * v));
      }
    }
    lds_barrier();
    Tile::store(lds_x, dx, cells, t, p.t1, p.L, p.c0, p.live);
    Tile::store(lds_d, ddt, cells, t, p.t1, p.L, p.c0, p.live);
    if (z) Tile::store(lds_z, dz, cells, t, p.t1, p.L, p.c0, p.live);
    for (int i = threadIdx.x; i < kSteps * 2 * NP; i += kSelThreads) {
      const int s = i / (2 * NP);
      if (t + s < p.L) sums[(t + s) * sums_t + i % (2 * NP)] = (lds_sum[0][i] + lds_sum[1][i]) + (lds_sum[2][i] + lds_sum[3][i]);
    }
    lds_barrier();
  }
  if (a.dh0 && live && p.seg == 0) store_row<J>(a.dh0 + cell * a.N, q * J, a.N, a.svec, c);
  if (live) write_states<J>(a.part_a + (p.seg * cells + cell) * NP + q * J, dA);
  sum_D = quad_sum(sum_D);
  sum_bias = quad_sum(sum_bias);
  if (live && q == 0) {
    float* more = a.part_a + a.segs * cells * NP + (p.seg * cells + cell) * 2;
    more[0] = sum_D;
    more[1] = sum_bias;
  }
}

// dB and dC from the tiles' sums, one thread a number; zero past a row's end.
template <typename DT>
__global__ __launch_bounds__(256) void sel_reduce_bc_kernel(SelectiveScanArgs a, int NP) {
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x, each = (int64_t)a.T * a.B * a.G * 2 * NP;
  if (i >= each) return;
  const int n = (int)(i % NP), which = (int)(i / NP % 2);
  const int64_t row = i / (2 * NP);                   // (t, b, group)
  const int b = (int)(row / a.G % a.B);
  const int64_t t = row / a.G / a.B;
  if (n >= a.N) return;
  float sum = 0.f;
  if (!a.lengths || t < a.lengths[b])
    for (int k = 0; k < a.group_tiles; ++k) sum += a.part_bc[k * each + i];
  DT* out = which ? (DT*)a.dC : (DT*)a.dB;
  out[row * a.N + n] = from_f32<DT>(sum);
}

// dA, dD and dbias: the sums of rows and segments, 64 numbers a workgroup,
// four threads each, whose sums are joined in order.
__global__ __launch_bounds__(256) void sel_reduce_a_kernel(SelectiveScanArgs a, int NP) {
  __shared__ float lds[256];
  const int64_t states = (int64_t)a.H * NP, i = blockIdx.x * (int64_t)64 + (threadIdx.x & 63);
  const int parts = a.segs * a.B, slot = threadIdx.x >> 6;
  const bool state = i < states, live = i < states + 2 * (int64_t)a.H;
  const int64_t k = i - states;                        // (channel, which) of the second array
  const float* from = state ? a.part_a + i : a.part_a + parts * states + k;
  const int64_t step = state ? states : 2 * (int64_t)a.H;
  float sum = 0.f;
  if (live) {
#pragma unroll 8
    for (int m = slot; m < parts; m += 4) sum += from[m * step];
  }
  lds[threadIdx.x] = sum;
  __syncthreads();
  if (slot || !live) return;
  sum = ((sum + lds[64 + threadIdx.x]) + lds[128 + threadIdx.x]) + lds[192 + threadIdx.x];
  if (state) {
    if (i % NP < a.N) a.dA[i / NP * a.N + i % NP] = sum;
  } else if (k % 2 == 0) {
    if (a.dD) a.dD[k / 2] = sum;
  } else if (a.dbias) {
    a.dbias[k / 2] = sum;
  }
}

template <typename DT, int J, bool VEC>
hipError_t run(const SelectiveScanArgs& a, hipStream_t st) {
  constexpr int NP = 4 * J;
  if (a.segs > 1) {
    launch_kernel(sel_compose_back_kernel<DT, J, VEC>, sel_grid(a), dim3(kSelThreads), 0, st, a);
    const hipError_t e = launch_sel_carry(a, a.dh_n, NP, true, st);
    if (e != hipSuccess) return e;
  }
  launch_kernel(sel_backward_kernel<DT, J, VEC>, sel_grid(a), dim3(kSelThreads), 0, st, a);
  const int64_t each = (int64_t)a.T * a.B * a.G * 2 * NP;
  launch_kernel(sel_reduce_bc_kernel<DT>, dim3((unsigned)((each + 255) / 256)), dim3(256), 0, st, a, NP);
  const int64_t sums = (int64_t)a.H * (NP + 2);
  launch_kernel(sel_reduce_a_kernel, dim3((unsigned)((sums + 63) / 64)), dim3(256), 0, st, a, NP);
  return hipGetLastError();
}

template <typename DT, int J>
hipError_t run_width(const SelectiveScanArgs& a, hipStream_t st) {
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

hipError_t launch_selective_scan_backward(SelectiveScanArgs a, bool bf, hipStream_t st) {
  sel_tiles(a);
  return bf ? run_states<bf16>(a, st) : run_states<float>(a, st);
}

}  // namespace rnnk
