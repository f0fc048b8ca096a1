// Cross attention, backward.
//
//   p  = 2^(s - lse),  dp = do v^T,  delta = sum over d of do o
//   ds = p (dp - delta),  dq = scale ds k,  dk = scale ds^T q,  dv = p^T do
//
// Two kernels that each form p again from the kept log-sum-exp: one owns
// query rows and walks the keys (delta, dq), the other owns keys and walks
// the query rows of all heads that share them (dk, dv). So every output has
// one owner and no sum depends on the order in which workgroups run.
//
// At large scores the log-sum-exp lse, a float, is rounded by more than the
// sums can bear (2^(s - lse) is off by a factor 2^(half a unit in its last
// place): 1e-3 at 2^13, 2 at 2^23). For such rows (large_lse) the first kernel
// adds up their probabilities as they come out, in a pass over the keys of its
// own, and keeps rest = log2 of the sum in delta's place; p is 2^(s - lse -
// rest) then, and the second kernel forms delta again from do and o. A
// workgroup without such rows does none of it; one with them takes 1.5 (fp32)
// to 3 times (bf16) as long.
//
// 1000 queries x 1000 keys, 32 ragged rows, 8/2 heads of 128, bf16, launches
// back to back: dq 188 us, dk and dv 292 us. The latter walks 310 equal key
// tiles on 256 compute units, so it takes as long as 512 would; dq and dk/dv in
// one launch, the query tiles filling the gap, took 4% more than apart (with
// delta's own launch) and was not taken.
#include <type_traits>

#include "attention_common.hpp"

namespace rnnk {
namespace {

// This lane's share (eight columns) of delta.
template <typename DT, bool FAST>
__device__ __forceinline__ float delta_part(const AttentionArgs& a, int64_t at, int col, const Frag<DT>& dO) {
  const Frag<DT> o = load8<DT, FAST>((const DT*)a.o + at, col, a.D, a.vec != 0);
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(o.get(j), dO.get(j), dot);
  if constexpr (sizeof(DT) == 2) {
    const Frag<DT> rest = load8<DT, FAST>((const DT*)a.o_rest + at, col, a.D, a.vec != 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(rest.get(j), dO.get(j), dot);
  }
  return dot;
}

// log2 of the sum of this lane's query row's probabilities as the kernels form
// them from the kept log-sum-exp. Called by whole waves.
template <typename DT, int DP, bool FAST>
__device__ __forceinline__ float lse_rest(const AttentionArgs& a, const DT* kb, int L, const Frag<DT> (&q)[DP / 32], float sl,
                                          float lse) {
  const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
  float sum = 0.f;
  for (int k0 = 0; k0 < L; k0 += 16) {
    const int key = k0 + i16;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < DP / 32; ++c)
      s = mma(key < L ? load8<DT, FAST>(kb + key * a.k_t, 32 * c + 8 * g, a.D, a.vec != 0) : zero_frag<DT>(), q[c], s);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k0 + 4 * g + j < L) sum += __builtin_amdgcn_exp2f(score_above(s[j], sl, lse));
  }
  return large_lse(lse) ? __builtin_amdgcn_logf(col_sum(sum)) : 0.f;
}

// Raw scores to base 2 above their row's log-sum-exp, of one row (a lane's
// four results belong to one) or of four. LARGE: there may be rows that need
// their rest. The kernels have their loops twice for it: a branch inside, that
// is never taken, costs 13% (1000 x 1000, 32 ragged rows, 8/2 heads of 128).
template <bool LARGE>
__device__ __forceinline__ void above_lse(f32x4& s, float sl, float lse, float rest) {
  if (LARGE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = score_above(s[j], sl, lse) - rest;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = __builtin_fmaf(s[j], sl, -lse);
  }
}
template <bool LARGE>
__device__ __forceinline__ void above_lse(f32x4& s, float sl, const f32x4& lse, const float* rest) {
  if (LARGE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = score_above(s[j], sl, lse[j]) - rest[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = __builtin_fmaf(s[j], sl, -lse[j]);
  }
}

// Whether any thread of the workgroup has a large log-sum-exp; a barrier.
template <int WAVES>
__device__ __forceinline__ bool any_large(bool mine, int* flags) {
  const int wave_has = __any(mine);
  if ((threadIdx.x & 63) == 0) flags[threadIdx.x >> 6] = wave_has;
  __syncthreads();
  int any = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) any |= flags[w];
  return __builtin_amdgcn_readfirstlane(any) != 0;
}

// For a tile of query rows some of which have a large log-sum-exp: takes their
// rest out of delta's place and puts delta there. Called by the whole
// workgroup of NT threads.
template <typename DT, int kRows, int NT>
__device__ __forceinline__ void settle_large_rows(const AttentionArgs& a, const QRows& rows, int b, int hk, int m0,
                                                  const DT* ldo, int ld, const float* llse, float* ldelta, float* lrest) {
  constexpr int kPer = NT / kRows;  // neighbouring threads of a row
  static_assert(NT % kRows == 0 && 64 % kPer == 0, "a row's threads are in one wave");
  const int r = threadIdx.x / kPer, part = threadIdx.x % kPer;
  const bool large = large_lse(llse[r]);  // not past the last row: infinite there
  float dot = 0.f;
  if (large) {
    const int64_t at = rows.dense(a, b, hk, m0 + r);
#pragma unroll 1
    for (int d = part; d < a.D; d += kPer) {
      float o = to_f32<DT>(((const DT*)a.o)[at + d]);
      if constexpr (sizeof(DT) == 2) o += to_f32<DT>(((const DT*)a.o_rest)[at + d]);
      dot = __builtin_fmaf(o, to_f32<DT>(ldo[r * ld + d]), dot);
    }
  }
#pragma unroll
  for (int k = 1; k < kPer; k <<= 1) dot += __shfl_xor(dot, k, 64);
  const float rest = ldelta[r];
  if (part == 0) {
    lrest[r] = large ? rest : 0.f;
    if (large) ldelta[r] = dot;
  }
  __syncthreads();
}

// Query rows across (16 per wave and tile), keys down: dq^T = K^T ds^T.
template <typename DT, int DP, int QT, int KT, bool FAST>
__global__ __launch_bounds__(kAttnThreads, 2) void attention_dq_kernel(AttentionArgs a) {
  constexpr int kC = DP / 32, kDT = DP / 16, kRows = 4 * QT * 16, kKeys = KT * 16;
  constexpr int kLdK = TileShape<DT, DP, true>::kLd, kLdV = TileShape<DT, DP, false>::kLd;
  extern __shared__ __align__(16) char lds[];
  DT* smem = reinterpret_cast<DT*>(lds);
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int tiles = (rows.M + kRows - 1) / kRows;
  const Work w = work_of(a, tiles);
  if (w.tile >= tiles) return;
  const int bh = w.bh, m0 = w.tile * kRows;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;
  const int L = key_count(a, b);
  const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;

  Frag<DT> q[QT][kC], dO[QT][kC];
  float lse[QT], delta[QT], rest_of[QT];
  bool large = false;  // a row of this wave
  const float sl = a.scale * kLog2e;
  f32x4 dq[QT][kDT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wave * QT + t) * 16 + i16;
    const bool on = m < rows.M;
    const int64_t at = rows.dense(a, b, hk, on ? m : 0);
    const DT* row = rows.in<DT>(qb, a.q_t, a.q_h, on ? m : 0);
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = 32 * c + 8 * g;
      q[t][c] = load8<DT, FAST>(row, col, a.D, vec);
      dO[t][c] = load8<DT, FAST>((const DT*)a.d_o + at, col, a.D, vec);
      if (!on) q[t][c] = dO[t][c] = zero_frag<DT>();
      dot += delta_part<DT, FAST>(a, at, col, dO[t][c]);
    }
    delta[t] = col_sum(dot);
    lse[t] = on && L > 0 ? a.lse[(int64_t)bh * rows.M + m] : 0.f;
    rest_of[t] = 0.f;
    if (__any(large_lse(lse[t]))) {
      rest_of[t] = lse_rest<DT, DP, FAST>(a, kb, L, q[t], sl, lse[t]);
      large = true;
    }
    if (on && g == 0) a.delta[(int64_t)bh * rows.M + m] = large_lse(lse[t]) ? rest_of[t] : delta[t];
#pragma unroll
    for (int d = 0; d < kDT; ++d) dq[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  TileLoad<DT, DP, kKeys, kLdK, FAST> nk;
  TileLoad<DT, DP, kKeys, kLdV, FAST> nv;
  constexpr int kTile = kKeys * (kLdK + kLdV);
  nk.load(kb, a.k_t, 0, L, a.D, vec);
  nv.load(vb, a.v_t, 0, L, a.D, vec);
  nk.put(smem);
  nv.put(smem + kKeys * kLdK);
  __shared__ int flags[kAttnThreads / 64];
  auto walk = [&](auto LARGE) {
    for (int k0 = 0; k0 < L; k0 += kKeys) {
      const DT* lk = smem + (k0 / kKeys & 1) * kTile;
      const DT* lv = lk + kKeys * kLdK;
      const bool more = k0 + kKeys < L;
      if (more) {
        nk.load(kb, a.k_t, k0 + kKeys, L, a.D, vec);
        nv.load(vb, a.v_t, k0 + kKeys, L, a.D, vec);
      }
      __builtin_amdgcn_sched_barrier(0);
      f32x4 s[QT][KT], dp[QT][KT];
#pragma unroll
      for (int n = 0; n < KT; ++n) {
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t][n] = dp[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const Frag<DT> kf = read_rows<DT>(lk, kLdK, n * 16 + i16, 32 * c + 8 * g);
          const Frag<DT> vf = read_rows<DT>(lv, kLdV, n * 16 + i16, 32 * c + 8 * g);
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            s[t][n] = mma(kf, q[t][c], s[t][n]);
            dp[t][n] = mma(vf, dO[t][c], dp[t][n]);
          }
        }
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          above_lse<LARGE()>(s[t][n], sl, lse[t], rest_of[t]);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t][n][j] = __builtin_amdgcn_exp2f(s[t][n][j]) * (dp[t][n][j] - delta[t]);
        }
      }
      if (!more) {  // keys past the row's end have a p that means nothing
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k0 + n * 16 + 4 * g + j >= L) {
#pragma unroll
              for (int t = 0; t < QT; ++t) s[t][n][j] = 0.f;
            }
      }
      // ds enters the product as its rounded value and the rest: the rounding
      // errors of a long row's ds would add up against a sum that cancels
#pragma unroll
      for (int n = 0; n < KT; n += 2) {
        Frag<DT> ds[QT], rest[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          ds[t] = stack<DT>(s[t][n], s[t][n + 1]);
          if constexpr (sizeof(DT) == 2) rest[t] = stack_rest(s[t][n], s[t][n + 1], ds[t]);
        }
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          const Frag<DT> kf = read_cols<DT>(lk, kLdK, n * 16, 16 * d, lane);
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            dq[t][d] = mma(kf, ds[t], dq[t][d]);
            if constexpr (sizeof(DT) == 2) dq[t][d] = mma(kf, rest[t], dq[t][d]);
          }
        }
      }
      if (more) {
        DT* dst = smem + (k0 / kKeys + 1 & 1) * kTile;
        nk.put(dst);
        nv.put(dst + kKeys * kLdK);
      }
      __syncthreads();
    }
  };
  if (any_large<kAttnThreads / 64>(large, flags))
    walk(std::true_type{});
  else
    walk(std::false_type{});
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wave * QT + t) * 16 + i16;
    if (m >= rows.M) continue;
    DT* dst = (DT*)a.dq + rows.dense(a, b, hk, m);
#pragma unroll
    for (int d = 0; d < kDT; ++d) store4<DT, FAST>(dst, 16 * d + 4 * g, a.D, vec, dq[t][d] * a.scale);
  }
}

// The same for few query rows: 16 a workgroup, whose waves divide the keys, 32
// at a time (see the forward pass): keys and values go from memory straight
// into fragments, and a wave's keys through its own piece of LDS for the
// product with ds.
template <typename DT, int DP>
struct DqStepShape {
  static constexpr int kLdK = TileShape<DT, DP, true>::kLd, kLdO = DP + 4;
  static constexpr int kBytesK = 4 * 32 * kLdK * (int)sizeof(DT), kBytesO = 4 * 16 * kLdO * (int)sizeof(float);
  static constexpr int kBytes = kBytesK > kBytesO ? kBytesK : kBytesO;
};
template <typename DT, int DP, bool FAST>
__global__ __launch_bounds__(kAttnThreads, sizeof(DT) == 4 && DP > 96 ? 1 : 2) void attention_dq_step_kernel(AttentionArgs a) {
  using S = DqStepShape<DT, DP>;
  constexpr int kC = DP / 32, kDT = DP / 16, kWaves = 4, kStep = 32, kLdK = S::kLdK, kLdO = S::kLdO;
  extern __shared__ __align__(16) char lds[];
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int tiles = (rows.M + 15) / 16;
  const Work w = work_of(a, tiles);
  if (w.tile >= tiles) return;
  const int bh = w.bh, m0 = w.tile * 16;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;
  const int L = key_count(a, b);
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;
  DT* lk = reinterpret_cast<DT*>(lds) + wave * kStep * kLdK;

  Frag<DT> k[2][kC], v[2][kC];
  auto load = [&](int k0) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int key = k0 + 16 * n + i16;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        k[n][c] = key < L ? load8<DT, FAST>(kb + key * a.k_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
        v[n][c] = key < L ? load8<DT, FAST>(vb + key * a.v_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
      }
    }
  };
  int k0 = wave * kStep;
  load(k0);
  const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
  const int mine = m0 + i16;
  const bool on = mine < rows.M;
  Frag<DT> q[kC], dO[kC];
  float dot = 0.f;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int col = 32 * c + 8 * g;
    q[c] = dO[c] = zero_frag<DT>();
    if (on) {
      const int64_t at = rows.dense(a, b, hk, mine);
      q[c] = load8<DT, FAST>(rows.in<DT>(qb, a.q_t, a.q_h, mine), col, a.D, vec);
      dO[c] = load8<DT, FAST>((const DT*)a.d_o + at, col, a.D, vec);
      dot += delta_part<DT, FAST>(a, at, col, dO[c]);
    }
  }
  const float delta = col_sum(dot);
  const float lse = on && L > 0 ? a.lse[(int64_t)bh * rows.M + mine] : 0.f;
  const float sl = a.scale * kLog2e;
  const bool large = __any(large_lse(lse));
  float rest_of = 0.f;
  if (large) rest_of = lse_rest<DT, DP, FAST>(a, kb, L, q, sl, lse);
  if (on && g == 0 && wave == 0) a.delta[(int64_t)bh * rows.M + mine] = large_lse(lse) ? rest_of : delta;
  f32x4 dq[kDT];
#pragma unroll
  for (int d = 0; d < kDT; ++d) dq[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (; k0 < L; k0 += kWaves * kStep) {
    f32x4 s[2], dp[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s[n] = dp[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        s[n] = mma(k[n][c], q[c], s[n]);
        dp[n] = mma(v[n][c], dO[c], dp[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int c = 0; c < kC; ++c) put8<DT>(lk + (16 * n + i16) * kLdK + 32 * c + 8 * g, k[n][c]);
    load(k0 + kWaves * kStep);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (large)
        above_lse<true>(s[n], sl, lse, rest_of);
      else
        above_lse<false>(s[n], sl, lse, rest_of);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = __builtin_amdgcn_exp2f(s[n][j]);
        s[n][j] = k0 + 16 * n + 4 * g + j < L ? p * (dp[n][j] - delta) : 0.f;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const Frag<DT> ds = stack<DT>(s[0], s[1]);
    Frag<DT> rest;
    if constexpr (sizeof(DT) == 2) rest = stack_rest(s[0], s[1], ds);
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      const Frag<DT> kf = read_cols<DT>(lk, kLdK, 0, 16 * d, lane);
      dq[d] = mma(kf, ds, dq[d]);
      if constexpr (sizeof(DT) == 2) dq[d] = mma(kf, rest, dq[d]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  // join the waves' parts of the keys, in order of their number
  float* jo = reinterpret_cast<float*>(lds);
  __syncthreads();
#pragma unroll
  for (int d = 0; d < kDT; ++d) *reinterpret_cast<f32x4*>(jo + (wave * 16 + i16) * kLdO + 16 * d + 4 * g) = dq[d];
  __syncthreads();
  for (int p = threadIdx.x; p < 16 * (DP / 4); p += kAttnThreads) {
    const int m = p / (DP / 4), col = p % (DP / 4) * 4;
    if (m0 + m >= rows.M) return;
    f32x4 acc = *reinterpret_cast<const f32x4*>(jo + m * kLdO + col);
#pragma unroll
    for (int x = 1; x < kWaves; ++x) acc += *reinterpret_cast<const f32x4*>(jo + (x * 16 + m) * kLdO + col);
    store4<DT, FAST>((DT*)a.dq + rows.dense(a, b, hk, m0 + m), col, a.D, vec, acc * a.scale);
  }
}

// Keys across (KT x 16 per wave), query rows down: dv^T = do^T p, dk^T = Q^T
// ds. The four waves are 4 / WM sets of keys times WM parts of a tile's rows,
// whose sums are joined at the end.
template <typename DT, int DP, int KT, int WM, int MT>
struct KvShape {
  static constexpr int kKeys = 4 / WM * KT * 16, kRows = WM * MT * 16;
  static constexpr int kLd = TileShape<DT, DP, true>::kLd;
  // a tile's query rows, their do, log-sum-exp, delta and the former's rest; kept twice
  static constexpr int kTile = 2 * kRows * kLd + 3 * kRows * (int)(sizeof(float) / sizeof(DT));
  static constexpr int kJoin = WM > 1 ? (WM - 1) * kKeys * (DP + 4) * (int)sizeof(float) : 0;
  static constexpr int kBytes = 2 * kTile * (int)sizeof(DT) > kJoin ? 2 * kTile * (int)sizeof(DT) : kJoin;
};

template <typename DT, int DP, int KT, int WM, int MT, bool FAST, bool REST>
__global__ __launch_bounds__(kAttnThreads, sizeof(DT) == 2 ? 2 : DP <= 64 ? 3 : DP <= 96 ? 2 : 1) void attention_dkv_kernel(AttentionArgs a) {
  using S = KvShape<DT, DP, KT, WM, MT>;
  constexpr int kC = DP / 32, kDT = DP / 16, kKeys = S::kKeys, kRows = S::kRows, kLd = S::kLd;
  extern __shared__ __align__(16) char lds[];
  DT* smem = reinterpret_cast<DT*>(lds);
  const int tiles = (a.Tk + kKeys - 1) / kKeys;
  const Work w = work_of(a, tiles);
  if (w.tile >= tiles) return;
  const int bh = w.bh, k0 = w.tile * kKeys;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const int wm = wave % WM, wk = wave / WM;
  const bool vec = a.vec != 0;
  const int L = key_count(a, b);

  f32x4 dk[KT][kDT], dv[KT][kDT];
#pragma unroll
  for (int n = 0; n < KT; ++n)
#pragma unroll
    for (int d = 0; d < kDT; ++d) dk[n][d] = dv[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (k0 < L) {
    const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
    const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;
    Frag<DT> k[KT][kC], v[KT][kC];
#pragma unroll
    for (int n = 0; n < KT; ++n) {
      const int key = k0 + (wk * KT + n) * 16 + i16;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        k[n][c] = key < L ? load8<DT, FAST>(kb + key * a.k_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
        v[n][c] = key < L ? load8<DT, FAST>(vb + key * a.v_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
      }
    }
    const float sl = a.scale * kLog2e;
    const float* stat = (threadIdx.x < kRows ? a.lse : a.delta) + (int64_t)bh * rows.M;
    const int srow = threadIdx.x % kRows;
    QueryLoad<DT, DP, kRows, kLd, FAST> nq, no;
    float nstat = 0.f;
    auto load = [&](int m0) {
      nq.load(m0, rows.M, a.D, vec);
      no.load(m0, rows.M, a.D, vec);
      // a row past the end: 2^-inf, so p = 0
      if (threadIdx.x < 2 * kRows)
        nstat = m0 + srow < rows.M ? stat[m0 + srow] : (threadIdx.x < kRows ? __builtin_inff() : 0.f);
    };
    auto put = [&](DT* dst) {
      nq.put(dst);
      no.put(dst + kRows * kLd);
      if (threadIdx.x < 2 * kRows) reinterpret_cast<float*>(dst + 2 * kRows * kLd)[threadIdx.x] = nstat;
    };
    nq.start((const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h, a.q_t, a.q_h, rows.G);
    no.start((const DT*)a.d_o + ((int64_t)b * a.heads + hk * rows.G) * a.D, (int64_t)a.B * a.heads * a.D, a.D, rows.G);
    load(0);
    bool large = false;
#pragma unroll 8
    for (int m = threadIdx.x; m < rows.M; m += kAttnThreads) large |= large_lse(a.lse[(int64_t)bh * rows.M + m]);
    put(smem);
    auto ahead = [&](int m0) {
      nq.next(rows.G);
      no.next(rows.G);
      load(m0 + kRows);
    };
    __shared__ int flags[kAttnThreads / 64];
    auto walk = [&](auto LARGE) {
      int turn = 0;
      for (int m0 = 0; m0 < rows.M; m0 += kRows, turn ^= 1) {
        const DT* lq = smem + turn * S::kTile;
        const DT* ldo = lq + kRows * kLd;
        const float* llse = reinterpret_cast<const float*>(ldo + kRows * kLd);
        const float *ldelta = llse + kRows, *lrest = ldelta + kRows;
        const bool more = m0 + kRows < rows.M;
        if (more && !LARGE()) ahead(m0);
        __builtin_amdgcn_sched_barrier(0);
        if (LARGE())
          settle_large_rows<DT, kRows, kAttnThreads>(a, rows, b, hk, m0, ldo, kLd, llse, const_cast<float*>(ldelta),
                                                 const_cast<float*>(lrest));
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2) {
          const int r0 = (wm * MT + mt) * 16;
          f32x4 s[2][KT], dp[2][KT];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int n = 0; n < KT; ++n) s[h][n] = dp[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kC; ++c) {
              const Frag<DT> qf = read_rows<DT>(lq, kLd, r0 + h * 16 + i16, 32 * c + 8 * g);
#pragma unroll
              for (int n = 0; n < KT; ++n) s[h][n] = mma(qf, k[n][c], s[h][n]);
              const Frag<DT> of = read_rows<DT>(ldo, kLd, r0 + h * 16 + i16, 32 * c + 8 * g);
#pragma unroll
              for (int n = 0; n < KT; ++n) dp[h][n] = mma(of, v[n][c], dp[h][n]);
            }
            const f32x4 lse = *reinterpret_cast<const f32x4*>(llse + r0 + h * 16 + 4 * g);
            const f32x4 de = *reinterpret_cast<const f32x4*>(ldelta + r0 + h * 16 + 4 * g);
            const float* rest_of = lrest + r0 + h * 16 + 4 * g;
#pragma unroll
            for (int n = 0; n < KT; ++n) {
              above_lse<LARGE()>(s[h][n], sl, lse, rest_of);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                s[h][n][j] = __builtin_amdgcn_exp2f(s[h][n][j]);
                dp[h][n][j] = s[h][n][j] * (dp[h][n][j] - de[j]);
              }
            }
          }
          Frag<DT> p[KT], ds[KT], p_rest[KT], ds_rest[KT];
#pragma unroll
          for (int n = 0; n < KT; ++n) {
            p[n] = stack<DT>(s[0][n], s[1][n]);
            ds[n] = stack<DT>(dp[0][n], dp[1][n]);
            if constexpr (REST) {
              p_rest[n] = stack_rest(s[0][n], s[1][n], p[n]);
              ds_rest[n] = stack_rest(dp[0][n], dp[1][n], ds[n]);
            }
          }
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            const Frag<DT> of = read_cols<DT>(ldo, kLd, r0, 16 * d, lane);
            const Frag<DT> qf = read_cols<DT>(lq, kLd, r0, 16 * d, lane);
#pragma unroll
            for (int n = 0; n < KT; ++n) {
              dv[n][d] = mma(of, p[n], dv[n][d]);
              dk[n][d] = mma(qf, ds[n], dk[n][d]);
              if constexpr (REST) {
                dv[n][d] = mma(of, p_rest[n], dv[n][d]);
                dk[n][d] = mma(qf, ds_rest[n], dk[n][d]);
              }
            }
          }
        }
        if (more && LARGE()) ahead(m0);  // fewer values are held meanwhile, so that the other loop has its registers
        if (more) put(smem + (turn ^ 1) * S::kTile);
        __syncthreads();
      }
    };
    if (any_large<kAttnThreads / 64>(large, flags))
      walk(std::true_type{});
    else
      walk(std::false_type{});
    if constexpr (WM > 1) {
      // join the parts of the rows, in order of their number
      constexpr int kLdJ = DP + 4;
      float* join = reinterpret_cast<float*>(lds);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (which == 1) __syncthreads();
        if (wm > 0) {
#pragma unroll
          for (int n = 0; n < KT; ++n)
#pragma unroll
            for (int d = 0; d < kDT; ++d)
              *reinterpret_cast<f32x4*>(join + (((wm - 1) * (4 / WM) + wk) * KT * 16 + n * 16 + i16) * kLdJ + 16 * d + 4 * g) =
                  which ? dv[n][d] : dk[n][d];
        }
        __syncthreads();
        if (wm == 0) {
#pragma unroll
          for (int w = 0; w < WM - 1; ++w)
#pragma unroll
            for (int n = 0; n < KT; ++n)
#pragma unroll
              for (int d = 0; d < kDT; ++d) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(
                    join + ((w * (4 / WM) + wk) * KT * 16 + n * 16 + i16) * kLdJ + 16 * d + 4 * g);
                if (which)
                  dv[n][d] += x;
                else
                  dk[n][d] += x;
              }
        }
      }
    }
  }
  if (wm != 0) return;
#pragma unroll
  for (int n = 0; n < KT; ++n) {
    const int key = k0 + (wk * KT + n) * 16 + i16;
    if (key >= a.Tk) continue;
    const bool on = key < L;
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    const int64_t at = (((int64_t)key * a.B + b) * a.kv_heads + hk) * a.D;
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      store4<DT, FAST>((DT*)a.dk + at, 16 * d + 4 * g, a.D, vec, on ? dk[n][d] * a.scale : z);
      store4<DT, FAST>((DT*)a.dv + at, 16 * d + 4 * g, a.D, vec, on ? dv[n][d] : z);
    }
  }
}

// The same for wide bf16 heads, where a wave cannot hold the sums of both
// gradients and two waves a SIMD at once: two teams of four waves own the same
// keys, one summing dv and one dk, and share the tiles of Q and do in LDS.
// Both form the scores (a quarter of the work more than forming them once); a
// SIMD runs a wave of each team, whose products, exponentials and LDS reads
// overlap. Measured at 1000 queries x 1000 keys, 32 ragged rows, 8/2 heads of
// 128: 292 us (144 GFLOP: 493 TFLOP/s); both sums in one wave (one wave a SIMD)
// took 1.2 and a launch for each 1.5 times as long.
template <typename DT, int DP, int KT, int MT, bool FAST, bool REST>
__global__ __launch_bounds__(512, 2) void attention_dkv_team_kernel(AttentionArgs a) {
  using S = KvShape<DT, DP, KT, 1, MT>;
  constexpr int kC = DP / 32, kDT = DP / 16, kKeys = S::kKeys, kRows = S::kRows, kLd = S::kLd;
  extern __shared__ __align__(16) char lds[];
  DT* smem = reinterpret_cast<DT*>(lds);
  const int tiles = (a.Tk + kKeys - 1) / kKeys;
  const Work w = work_of(a, tiles);
  if (w.tile >= tiles) return;
  const int bh = w.bh, k0 = w.tile * kKeys;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const int wk = wave & 3;
  const bool for_dk = wave >= 4;
  const bool vec = a.vec != 0;
  const int L = key_count(a, b);

  f32x4 acc[KT][kDT];
#pragma unroll
  for (int n = 0; n < KT; ++n)
#pragma unroll
    for (int d = 0; d < kDT; ++d) acc[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (k0 < L) {
    const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
    const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;
    Frag<DT> k[KT][kC], v[KT][kC];
#pragma unroll
    for (int n = 0; n < KT; ++n) {
      const int key = k0 + (wk * KT + n) * 16 + i16;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        k[n][c] = key < L ? load8<DT, FAST>(kb + key * a.k_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
        v[n][c] = key < L ? load8<DT, FAST>(vb + key * a.v_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
      }
    }
    const float sl = a.scale * kLog2e;
    const float* stat = (threadIdx.x < kRows ? a.lse : a.delta) + (int64_t)bh * rows.M;
    const int srow = threadIdx.x % kRows;
    QueryLoad<DT, DP, kRows, kLd, FAST, 512> nq, no;
    float nstat = 0.f;
    auto load = [&](int m0) {
      nq.load(m0, rows.M, a.D, vec);
      no.load(m0, rows.M, a.D, vec);
      // a row past the end: 2^-inf, so p = 0
      if (threadIdx.x < 2 * kRows)
        nstat = m0 + srow < rows.M ? stat[m0 + srow] : (threadIdx.x < kRows ? __builtin_inff() : 0.f);
    };
    auto put = [&](DT* dst) {
      nq.put(dst);
      no.put(dst + kRows * kLd);
      if (threadIdx.x < 2 * kRows) reinterpret_cast<float*>(dst + 2 * kRows * kLd)[threadIdx.x] = nstat;
    };
    nq.start((const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h, a.q_t, a.q_h, rows.G);
    no.start((const DT*)a.d_o + ((int64_t)b * a.heads + hk * rows.G) * a.D, (int64_t)a.B * a.heads * a.D, a.D, rows.G);
    load(0);
    bool large = false;
#pragma unroll 8
    for (int m = threadIdx.x; m < rows.M; m += 512) large |= large_lse(a.lse[(int64_t)bh * rows.M + m]);
    put(smem);
    auto ahead = [&](int m0) {
      nq.next(rows.G);
      no.next(rows.G);
      load(m0 + kRows);
    };
    __shared__ int flags[512 / 64];
    auto walk = [&](auto LARGE) {
      int turn = 0;
      for (int m0 = 0; m0 < rows.M; m0 += kRows, turn ^= 1) {
        const DT* lq = smem + turn * S::kTile;
        const DT* ldo = lq + kRows * kLd;
        const float* llse = reinterpret_cast<const float*>(ldo + kRows * kLd);
        const float *ldelta = llse + kRows, *lrest = ldelta + kRows;
        const bool more = m0 + kRows < rows.M;
        if (more && !LARGE()) ahead(m0);
        const DT* lx = for_dk ? lq : ldo;
        if (LARGE())
          settle_large_rows<DT, kRows, 512>(a, rows, b, hk, m0, ldo, kLd, llse, const_cast<float*>(ldelta),
                                                 const_cast<float*>(lrest));
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2) {
          f32x4 s[2][KT];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r0 = (mt + h) * 16;
#pragma unroll
            for (int n = 0; n < KT; ++n) s[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kC; ++c) {
              const Frag<DT> qf = read_rows<DT>(lq, kLd, r0 + i16, 32 * c + 8 * g);
#pragma unroll
              for (int n = 0; n < KT; ++n) s[h][n] = mma(qf, k[n][c], s[h][n]);
            }
            const f32x4 lse = *reinterpret_cast<const f32x4*>(llse + r0 + 4 * g);
            const float* rest_of = lrest + r0 + 4 * g;
#pragma unroll
            for (int n = 0; n < KT; ++n) {
              above_lse<LARGE()>(s[h][n], sl, lse, rest_of);
#pragma unroll
              for (int j = 0; j < 4; ++j) s[h][n][j] = __builtin_amdgcn_exp2f(s[h][n][j]);
            }
          }
          if (for_dk) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r0 = (mt + h) * 16;
              f32x4 dp[KT];
#pragma unroll
              for (int n = 0; n < KT; ++n) dp[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int c = 0; c < kC; ++c) {
                const Frag<DT> of = read_rows<DT>(ldo, kLd, r0 + i16, 32 * c + 8 * g);
#pragma unroll
                for (int n = 0; n < KT; ++n) dp[n] = mma(of, v[n][c], dp[n]);
              }
              const f32x4 de = *reinterpret_cast<const f32x4*>(ldelta + r0 + 4 * g);
#pragma unroll
              for (int n = 0; n < KT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[h][n][j] *= dp[n][j] - de[j];
            }
          }
          Frag<DT> x[KT], rest[KT];
#pragma unroll
          for (int n = 0; n < KT; ++n) {
            x[n] = stack<DT>(s[0][n], s[1][n]);
            if constexpr (REST) rest[n] = stack_rest(s[0][n], s[1][n], x[n]);
          }
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            const Frag<DT> f = read_cols<DT>(lx, kLd, mt * 16, 16 * d, lane);
#pragma unroll
            for (int n = 0; n < KT; ++n) {
              acc[n][d] = mma(f, x[n], acc[n][d]);
              if constexpr (REST) acc[n][d] = mma(f, rest[n], acc[n][d]);
            }
          }
        }
        if (more && LARGE()) ahead(m0);  // fewer values are held meanwhile, so that the other loop has its registers
        if (more) put(smem + (turn ^ 1) * S::kTile);
        __syncthreads();
      }
    };
    if (any_large<512 / 64>(large, flags))
      walk(std::true_type{});
    else
      walk(std::false_type{});
  }
  const float mul = for_dk ? a.scale : 1.0f;
  DT* out = (DT*)(for_dk ? a.dk : a.dv);
#pragma unroll
  for (int n = 0; n < KT; ++n) {
    const int key = k0 + (wk * KT + n) * 16 + i16;
    if (key >= a.Tk) continue;
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    DT* dst = out + (((int64_t)key * a.B + b) * a.kv_heads + hk) * a.D;
#pragma unroll
    for (int d = 0; d < kDT; ++d) store4<DT, FAST>(dst, 16 * d + 4 * g, a.D, vec, key < L ? acc[n][d] * mul : z);
  }
}

// p and ds are rounded to bf16 for the products of dk and dv (one rounding of
// each value, of the relative size of the gradients' own, so that these come
// out sqrt(2) times as far off as by their own rounding alone) where the
// launch fills the device: with the rest of the rounding as a second product
// dk and dv take 372 us for 292 at 1000 x 1000, 32 ragged rows, 8/2 heads of
// 128, and with heads of 32 the whole backward pass 218 for 149. A launch with fewer workgroups than compute units has the time for it.
// include/rnn.h states the rule, which is part of what a caller gets.
bool keep_rest(const AttentionArgs& a, int64_t tiles) { return tiles * a.B * a.kv_heads <= a.cus; }

template <typename DT, int DP, int KT, int WM, int MT>
hipError_t run_kv(const AttentionArgs& a, bool fast, hipStream_t st) {
  using S = KvShape<DT, DP, KT, WM, MT>;
  constexpr bool kBf = sizeof(DT) == 2;
  const int64_t tiles = ((int64_t)a.Tk + S::kKeys - 1) / S::kKeys;
  const bool rest = kBf && keep_rest(a, tiles);
  const auto kernel = rest ? (fast ? attention_dkv_kernel<DT, DP, KT, WM, MT, true, kBf> : attention_dkv_kernel<DT, DP, KT, WM, MT, false, kBf>)
                           : (fast ? attention_dkv_kernel<DT, DP, KT, WM, MT, true, false> : attention_dkv_kernel<DT, DP, KT, WM, MT, false, false>);
  const hipError_t e = allow_lds(kernel, S::kBytes);
  if (e != hipSuccess) return e;
  launch_kernel(kernel, dim3((unsigned)work_grid(a, tiles)), dim3(kAttnThreads), S::kBytes, st, a);
  return hipGetLastError();
}

template <typename DT, int DP, int KT, int MT>
hipError_t run_kv_team(const AttentionArgs& a, bool fast, hipStream_t st) {
  using S = KvShape<DT, DP, KT, 1, MT>;
  const int64_t tiles = ((int64_t)a.Tk + S::kKeys - 1) / S::kKeys;
  const bool rest = keep_rest(a, tiles);
  const auto kernel = rest ? (fast ? attention_dkv_team_kernel<DT, DP, KT, MT, true, true> : attention_dkv_team_kernel<DT, DP, KT, MT, false, true>)
                           : (fast ? attention_dkv_team_kernel<DT, DP, KT, MT, true, false> : attention_dkv_team_kernel<DT, DP, KT, MT, false, false>);
  const hipError_t e = allow_lds(kernel, S::kBytes);
  if (e != hipSuccess) return e;
  launch_kernel(kernel, dim3((unsigned)work_grid(a, tiles)), dim3(512), S::kBytes, st, a);
  return hipGetLastError();
}

template <typename DT, int DP>
hipError_t run(const AttentionArgs& a, hipStream_t st) {
  constexpr int QT = sizeof(DT) == 2 ? 2 : 1, KT = 2;
  const int64_t M = (int64_t)a.Tq * (a.heads / a.kv_heads);
  constexpr int kLdT = TileShape<DT, DP, true>::kLd, kLdR = TileShape<DT, DP, false>::kLd;
  constexpr int kLdsQ = 2 * KT * 16 * (kLdT + kLdR) * (int)sizeof(DT);
  const bool fast = a.vec && a.near && a.D == DP;
  // the tiling of the query rows follows the forward pass's rule
  if (attention_plan(a.B, a.Tq, a.Tk, a.heads, a.kv_heads, sizeof(DT) == 2, a.cus).narrow) {
    const auto dq = fast ? attention_dq_step_kernel<DT, DP, true> : attention_dq_step_kernel<DT, DP, false>;
    constexpr int kLds = DqStepShape<DT, DP>::kBytes;
    const hipError_t e = allow_lds(dq, kLds);
    if (e != hipSuccess) return e;
    launch_kernel(dq, dim3((unsigned)work_grid(a, (M + 15) / 16)), dim3(kAttnThreads), kLds, st, a);
  } else {
    const auto dq = fast ? attention_dq_kernel<DT, DP, QT, KT, true> : attention_dq_kernel<DT, DP, QT, KT, false>;
    const hipError_t e = allow_lds(dq, kLdsQ);
    if (e != hipSuccess) return e;
    launch_kernel(dq, dim3((unsigned)work_grid(a, (M + 64 * QT - 1) / (64 * QT))), dim3(kAttnThreads), kLdsQ, st, a);
  }
  if constexpr (sizeof(DT) == 4)
    return run_kv<DT, DP, 1, 1, 2>(a, fast, st);
  else if constexpr (DP <= 64)
    return run_kv<DT, DP, 2, 2, 2>(a, fast, st);
  else
    return run_kv_team<DT, DP, 2, 4>(a, fast, st);
}

template <typename DT>
hipError_t run_t(const AttentionArgs& a, hipStream_t st) {
  if (a.D <= 32) return run<DT, 32>(a, st);
  if (a.D <= 64) return run<DT, 64>(a, st);
  if (a.D <= 96) return run<DT, 96>(a, st);
  return run<DT, 128>(a, st);
}

}  // namespace

hipError_t launch_attention_backward(const AttentionArgs& a, bool bf, hipStream_t st) {
  return bf ? run_t<bf16>(a, st) : run_t<float>(a, st);
}

}  // namespace rnnk
