// Cross attention, backward.
//
//   p  = 2^(s - lse),  dp = do v^T,  delta = sum over d of do o
//   ds = p (dp - delta),  dq = scale ds k,  dk = scale ds^T q,  dv = p^T do
//
// Two kernels that each form p again from the kept log-sum-exp: one owns
// query rows and walks the keys (delta, dq), the other owns keys and walks
// the query rows of all heads that share them (dk, dv). So every output has
// one owner and no sum depends on the order in which workgroups run.
#include "attention_common.hpp"

namespace rnnk {
namespace {

// Query rows across (16 per wave and tile), keys down: dq^T = K^T ds^T.
template <typename DT, int DP, int QT, int KT>
__global__ __launch_bounds__(kAttnThreads) void attention_dq_kernel(AttentionArgs a) {
  constexpr int kC = DP / 32, kDT = DP / 16, kRows = 4 * QT * 16, kKeys = KT * 16;
  constexpr int kLdK = TileShape<DT, DP, true>::kLd, kLdV = TileShape<DT, DP, false>::kLd;
  extern __shared__ __align__(16) char smem[];
  DT* lk = reinterpret_cast<DT*>(smem);
  DT* lv = lk + kKeys * kLdK;
  const int groups = a.B * a.kv_heads;
  const int bh = blockIdx.x % groups, m0 = blockIdx.x / groups * kRows;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;
  const int L = key_count(a, b);
  const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;

  Frag<DT> q[QT][kC], dO[QT][kC];
  float lse[QT], delta[QT];
  f32x4 dq[QT][kDT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wave * QT + t) * 16 + i16;
    const bool on = m < rows.M;
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = 32 * c + 8 * g;
      q[t][c] = dO[t][c] = zero_frag<DT>();
      if (on) {
        const int64_t at = rows.dense(a, b, hk, m);
        q[t][c] = load8<DT>(rows.in<DT>(qb, a.q_t, a.q_h, m), col, a.D, vec);
        dO[t][c] = load8<DT>((const DT*)a.d_o + at, col, a.D, vec);
        const Frag<DT> o = load8<DT>((const DT*)a.o + at, col, a.D, vec);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(o.get(j), dO[t][c].get(j), dot);
      }
    }
    delta[t] = col_sum(dot);
    lse[t] = on && L > 0 ? a.lse[(int64_t)bh * rows.M + m] : 0.f;
    if (on && g == 0) a.delta[(int64_t)bh * rows.M + m] = delta[t];
#pragma unroll
    for (int d = 0; d < kDT; ++d) dq[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float sl = a.scale * kLog2e;

  for (int k0 = 0; k0 < L; k0 += kKeys) {
    __syncthreads();
    stage<DT, DP, kKeys, kLdK>(lk, a.D, vec, [&](int r) { return k0 + r < L ? kb + (k0 + r) * a.k_t : nullptr; });
    stage<DT, DP, kKeys, kLdV>(lv, a.D, vec, [&](int r) { return k0 + r < L ? vb + (k0 + r) * a.v_t : nullptr; });
    __syncthreads();
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
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = __builtin_amdgcn_exp2f(s[t][n][j] * sl - lse[t]);
          s[t][n][j] = k0 + n * 16 + 4 * g + j < L ? p * (dp[t][n][j] - delta[t]) : 0.f;
        }
    }
    // ds is rounded to the storage type for the product (see the forward's p)
#pragma unroll
    for (int n = 0; n < KT; n += 2) {
      Frag<DT> ds[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) ds[t] = stack<DT>(s[t][n], s[t][n + 1]);
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const Frag<DT> kf = read_cols<DT>(lk, kLdK, n * 16, 16 * d, lane);
#pragma unroll
        for (int t = 0; t < QT; ++t) dq[t][d] = mma(kf, ds[t], dq[t][d]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wave * QT + t) * 16 + i16;
    if (m >= rows.M) continue;
    DT* dst = (DT*)a.dq + rows.dense(a, b, hk, m);
#pragma unroll
    for (int d = 0; d < kDT; ++d) store4<DT>(dst, 16 * d + 4 * g, a.D, vec, dq[t][d] * a.scale);
  }
}

// Keys across (16 per wave and tile), query rows down: dv^T = do^T p,
// dk^T = Q^T ds.
template <typename DT, int DP, int KT, int MT>
__global__ __launch_bounds__(kAttnThreads) void attention_dkv_kernel(AttentionArgs a) {
  constexpr int kC = DP / 32, kDT = DP / 16, kKeys = 4 * KT * 16, kRows = MT * 16;
  constexpr int kLd = TileShape<DT, DP, true>::kLd;
  extern __shared__ __align__(16) char smem[];
  DT* lq = reinterpret_cast<DT*>(smem);
  DT* ldo = lq + kRows * kLd;
  float* llse = reinterpret_cast<float*>(ldo + kRows * kLd);
  float* ldelta = llse + kRows;
  const int groups = a.B * a.kv_heads;
  const int bh = blockIdx.x % groups, k0 = blockIdx.x / groups * kKeys;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;
  const int L = key_count(a, b);
  const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;

  Frag<DT> k[KT][kC], v[KT][kC];
  f32x4 dk[KT][kDT], dv[KT][kDT];
#pragma unroll
  for (int n = 0; n < KT; ++n) {
    const int key = k0 + (wave * KT + n) * 16 + i16;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      k[n][c] = v[n][c] = zero_frag<DT>();
      if (key < L) {
        k[n][c] = load8<DT>(kb + key * a.k_t, 32 * c + 8 * g, a.D, vec);
        v[n][c] = load8<DT>(vb + key * a.v_t, 32 * c + 8 * g, a.D, vec);
      }
    }
#pragma unroll
    for (int d = 0; d < kDT; ++d) dk[n][d] = dv[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float sl = a.scale * kLog2e;

  if (k0 < L) {
    for (int m0 = 0; m0 < rows.M; m0 += kRows) {
      __syncthreads();
      stage<DT, DP, kRows, kLd>(lq, a.D, vec,
                                [&](int r) { return m0 + r < rows.M ? rows.in<DT>(qb, a.q_t, a.q_h, m0 + r) : nullptr; });
      stage<DT, DP, kRows, kLd>(ldo, a.D, vec, [&](int r) {
        return m0 + r < rows.M ? (const DT*)a.d_o + rows.dense(a, b, hk, m0 + r) : nullptr;
      });
      for (int r = threadIdx.x; r < kRows; r += kAttnThreads) {
        const bool on = m0 + r < rows.M;
        const int64_t at = (int64_t)bh * rows.M + m0 + r;
        llse[r] = on ? a.lse[at] : __builtin_inff();  // 2^-inf: a row past the end has p = 0
        ldelta[r] = on ? a.delta[at] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; mt += 2) {
        f32x4 s[2][KT], dp[2][KT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int n = 0; n < KT; ++n) s[h][n] = dp[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const Frag<DT> qf = read_rows<DT>(lq, kLd, (mt + h) * 16 + i16, 32 * c + 8 * g);
            const Frag<DT> of = read_rows<DT>(ldo, kLd, (mt + h) * 16 + i16, 32 * c + 8 * g);
#pragma unroll
            for (int n = 0; n < KT; ++n) {
              s[h][n] = mma(qf, k[n][c], s[h][n]);
              dp[h][n] = mma(of, v[n][c], dp[h][n]);
            }
          }
          const f32x4 lse = *reinterpret_cast<const f32x4*>(llse + (mt + h) * 16 + 4 * g);
          const f32x4 de = *reinterpret_cast<const f32x4*>(ldelta + (mt + h) * 16 + 4 * g);
#pragma unroll
          for (int n = 0; n < KT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p = __builtin_amdgcn_exp2f(s[h][n][j] * sl - lse[j]);
              s[h][n][j] = p;
              dp[h][n][j] = p * (dp[h][n][j] - de[j]);
            }
        }
        Frag<DT> p[KT], ds[KT];
#pragma unroll
        for (int n = 0; n < KT; ++n) {
          p[n] = stack<DT>(s[0][n], s[1][n]);
          ds[n] = stack<DT>(dp[0][n], dp[1][n]);
        }
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          const Frag<DT> of = read_cols<DT>(ldo, kLd, mt * 16, 16 * d, lane);
          const Frag<DT> qf = read_cols<DT>(lq, kLd, mt * 16, 16 * d, lane);
#pragma unroll
          for (int n = 0; n < KT; ++n) {
            dv[n][d] = mma(of, p[n], dv[n][d]);
            dk[n][d] = mma(qf, ds[n], dk[n][d]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < KT; ++n) {
    const int key = k0 + (wave * KT + n) * 16 + i16;
    if (key >= a.Tk) continue;
    const bool on = key < L;
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    const int64_t at = (((int64_t)key * a.B + b) * a.kv_heads + hk) * a.D;
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      store4<DT>((DT*)a.dk + at, 16 * d + 4 * g, a.D, vec, on ? dk[n][d] * a.scale : z);
      store4<DT>((DT*)a.dv + at, 16 * d + 4 * g, a.D, vec, on ? dv[n][d] : z);
    }
  }
}

template <typename DT, int DP>
hipError_t run(const AttentionArgs& a, hipStream_t st) {
  constexpr int QT = 1, KT = 2, KV = 1, MT = 4;
  const int64_t M = (int64_t)a.Tq * (a.heads / a.kv_heads), groups = (int64_t)a.B * a.kv_heads;
  constexpr int kLdT = TileShape<DT, DP, true>::kLd, kLdR = TileShape<DT, DP, false>::kLd;
  constexpr int kLdsQ = KT * 16 * (kLdT + kLdR) * (int)sizeof(DT);
  constexpr int kLdsKv = MT * 16 * (2 * kLdT * (int)sizeof(DT) + 2 * (int)sizeof(float));
  hipError_t e = allow_lds(attention_dq_kernel<DT, DP, QT, KT>, kLdsQ);
  if (e == hipSuccess) e = allow_lds(attention_dkv_kernel<DT, DP, KV, MT>, kLdsKv);
  if (e != hipSuccess) return e;
  launch_kernel(attention_dq_kernel<DT, DP, QT, KT>, dim3((unsigned)((M + 64 * QT - 1) / (64 * QT) * groups)),
                dim3(kAttnThreads), kLdsQ, st, a);
  launch_kernel(attention_dkv_kernel<DT, DP, KV, MT>, dim3((unsigned)(((int64_t)a.Tk + 64 * KV - 1) / (64 * KV) * groups)),
                dim3(kAttnThreads), kLdsKv, st, a);
  return hipGetLastError();
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
