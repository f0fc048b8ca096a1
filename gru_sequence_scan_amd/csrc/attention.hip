// Cross attention, forward.
//
//   o = softmax(scale q k^T) v   over the first L_b keys of a batch row
//
// One pass over the keys with a running maximum m and sum l per query row
// (in base 2: p = 2^(s - m), s = scale log2(e) q k):
//   m' = max(m, max s),  l' = 2^(m - m') l + sum p,  o' = 2^(m - m') o + p v
//
// The scores are formed transposed, keys down and query rows across (S^T =
// K Q^T), so that a lane keeps one query row: its statistics need two
// exchanges per tile, and p is already the operand of o^T = V^T P^T. The
// query heads that share a key head are rows of the same tile, so K and V
// are read once for all of them; a single-token call has as many rows as
// that group has heads.
#include "attention_common.hpp"

namespace rnnk {
namespace {

// WQ x WK waves: WQ sets of QT x 16 query rows, WK parts of the tile's keys,
// KT x 16 keys each.
template <typename DT, int DP, int WQ, int WK, int QT, int KT>
struct Shape {
  static constexpr int kRows = WQ * QT * 16;
  static constexpr int kKeys = WK * KT * 16;
  static constexpr int kLdK = TileShape<DT, DP, false>::kLd;
  static constexpr int kLdV = TileShape<DT, DP, true>::kLd;
  static constexpr int kTileBytes = kKeys * (kLdK + kLdV) * (int)sizeof(DT);
  // the join of WK parts: per wave O^T [QT 16][DP + 1 pad] fp32 and m, l
  static constexpr int kJoinBytes = WK > 1 ? WK * WQ * QT * 16 * (DP + 4 + 2) * 4 : 0;
  static constexpr int kBytes = kTileBytes > kJoinBytes ? kTileBytes : kJoinBytes;
};

template <typename DT, int DP, int WQ, int WK, int QT, int KT>
__global__ __launch_bounds__(kAttnThreads) void attention_kernel(AttentionArgs a) {
  using S = Shape<DT, DP, WQ, WK, QT, KT>;
  static_assert(WQ * WK * 64 == kAttnThreads, "four waves");
  static_assert(KT % 2 == 0, "pairs of key tiles make a fragment");
  constexpr int kC = DP / 32, kDT = DP / 16;
  extern __shared__ __align__(16) char smem[];
  DT* lk = reinterpret_cast<DT*>(smem);
  DT* lv = lk + S::kKeys * S::kLdK;

  const int groups = a.B * a.kv_heads;
  int id = blockIdx.x;
  const int bh = id % groups;  // neighbours in launch order (one XCD in turn) keep one (row, head)'s keys in their L2
  id /= groups;
  const int split = id % a.splits, m0 = id / a.splits * S::kRows;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wq = wave % WQ, wk = wave / WQ, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;

  const int L = key_count(a, b);
  const int tiles = (L + S::kKeys - 1) / S::kKeys;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int first = split * per, last = first + per < tiles ? first + per : tiles;

  const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;

  Frag<DT> q[QT][kC];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wq * QT + t) * 16 + i16;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      q[t][c] = m < rows.M ? load8<DT>(rows.in<DT>(qb, a.q_t, a.q_h, m), 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
  }
  f32x4 o[QT][kDT];
  float mx[QT], sum[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    // the lowest finite value: subtracting it never makes inf - inf
    mx[t] = -3.402823466e38f;
    sum[t] = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float sl = a.scale * kLog2e;

  for (int tile = first; tile < last; ++tile) {
    const int k0 = tile * S::kKeys;
    __syncthreads();
    stage<DT, DP, S::kKeys, S::kLdK>(lk, a.D, vec, [&](int r) { return k0 + r < L ? kb + (k0 + r) * a.k_t : nullptr; });
    stage<DT, DP, S::kKeys, S::kLdV>(lv, a.D, vec, [&](int r) { return k0 + r < L ? vb + (k0 + r) * a.v_t : nullptr; });
    __syncthreads();
    f32x4 s[QT][KT];
#pragma unroll
    for (int n = 0; n < KT; ++n) {
#pragma unroll
      for (int t = 0; t < QT; ++t) s[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const Frag<DT> kf = read_rows<DT>(lk, S::kLdK, (wk * KT + n) * 16 + i16, 32 * c + 8 * g);
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t][n] = mma(kf, q[t][c], s[t][n]);
      }
    }
    const bool edge = k0 + S::kKeys > L;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float top = mx[t];
#pragma unroll
      for (int n = 0; n < KT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[t][n][j] *= sl;
          if (edge && k0 + (wk * KT + n) * 16 + 4 * g + j >= L) s[t][n][j] = -__builtin_inff();
          top = __builtin_fmaxf(top, s[t][n][j]);
        }
      top = col_max(top);
      const float keep = __builtin_amdgcn_exp2f(mx[t] - top);
      mx[t] = top;
      float part = 0.f;
#pragma unroll
      for (int n = 0; n < KT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[t][n][j] = __builtin_amdgcn_exp2f(s[t][n][j] - top);
          part += s[t][n][j];
        }
      sum[t] = sum[t] * keep + part;  // this lane's keys; the four lanes of a row are joined at the end
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[t][d] *= keep;
    }
    // p is rounded to the storage type here (one rounding of a value in
    // [0, 1], no worse than the rounding of o); its sum keeps 32 bits
#pragma unroll
    for (int n = 0; n < KT; n += 2) {
      Frag<DT> p[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) p[t] = stack<DT>(s[t][n], s[t][n + 1]);
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const Frag<DT> vf = read_cols<DT>(lv, S::kLdV, (wk * KT + n) * 16, 16 * d, lane);
#pragma unroll
        for (int t = 0; t < QT; ++t) o[t][d] = mma(vf, p[t], o[t][d]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) sum[t] = col_sum(sum[t]);

  if constexpr (WK > 1) {
    // join the waves' parts of the keys, in order of their number
    constexpr int kLdO = DP + 4;
    float* jo = reinterpret_cast<float*>(smem);
    float* jm = jo + WK * S::kRows * kLdO;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int r = wk * S::kRows + (wq * QT + t) * 16 + i16;
#pragma unroll
      for (int d = 0; d < kDT; ++d) *reinterpret_cast<f32x4*>(jo + r * kLdO + 16 * d + 4 * g) = o[t][d];
      if (g == 0) jm[2 * r] = mx[t], jm[2 * r + 1] = sum[t];
    }
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int r = (wq * QT + t) * 16 + i16;
      float top = mx[t];
#pragma unroll
      for (int w = 1; w < WK; ++w) top = __builtin_fmaxf(top, jm[2 * (w * S::kRows + r)]);
      const float keep = __builtin_amdgcn_exp2f(mx[t] - top);
      sum[t] *= keep;
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[t][d] *= keep;
#pragma unroll
      for (int w = 1; w < WK; ++w) {
        const int rr = w * S::kRows + r;
        const float f = __builtin_amdgcn_exp2f(jm[2 * rr] - top);
        sum[t] += f * jm[2 * rr + 1];
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(jo + rr * kLdO + 16 * d + 4 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[t][d][j] += f * v[j];
        }
      }
      mx[t] = top;
    }
  }

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wq * QT + t) * 16 + i16;
    if (m >= rows.M) continue;
    if (a.splits > 1) {
      const int64_t r = ((int64_t)split * groups + bh) * rows.M + m;
#pragma unroll
      for (int d = 0; d < kDT; ++d) store4<float>(a.part_o + r * a.D, 16 * d + 4 * g, a.D, a.D % 4 == 0, o[t][d]);
      if (g == 0) a.part_ml[2 * r] = mx[t], a.part_ml[2 * r + 1] = sum[t];
    } else {
      const float inv = sum[t] > 0.f ? 1.0f / sum[t] : (L > 0 ? __builtin_nanf("") : 0.f);
      DT* dst = (DT*)a.o + rows.dense(a, b, hk, m);
#pragma unroll
      for (int d = 0; d < kDT; ++d) store4<DT>(dst, 16 * d + 4 * g, a.D, vec, o[t][d] * inv);
      if (a.lse && g == 0) a.lse[(int64_t)bh * rows.M + m] = mx[t] + __builtin_amdgcn_logf(sum[t]);
    }
  }
}

// Joins the splits' partial results, in order: one wave per query row.
template <typename DT>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttentionArgs a) {
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int groups = a.B * a.kv_heads, lane = threadIdx.x & 63;
  const int64_t n = (int64_t)groups * rows.M;
  const int64_t r = blockIdx.x * (int64_t)(kAttnThreads / 64) + (threadIdx.x >> 6);
  if (r >= n) return;
  const int bh = (int)(r / rows.M), m = (int)(r % rows.M);
  const int L = key_count(a, bh / a.kv_heads);
  float top = -3.402823466e38f, sum = 0.f;
  for (int s = 0; s < a.splits; ++s) top = __builtin_fmaxf(top, a.part_ml[2 * (s * n + r)]);
  float acc[2] = {0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * (s * n + r)] - top);
    sum += f * a.part_ml[2 * (s * n + r) + 1];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + 64 * k < a.D) acc[k] += f * a.part_o[(s * n + r) * a.D + lane + 64 * k];
  }
  const float inv = sum > 0.f ? 1.0f / sum : (L > 0 ? __builtin_nanf("") : 0.f);
  DT* dst = (DT*)a.o + rows.dense(a, bh / a.kv_heads, bh % a.kv_heads, m);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 64 * k < a.D) dst[lane + 64 * k] = from_f32<DT>(acc[k] * inv);
  if (a.lse && lane == 0) a.lse[r] = top + __builtin_amdgcn_logf(sum);
}

template <typename DT, int DP, int WQ, int WK, int QT, int KT>
hipError_t run(const AttentionArgs& a, hipStream_t st) {
  using S = Shape<DT, DP, WQ, WK, QT, KT>;
  const int64_t M = (int64_t)a.Tq * (a.heads / a.kv_heads);
  const int64_t grid = (M + S::kRows - 1) / S::kRows * a.splits * a.B * a.kv_heads;
  const hipError_t e = allow_lds(attention_kernel<DT, DP, WQ, WK, QT, KT>, S::kBytes);
  if (e != hipSuccess) return e;
  launch_kernel(attention_kernel<DT, DP, WQ, WK, QT, KT>, dim3((unsigned)grid), dim3(kAttnThreads), S::kBytes, st, a);
  if (a.splits > 1) {
    const int64_t r = M * a.B * a.kv_heads;
    launch_kernel(attention_join_kernel<DT>, dim3((unsigned)((r + 3) / 4)), dim3(kAttnThreads), 0, st, a);
  }
  return hipGetLastError();
}

template <typename DT, int DP>
hipError_t run_d(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  if (p.narrow) return run<DT, DP, 1, 4, 1, 2>(a, st);
  if constexpr (sizeof(DT) == 2)
    return run<DT, DP, 4, 1, 2, 4>(a, st);
  else
    return run<DT, DP, 4, 1, 1, 2>(a, st);
}

template <typename DT>
hipError_t run_t(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  if (a.D <= 32) return run_d<DT, 32>(a, p, st);
  if (a.D <= 64) return run_d<DT, 64>(a, p, st);
  if (a.D <= 96) return run_d<DT, 96>(a, p, st);
  return run_d<DT, 128>(a, p, st);
}

}  // namespace

AttentionPlan attention_plan(int B, int Tq, int Tk, int heads, int kv_heads, bool bf, int cus) {
  const int64_t M = (int64_t)Tq * (heads / kv_heads);
  AttentionPlan p{};
  p.narrow = M <= 16;
  p.rows = p.narrow ? 16 : bf ? 128 : 64;
  const int keys = p.narrow ? 128 : bf ? 64 : 32;
  // Split the keys while the launch has fewer workgroups than two a compute
  // unit and a split keeps two tiles or more.
  const int64_t groups = (M + p.rows - 1) / p.rows * B * kv_heads;
  const int64_t tiles = ((int64_t)Tk + keys - 1) / keys;
  int64_t want = (2ll * cus + groups - 1) / groups;
  if (want > tiles / 2) want = tiles / 2;
  if (want > 64) want = 64;
  p.splits = want < 1 ? 1 : (int)want;
  return p;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, bool bf, hipStream_t st) {
  return bf ? run_t<bf16>(a, p, st) : run_t<float>(a, p, st);
}

}  // namespace rnnk
