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

// The running maximum of no scores: finite, so that subtracting it from the
// -inf of a masked score never makes inf - inf.
constexpr float kLowest = -3.402823466e38f;

// WQ x WK waves: WQ sets of QT x 16 query rows, WK parts of the tile's keys,
// KT x 16 keys each.
template <typename DT, int DP, int WQ, int WK, int QT, int KT>
struct Shape {
  static constexpr int kRows = WQ * QT * 16;
  static constexpr int kKeys = WK * KT * 16;
  static constexpr int kLdK = TileShape<DT, DP, false>::kLd;
  static constexpr int kLdV = TileShape<DT, DP, true>::kLd;
  static constexpr int kTile = kKeys * (kLdK + kLdV);  // a tile of keys and its values, kept twice
  static constexpr int kTileBytes = 2 * kTile * (int)sizeof(DT);
  // the join of WK parts: per wave O^T [QT 16][DP + 1 pad] fp32 and m, l
  static constexpr int kJoinBytes = WK > 1 ? WK * WQ * QT * 16 * (DP + 4 + 2) * 4 : 0;
  static constexpr int kBytes = kTileBytes > kJoinBytes ? kTileBytes : kJoinBytes;
  static_assert(kBytes <= 160 * 1024, "LDS of a compute unit");
};

template <typename DT, int DP, int WQ, int WK, int QT, int KT, bool FAST>
__global__ __launch_bounds__(kAttnThreads, 2) void attention_kernel(AttentionArgs a) {
  using S = Shape<DT, DP, WQ, WK, QT, KT>;
  static_assert(WQ * WK * 64 == kAttnThreads, "four waves");
  static_assert(KT % 2 == 0, "pairs of key tiles make a fragment");
  constexpr int kC = DP / 32, kDT = DP / 16;
  extern __shared__ __align__(16) char smem[];
  DT* lk = reinterpret_cast<DT*>(smem);
  DT* lv = lk + S::kKeys * S::kLdK;

  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int tiles_all = (rows.M + S::kRows - 1) / S::kRows * a.splits;
  const Work w = work_of(a, tiles_all);
  if (w.tile >= tiles_all) return;
  const int groups = a.B * a.kv_heads, bh = w.bh;
  const int split = w.tile % a.splits, m0 = w.tile / a.splits * S::kRows;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
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
      q[t][c] = m < rows.M ? load8<DT, FAST>(rows.in<DT>(qb, a.q_t, a.q_h, m), 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
  }
  f32x4 o[QT][kDT];
  float mx[QT], sum[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    mx[t] = kLowest;
    sum[t] = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // A negative scale is taken into q (exactly), a zero one replaced by the
  // smallest positive (2^(s sl) rounds to 1 alike): scores are compared before
  // they are scaled, and the scale rides in the exponent's multiply-add.
  const float sl = __builtin_fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1.17549435e-38f);
  if (a.scale < 0.f) {
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) q[t][c].set(j, -q[t][c].get(j));
  }

  TileLoad<DT, DP, S::kKeys, S::kLdK, FAST> nk;
  TileLoad<DT, DP, S::kKeys, S::kLdV, FAST> nv;
  if (first < last) {
    nk.load(kb, a.k_t, first * S::kKeys, L, a.D, vec);
    nv.load(vb, a.v_t, first * S::kKeys, L, a.D, vec);
    nk.put(lk);
    nv.put(lv);
  }
  __syncthreads();
  for (int tile = first; tile < last; ++tile) {
    const int k0 = tile * S::kKeys;
    const DT* ck = lk + (tile - first & 1) * S::kTile;
    const DT* cv = ck + S::kKeys * S::kLdK;
    if (tile + 1 < last) {
      nk.load(kb, a.k_t, k0 + S::kKeys, L, a.D, vec);
      nv.load(vb, a.v_t, k0 + S::kKeys, L, a.D, vec);
    }
    __builtin_amdgcn_sched_barrier(0);
    f32x4 s[QT][KT];
#pragma unroll
    for (int n = 0; n < KT; ++n) {
#pragma unroll
      for (int t = 0; t < QT; ++t) s[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const Frag<DT> kf = read_rows<DT>(ck, S::kLdK, (wk * KT + n) * 16 + i16, 32 * c + 8 * g);
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t][n] = mma(kf, q[t][c], s[t][n]);
      }
    }
    if (k0 + S::kKeys > L) {
#pragma unroll
      for (int n = 0; n < KT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + (wk * KT + n) * 16 + 4 * g + j >= L) {
#pragma unroll
            for (int t = 0; t < QT; ++t) s[t][n][j] = -__builtin_inff();
          }
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float top = s[t][0][0];
#pragma unroll
      for (int n = 0; n < KT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[t][n][j]);
      // The maximum that is subtracted only has to keep 2^(s - m) in range:
      // it moves when a score passes it by more than 2^kSlack, so most tiles
      // skip the exchange between lanes and the rescaling of o.
      constexpr float kSlack = 8.0f;
      if (__any((top - mx[t]) * sl > kSlack)) {
        top = __builtin_fmaxf(mx[t], col_max(top));
        const float keep = __builtin_amdgcn_exp2f((mx[t] - top) * sl);
        mx[t] = top;
        sum[t] *= keep;
#pragma unroll
        for (int d = 0; d < kDT; ++d) o[t][d] *= keep;
      }
      // s sl - m sl in one multiply-add: the rounding of m sl is the same
      // factor in every p and in their sum. Past 2^20 that rounding is no
      // longer small against 1, and the difference is taken first.
      const float shift = __builtin_fmaxf(mx[t] * sl, kLowest);
      float part = 0.f;
      if (__any(__builtin_fabsf(shift) > 1048576.0f)) {
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t][n][j] = (s[t][n][j] - mx[t]) * sl;
      } else {
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t][n][j] = __builtin_fmaf(s[t][n][j], sl, -shift);
      }
#pragma unroll
      for (int n = 0; n < KT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[t][n][j] = __builtin_amdgcn_exp2f(s[t][n][j]);
          part += s[t][n][j];
        }
      sum[t] += part;  // this lane's keys; the four lanes of a row are joined at the end
    }
    // p is rounded to the storage type here (one rounding of each value, of
    // the relative size of o's own); its sum keeps 32 bits
#pragma unroll
    for (int n = 0; n < KT; n += 2) {
      Frag<DT> p[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) p[t] = stack<DT>(s[t][n], s[t][n + 1]);
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const Frag<DT> vf = read_cols<DT>(cv, S::kLdV, (wk * KT + n) * 16, 16 * d, lane);
#pragma unroll
        for (int t = 0; t < QT; ++t) o[t][d] = mma(vf, p[t], o[t][d]);
      }
    }
    if (tile + 1 < last) {
      DT* dst = lk + (tile + 1 - first & 1) * S::kTile;
      nk.put(dst);
      nv.put(dst + S::kKeys * S::kLdK);
    }
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    sum[t] = col_sum(sum[t]);
    mx[t] = __builtin_fmaxf(mx[t] * sl, kLowest);  // base-2 units from here on, as it was subtracted
  }

  if constexpr (WK > 1) {
    // join the waves' parts of the keys, in order of their number
    constexpr int kLdO = DP + 4;
    float* jo = reinterpret_cast<float*>(smem);
    float* jm = jo + WK * S::kRows * kLdO;
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
      for (int d = 0; d < kDT; ++d) store4<float, FAST>(a.part_o + r * a.D, 16 * d + 4 * g, a.D, a.D % 4 == 0, o[t][d]);
      if (g == 0) a.part_ml[2 * r] = mx[t], a.part_ml[2 * r + 1] = sum[t];
    } else {
      const float inv = sum[t] > 0.f ? 1.0f / sum[t] : (L > 0 ? __builtin_nanf("") : 0.f);
      DT* dst = (DT*)a.o + rows.dense(a, b, hk, m);
#pragma unroll
      for (int d = 0; d < kDT; ++d) store4<DT, FAST>(dst, 16 * d + 4 * g, a.D, vec, o[t][d] * inv);
      if (a.lse && g == 0) a.lse[(int64_t)bh * rows.M + m] = mx[t] + __builtin_amdgcn_logf(sum[t]);
    }
  }
}

// Joins the splits' partial results of one query row: 32 threads across the
// row (four elements each), 8 along the splits, whose sums meet in LDS.
template <typename DT>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttentionArgs a) {
  __shared__ f32x4 lds[kAttnThreads];
  __shared__ float lsum[8];
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int64_t n = (int64_t)a.B * a.kv_heads * rows.M, r = blockIdx.x;
  const int bh = (int)(r / rows.M), m = (int)(r % rows.M);
  const int c = (threadIdx.x & 31) * 4, part = threadIdx.x >> 5;
  // at most 64 splits: a lane each
  const int lane = threadIdx.x & 63;
  float top = lane < a.splits ? a.part_ml[2 * (lane * n + r)] : kLowest;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, k, 64));
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
#pragma unroll 4
  for (int s = part; s < a.splits; s += 8) {
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * (s * n + r)] - top);
    sum += f * a.part_ml[2 * (s * n + r) + 1];
    const float* src = a.part_o + (s * n + r) * a.D;
    if (a.D % 4 == 0) {
      if (c < a.D) acc += f * *reinterpret_cast<const f32x4*>(src + c);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < a.D) acc[j] += f * src[c + j];
    }
  }
  lds[threadIdx.x] = acc;
  if ((threadIdx.x & 31) == 0) lsum[part] = sum;
  __syncthreads();
  if (part != 0) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    acc += lds[k * 32 + threadIdx.x];
    sum += lsum[k];
  }
  const float inv = sum > 0.f ? 1.0f / sum : (key_count(a, bh / a.kv_heads) > 0 ? __builtin_nanf("") : 0.f);
  store4<DT, false>((DT*)a.o + rows.dense(a, bh / a.kv_heads, bh % a.kv_heads, m), c, a.D, a.vec != 0, acc * inv);
  if (a.lse && threadIdx.x == 0) a.lse[r] = top + __builtin_amdgcn_logf(sum);
}

template <typename DT, int DP, int WQ, int WK, int QT, int KT>
hipError_t run(const AttentionArgs& a, hipStream_t st) {
  using S = Shape<DT, DP, WQ, WK, QT, KT>;
  const auto kernel = a.vec && a.near && a.D == DP ? attention_kernel<DT, DP, WQ, WK, QT, KT, true>
                                         : attention_kernel<DT, DP, WQ, WK, QT, KT, false>;
  const int64_t M = (int64_t)a.Tq * (a.heads / a.kv_heads);
  const int64_t grid = work_grid(a, (M + S::kRows - 1) / S::kRows * a.splits);
  const hipError_t e = allow_lds(kernel, S::kBytes);
  if (e != hipSuccess) return e;
  launch_kernel(kernel, dim3((unsigned)grid), dim3(kAttnThreads), S::kBytes, st, a);
  if (a.splits > 1)
    launch_kernel(attention_join_kernel<DT>, dim3((unsigned)(M * a.B * a.kv_heads)), dim3(kAttnThreads), 0, st, a);
  return hipGetLastError();
}

template <typename DT, int DP>
hipError_t run_d(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  if (p.narrow) {
    // two fp32 tiles of 128 wide keys would not fit in LDS
    if constexpr (sizeof(DT) == 4 && DP > 64)
      return run<DT, DP, 2, 2, 1, 2>(a, st);
    else
      return run<DT, DP, 1, 4, 1, 2>(a, st);
  }
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
  // Split the keys while the launch has fewer workgroups than compute units
  // and a split keeps two tiles or more.
  const int64_t groups = (M + p.rows - 1) / p.rows * B * kv_heads;
  const int64_t tiles = ((int64_t)Tk + keys - 1) / keys;
  int64_t want = cus / groups;
  if (want > tiles / 2) want = tiles / 2;
  if (want > 64) want = 64;
  p.splits = want < 1 ? 1 : (int)want;
  return p;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, bool bf, hipStream_t st) {
  return bf ? run_t<bf16>(a, p, st) : run_t<float>(a, p, st);
}

}  // namespace rnnk
