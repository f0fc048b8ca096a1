// Cross attention, forward.
//
//   o = softmax(scale q k^T) v   over the first L_b keys of a batch row
//
// One pass over the keys with a running reference r (the maximum, or near it)
// and sum l per query row (in base 2: p = 2^(s - r), s = scale log2(e) q k):
//   r' = max(r, max s),  l' = 2^(r - r') l + sum p,  o' = 2^(r - r') o + p v
// r is a float, and everything refers to that float itself, not to the product
// it was rounded from: the tiles before and after it moves, the waves and the
// splits that are joined, and the log-sum-exp. So its rounding, which at large
// scores is not small against 1, cancels in p / l.
//
// The scores are formed transposed, keys down and query rows across (S^T =
// K Q^T), so that a lane keeps one query row: its statistics need two
// exchanges per tile, and p is already the operand of o^T = V^T P^T. The
// query heads that share a key head are rows of the same tile, so K and V
// are read once for all of them; a single-token call has as many rows as
// that group has heads.
//
// 1000 queries x 1000 keys, 32 rows, 8/2 heads of 128, bf16, launches back to
// back: 197 us (665 TFLOP/s of 4 Tq Tk D a head), ragged in training 157 us.
// Neither the matrix units (34% of the SIMD cycles) nor LDS (a quarter) is full:
// two waves a SIMD take turns at products, exponentials and LDS reads and hide
// only part of each other. fp32 at 1000 x 1000, 8 rows, 4 heads of 64: 79 us
// (104 of the 154 TFLOP/s that a large fp32 product reaches).
#include "attention_common.hpp"

namespace rnnk {
namespace {

constexpr int kMaxSplits = 256;

// Four waves of QT x 16 query rows share tiles of KT x 16 keys.
template <typename DT, int DP, int QT, int KT>
struct Shape {
  static constexpr int kRows = 4 * QT * 16;
  static constexpr int kKeys = KT * 16;
  static constexpr int kLdK = TileShape<DT, DP, false>::kLd;
  static constexpr int kLdV = TileShape<DT, DP, true>::kLd;
  static constexpr int kTile = kKeys * (kLdK + kLdV);  // a tile of keys and its values, kept twice
  static constexpr int kBytes = 2 * kTile * (int)sizeof(DT);
  static_assert(kBytes <= 160 * 1024, "LDS of a compute unit");
};

// A negative scale is taken into q (exactly), a zero one replaced by the
// smallest positive (2^(s sl) rounds to 1 alike): scores are compared before
// they are scaled, and the scale rides in the exponent's multiply-add.
template <typename DT, int N>
__device__ __forceinline__ float base2_scale(float scale, Frag<DT> (&q)[N]) {
  if (scale < 0.f) {
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[c].set(j, -q[c].get(j));
  }
  return __builtin_fmaxf(__builtin_fabsf(scale) * kLog2e, 1.17549435e-38f);
}

// Scores of KT tiles of keys (raw, -inf where masked) to probabilities:
// updates the reference and the sum of this lane's query row and rescales its
// part of o. The reference is -inf before the row's first tile and finite from
// then on, so that a masked score never makes inf - inf.
template <int KT, int NO>
__device__ __forceinline__ void softmax_step(f32x4 (&s)[KT], float sl, float* ref, float* sum, f32x4 (&o)[NO]) {
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < KT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[n][j]);
  // The reference only has to keep 2^(s - r) in range: it moves when a score
  // passes it by more than 2^kSlack, so most tiles skip the exchange between
  // lanes and the rescaling of o.
  constexpr float kSlack = 8.0f;
  if (__any(!(__builtin_fmaf(top, sl, -*ref) <= kSlack))) {
    const float next = __builtin_fmaxf(*ref, base2_score(col_max(top), sl));
    const float keep = __builtin_amdgcn_exp2f(*ref - next);
    *ref = next;
    *sum *= keep;
#pragma unroll
    for (int d = 0; d < NO; ++d) o[d] *= keep;
  }
  if (__any(__builtin_fabsf(*ref) > kCoarse)) {
#pragma unroll
    for (int n = 0; n < KT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[n][j] = score_above(s[n][j], sl, *ref);
  } else {
#pragma unroll
    for (int n = 0; n < KT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[n][j] = __builtin_fmaf(s[n][j], sl, -*ref);
  }
  float part = 0.f;
#pragma unroll
  for (int n = 0; n < KT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[n][j] = __builtin_amdgcn_exp2f(s[n][j]);
      part += s[n][j];
    }
  *sum += part;  // this lane's keys; the four lanes of a row are joined at the end
}

// Four elements of o and, in training, what their rounding leaves: delta in
// the backward pass is a sum over o that is taken from values of its own
// size, where the error of a rounded o would show.
template <typename DT, bool FAST>
__device__ __forceinline__ void write_o(const AttentionArgs& a, int64_t at, int col, const f32x4& o) {
  store4<DT, FAST>((DT*)a.o + at, col, a.D, a.vec != 0, o);
  if constexpr (sizeof(DT) == 2) {
    if (a.o_rest) {
      f32x4 rest;
#pragma unroll
      for (int j = 0; j < 4; ++j) rest[j] = o[j] - (float)(bf16)o[j];
      store4<DT, FAST>((DT*)a.o_rest + at, col, a.D, a.vec != 0, rest);
    }
  }
}

// Four elements of each of N column tiles of a query row's result (sum over all lanes), or of its part
// where the keys are split.
template <typename DT, bool FAST, int N>
__device__ __forceinline__ void write_part(const AttentionArgs& a, const QRows& rows, int bh, int split, int m, int L, int col,
                                           float ref, float sum, const f32x4 (&o)[N]) {
  if (a.splits > 1) {
    const int64_t r = ((int64_t)split * a.B * a.kv_heads + bh) * rows.M + m;
#pragma unroll
    for (int d = 0; d < N; ++d) store4<float, FAST>(a.part_o + r * a.D, 16 * d + col, a.D, a.D % 4 == 0, o[d]);
    if (col == 0) a.part_ml[2 * r] = ref, a.part_ml[2 * r + 1] = sum;
    return;
  }
  const float inv = sum > 0.f ? 1.0f / sum : (L > 0 ? __builtin_nanf("") : 0.f);
  const int64_t at = rows.dense(a, bh / a.kv_heads, bh % a.kv_heads, m);
#pragma unroll
  for (int d = 0; d < N; ++d) write_o<DT, FAST>(a, at, 16 * d + col, o[d] * inv);
  if (a.lse && col == 0) a.lse[(int64_t)bh * rows.M + m] = ref + __builtin_amdgcn_logf(sum);
}

template <typename DT, int DP, int QT, int KT, bool FAST>
__global__ __launch_bounds__(kAttnThreads, 2) void attention_kernel(AttentionArgs a) {
  using S = Shape<DT, DP, QT, KT>;
  static_assert(KT % 2 == 0, "pairs of key tiles make a fragment");
  constexpr int kC = DP / 32, kDT = DP / 16;
  extern __shared__ __align__(16) char smem[];
  DT* lk = reinterpret_cast<DT*>(smem);
  DT* lv = lk + S::kKeys * S::kLdK;

  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int tiles_all = (rows.M + S::kRows - 1) / S::kRows * a.splits;
  const Work w = work_of(a, tiles_all);
  if (w.tile >= tiles_all) return;
  const int bh = w.bh, split = w.tile % a.splits, m0 = w.tile / a.splits * S::kRows;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;

  const int L = key_count(a, b);
  const int tiles = (L + S::kKeys - 1) / S::kKeys;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int first = split * per, last = first + per < tiles ? first + per : tiles;

  const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;

  Frag<DT> q[QT][kC];
  f32x4 o[QT][kDT];
  float ref[QT], sum[QT], sl = 0.f;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = m0 + (wave * QT + t) * 16 + i16;
    const DT* row = rows.in<DT>(qb, a.q_t, a.q_h, m < rows.M ? m : 0);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      q[t][c] = load8<DT, FAST>(row, 32 * c + 8 * g, a.D, vec);
      if (m >= rows.M) q[t][c] = zero_frag<DT>();
    }
    sl = base2_scale<DT, kC>(a.scale, q[t]);
    ref[t] = -__builtin_inff();
    sum[t] = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
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
    // the wave whose products are ready goes first: the other's exponentials
    // fill in (2 to 4% at 1000 to 2048 keys)
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int n = 0; n < KT; ++n) {
#pragma unroll
      for (int t = 0; t < QT; ++t) s[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const Frag<DT> kf = read_rows<DT>(ck, S::kLdK, n * 16 + i16, 32 * c + 8 * g);
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t][n] = mma(kf, q[t][c], s[t][n]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (k0 + S::kKeys > L) {
#pragma unroll
      for (int n = 0; n < KT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + n * 16 + 4 * g + j >= L) {
#pragma unroll
            for (int t = 0; t < QT; ++t) s[t][n][j] = -__builtin_inff();
          }
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) softmax_step<KT, kDT>(s[t], sl, &ref[t], &sum[t], o[t]);
    // p in bf16 enters the product as its rounded value and the rest of the
    // rounding, so that o is as exact as its own rounding. With the rounded
    // value alone 1000 x 1000, 32 ragged rows, 8/2 heads of 128 takes 133 us
    // for 157, with o 1.4 times as far off and the backward pass's delta, a
    // sum over o, up to 1.9 times where there are few keys.
#pragma unroll
    for (int n = 0; n < KT; n += 2) {
      constexpr bool kRest = sizeof(DT) == 2;
      Frag<DT> p[QT], rest[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        p[t] = stack<DT>(s[t][n], s[t][n + 1]);
        if constexpr (kRest) rest[t] = stack_rest(s[t][n], s[t][n + 1], p[t]);
      }
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const Frag<DT> vf = read_cols<DT>(cv, S::kLdV, n * 16, 16 * d, lane);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          o[t][d] = mma(vf, p[t], o[t][d]);
          if constexpr (kRest) o[t][d] = mma(vf, rest[t], o[t][d]);
        }
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
    const int m = m0 + (wave * QT + t) * 16 + i16;
    const float total = col_sum(sum[t]);
    if (m < rows.M) write_part<DT, FAST, kDT>(a, rows, bh, split, m, L, 4 * g, ref[t], total, o[t]);
  }
}

// 16 query rows a workgroup (one token, with the heads that share a key head;
// or a few tiles of them where wider ones would leave compute units idle;
// for one tile bound by the reading of K and V, each used once: 64 requests
// over 2000 states of 8 heads of 64, bf16, 44 to 47 us = 5.6 to 6 TB/s, more
// than a large copy; over 500 ragged ones 10 us, mostly latency; fp32, 2000
// states, 97 us = 5.4 TB/s). The waves
// divide the keys, 32 at a time, and never wait for each other before the
// end: keys go from memory straight into fragments, values through a wave's
// own piece of LDS, which turns them. A step's keys are loaded as soon as the
// ones before have been used, and its values likewise.
constexpr int kStepKeys = 32, kStepThreads = 256;
template <typename DT, int DP>
struct StepShape {
  static constexpr int kWaves = kStepThreads / 64;
  static constexpr int kLdV = TileShape<DT, DP, true>::kLd, kLdO = DP + 4;
  static constexpr int kBytesV = kWaves * kStepKeys * kLdV * (int)sizeof(DT), kBytesO = kWaves * 16 * (kLdO + 2) * 4;
  static constexpr int kBytes = kBytesV > kBytesO ? kBytesV : kBytesO;
};
template <typename DT, int DP, bool FAST>
__global__ __launch_bounds__(kStepThreads, 2) void attention_step_kernel(AttentionArgs a) {
  using S = StepShape<DT, DP>;
  constexpr int kC = DP / 32, kDT = DP / 16, kWaves = S::kWaves, kLdV = S::kLdV, kLdO = S::kLdO;
  constexpr int kCols = DP / 8, kV = kStepKeys * kCols / 64;  // a lane's pieces of a step's values
  extern __shared__ __align__(16) char smem[];

  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int tiles_all = (rows.M + 15) / 16 * a.splits;
  const Work w = work_of(a, tiles_all);
  if (w.tile >= tiles_all) return;
  const int bh = w.bh, split = w.tile % a.splits, m0 = w.tile / a.splits * 16;
  const int b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
  const bool vec = a.vec != 0;
  const DT* kb = (const DT*)a.k + b * a.k_b + hk * a.k_h;
  const DT* vb = (const DT*)a.v + b * a.v_b + hk * a.v_h;
  DT* lv = reinterpret_cast<DT*>(smem) + wave * kStepKeys * kLdV;

  const int L = key_count(a, b);
  const int per = ((L + a.splits - 1) / a.splits + kStepKeys - 1) / kStepKeys * kStepKeys;
  const int first = split * per, last = first + per < L ? first + per : L;

  Frag<DT> k[2][kC], v[kV];
  auto load_k = [&](int k0) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int key = k0 + 16 * n + i16;
#pragma unroll
      for (int c = 0; c < kC; ++c)
        k[n][c] = key < last ? load8<DT, FAST>(kb + key * a.k_t, 32 * c + 8 * g, a.D, vec) : zero_frag<DT>();
    }
  };
  auto load_v = [&](int k0) {
#pragma unroll
    for (int n = 0; n < kV; ++n) {
      const int p = n * 64 + lane, key = k0 + p / kCols;
      v[n] = key < last ? load8<DT, FAST>(vb + key * a.v_t, p % kCols * 8, a.D, vec) : zero_frag<DT>();
    }
  };
  int k0 = first + wave * kStepKeys;
  load_k(k0);
  load_v(k0);
  Frag<DT> q[kC];
  {
    const DT* qb = (const DT*)a.q + b * a.q_b + (int64_t)hk * rows.G * a.q_h;
    const bool on = m0 + i16 < rows.M;
    const DT* row = rows.in<DT>(qb, a.q_t, a.q_h, on ? m0 + i16 : 0);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      q[c] = load8<DT, FAST>(row, 32 * c + 8 * g, a.D, vec);
      if (!on) q[c] = zero_frag<DT>();
    }
  }
  const float sl = base2_scale<DT, kC>(a.scale, q);
  f32x4 o[kDT];
#pragma unroll
  for (int d = 0; d < kDT; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  float ref = -__builtin_inff(), sum = 0.f;
  for (; k0 < last; k0 += kWaves * kStepKeys) {
    f32x4 s[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) s[n] = mma(k[n][c], q[c], s[n]);
    }
    load_k(k0 + kWaves * kStepKeys);
    if (k0 + kStepKeys > last) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + n * 16 + 4 * g + j >= last) s[n][j] = -__builtin_inff();
    }
    softmax_step<2, kDT>(s, sl, &ref, &sum, o);
    // the wave's own reads of the step before are done: they fed products
    // that were issued before these writes
#pragma unroll
    for (int n = 0; n < kV; ++n) {
      const int p = n * 64 + lane;
      put8<DT>(lv + p / kCols * kLdV + p % kCols * 8, v[n]);
    }
    load_v(k0 + kWaves * kStepKeys);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const Frag<DT> p = stack<DT>(s[0], s[1]);
    Frag<DT> rest;
    if constexpr (sizeof(DT) == 2) rest = stack_rest(s[0], s[1], p);  // p is not rounded here: the products are not what takes time
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      const Frag<DT> vf = read_cols<DT>(lv, kLdV, 0, 16 * d, lane);
      o[d] = mma(vf, p, o[d]);
      if constexpr (sizeof(DT) == 2) o[d] = mma(vf, rest, o[d]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  sum = col_sum(sum);

  // join the waves' parts, in order of their number: four elements of a row
  // per thread
  float* jo = reinterpret_cast<float*>(smem);
  float* jm = jo + kWaves * 16 * kLdO;
  __syncthreads();
  const int r = wave * 16 + i16;
#pragma unroll
  for (int d = 0; d < kDT; ++d) *reinterpret_cast<f32x4*>(jo + r * kLdO + 16 * d + 4 * g) = o[d];
  if (g == 0) jm[2 * r] = ref, jm[2 * r + 1] = sum;
  __syncthreads();
  for (int k = threadIdx.x; k < 16 * (DP / 4); k += kStepThreads) {
    const int m = k / (DP / 4), col = k % (DP / 4) * 4;
    if (m0 + m >= rows.M) return;
    float top = kLowest;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) top = __builtin_fmaxf(top, jm[2 * (x * 16 + m)]);
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    float total = 0.f;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
      const int rr = x * 16 + m;
      const float f = __builtin_amdgcn_exp2f(jm[2 * rr] - top);
      total += f * jm[2 * rr + 1];
      acc[0] += f * *reinterpret_cast<const f32x4*>(jo + rr * kLdO + col);
    }
    write_part<DT, FAST, 1>(a, rows, bh, split, m0 + m, L, col, top, total, acc);
  }
}

// Joins the splits' partial results of one query row: a thread per split for
// the weights, then 32 threads across the row (four elements each) by 8 along
// the splits, whose sums meet in LDS.
template <typename DT>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttentionArgs a) {
  static_assert(kMaxSplits <= kAttnThreads, "a thread per split");
  __shared__ f32x4 lds[kAttnThreads];
  __shared__ float weight[kAttnThreads], wtop[4], wsum[4];
  const QRows rows{a.Tq * (a.heads / a.kv_heads), a.heads / a.kv_heads};
  const int64_t n = (int64_t)a.B * a.kv_heads * rows.M, r = blockIdx.x;
  const int bh = (int)(r / rows.M), m = (int)(r % rows.M);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const bool on = (int)threadIdx.x < a.splits;
  const float mine = on ? a.part_ml[2 * (threadIdx.x * n + r)] : kLowest;
  const float part = on ? a.part_ml[2 * (threadIdx.x * n + r) + 1] : 0.f;
  float top = __builtin_fmaxf(mine, kLowest);  // finite where every part is empty
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, k, 64));
  if (lane == 0) wtop[wave] = top;
  __syncthreads();
  top = __builtin_fmaxf(__builtin_fmaxf(wtop[0], wtop[1]), __builtin_fmaxf(wtop[2], wtop[3]));
  const float f = __builtin_amdgcn_exp2f(mine - top);
  weight[threadIdx.x] = f;
  float sum = f * part;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k, 64);
  if (lane == 0) wsum[wave] = sum;
  __syncthreads();
  const int c = (threadIdx.x & 31) * 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (a.D % 4 == 0) {
    if (c < a.D) {
#pragma unroll 8
      for (int s = threadIdx.x >> 5; s < a.splits; s += 8)
        acc += weight[s] * *reinterpret_cast<const f32x4*>(a.part_o + (s * n + r) * a.D + c);
    }
  } else {
    for (int s = threadIdx.x >> 5; s < a.splits; s += 8)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < a.D) acc[j] += weight[s] * a.part_o[(s * n + r) * a.D + c + j];
  }
  lds[threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.x >= 32) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) acc += lds[k * 32 + threadIdx.x];
  sum = (wsum[0] + wsum[1]) + (wsum[2] + wsum[3]);
  const float inv = sum > 0.f ? 1.0f / sum : (key_count(a, bh / a.kv_heads) > 0 ? __builtin_nanf("") : 0.f);
  write_o<DT, false>(a, rows.dense(a, bh / a.kv_heads, bh % a.kv_heads, m), c, acc * inv);
  if (a.lse && threadIdx.x == 0) a.lse[r] = top + __builtin_amdgcn_logf(sum);
}

template <typename DT, int DP>
hipError_t run(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  constexpr int QT = sizeof(DT) == 2 ? 2 : 1, KT = sizeof(DT) == 2 ? 4 : 2;
  using S = Shape<DT, DP, QT, KT>;
  const bool fast = a.vec && a.near && a.D == DP;
  const int64_t M = (int64_t)a.Tq * (a.heads / a.kv_heads);
  if (p.narrow) {
    const auto kernel = fast ? attention_step_kernel<DT, DP, true> : attention_step_kernel<DT, DP, false>;
    const hipError_t e = allow_lds(kernel, StepShape<DT, DP>::kBytes);
    if (e != hipSuccess) return e;
    launch_kernel(kernel, dim3((unsigned)work_grid(a, (M + 15) / 16 * a.splits)), dim3(kStepThreads), StepShape<DT, DP>::kBytes, st, a);
  } else {
    const auto kernel = fast ? attention_kernel<DT, DP, QT, KT, true> : attention_kernel<DT, DP, QT, KT, false>;
    const hipError_t e = allow_lds(kernel, S::kBytes);
    if (e != hipSuccess) return e;
    launch_kernel(kernel, dim3((unsigned)work_grid(a, (M + S::kRows - 1) / S::kRows * a.splits)), dim3(kAttnThreads),
                  S::kBytes, st, a);
  }
  if (a.splits > 1)
    launch_kernel(attention_join_kernel<DT>, dim3((unsigned)(M * a.B * a.kv_heads)), dim3(kAttnThreads), 0, st, a);
  return hipGetLastError();
}

template <typename DT>
hipError_t run_t(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  if (a.D <= 32) return run<DT, 32>(a, p, st);
  if (a.D <= 64) return run<DT, 64>(a, p, st);
  if (a.D <= 96) return run<DT, 96>(a, p, st);
  return run<DT, 128>(a, p, st);
}

}  // namespace

AttentionPlan attention_plan(int B, int Tq, int Tk, int heads, int kv_heads, bool bf, int cus) {
  const int64_t M = (int64_t)Tq * (heads / kv_heads);
  AttentionPlan p{};
  const int wide = bf ? 128 : 64;
  const int64_t heads_all = (int64_t)B * kv_heads;
  // Narrow also while its workgroups are at most three a compute unit and walk
  // few steps. Measured (us, narrow / wide tiles, 4 heads), forward at 500
  // keys: heads of 64, 512 workgroups, bf16 10.4 / 23.5, fp32 19.3 / 30.0; 768:
  // 12.5 / 16.2, 25.5 / 30.7; 992: 15.2 / 16.3, 31.5 / 31.5; heads of 128, 768:
  // 21.5 / 22.5, 50.5 / 49.5; 992: 26.5 / 23.1, 64.2 / 52.0. Backward, whose dq
  // follows the same rule (1000 keys): heads of 64, 512 workgroups, bf16 47.8 /
  // 56.4, fp32 99 / 130; 768: 67.7 / 69.5, 139 / 151; 992: 85.0 / 78.5, 178 /
  // 178; heads of 128, 768: 130 / 126, 351 / 363; 992: 168 / 151, 464 / 426.
  // 4000 keys, 8 heads of 128, 152 workgroups, bf16, forward: 42.6 / 28.8.
  p.narrow = M <= 16 || ((M + 15) / 16 * heads_all <= 3ll * cus && Tk <= 8 * kStepKeys * kStepThreads / 64);
  const int rows = p.narrow ? 16 : wide;
  // A split of the keys keeps two tiles (narrow: a step of every wave) or more.
  const int keys = p.narrow ? kStepKeys * kStepThreads / 64 : bf ? 128 : 64;
  const int64_t groups = (M + rows - 1) / rows * heads_all;
  // Split while there are fewer workgroups than compute units.
  int64_t want = cus / groups;
  if (want > Tk / keys) want = Tk / keys;
  if (want > kMaxSplits) want = kMaxSplits;
  p.splits = want < 1 ? 1 : (int)want;
  return p;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, bool bf, hipStream_t st) {
  return bf ? run_t<bf16>(a, p, st) : run_t<float>(a, p, st);
}

}  // namespace rnnk
