// Gated feed-forward: the kernels for few rows, and the copies and sums around
// the products (feed_forward_gemm.hpp; how those are tiled and split is in
// feed_forward_plan.hpp).
//
//   g | u = x W_in^T,  h = act(g) u,  y = h W_out^T (+ residual)
//
//   dh = dy W_out,  dg = dh u act'(g),  du = dh act(g)
//   dx = [dg du] W_in,  dW_in = [dg du]^T x,  dW_out = dy^T h
//
// g and u meet in the first product's accumulators and dg and du come out of
// dh's: neither g and u (in the forward alone) nor dh is ever in memory. h, dg
// and du are rounded to the storage type once, where they leave the
// accumulators: they are operands of matrix instructions of that type. So y,
// dx and the weights' gradients carry one rounding of their terms beside
// their own, sqrt(2) times the latter alone. Training keeps g and u in fp32
// (8 bytes a hidden unit and row): rounded, they would put two more roundings
// into every gradient.
#include "attention_common.hpp"
#include "feed_forward_gemm.hpp"

namespace rnnk {
namespace {

// ---------------------------------------------------------------------------
// Few rows. The weights' way from memory is what counts: a workgroup takes 16
// hidden units (32 rows of W_in), or 16 outputs, over all rows of x, its waves
// divide the summed dimension, and their sums meet in LDS. The weights are the
// first operand of the 16x16 instructions and go straight from memory into
// registers; a result lane holds four neighbouring hidden units of one row.
// One row, 1024 x 2816, bf16: 5.5 us for g | u (2.1 TB/s of weights) and 5.8
// for y, most of it the way of one load and of the sums through LDS; fp32 9.5
// and 9.6. 64 rows, 1024 x 4096, bf16: 10.6, 8.6 and 3.9 us for adding up the
// divided sums, fp32 23.0, 14.7 and 4.0: with four blocks of rows the registers
// hold two of a wave's steps, so that its four are two trips to memory.
// ---------------------------------------------------------------------------
constexpr int kInWaves = 8, kOutWaves = 16;

template <typename DT>
__device__ __forceinline__ void store4(DT* p, const f32x4& v, int n) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (r < n) p[r] = from_f32<DT>(v[r]);
}

// Eight elements of a row of K from `col` on, zeros behind its end. Rows may
// begin at any element: they are read 16 bytes a load all the same, which
// global memory takes at any address, and nothing about a load is conditional:
// what would pass the row's end is read so that it stops there, and moved down
// where it is used. One row, 1024 x 2816: 11.4 us of both products in bf16 and
// 18.0 in fp32; 1024 x 2815, whose rows of W_out begin anywhere: 16.7 and 18.5
// (36 and 41 with one element a load, and every operand read so where one of
// them was not aligned); 64 rows, 2047 x 8191, fp32: 136 (215; 127 at 2048 x 8192).
template <typename DT>
struct FewChunk {
  static constexpr int E = 16 / (int)sizeof(DT), kLoads = 8 / E;
  struct __attribute__((packed, aligned(sizeof(DT)))) Any {
    u32x4 v;
  };
  u32x4 r[kLoads];
  __device__ __forceinline__ void load(const DT* row, int col, int K) {
    if (K < E) {  // a row of less than 16 bytes
#pragma unroll
      for (int h = 0; h < kLoads; ++h) {
        DT v[E];
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = col + h * E + j < K ? row[col + h * E + j] : (DT)0.f;
        __builtin_memcpy(&r[h], v, 16);
      }
      return;
    }
#pragma unroll
    for (int h = 0; h < kLoads; ++h) {
      const int c = col + h * E;
      r[h] = reinterpret_cast<const Any*>(row + (c + E <= K ? c : K - E))->v;
    }
  }
  __device__ __forceinline__ void end(int col, int K) {
    if (K < E) return;
#pragma unroll
    for (int h = 0; h < kLoads; ++h) {
      const int over = col + (h + 1) * E - K, by = over < 0 ? 0 : over < E ? over : E;  // elements that are not the row's
      u32x4 v = r[h];
      if constexpr (sizeof(DT) == 2) {
        if (by & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
      }
      constexpr int kOne = 4 / (int)sizeof(DT);  // elements of a word
      if (by & kOne) v = u32x4{v[1], v[2], v[3], 0u};
      if (by & 2 * kOne) v = u32x4{v[2], v[3], 0u, 0u};
      if (by & 4 * kOne) v = u32x4{0u, 0u, 0u, 0u};
      r[h] = v;
    }
  }
  __device__ __forceinline__ Frag<DT> frag() const {
    Frag<DT> f;
    __builtin_memcpy(&f.v, r, sizeof(r));
    return f;
  }
};

// acc[w][t] = the weights' rows (w of 16 each) times 16 rows of x (t), over
// this wave's share of the steps [first, steps) of 32.
template <typename DT, int NW, int MT, int WAVES, int DEEP>
__device__ __forceinline__ void few_product(f32x4 (&acc)[NW][MT], const DT* (&wrow)[NW], const DT* (&xrow)[MT], int K, int KX,
                                            int first, int steps, int wave, int group) {
#pragma unroll
  for (int w = 0; w < NW; ++w)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[w][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = first + wave; s0 < steps; s0 += WAVES * DEEP) {
    FewChunk<DT> fw[DEEP][NW], fx[DEEP][MT];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int step = s0 + d * WAVES, col = step * 32 + 8 * group;
      if (step >= steps) break;
#pragma unroll
      for (int w = 0; w < NW; ++w) fw[d][w].load(wrow[w], col, K);
#pragma unroll
      for (int t = 0; t < MT; ++t) fx[d][t].load(xrow[t], col, KX);
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int step = s0 + d * WAVES, col = step * 32 + 8 * group;
      if (step >= steps) break;
      if (step * 32 + 32 > K) {
#pragma unroll
        for (int w = 0; w < NW; ++w) fw[d][w].end(col, K);
      }
      if (step * 32 + 32 > KX) {
#pragma unroll
        for (int t = 0; t < MT; ++t) fx[d][t].end(col, KX);
      }
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[w][t] = mma(fw[d][w].frag(), fx[d][t].frag(), acc[w][t]);
    }
  }
}

template <typename DT, int MT>
__global__ __launch_bounds__(kInWaves * 64) void feed_few_in_kernel(FeedFewArgs a) {
  __shared__ f32x4 sums[kInWaves][2 * MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, group = lane >> 4;
  const int f0 = blockIdx.x * 16;
  const DT *wrow[2], *xrow[MT];
  const int f = f0 + i < a.F ? f0 + i : a.F - 1;
  wrow[0] = (const DT*)a.w_in + (int64_t)f * a.ld_in;
  wrow[1] = (const DT*)a.w_in + ((int64_t)a.F + f) * a.ld_in;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = 16 * t + i < a.rows ? 16 * t + i : a.rows - 1;
    xrow[t] = (const DT*)a.x + m * a.ldx;
  }
  f32x4 acc[2][MT];
  few_product<DT, 2, MT, kInWaves, MT <= 2 ? 4 : 2>(acc, wrow, xrow, a.n, a.n, 0, (a.n + 31) / 32, wave, group);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    sums[wave][t][lane] = acc[0][t];
    sums[wave][MT + t][lane] = acc[1][t];
  }
  __syncthreads();
  if (wave >= MT) return;
  f32x4 g = sums[0][wave][lane], u = sums[0][MT + wave][lane];
#pragma unroll
  for (int k = 1; k < kInWaves; ++k) {
    g += sums[k][wave][lane];
    u += sums[k][MT + wave][lane];
  }
  const int m = 16 * wave + i, fo = f0 + 4 * group;
  f32x4 h;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (fo + r >= a.F) g[r] = u[r] = 0.f;
    h[r] = activate(g[r], a.act).act * u[r];
  }
  if (m >= a.rows) return;
  store4((DT*)a.h + (int64_t)m * a.Fp + fo, h, a.Fp - fo);
  if (a.gu) {  // F is padded to whole fours
    float* gu = a.gu + (int64_t)m * 2 * a.Fp + fo;
    *reinterpret_cast<f32x4*>(gu) = g;
    *reinterpret_cast<f32x4*>(gu + a.Fp) = u;
  }
}

template <typename DT, int MT>
__global__ __launch_bounds__(kOutWaves * 64) void feed_few_out_kernel(FeedFewArgs a) {
  __shared__ f32x4 sums[kOutWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, group = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int steps = (a.F + 31) / 32, each = (steps + a.splits - 1) / a.splits, first = blockIdx.y * each;
  const DT *wrow[1], *xrow[MT];
  wrow[0] = (const DT*)a.w_out + (int64_t)(n0 + i < a.n_out ? n0 + i : a.n_out - 1) * a.ld_out;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = 16 * t + i < a.rows ? 16 * t + i : a.rows - 1;
    xrow[t] = (const DT*)a.h + (int64_t)m * a.Fp;
  }
  f32x4 acc[1][MT];
  few_product<DT, 1, MT, kOutWaves, MT <= 2 ? 4 : 2>(acc, wrow, xrow, a.F, a.Fp, first,
                                                     steps - first < each ? steps : first + each, wave, group);
#pragma unroll
  for (int t = 0; t < MT; ++t) sums[wave][t][lane] = acc[0][t];
  __syncthreads();
  if (wave >= MT) return;
  f32x4 y = sums[0][wave][lane];
#pragma unroll
  for (int k = 1; k < kOutWaves; ++k) y += sums[k][wave][lane];
  const int m = 16 * wave + i, n = n0 + 4 * group;
  if (m >= a.rows) return;
  if (a.splits > 1) {
    store4(a.part + ((int64_t)blockIdx.y * a.rows + m) * a.n_out + n, y, a.n_out - n);
    return;
  }
  if (a.residual) {
    const DT* r = (const DT*)a.residual + m * a.ldr + n;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < a.n_out) y[k] += to_f32<DT>(r[k]);
  }
  store4((DT*)a.y + (int64_t)m * a.n_out + n, y, a.n_out - n);
}

template <typename DT, int MT>
hipError_t few(const FeedFewArgs& a, hipStream_t st) {
  launch_kernel(feed_few_in_kernel<DT, MT>, dim3((unsigned)((a.Fp + 15) / 16)), dim3(kInWaves * 64), 0, st, a);
  launch_kernel(feed_few_out_kernel<DT, MT>, dim3((unsigned)((a.n_out + 15) / 16), (unsigned)a.splits), dim3(kOutWaves * 64), 0,
                st, a);
  if (a.splits == 1) return hipGetLastError();
  FeedArgs j{};
  j.M = a.rows; j.N = a.n_out; j.splits = a.splits; j.part = a.part;
  j.out = a.y; j.ldo = a.n_out; j.residual = a.residual; j.ldr = a.ldr;
  return launch_feed_join(kFeedOut, j, sizeof(DT) == 2, st);
}

template <typename DT>
hipError_t few_rows(const FeedFewArgs& a, hipStream_t st) {
  return a.rows <= 16 ? few<DT, 1>(a, st) : a.rows <= 32 ? few<DT, 2>(a, st) : few<DT, 4>(a, st);
}

// ---------------------------------------------------------------------------
// Copies and sums around the products
// ---------------------------------------------------------------------------
template <typename DT>
__global__ __launch_bounds__(256) void feed_pack_kernel(FeedPackArgs a) {
  const auto t = a.t[blockIdx.y];
  for (int64_t row = blockIdx.x; row < t.rows; row += gridDim.x)
    for (int c = threadIdx.x; c < t.pitch; c += 256)
      ((DT*)t.to)[row * t.pitch + c] = c < t.cols ? ((const DT*)t.from)[row * t.ld + c] : (DT)0.f;
}

// out = residual + the partial products, in their order: four columns a
// thread, or one where rows are not multiples of four.
template <typename DT, int E>
__global__ __launch_bounds__(256) void feed_join_kernel(FeedArgs a) {
  const int64_t plane = (int64_t)a.M * a.N, count = plane / E;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i * E / a.N, n = i * E % a.N;
    int64_t row = m;
    if (a.rows_split) {
      const bool second = m >= a.rows_split;
      row = second ? m - a.rows_split + a.F : m;
      if (row >= (second ? 2 * (int64_t)a.F : a.F)) continue;
    }
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const float* p = a.part + s * plane + i * E;
      if constexpr (E == 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += v[e];
      } else {
        sum[0] += p[0];
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (a.residual) sum[e] += to_f32<DT>(((const DT*)a.residual)[row * a.ldr + n + e]);
      ((DT*)a.out)[row * a.ldo + n + e] = from_f32<DT>(sum[e]);
    }
  }
}

// The same for the products whose results go through the activation: four
// hidden units a thread.
template <typename DT, bool BACK>
__global__ __launch_bounds__(256) void feed_join_act_kernel(FeedArgs a) {
  const int per = a.Fp / 4;
  const int64_t count = (int64_t)a.M * per, plane = (int64_t)a.M * a.Fp * (BACK ? 1 : 2);
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per;
    const int f = (int)(i % per) * 4;
    const float* p = a.part + m * a.Fp * (BACK ? 1 : 2) + f;
    f32x4 g = {0.f, 0.f, 0.f, 0.f}, u = g, dh = g;
    for (int s = 0; s < a.splits; ++s, p += plane) {
      if (BACK) {
        dh += *reinterpret_cast<const f32x4*>(p);
      } else {
        g += *reinterpret_cast<const f32x4*>(p);
        u += *reinterpret_cast<const f32x4*>(p + a.Fp);
      }
    }
    float* gu = a.gu ? a.gu + m * 2 * a.Fp + f : nullptr;
    if (BACK) {
      g = *reinterpret_cast<const f32x4*>(gu);
      u = *reinterpret_cast<const f32x4*>(gu + a.Fp);
    }
    DT* out = (DT*)a.out + m * a.ldo + f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool on = f + e < a.F;
      if (!on) g[e] = u[e] = dh[e] = 0.f;
      const Activated r = activate(g[e], a.act);
      out[e] = from_f32<DT>(BACK ? dh[e] * u[e] * r.slope : r.act * u[e]);
      if (BACK) out[a.Fp + e] = from_f32<DT>(dh[e] * r.act);
    }
    if (!BACK && gu) {
      *reinterpret_cast<f32x4*>(gu) = g;
      *reinterpret_cast<f32x4*>(gu + a.Fp) = u;
    }
  }
}

template <typename DT>
hipError_t join(int op, const FeedArgs& a, hipStream_t st) {
  if (op == kFeedIn || op == kFeedDh) {
    const int64_t n = ((int64_t)a.M * (a.Fp / 4) + 255) / 256;
    const dim3 blocks((unsigned)(n < 4096 ? n : 4096));
    if (op == kFeedDh)
      launch_kernel(feed_join_act_kernel<DT, true>, blocks, dim3(256), 0, st, a);
    else
      launch_kernel(feed_join_act_kernel<DT, false>, blocks, dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const bool four = a.N % 4 == 0;
  const int64_t blocks = ((int64_t)a.M * a.N / (four ? 4 : 1) + 255) / 256;
  const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
  if (four)
    launch_kernel(feed_join_kernel<DT, 4>, grid, dim3(256), 0, st, a);
  else
    launch_kernel(feed_join_kernel<DT, 1>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// A workgroup of the second product reads all hidden values (F of each row)
// beside its 16 rows of weights: with more than 16 rows that is what bounds it,
// so the summed dimension is divided over as many workgroups as the device has
// compute units, and a third launch adds up. 64 rows, F = 4096, 1024 outputs,
// bf16: 21 us undivided; with 16 rows and less the launch would cost more.
int feed_few_splits(int64_t rows, int F, int n_out, int cus) {
  if (rows <= 16) return 1;
  const int tiles = (n_out + 15) / 16, steps = (F + 31) / 32;
  int want = cus / tiles;
  if (want > steps / 16) want = steps / 16;  // a step for every wave
  if (want < 2) return 1;
  const int each = (steps + want - 1) / want;
  return (steps + each - 1) / each;
}

hipError_t launch_feed_few(const FeedFewArgs& a, bool bf, hipStream_t st) {
  return bf ? few_rows<bf16>(a, st) : few_rows<float>(a, st);
}

hipError_t launch_feed_pack(const FeedPackArgs& a, bool bf, hipStream_t st) {
  int64_t rows = 1;
  for (int i = 0; i < a.count; ++i) rows = rows > a.t[i].rows ? rows : a.t[i].rows;
  const dim3 grid((unsigned)(rows < 8192 ? rows : 8192), (unsigned)a.count);
  if (bf)
    launch_kernel(feed_pack_kernel<bf16>, grid, dim3(256), 0, st, a);
  else
    launch_kernel(feed_pack_kernel<float>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_feed_join(int op, const FeedArgs& a, bool bf, hipStream_t st) {
  return bf ? join<bf16>(op, a, st) : join<float>(op, a, st);
}

}  // namespace rnnk
