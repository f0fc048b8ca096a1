// The products of the gated feed-forward, one kernel template.
//
// C[m, n] = sum_k A[m, k] B[n, k]: an operand lies with k running along its
// rows, or across them. A workgroup makes a tile of 256 x 256 (eight waves of
// 128 x 64, one workgroup a compute unit) or 128 x 128 (four of 64 x 64, two
// workgroups) outputs on the 32x32 matrix instructions, k in steps of 128
// bytes. A step's operands go straight from memory into LDS (16 bytes a lane),
// in five places that hold one operand's step each: while a step is multiplied
// one operand of the next is there, the other and one more are on their way,
// issued between the products. One barrier a step says that the next step has
// arrived and that this one's places are free.
//
// In LDS an operand that runs along k is [rows][128 bytes], the 16-byte chunk
// c of row r at c ^ ((r >> 1) & 7), so that 16 neighbouring rows' reads of a
// chunk fall on different banks. One that runs across is [k][tile columns];
// bf16 takes it through the transposing read (4 x 16 blocks), whose 32-byte
// columns u lie at u ^ turn(k) for the same reason. The order of k inside a
// step is the same for both operands, which is all that a product asks of it.
//
// What is behind a row's end along k is zero in LDS: the last step of such an
// operand goes through registers. Rows and columns behind the output's are
// some row or column again and are not stored.
//
// Workgroups stay for several tiles: the first steps of the next one are
// fetched while the last of this one are multiplied and its results are
// stored. Neighbouring tiles (8 rows of tiles, then the next column) go to one
// XCD at a time, whose L2 they share.
//
// Products of few tiles take eight waves on 128 x 128 and nine places (more
// steps on their way for a workgroup that is alone on its compute unit): 333
// rows, 1024 x 2816, bf16: 38 us of kernels in tiles of four waves, 33 so.
//
// Measured at 32000 rows, 1024 x 2816, bf16 (us, TFLOP/s, share of the compute
// units' matrix cycles): g | u 445, 829, 43% (it writes 0.9 GB of g, u and h);
// y 213, 868, 43%; dh with dg and du 445 to 496, 390, 17% (1.2 GB read, 0.5
// written: bound by memory); dx 412, 896, 42%; dW_in 453, 815, 44%; dW_out
// 235, 786, 43%. What bounds the others: a step of 256 x 256 in bf16 takes 2060
// clocks of a compute unit's matrix units and 2050 of its LDS port (196 kB read,
// 64 kB written, 128 bytes a clock), and a step of y 2.5 us, both and more: the
// two run largely one after the other, since every step begins behind its barrier
// with all waves reading. (Alone the loads of dx take 250 us and its products
// 257.) The card's power is the smaller part: at 8192^3 the same kernel takes
// 976 us on random numbers and 768 on zeros, a library product 793 and 485; of
// y's size the library takes 141 us. Not faster:
// steps of 64 bytes with two workgroups (2408 us for all six against 2200) or
// with a longer ring (2459), 16 waves, operands through registers, k begun at
// another place in each workgroup. fp32 at 19334 rows, 512 x 1368: 105 to 121
// TFLOP/s of 153, dh 80 (bound by memory); products of few tiles reach 50 to 80,
// since whole tiles leave places empty (400 rows, 1024 x 2816: g | u 74 us).
#pragma once

#include <type_traits>

#include "../../include/rnn.h"
#include "device_common.hpp"
#include "state_block_kernels.hpp"

namespace rnnk {
namespace {

typedef short feed_s16x4 __attribute__((ext_vector_type(4)));
typedef short feed_s16x8 __attribute__((ext_vector_type(8)));

// act(g) and its slope. gelu(g) = g (1 + tanh(u)) / 2 = g sigma(2 u).
struct Activated {
  float act, slope;
};
__device__ __forceinline__ Activated activate(float g, int kind) {
  Activated r;
  if (kind == RNN_ACT_GELU_TANH) {
    // beyond +-40 sigma is 0 or 1 and its slope 0 in fp32 (2 u is past 4600 there),
    // while g^2 would overflow for large gates and make the slope 0 times infinity
    constexpr float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float b = g > 40.0f ? 40.0f : g < -40.0f ? -40.0f : g, b2 = b * b;  // (what is no number stays so)
    const SigmoidPair p = fsigmoid_pair(c * b * __builtin_fmaf(0.044715f, b2, 1.0f));
    r.act = g * p.s;
    r.slope = __builtin_fmaf(b * p.s * p.no, c * __builtin_fmaf(3.0f * 0.044715f, b2, 1.0f), p.s);
  } else {
    const SigmoidPair p = fsigmoid_pair(g);
    r.act = kind == RNN_ACT_SIGMOID ? p.s : g * p.s;
    r.slope = kind == RNN_ACT_SIGMOID ? p.s * p.no : __builtin_fmaf(g * p.s, p.no, p.s);
  }
  return r;
}

// Tiles: kTileBig; kTileSmall, two workgroups a compute unit; kTileDeep, small
// ones alone on their compute unit, with eight waves (of 32 x 64) and more
// steps on their way, for products with few tiles.
template <int TILE>
struct FeedTile {
  static constexpr bool kBig = TILE == kTileBig;
  static constexpr int kRows = kBig ? 256 : 128;      // of either operand
  static constexpr int kThreads = TILE == kTileSmall ? 256 : 512;
  static constexpr int kWavesN = kRows / 64;          // waves across
  static constexpr int MI = kRows / 32 * kWavesN / (kThreads / 64);  // 32-row blocks of a wave; two across
  static constexpr int kBytes = kRows * 128;          // one operand's step
  static constexpr int kAhead = TILE == kTileDeep ? 4 : 2;  // steps that A's loads run ahead; B's one less
  static constexpr int kSlots = 2 * kAhead + 1, kLds = kSlots * kBytes;
  static constexpr int kTimes = kBytes / 16 / kThreads;     // 16-byte loads of a thread
  static constexpr int kResident = TILE == kTileSmall ? 512 : 256;  // workgroups that a device of 256 compute units holds
};

// 16-byte loads that bring an operand's step into LDS. A thread's addresses
// are 32-bit distances from the step's, which is the same for all.
template <typename DT, int TILE, bool ALONG>
struct Operand {
  using T = FeedTile<TILE>;
  static constexpr int E = 16 / (int)sizeof(DT);              // elements of a chunk
  static constexpr int kStep = 128 / (int)sizeof(DT);         // k of a step
  static constexpr int kChunks = T::kRows / E;                // of a k row (across)
  static constexpr int kSweep = ALONG ? T::kThreads / 8 : T::kThreads / kChunks;  // rows between a thread's loads
  const char* base;                                           // the tile's first element (the same for a wave)
  int64_t partner;                                            // ... and how far from it the other rows of pairs are
  uint32_t at[ALONG ? T::kTimes : 1];
  // 32-byte column u of k row k is at u ^ turn(k): four rows on different
  // banks, also where two neighbouring columns are read at once
  static __device__ __forceinline__ int turn(int k) { return (k & 3) ^ ((k & 1) << 2); }
  // first k (along) or k row (across) of this thread in a step
  static __device__ __forceinline__ int chunk() {
    const int t = threadIdx.x;
    return ALONG ? ((t & 7) ^ ((t >> 4) & 7)) * E : t / kChunks;
  }

  // The tile's rows from row0 on, `rows` there are; PAIRS: 32 of them, then 32
  // that are `apart` rows behind those, then the next 32 and so on.
  template <bool PAIRS>
  __device__ __forceinline__ void place_along(const void* p, int64_t ld, int row0, int rows, int apart) {
    base = (const char*)p + row0 * ld * (int64_t)sizeof(DT);
    partner = PAIRS ? apart * ld * (int64_t)sizeof(DT) : 0;
    if (T::kThreads == 512) {  // a wave's rows are all on one side: 8 of every 64
      if (__builtin_amdgcn_readfirstlane(threadIdx.x) & 256) base += partner;
      partner = 0;
    }
#pragma unroll
    for (int i = 0; i < T::kTimes; ++i) {
      const int r = (threadIdx.x >> 3) + i * kSweep, n = PAIRS ? (r >> 6) * 32 + (r & 31) : r;
      const int row = row0 + n < rows ? n : rows - 1 - row0;
      at[ALONG ? i : 0] = (uint32_t)((row * ld + chunk()) * (int64_t)sizeof(DT));
    }
  }
  // The tile's columns from col0 on, `cols` there are in memory.
  __device__ __forceinline__ void place_across(const void* p, int64_t ld, int col0, int cols) {
    const int t = threadIdx.x, k = t / kChunks, pos = t % kChunks;
    const int c = (sizeof(DT) == 2 ? ((pos >> 1) ^ turn(k)) * 2 + (pos & 1) : pos) * E;
    base = (const char*)p + (int64_t)col0 * (int64_t)sizeof(DT);
    partner = 0;
    at[0] = (uint32_t)((k * ld + (col0 + c + E <= cols ? c : cols - E - col0)) * (int64_t)sizeof(DT));
  }

  // Load i of a step whose first k is k0 and (across) first row row0.
  __device__ __forceinline__ const char* from(int i, int k0, int64_t row0, int64_t ld) const {
    const char* step = base + (ALONG ? (int64_t)k0 : (row0 + i * kSweep) * ld) * (int64_t)sizeof(DT);
    if (T::kThreads == 256 && ALONG && i % 2) step += partner;  // every other 32 rows
    return step + at[ALONG ? i : 0];
  }
  // ... that is there as a whole
  __device__ __forceinline__ void load(char* lds, int i, int k0, int64_t row0, int64_t ld) const {
    [[maybe_unused]] char* to = lds + (threadIdx.x >> 6) * 1024 + i * T::kThreads * 16;
    [[maybe_unused]] const char* p = from(i, k0, row0, ld);
#ifdef __HIP_DEVICE_COMPILE__  // the host's pass does not know LDS pointers and drops kernels over them
    __builtin_amdgcn_global_load_lds(p, to, 16, 0, 0);
#endif
  }
  __device__ __forceinline__ void fetch(char* lds, int k0, int64_t row0, int limit, int64_t ld) const {
    if (k0 + kStep <= limit) {
#pragma unroll
      for (int i = 0; i < T::kTimes; ++i) load(lds, i, k0, row0, ld);
    } else {
      u32x4 v[T::kTimes];
      const int c = chunk();
#pragma unroll
      for (int i = 0; i < T::kTimes; ++i) {
        const int k = k0 + c + (ALONG ? 0 : i * kSweep);
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (k < limit) v[i] = *reinterpret_cast<const u32x4*>(from(i, k0, row0, ld));
      }
      // A wave none of whose rows are left has loaded nothing here: without a
      // wait of its own the loads that step_barrier counts could be older ones.
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < T::kTimes; ++i) *reinterpret_cast<u32x4*>(lds + (i * T::kThreads + threadIdx.x) * 16) = v[i];
    }
  }
};

// A wave's fragment of 32 rows for part s of a step (a quarter in both types).
template <typename DT>
struct FeedFrag;
template <>
struct FeedFrag<bf16> {
  bf16x8 v;
};
template <>
struct FeedFrag<float> {
  float v[4];
};

template <bool ALONG, int ROWS>
__device__ __forceinline__ void read_frag(FeedFrag<bf16>& f, const char* lds, int r0, int s, int lane) {
  const int half = lane >> 5, l32 = lane & 31;
  if constexpr (ALONG) {
    f.v = *reinterpret_cast<const bf16x8*>(lds + (r0 + l32) * 128 + (((2 * s + half) ^ ((l32 >> 1) & 7)) << 4));
  } else {
    typedef __attribute__((address_space(3))) feed_s16x4* LdsPtr;
    const int i = lane & 15, unit = (r0 >> 4) + ((lane >> 4) & 1), k = 16 * s + 8 * half + (i >> 2);
    const char* p = lds + k * (ROWS * 2) + ((unit ^ Operand<bf16, kTileBig, false>::turn(k)) << 5) + ((i & 3) << 3);
    const feed_s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p));
    const feed_s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p + 4 * ROWS * 2));
    f.v = __builtin_bit_cast(bf16x8, (feed_s16x8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}
template <bool ALONG, int ROWS>
__device__ __forceinline__ void read_frag(FeedFrag<float>& f, const char* lds, int r0, int s, int lane) {
  const int half = lane >> 5, l32 = lane & 31;
  if constexpr (ALONG) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(lds + (r0 + l32) * 128 + (((2 * s + half) ^ ((l32 >> 1) & 7)) << 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = v[e];
  } else {
    const float* p = reinterpret_cast<const float*>(lds) + (4 * (2 * s + half)) * ROWS + r0 + l32;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = p[e * ROWS];
  }
}

__device__ __forceinline__ f32x16 feed_mma(const FeedFrag<bf16>& a, const FeedFrag<bf16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 feed_mma(const FeedFrag<float>& a, const FeedFrag<float>& b, f32x16 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[e], b.v[e], c, 0, 0, 0);
  return c;
}

// Waits until all but the last LATER loads have arrived (loads and stores end
// in order), then for the other waves.
template <int LATER>
__device__ __forceinline__ void step_barrier() {
  static_assert(LATER < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (LATER & 15) | LATER >> 4 << 14);  // vmcnt(LATER), lgkmcnt(0), expcnt at its maximum
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int OP>
struct FeedShape {
  static constexpr bool kAlongA = OP == kFeedIn || OP == kFeedOut || OP == kFeedDh || OP == kFeedDx;
  static constexpr bool kAlongB = OP == kFeedIn || OP == kFeedOut;
};

// One piece of work: a tile of the output and a range of steps.
struct FeedItem {
  int m0, n0, split, k0, k1;
};
template <int TILE, int OP>
__device__ __forceinline__ FeedItem feed_item(const FeedArgs& a, int tiles_m, int tiles_n, int id) {
  constexpr int kRows = FeedTile<TILE>::kRows, kCols = OP == kFeedIn ? kRows / 2 : kRows;
  const int tiles = tiles_m * tiles_n;
  FeedItem w;
  w.split = id / tiles;
  int t = id % tiles;
  constexpr int kGroup = 8;
  const int per = kGroup * tiles_n, group = t / per, first = group * kGroup;
  const int down = tiles_m - first < kGroup ? tiles_m - first : kGroup;
  t -= group * per;
  w.m0 = (first + t % down) * kRows;
  w.n0 = t / down * kCols;
  const int each = (a.steps + a.splits - 1) / a.splits;
  w.k0 = w.split * each;
  w.k1 = a.steps - w.k0 < each ? a.steps : w.k0 + each;
  return w;
}

// Eight results of a lane: column n, rows 8 (v / 4) + v % 4 of `out`, where
// half a 32 x 32 block begins. In bf16 lanes change every other row's result
// with their neighbour, so that each stores two columns at a time (PAIRS: rows
// and n allow it).
template <typename DT, bool PAIRS>
__device__ __forceinline__ void store_half(DT* out, int64_t ld, const float (&val)[8], int lane) {
  if constexpr (PAIRS && sizeof(DT) == 2) {
    const bool odd = lane & 1;
    bf16* p = out + (odd ? ld - 1 : 0);
#pragma unroll
    for (int v = 0; v < 8; v += 2) {
      const float keep = odd ? val[v + 1] : val[v], give = odd ? val[v] : val[v + 1];
      const int there = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, give), 0xB1, 0xF, 0xF, true);
      const float got = __builtin_bit_cast(float, there);
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<bf16x2*>(p + (8 * (v >> 2) + (v & 3)) * ld) = bf16x2{(bf16)(odd ? got : keep), (bf16)(odd ? keep : got)};
    }
  } else {
#pragma unroll
    for (int v = 0; v < 8; ++v) out[(8 * (v >> 2) + (v & 3)) * ld] = from_f32<DT>(val[v]);
  }
}
template <typename DT>
__device__ __forceinline__ void store_half(DT* out, int64_t ld, const float (&val)[8], int lane, bool pairs) {
  if (pairs)
    store_half<DT, true>(out, ld, val, lane);
  else
    store_half<DT, false>(out, ld, val, lane);
}

// A tile's way out of the accumulators. A lane holds column lane % 32 and rows
// 8 (v / 4) + 4 (lane / 32) + v % 4 of each 32 x 32 block. WHOLE: every row
// and column of the tile exists; it leaves in halves of a block, and what a
// half needs from memory is asked for while the one before it is worked on.
template <typename DT, int TILE, int OP, bool WHOLE>
__device__ __forceinline__ void feed_results(const FeedArgs& a, const FeedItem& w,
                                             const f32x16 (&acc)[FeedTile<TILE>::MI][2], int wm, int wn, int lane) {
  constexpr int MI = FeedTile<TILE>::MI, kAcross = OP == kFeedIn ? 1 : 2, kBlocks = kAcross * MI;
  const int m_base = w.m0 + wm * MI * 32 + 4 * (lane >> 5), n_base = w.n0 + wn * (OP == kFeedIn ? 32 : 64) + (lane & 31);
  if constexpr (WHOLE) {
    const bool pairs = sizeof(DT) == 2 && a.ldo % 2 == 0 && ((uintptr_t)a.out & 3) == 0;
    const bool add = OP == kFeedOut && a.residual && a.splits == 1;
    float more[2][8], more_u[OP == kFeedDh ? 2 : 1][8];
    auto ask = [&](int k) {
      const int64_t m = m_base + k / (2 * kAcross) * 32 + k % 2 * 16, n = n_base + k / 2 % kAcross * 32;
      if constexpr (OP == kFeedDh) {
        const float* p = a.gu + m * 2 * a.Fp + n;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float* q = p + (int64_t)(8 * (v >> 2) + (v & 3)) * 2 * a.Fp;
          more[k & 1][v] = q[0];
          more_u[k & 1][v] = q[a.Fp];
        }
      } else if constexpr (OP == kFeedOut) {
        const DT* p = (const DT*)a.residual + m * a.ldr + n;
#pragma unroll
        for (int v = 0; v < 8; ++v) more[k & 1][v] = to_f32<DT>(p[(8 * (v >> 2) + (v & 3)) * a.ldr]);
      }
    };
    const bool asks = OP == kFeedDh ? a.splits == 1 : add;
    if (asks) ask(0);
#pragma unroll
    for (int k = 0; k < 2 * kBlocks; ++k) {
      const int i = k / (2 * kAcross), j = k / 2 % kAcross, v0 = k % 2 * 8;
      const int64_t m = m_base + i * 32 + k % 2 * 16, n = n_base + j * 32;
      if (asks && k + 1 < 2 * kBlocks) ask(k + 1);
      float val[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) val[v] = acc[i][j][v0 + v];
      if constexpr (OP == kFeedIn) {
        float u[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) u[v] = acc[i][1][v0 + v];
        if (a.splits > 1) {
          float* p = a.part + ((int64_t)w.split * a.M + m) * 2 * a.Fp + n;
          store_half<float, false>(p, 2 * (int64_t)a.Fp, val, lane);
          store_half<float, false>(p + a.Fp, 2 * (int64_t)a.Fp, u, lane);
          continue;
        }
        if (a.gu) {
          float* p = a.gu + m * 2 * a.Fp + n;
          store_half<float, false>(p, 2 * (int64_t)a.Fp, val, lane);
          store_half<float, false>(p + a.Fp, 2 * (int64_t)a.Fp, u, lane);
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) u[v] *= activate(val[v], a.act).act;
        store_half<DT>((DT*)a.out + m * a.ldo + n, a.ldo, u, lane, pairs);
      } else if (a.splits > 1) {
        store_half<float, false>(a.part + ((int64_t)w.split * a.M + m) * a.N + n, a.N, val, lane);
      } else if constexpr (OP == kFeedDh) {
        float du[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const Activated r = activate(more[k & 1][v], a.act);
          du[v] = val[v] * r.act;
          val[v] *= more_u[k & 1][v] * r.slope;
        }
        DT* out = (DT*)a.out + m * a.ldo + n;
        store_half<DT>(out, a.ldo, val, lane, pairs);
        store_half<DT>(out + a.Fp, a.ldo, du, lane, pairs);
      } else {
        // a block's rows lie on one side of the gate's last (padded) one
        const bool second = OP == kFeedDwIn && m >= a.Fp;
        const int64_t f = second ? m - a.Fp : m, row = second ? f + a.F : m;
        DT* out = (DT*)a.out + row * a.ldo + n;
        if (add) {
#pragma unroll
          for (int v = 0; v < 8; ++v) val[v] += more[k & 1][v];
        }
        if (OP == kFeedDwIn && f + 16 > a.F) {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            if (f + 8 * (v >> 2) + (v & 3) < a.F) out[(8 * (v >> 2) + (v & 3)) * a.ldo] = from_f32<DT>(val[v]);
        } else {
          store_half<DT>(out, a.ldo, val, lane, pairs);
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      const int i = k / kAcross, j = k % kAcross;
      const int n = n_base + j * 32;
      if (n >= (OP == kFeedIn ? a.Fp : a.N)) continue;
      // what the block needs from memory, all on its way at once (the last row again for those behind it):
      // dh of 1759 rows, 1112 x 264, bf16, whose tiles all lie at an edge, 42 -> 31 us
      float more[16], more_u[OP == kFeedDh ? 16 : 1];
      if (OP == kFeedDh ? a.splits == 1 : OP == kFeedOut && a.residual && a.splits == 1) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          int64_t m = m_base + i * 32 + 8 * (v >> 2) + (v & 3);
          m = m < a.M ? m : a.M - 1;
          if constexpr (OP == kFeedDh) {
            const float* gu = a.gu + m * 2 * a.Fp + n;
            more[v] = gu[0];
            more_u[v] = gu[a.Fp];
          } else if constexpr (OP == kFeedOut) {
            more[v] = to_f32<DT>(((const DT*)a.residual)[m * a.ldr + n]);
          }
        }
      }
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t m = m_base + i * 32 + 8 * (v >> 2) + (v & 3);
        if (m >= a.M) continue;
        const float val = acc[i][j][v];
        if (a.splits > 1) {
          if constexpr (OP == kFeedIn) {
            float* p = a.part + ((int64_t)w.split * a.M + m) * 2 * a.Fp + n;
            p[0] = val;
            p[a.Fp] = acc[i][1][v];
          } else {
            a.part[((int64_t)w.split * a.M + m) * a.N + n] = val;
          }
        } else if constexpr (OP == kFeedIn) {
          const bool on = n < a.F;
          const float g = on ? val : 0.f, u = on ? acc[i][1][v] : 0.f;
          ((DT*)a.out)[m * a.ldo + n] = from_f32<DT>(activate(g, a.act).act * u);
          if (a.gu) {
            a.gu[m * 2 * a.Fp + n] = g;
            a.gu[m * 2 * a.Fp + a.Fp + n] = u;
          }
        } else if constexpr (OP == kFeedDh) {
          const Activated r = activate(more[v], a.act);
          const bool on = n < a.F;
          DT* out = (DT*)a.out + m * a.ldo + n;
          out[0] = from_f32<DT>(on ? val * more_u[v] * r.slope : 0.f);
          out[a.Fp] = from_f32<DT>(on ? val * r.act : 0.f);
        } else {
          int64_t row = m;
          if (OP == kFeedDwIn) {
            const bool second = m >= a.Fp;
            row = second ? m - a.Fp + a.F : m;
            if (row >= (second ? 2 * (int64_t)a.F : a.F)) continue;
          }
          ((DT*)a.out)[row * a.ldo + n] = from_f32<DT>(OP == kFeedOut && a.residual ? val + more[v] : val);
        }
      }
    }
  }
}

// One operand's loads, which run ahead of the products.
template <typename DT, int TILE, int OP, bool IS_A>
struct FeedStream {
  static constexpr bool kAlong = IS_A ? FeedShape<OP>::kAlongA : FeedShape<OP>::kAlongB;
  static constexpr int kStep = 128 / (int)sizeof(DT);
  Operand<DT, TILE, kAlong> op;
  int id, kt, end, slot;  // the next step to fetch and where it goes
  __device__ __forceinline__ void place(const FeedArgs& a, int tiles_m, int tiles_n) {
    const FeedItem w = feed_item<TILE, OP>(a, tiles_m, tiles_n, id);
    kt = w.k0;
    end = w.k1;
    if (IS_A) {
      if (kAlong)
        op.template place_along<false>(a.A, a.lda, w.m0, a.M, 0);
      else
        op.place_across(a.A, a.lda, w.m0, a.cols_a);
    } else {
      if (kAlong)
        op.template place_along<OP == kFeedIn>(a.B, a.ldb, w.n0, OP == kFeedIn ? a.F : a.N, a.F);
      else
        op.place_across(a.B, a.ldb, w.n0, a.cols_b);
    }
  }
  // Goes on to the next item where this one's steps are all fetched; whether
  // there is a step left.
  __device__ __forceinline__ bool ready(const FeedArgs& a, int tiles_m, int tiles_n, int items) {
    if (kt == end && id < items) {
      id += gridDim.x;
      if (id < items) place(a, tiles_m, tiles_n);
    }
    return id < items;
  }
  // The step's first k, how far k goes and the operand's row (across): those
  // of the gate's weights and of its partner's, F each, follow each other.
  __device__ __forceinline__ void where(const FeedArgs& a, int* k, int* row, int* limit) const {
    *k = *row = kt * kStep;
    *limit = IS_A ? a.KA : a.KB;
    if (OP == kFeedDx && !IS_A) {
      *limit = a.F;
      if (*k >= a.Fp) {
        *k -= a.Fp;
        *row = *k + a.F;
      }
    }
  }
  __device__ __forceinline__ bool whole(const FeedArgs& a) const {
    int k, row, limit;
    where(a, &k, &row, &limit);
    return k + kStep <= limit;
  }
  __device__ __forceinline__ char* to(char* lds) const { return lds + slot * FeedTile<TILE>::kBytes; }
  __device__ __forceinline__ void load(const FeedArgs& a, char* lds, int i) const {
    int k, row, limit;
    where(a, &k, &row, &limit);
    op.load(to(lds), i, k, row, IS_A ? a.lda : a.ldb);
  }
  __device__ __forceinline__ void next() {
    ++kt;
    slot = slot + 2 < FeedTile<TILE>::kSlots ? slot + 2 : slot + 2 - FeedTile<TILE>::kSlots;
  }
  __device__ __forceinline__ void fetch(const FeedArgs& a, char* lds) {
    int k, row, limit;
    where(a, &k, &row, &limit);
    op.fetch(to(lds), k, row, limit, IS_A ? a.lda : a.ldb);
    next();
  }
};

template <typename DT, int TILE, int OP>
__global__ __launch_bounds__(FeedTile<TILE>::kThreads, 2) void feed_kernel(FeedArgs a, int tiles_m, int tiles_n) {
  using T = FeedTile<TILE>;
  using S = FeedShape<OP>;
  constexpr int MI = T::MI;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::kWavesN, wn = wave % T::kWavesN;
  const int items = tiles_m * tiles_n * a.splits;
  // this round's items of one XCD are neighbours
  const int grid = gridDim.x, whole_grid = grid / 8 * 8;
  const int mine = (int)blockIdx.x < whole_grid ? (blockIdx.x % 8) * (whole_grid / 8) + blockIdx.x / 8 : blockIdx.x;
  if (mine >= items) return;

  // Slots of LDS are taken in turn: A 0, B 0, A 1, B 1, ... While step t is
  // multiplied, B t + kAhead - 1 and A t + kAhead go to the two places that
  // step t - 1 left; what lies between is there or on its way.
  FeedStream<DT, TILE, OP, true> sa;
  FeedStream<DT, TILE, OP, false> sb;
  sa.id = sb.id = mine;
  sa.slot = 0;
  sb.slot = 1;
  sa.place(a, tiles_m, tiles_n);
  sb.place(a, tiles_m, tiles_n);
#pragma unroll
  for (int i = 0; i < T::kAhead; ++i) {
    if (sa.ready(a, tiles_m, tiles_n, items)) sa.fetch(a, lds);
    if (i < T::kAhead - 1 && sb.ready(a, tiles_m, tiles_n, items)) sb.fetch(a, lds);
  }
  step_barrier<0>();
  constexpr int kLater = T::kTimes * feed_later(T::kAhead, true, true, true, 0);
  static_assert(T::kAhead == 2 || T::kAhead == 4, "the waits of the last steps are written for these");
  int slot = 0;
  for (int id = mine; id < items; id += grid) {
    const FeedItem w = feed_item<TILE, OP>(a, tiles_m, tiles_n, id);
    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    // One step: its products, and between them the loads (FETCH) and the next
    // quarter's reads.
    auto multiply = [&](auto fetch_tag) {
      constexpr bool FETCH = decltype(fetch_tag)::value;
      const char *at_a = lds + slot * T::kBytes, *at_b = lds + (slot == T::kSlots - 1 ? 0 : slot + 1) * T::kBytes;
      FeedFrag<DT> fa[2][MI], fb[2][2];
      auto read = [&](int s) {
#pragma unroll
        for (int j = 0; j < 2; ++j) read_frag<S::kAlongB, T::kRows>(fb[s & 1][j], at_b, wn * 64 + j * 32, s, lane);
#pragma unroll
        for (int i = 0; i < MI; ++i) read_frag<S::kAlongA, T::kRows>(fa[s & 1][i], at_a, wm * MI * 32 + i * 32, s, lane);
      };
      read(0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < 3) read(s + 1);
        if constexpr (FETCH) {
#pragma unroll
          for (int i = 0; i < T::kTimes / 2; ++i) {
            if (s < 2)
              sb.load(a, lds, s * (T::kTimes / 2) + i);
            else
              sa.load(a, lds, (s - 2) * (T::kTimes / 2) + i);
          }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = feed_mma(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
      }
      if constexpr (sizeof(DT) == 2) {
        constexpr int kReads = MI * (S::kAlongA ? 1 : 2) + 2 * (S::kAlongB ? 1 : 2), kEach = (kReads + 2 * MI - 1) / (2 * MI);
        __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int m = 0; m < 2 * MI; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (s < 3 && m * kEach < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
            if (FETCH && m >= 2 * MI - T::kTimes / 2) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
          }
        }
      }
    };
    // What the next step needs has arrived where the steps end: a tile's stores
    // are behind that wait.
    for (int kt = w.k0; kt < w.k1;) {
      bool fast = true;
      for (; kt < w.k1 && fast; ++kt) {
        const bool more_b = sb.ready(a, tiles_m, tiles_n, items), more_a = sa.ready(a, tiles_m, tiles_n, items);
        fast = more_a && more_b && sa.whole(a) && sb.whole(a);
        if (!fast) break;
        multiply(std::true_type{});
        sb.next();
        sa.next();
        step_barrier<kLater>();
        slot = slot + 2 < T::kSlots ? slot + 2 : slot + 2 - T::kSlots;
      }
      if (kt < w.k1) {
        // a step that goes through registers, or one of the workgroup's last
        const bool more_a = sa.id < items, more_b = sb.id < items;
        const bool direct = (!more_a || sa.whole(a)) && (!more_b || sb.whole(a));
        if (more_b) sb.fetch(a, lds);
        if (more_a) sa.fetch(a, lds);
        multiply(std::false_type{});
        const int later = feed_later(T::kAhead, more_a, more_b, direct, w.k1 - 1 - kt);
        if (T::kAhead > 2 && later == 4)
          step_barrier<(T::kAhead > 2 ? 4 * T::kTimes : 0)>();
        else if (T::kAhead > 2 && later == 2)
          step_barrier<(T::kAhead > 2 ? 2 * T::kTimes : 0)>();
        else
          step_barrier<0>();
        slot = slot + 2 < T::kSlots ? slot + 2 : slot + 2 - T::kSlots;
        ++kt;
      }
    }
    const int last = OP == kFeedIn || OP == kFeedDh ? a.F : a.N;
    const bool whole = w.m0 + T::kRows <= a.M && w.n0 + (OP == kFeedIn ? T::kRows / 2 : T::kRows) <= last;
    if (whole)
      feed_results<DT, TILE, OP, true>(a, w, acc, wm, wn, lane);
    else
      feed_results<DT, TILE, OP, false>(a, w, acc, wm, wn, lane);
  }
}

template <typename DT, int TILE, int OP>
hipError_t launch_feed_op(const FeedArgs& a, hipStream_t st) {
  using T = FeedTile<TILE>;
  constexpr int kCols = OP == kFeedIn ? T::kRows / 2 : T::kRows;
  const int tiles_m = (a.M + T::kRows - 1) / T::kRows, tiles_n = (a.N + kCols - 1) / kCols;
  const int64_t items = (int64_t)tiles_m * tiles_n * a.splits;
  auto kernel = feed_kernel<DT, TILE, OP>;
  if (T::kLds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    if (e != hipSuccess) return e;
  }
  launch_kernel(kernel, dim3((unsigned)(items < T::kResident ? items : T::kResident)), dim3(T::kThreads), T::kLds, st, a, tiles_m,
                tiles_n);
  if (a.splits > 1) return launch_feed_join(OP, a, sizeof(DT) == 2, st);
  return hipGetLastError();
}

template <typename DT, int TILE>
hipError_t launch_feed_tile(int op, const FeedArgs& a, hipStream_t st) {
  switch (op) {
    case kFeedIn: return launch_feed_op<DT, TILE, kFeedIn>(a, st);
    case kFeedOut: return launch_feed_op<DT, TILE, kFeedOut>(a, st);
    case kFeedDh: return launch_feed_op<DT, TILE, kFeedDh>(a, st);
    case kFeedDx: return launch_feed_op<DT, TILE, kFeedDx>(a, st);
    case kFeedDwIn: return launch_feed_op<DT, TILE, kFeedDwIn>(a, st);
    default: return launch_feed_op<DT, TILE, kFeedDwOut>(a, st);
  }
}

template <typename DT>
hipError_t launch_feed_type(int op, const FeedArgs& a, const FeedPlan& p, hipStream_t st) {
  return p.tile == kTileBig    ? launch_feed_tile<DT, kTileBig>(op, a, st)
         : p.tile == kTileDeep ? launch_feed_tile<DT, kTileDeep>(op, a, st)
                               : launch_feed_tile<DT, kTileSmall>(op, a, st);
}

}  // namespace
}  // namespace rnnk
