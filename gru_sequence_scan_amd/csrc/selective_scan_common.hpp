// Building blocks of the selective scan's kernels.
//
// A workgroup of 256 threads owns 64 channels of one batch row: four lanes a
// channel, each with J of the channel's states (n = J q .. J q + J - 1 for
// lane q of the four). Per-step scalars of a channel (its step, its input, its
// gate) are formed by one lane for each of four steps and handed round by lane
// permutations; sums over a channel's states go the other way, so that lane q
// ends with the sum that belongs to step q.
#pragma once

#include "device_common.hpp"
#include "state_block_kernels.hpp"

namespace rnnk {

constexpr int kSelThreads = 256;

// B and C are read from LDS two steps before they are used; this barrier of
// the compiler's keeps those reads where they stand (all but LDS accesses may
// pass), and registers are handed out for this many waves a SIMD, since the
// compiler would save them for more by moving the reads back. With what a
// step's scalars need formed for 16 steps at once: 1000 steps of 32 x 1024 x
// 16 in bf16 185 -> 169 us.
constexpr int kAhead = 2;
constexpr int kSelKeepReads = 0x47F;
constexpr int sel_waves(int J) { return J <= 4 ? 4 : J == 8 ? 3 : 2; }

template <typename DT, int E>
struct alignas(sizeof(DT) * E) SelVec {
  DT v[E];
};

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// Lane s's value of each four lanes.
template <int S>
__device__ __forceinline__ float quad_from(float v) {
  return dpp<S * 0x55>(v);
}
__device__ __forceinline__ float quad_from(float v, int s) {  // s known once loops are unrolled
  return s == 0 ? quad_from<0>(v) : s == 1 ? quad_from<1>(v) : s == 2 ? quad_from<2>(v) : quad_from<3>(v);
}
__device__ __forceinline__ float quad_sum(float v) {
  v += dpp<0xB1>(v);        // lanes 1 0 3 2
  return v + dpp<0x4E>(v);  // lanes 2 3 0 1
}
// Lane q of each four gets the sum over them of v[q].
__device__ __forceinline__ float quad_scatter(const float (&v)[4], int q) {
  const bool odd = q & 1, high = q & 2;
  const float a = (odd ? v[1] : v[0]) + dpp<0xB1>(odd ? v[0] : v[1]);
  const float b = (odd ? v[3] : v[2]) + dpp<0xB1>(odd ? v[2] : v[3]);
  return (high ? b : a) + dpp<0x4E>(high ? a : b);
}

typedef unsigned sel_u32x2 __attribute__((ext_vector_type(2)));

// Over the 16 channels of a wave (lane bits 2 to 5): the lanes of channel c
// get the sum over the channels of v[c], lane by lane of the four.
__device__ __forceinline__ float channel_scatter(float (&v)[16], int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the upper 32 lanes of the first change places with the lower of the second
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v[i]), __builtin_bit_cast(unsigned, v[i + 8]),
                                                    false, false);
    const unsigned lo = r[0], hi = r[1];
    v[i] = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v[i]), __builtin_bit_cast(unsigned, v[i + 4]),
                                                    false, false);
    const unsigned lo = r[0], hi = r[1];
    v[i] = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
  }
  const bool b3 = lane & 8, b2 = lane & 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = (b3 ? v[i + 2] : v[i]) + dpp<0x128>(b3 ? v[i] : v[i + 2]);  // rotated by 8 of 16 lanes
  // four lanes on: the mirror of eight, and the four lanes turned back
  return (b2 ? v[1] : v[0]) + dpp<0x141>(dpp<0x1B>(b2 ? v[0] : v[1]));
}

// A step's length from its raw value: softplus(raw) = max(raw, 0) + log(1 + y),
// y = exp(-|raw|), or raw itself. log(1 + y) = log(u) y / (u - 1) with u = 1 + y
// rounded (Kahan): the error of u cancels, so small steps keep their own accuracy.
__device__ __forceinline__ float step_length(float raw, int soft) {
  if (!soft) return raw;
  const float y = fexp(-__builtin_fabsf(raw)), u = 1.0f + y;
  const float l = __builtin_amdgcn_logf(u) * kLn2 * (y * __builtin_amdgcn_rcpf(u - 1.0f));
  return __builtin_fmaxf(raw, 0.0f) + (u == 1.0f ? y : l);
}

// Where a workgroup works.
struct SelPlace {
  int b, L, seg, t0, t1;   // batch row, its length, segment, its steps [t0, t1)
  int group, gt;           // group of channels, tile in the group
  int c0, live;            // first channel and how many of the 64 exist
  __device__ __forceinline__ explicit SelPlace(const SelectiveScanArgs& a) {
    // Workgroup ids are dealt to the XCDs in turn: the tiles of one (row,
    // segment), which share B, C and the cache lines at their edges, go to one
    // XCD one after the other.
    const unsigned slot = blockIdx.x / a.xcds, unit = slot / a.tiles * a.xcds + blockIdx.x % a.xcds;
    const int ct = slot % a.tiles;
    b = unit % a.B;
    seg = unit / a.B;
    group = ct / a.group_tiles;
    gt = ct % a.group_tiles;
    const int per = a.H / a.G;
    c0 = group * per + gt * kSelTile;
    live = per - gt * kSelTile < kSelTile ? per - gt * kSelTile : kSelTile;
    t0 = seg * a.seg_steps;
    t1 = a.T - t0 < a.seg_steps ? a.T : t0 + a.seg_steps;
    if (seg < a.segs) {
      const int n = a.lengths ? a.lengths[b] : a.T;
      L = n < 0 ? 0 : (n > a.T ? a.T : n);
    }
  }
};

// A thread's share of a tile of STEPS x 64 elements in memory: E neighbouring
// channels of a step in one access (or one by one where rows are not aligned).
// Nothing is conditional: a step past the row's end reads the last one again,
// a channel past the last one the first.
template <typename DT, int STEPS, bool VEC>
struct SelTile {
  static constexpr int kShare = kSelTile * STEPS / kSelThreads, kWide = 16 / (int)sizeof(DT);  // of a thread, of an access
  static constexpr int E = kShare < kWide ? kShare : kWide;
  static constexpr int kPer = kSelTile / E;                               // accesses of a step
  static constexpr int kTimes = STEPS * kPer / kSelThreads;               // accesses of a thread
  static constexpr int kLd = kSelTile + 16;                               // a step's row in LDS: four steps fall on different banks
  static constexpr int kWords = E * (int)sizeof(DT) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  Words r[kTimes];
  __device__ __forceinline__ void load(const void* base, int64_t ld_t, int t0, int last, int c0, int live) {
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int id = i * kSelThreads + (int)threadIdx.x, t = t0 + id / kPer, c = id % kPer * E;
      const DT* p = (const DT*)base + (int64_t)(t < last ? t : last) * ld_t + c0;
      if (VEC) {
        r[i] = *reinterpret_cast<const Words*>(p + (c < live ? c : 0));
      } else {
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          if constexpr (sizeof(DT) == 4) {
            const float v = p[c + w < live ? c + w : 0];
            r[i][w] = __builtin_bit_cast(uint32_t, v);
          } else {
            const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
            const uint32_t lo = u[c + 2 * w < live ? c + 2 * w : 0], hi = u[c + 2 * w + 1 < live ? c + 2 * w + 1 : 0];
            r[i][w] = lo | hi << 16;
          }
        }
      }
    }
  }
  __device__ __forceinline__ void put(DT* lds) const {
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int id = i * kSelThreads + (int)threadIdx.x;
      *reinterpret_cast<Words*>(lds + id / kPer * kLd + id % kPer * E) = r[i];
    }
  }
  // A tile of results from LDS to memory; zeros for steps from L on.
  static __device__ __forceinline__ void store(const DT* lds, void* base, int64_t ld_t, int t0, int t1, int L, int c0, int live) {
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int id = i * kSelThreads + (int)threadIdx.x, t = t0 + id / kPer, c = id % kPer * E;
      if (t >= t1) continue;
      const DT* from = lds + id / kPer * kLd + c;
      DT* p = (DT*)base + t * ld_t + c0 + c;
      if (VEC) {
        const Words v = *reinterpret_cast<const Words*>(from);
        if (c < live) *reinterpret_cast<Words*>(p) = t < L ? v : Words(0u);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (c + e < live) p[e] = t < L ? from[e] : (DT)0.f;
      }
    }
  }
};

// STEPS rows of B or C, as fp32 in LDS: zero from the row's end on and past N.
template <typename DT, int STEPS, int NP>
struct SelRows {
  static constexpr int kTimes = (STEPS * NP + kSelThreads - 1) / kSelThreads;
  DT r[kTimes];
  __device__ __forceinline__ void load(const void* base, int64_t ld_t, int t0, int last, int N) {
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int id = i * kSelThreads + (int)threadIdx.x, t = t0 + id / NP, n = id % NP;
      r[i] = ((const DT*)base)[(int64_t)(t < last ? t : last) * ld_t + (n < N ? n : 0)];
    }
  }
  __device__ __forceinline__ void put(float* lds, int t0, int L, int N) const {
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int id = i * kSelThreads + (int)threadIdx.x;
      if (STEPS * NP % kSelThreads == 0 || id < STEPS * NP)
        lds[id] = t0 + id / NP < L && id % NP < N ? to_f32<DT>(r[i]) : 0.f;
    }
  }
};

// J neighbouring floats.
template <int J>
__device__ __forceinline__ void read_states(const float* p, float (&v)[J]) {
  constexpr int W = J < 4 ? J : 4;
#pragma unroll
  for (int j = 0; j < J; j += W) {
    const SelVec<float, W> r = *reinterpret_cast<const SelVec<float, W>*>(p + j);
#pragma unroll
    for (int i = 0; i < W; ++i) v[j + i] = r.v[i];
  }
}
template <int J>
__device__ __forceinline__ void write_states(float* p, const float (&v)[J]) {
  constexpr int W = J < 4 ? J : 4;
#pragma unroll
  for (int j = 0; j < J; j += W) {
    SelVec<float, W> r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i] = v[j + i];
    *reinterpret_cast<SelVec<float, W>*>(p + j) = r;
  }
}
// The same of a tensor [.., N] whose rows may be shorter than the lanes hold
// (vec: they are not, and aligned); zeros behind N and without a tensor.
template <int J>
__device__ __forceinline__ void load_row(const float* row, int n0, int N, bool vec, float (&v)[J]) {
  if (!row) {
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = 0.f;
  } else if (vec) {
    read_states<J>(row + n0, v);
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = row[n0 + j < N ? n0 + j : N - 1];
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = n0 + j < N ? v[j] : 0.f;
  }
}
template <int J>
__device__ __forceinline__ void store_row(float* row, int n0, int N, bool vec, const float (&v)[J]) {
  if (vec) {
    write_states<J>(row + n0, v);
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (n0 + j < N) row[n0 + j] = v[j];
  }
}

// The grid of a launch over (row, segment)s and tiles of channels.
inline dim3 sel_grid(const SelectiveScanArgs& a) {
  const int64_t units = (int64_t)a.B * a.segs;
  return dim3((unsigned)((units + a.xcds - 1) / a.xcds * a.xcds * a.tiles));
}
inline void sel_tiles(SelectiveScanArgs& a) {
  a.group_tiles = sel_group_tiles(a.H, a.G);
  a.tiles = a.group_tiles * a.G;
  if ((int64_t)a.B * a.segs < a.xcds) a.xcds = 1;  // fewer (row, segment)s than XCDs: spread their tiles instead
}
hipError_t launch_sel_carry(const SelectiveScanArgs& a, const float* first, int NP, bool back, hipStream_t st);

}  // namespace rnnk
