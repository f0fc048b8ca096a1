// Building blocks of the cross-attention kernels.
//
// Products run on the 16x16 matrix instructions. An operand fragment is eight
// elements per lane: lane l holds row (or column) l % 16 and the eight
// elements of the summed dimension that belong to its group g = l / 16. Which
// eight they are does not matter as long as both operands agree; a fp32
// fragment is fed to eight 16x16x4 instructions, a bf16 one to a single
// 16x16x32. A 16x16 result has column l % 16 and rows 4 g .. 4 g + 3 in a
// lane. So two results stacked along their rows are, lane by lane, an operand
// fragment whose summed dimension is those 32 rows, in the order
// 4 g + j (j < 4) and 16 + 4 g + j - 4 (j >= 4): probabilities go from one
// product into the next without leaving their registers.
#pragma once

#include "block_kernels.hpp"
#include "device_common.hpp"

namespace rnnk {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;

// Launches beyond 64 KiB of LDS have to be asked for.
template <typename F>
inline hipError_t allow_lds(F kernel, int bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename DT>
struct Frag;
template <>
struct Frag<bf16> {
  bf16x8 v;
  __device__ __forceinline__ void set(int j, float x) { v[j] = (bf16)x; }
  __device__ __forceinline__ float get(int j) const { return (float)v[j]; }
};
template <>
struct Frag<float> {
  float v[8];
  __device__ __forceinline__ void set(int j, float x) { v[j] = x; }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16>& a, const Frag<bf16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}

// Rows of a tile in LDS lie DP elements plus a pad apart. With 16 bytes of
// pad a wave's fragment reads (16 rows, 16 bytes each) fall on different
// banks, with 32 bytes the transposed reads of bf16 tiles (8 rows, 32 bytes
// each) do; a bf16 tile read both ways takes the pad of its more frequent
// use.
template <typename DT, int DP, bool TR>
struct TileShape {
  static constexpr int kPad = (TR && sizeof(DT) == 2 ? 32 : 16) / sizeof(DT);
  static constexpr int kLd = DP + kPad;
};

// Eight neighbouring elements of row `row`, from column col0 + 8 g.
template <typename DT>
__device__ __forceinline__ Frag<DT> read_rows(const DT* lds, int ld, int row, int col);
template <>
__device__ __forceinline__ Frag<bf16> read_rows<bf16>(const bf16* lds, int ld, int row, int col) {
  Frag<bf16> f;
  f.v = *reinterpret_cast<const bf16x8*>(lds + row * ld + col);
  return f;
}
template <>
__device__ __forceinline__ Frag<float> read_rows<float>(const float* lds, int ld, int row, int col) {
  Frag<float> f;
  const f32x4 a = *reinterpret_cast<const f32x4*>(lds + row * ld + col);
  const f32x4 b = *reinterpret_cast<const f32x4*>(lds + row * ld + col + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
  return f;
}

// The transposed fragment: column col0 + l % 16 of the 32 rows from row0 on,
// in the order of stacked results (see above).
template <typename DT>
__device__ __forceinline__ Frag<DT> read_cols(const DT* lds, int ld, int row0, int col0, int lane);
template <>
__device__ __forceinline__ Frag<bf16> read_cols<bf16>(const bf16* lds, int ld, int row0, int col0, int lane) {
  // The transposing read hands 16 lanes the columns of the 4 x 16 block that
  // their 8-byte reads make up, four lanes a row.
  typedef __attribute__((address_space(3))) s16x4* LdsPtr;
  const int g = lane >> 4, i = lane & 15;
  const bf16* p = lds + (row0 + 4 * g + (i >> 2)) * ld + col0 + 4 * (i & 3);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p + 16 * ld));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  Frag<bf16> f;
  f.v = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  return f;
}
template <>
__device__ __forceinline__ Frag<float> read_cols<float>(const float* lds, int ld, int row0, int col0, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const float* p = lds + (row0 + 4 * g) * ld + col0 + i;
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = p[j * ld], f.v[4 + j] = p[(16 + j) * ld];
  return f;
}

// Two stacked results as the fragment they are.
template <typename DT>
__device__ __forceinline__ Frag<DT> stack(const f32x4& a, const f32x4& b) {
  Frag<DT> f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.set(j, a[j]);
    f.set(4 + j, b[j]);
  }
  return f;
}

// What the rounding of stack() leaves.
__device__ __forceinline__ Frag<bf16> stack_rest(const f32x4& a, const f32x4& b, const Frag<bf16>& f) {
  Frag<bf16> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.set(j, a[j] - f.get(j));
    r.set(4 + j, b[j] - f.get(4 + j));
  }
  return r;
}

// Max and sum over the four lanes that hold a column (l % 16 alike): the
// swaps hand every lane its own value and the one 16 or 32 lanes away.
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void swap16(float v, float* a, float* b) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const u32x2 r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned r0 = r[0], r1 = r[1];  // a bit cast of a vector's element reads its first
  *a = __builtin_bit_cast(float, r0);
  *b = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ void swap32(float v, float* a, float* b) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned r0 = r[0], r1 = r[1];
  *a = __builtin_bit_cast(float, r0);
  *b = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ float col_max(float v) {
  float a, b;
  swap16(v, &a, &b);
  swap32(__builtin_fmaxf(a, b), &a, &b);
  return __builtin_fmaxf(a, b);
}
__device__ __forceinline__ float col_sum(float v) {
  float a, b;
  swap16(v, &a, &b);
  swap32(a + b, &a, &b);
  return a + b;
}

// Scores in base 2, s sl for the raw score s and sl = scale log2(e), relative
// to a reference r: one multiply-add, exact but for its last rounding. r is
// such a product rounded, so that even the largest score lies half a unit in
// r's last place from it; past kCoarse (16 there, and the spacing of scores
// 32: only equal ones share the weight) products are rounded like r instead,
// and clamped to finite values.
constexpr float kLowest = -3.402823466e38f, kHighest = 3.402823466e38f;
constexpr float kCoarse = 536870912.0f;  // 2^29
__device__ __forceinline__ float base2_score(float s, float sl) {
  return __builtin_fmaxf(kLowest, __builtin_fminf(kHighest, s * sl));
}
__device__ __forceinline__ float score_above(float s, float sl, float r) {
  if (__builtin_fabsf(r) <= kCoarse || !__builtin_isfinite(s)) return __builtin_fmaf(s, sl, -r);
  return base2_score(s, sl) - r;
}
// The kept log-sum-exp of a row is a float too. Up to 256 half a unit in its
// last place (2^-17) is small beside what fp32 scores of that size carry
// themselves; past it the backward pass makes up for it.
__device__ __forceinline__ bool large_lse(float lse) {
  return __builtin_fabsf(lse) > 256.0f && __builtin_isfinite(lse);
}

// Eight elements of a row in global memory from column col on; columns past D
// are zero. `vec`: rows take 16-byte accesses and D is a multiple of them.
// FAST kernels are for rows that do and fill their tiles (D = DP): no access
// has a condition on its column then.
template <typename DT, bool FAST>
__device__ __forceinline__ Frag<DT> load8(const DT* row, int col, int D, bool vec) {
  Frag<DT> f;
  if constexpr (FAST) {
    if constexpr (sizeof(DT) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(row + col);
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(row + col), b = *reinterpret_cast<const f32x4*>(row + col + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
    }
    return f;
  }
  if (vec) {
    if constexpr (sizeof(DT) == 2) {
      const u32x4 z = {0, 0, 0, 0};
      f.v = __builtin_bit_cast(bf16x8, col < D ? *reinterpret_cast<const u32x4*>(row + col) : z);
    } else {
      const f32x4 z = {0.f, 0.f, 0.f, 0.f};
      const f32x4 a = col < D ? *reinterpret_cast<const f32x4*>(row + col) : z;
      const f32x4 b = col + 4 < D ? *reinterpret_cast<const f32x4*>(row + col + 4) : z;
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.set(j, col + j < D ? to_f32<DT>(row[col + j]) : 0.f);
  }
  return f;
}

template <typename DT>
__device__ __forceinline__ Frag<DT> zero_frag() {
  Frag<DT> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.set(j, 0.f);
  return f;
}

template <typename DT>
__device__ __forceinline__ void put8(DT* lds, const Frag<DT>& f) {
  if constexpr (sizeof(DT) == 2) {
    *reinterpret_cast<bf16x8*>(lds) = f.v;
  } else {
    *reinterpret_cast<f32x4*>(lds) = f32x4{f.v[0], f.v[1], f.v[2], f.v[3]};
    *reinterpret_cast<f32x4*>(lds + 4) = f32x4{f.v[4], f.v[5], f.v[6], f.v[7]};
  }
}

// Four results of a lane (neighbouring columns of one row) to global memory.
template <typename DT, bool FAST>
__device__ __forceinline__ void store4(DT* row, int col, int D, bool vec, const f32x4& v) {
  if (FAST || vec) {
    if (FAST || col < D) {
      if constexpr (sizeof(DT) == 2) {
        bf16x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (bf16)v[j];
        *reinterpret_cast<bf16x4*>(row + col) = o;
      } else {
        *reinterpret_cast<f32x4*>(row + col) = v;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < D) row[col + j] = from_f32<DT>(v[j]);
  }
}

// A row's offset: FAST kernels are launched only where every offset inside a
// (batch row, key head) of q, do and of a tile of k and v fits 31 bits of
// bytes, so that a load takes a scalar base and a 32-bit offset.
template <bool FAST>
struct Offset {
  typedef int64_t type;
};
template <>
struct Offset<true> {
  typedef uint32_t type;
};

// A tile of rows row0 .. row0 + ROWS - 1 of an array whose rows lie `stride`
// apart, zero from row `limit` on, from global memory into LDS: in two
// halves, so that a tile's loads are in flight while the one before it is
// worked on.
template <typename DT, int DP, int ROWS, int LD, bool FAST>
struct TileLoad {
  typedef typename Offset<FAST>::type Off;
  static constexpr int kCols = DP / 8, kTotal = ROWS * kCols, kIters = (kTotal + kAttnThreads - 1) / kAttnThreads;
  Frag<DT> f[kIters];
  __device__ __forceinline__ static Off at(int n, Off stride) {
    const int k = n * kAttnThreads + threadIdx.x;
    return (Off)(k / kCols) * stride + (Off)((k % kCols) * 8);
  }
  __device__ __forceinline__ void load(const DT* base, int64_t stride, int row0, int limit, int D, bool vec) {
    base += row0 * stride;
    if (FAST && row0 + ROWS <= limit) {  // the same for the whole workgroup: no condition per row
#pragma unroll
      for (int n = 0; n < kIters; ++n)
        if (kTotal % kAttnThreads == 0 || n * kAttnThreads + (int)threadIdx.x < kTotal)
          f[n] = load8<DT, FAST>(base + at(n, (Off)stride), 0, D, vec);
      return;
    }
#pragma unroll
    for (int n = 0; n < kIters; ++n) {
      const int k = n * kAttnThreads + threadIdx.x, c = k % kCols * 8;
      const bool on = (kTotal % kAttnThreads == 0 || k < kTotal) && row0 + k / kCols < limit;
      f[n] = on ? load8<DT, FAST>(base + at(n, (Off)stride) - c, c, D, vec) : zero_frag<DT>();
    }
  }
  __device__ __forceinline__ void put(DT* lds) const {
#pragma unroll
    for (int n = 0; n < kIters; ++n) {
      const int k = n * kAttnThreads + threadIdx.x;
      if (kTotal % kAttnThreads == 0 || k < kTotal) put8<DT>(lds + k / kCols * LD + (k % kCols) * 8, f[n]);
    }
  }
};

// Query rows of one key head: row m is step m / G of query head hk G + m % G.
struct QRows {
  int M, G;
  template <typename DT>
  __device__ __forceinline__ const DT* in(const void* p, int64_t st, int64_t sh, int m) const {
    const int t = m / G;
    return (const DT*)p + t * st + (m - t * G) * sh;
  }
  // offset of row m in a dense [Tq, B, heads, D]
  __device__ __forceinline__ int64_t dense(const AttentionArgs& a, int b, int hk, int m) const {
    const int t = m / G;
    return (((int64_t)t * a.B + b) * a.heads + hk * G + (m - t * G)) * a.D;
  }
};

// The same for consecutive tiles of query rows: a thread carries each of its
// rows along as (head in the group, offset), so that no tile divides, and
// where G divides ROWS only the scalar base moves.
template <typename DT, int DP, int ROWS, int LD, bool FAST, int NT = kAttnThreads>
struct QueryLoad {
  typedef typename Offset<FAST>::type Off;
  static constexpr int kCols = DP / 8, kTotal = ROWS * kCols, kIters = (kTotal + NT - 1) / NT;
  Frag<DT> f[kIters];
  int h[kIters];
  Off off[kIters];
  const DT* base;
  int64_t step;  // of the base, per tile
  Off shift, wrap;
  int dh;
  __device__ __forceinline__ void start(const DT* p, int64_t st, int64_t sh, int G) {
    base = p;
    const int dt = ROWS / G;
    dh = ROWS - dt * G;
    step = dt * st;
    shift = (Off)dh * (Off)sh;
    wrap = (Off)st - (Off)G * (Off)sh;
#pragma unroll
    for (int n = 0; n < kIters; ++n) {
      const int m = (n * NT + (int)threadIdx.x) / kCols, t = m / G;
      h[n] = m - t * G;
      off[n] = (Off)t * (Off)st + (Off)h[n] * (Off)sh;
    }
  }
  __device__ __forceinline__ void next(int G) {
    base += step;
    if (dh != 0) {
#pragma unroll
      for (int n = 0; n < kIters; ++n) {
        h[n] += dh;
        const bool over = h[n] >= G;
        off[n] += over ? shift + wrap : shift;
        if (over) h[n] -= G;
      }
    }
  }
  __device__ __forceinline__ void load(int m0, int M, int D, bool vec) {
    if (FAST && m0 + ROWS <= M) {
#pragma unroll
      for (int n = 0; n < kIters; ++n) {
        const int k = n * NT + threadIdx.x;
        if (kTotal % NT == 0 || k < kTotal)
          f[n] = load8<DT, FAST>(base + (Off)(off[n] + (Off)(k % kCols * 8)), 0, D, vec);
      }
      return;
    }
#pragma unroll
    for (int n = 0; n < kIters; ++n) {
      const int k = n * NT + threadIdx.x;
      const bool on = (kTotal % NT == 0 || k < kTotal) && m0 + k / kCols < M;
      f[n] = on ? load8<DT, FAST>(base + off[n], k % kCols * 8, D, vec) : zero_frag<DT>();
    }
  }
  __device__ __forceinline__ void put(DT* lds) const {
#pragma unroll
    for (int n = 0; n < kIters; ++n) {
      const int k = n * NT + threadIdx.x;
      if (kTotal % NT == 0 || k < kTotal) put8<DT>(lds + k / kCols * LD + (k % kCols) * 8, f[n]);
    }
  }
};

// Which tile a workgroup owns. Workgroup ids are dealt to the XCDs in turn.
// The tiles of one (batch row, key head) are cut into up to kParts parts
// (every kParts-th tile); a part's tiles run on one XCD one after the other,
// so that they share its L2, and the parts of a row fall on different XCDs,
// so that rows of different lengths load the XCDs evenly. Each part begins
// one tile further on than the one before it: an XCD's compute units are
// dealt workgroups in turn too, and the last tiles of a short row are idle.
struct Work {
  int bh, tile;  // tile < tiles, or the workgroup has none
};
constexpr int kParts = 4;
// With 16 (row, key head)s an XCD the rows' lengths even out by themselves,
// and a row's tiles stay together.
inline __host__ __device__ int part_count(const AttentionArgs& a, int tiles) {
  if (a.B * a.kv_heads >= 16 * a.xcds) return 1;
  return tiles < kParts ? tiles : kParts;
}
__device__ __forceinline__ Work work_of(const AttentionArgs& a, int tiles) {
  const int parts = part_count(a, tiles), each = (tiles + parts - 1) / parts;
  const int xcd = blockIdx.x % a.xcds, slot = blockIdx.x / a.xcds;
  const int turn = slot / each, unit = turn * a.xcds + xcd, within = (slot + turn) % each;
  Work w;
  w.bh = unit / parts;
  w.tile = within * parts + unit % parts;
  if (w.bh >= a.B * a.kv_heads) w.tile = tiles;
  return w;
}
inline int64_t work_grid(const AttentionArgs& a, int64_t tiles) {
  const int parts = part_count(a, (int)tiles);
  const int64_t each = (tiles + parts - 1) / parts, units = (int64_t)a.B * a.kv_heads * parts;
  return (units + a.xcds - 1) / a.xcds * a.xcds * each;
}

__device__ __forceinline__ int key_count(const AttentionArgs& a, int b) {
  const int n = a.lengths ? a.lengths[b] : a.Tk;
  return n < 0 ? 0 : (n > a.Tk ? a.Tk : n);
}

}  // namespace rnnk
