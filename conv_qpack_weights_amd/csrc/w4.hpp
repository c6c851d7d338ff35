// w4.hpp -- what the weight-only int4 products share: the blob's view, the
// rows of an expert's tile, operand fragments, int4 to float.
//
// The blob (see qpack_weights in the header): channel n, 128-K block b at
// ((n/16)*nblk + b)*1024 + (n%16)*64; the word at byte 16c + 4t of it holds
// k = 128b + 32t + 8c + j in the low nibble of byte j and k + 4 in the high
// one.  Lane l of a v_mfma_*_16x16x32 operand holds row l%16 and the eight
// reduction indexes 8*(l/16) ..: so lane l's 16-byte load at chunk c = l/16 of
// channel l%16 is, word by word, the operand of the block's four 32-K steps,
// and a wave's load is one contiguous kilobyte.
#pragma once

#include "dev_util.hpp"
#include "float_types.hpp"
#include "qp_internal.hpp"

namespace qp {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// kind: 0 f32 scales, 1 bf16 scales, 2 f32 scales and offsets
struct W4View {
  const uint8_t* blob;     // expert 0
  int64_t expert_stride;   // bytes
  int64_t data_off, scale_off, offs_off;
  int64_t N, Npad, K, nblk;
  int64_t G4;              // quads of groups per channel
  int32_t group;
};

// Rows grouped by expert: rows [offsets[e], offsets[e+1]) are expert e's.
// offsets null: one expert with all rows.  map: row r of the product reads
// row map[r]/map_div of X, if that is one of its x_rows rows.
struct W4Rows {
  const int32_t* offsets;
  int32_t experts;
  int64_t M;
  const int32_t* map;
  int64_t map_div, x_rows;
};

constexpr int64_t kW4MaxRows = INT64_C(1) << 30;  // row numbers and tile counts in 32 bits

struct W4Tile {
  int32_t expert;   // == experts: rows of no expert (stored as zeros); -1: nothing
  int64_t r0, r1;   // rows
};

// How many BM-row tiles any split of M rows over the experts (and the rows of
// no expert) can have.
inline int64_t w4_tile_slots(const W4Rows& r, int64_t BM) {
  if (!r.offsets) return ceil_div(r.M, BM);
  const int64_t parts = r.experts + 1 < r.M ? r.experts + 1 : r.M;
  return (r.M + (BM - 1) * parts) / BM;
}

// Tile number `slot` of the rows: the experts' tiles in order, then those of
// the rows past offsets[experts].  Every wave works it out for itself: a lane
// per expert, a running sum over the wave.  Offsets are clamped to [0, M], so
// that no offsets can send a tile outside the rows.
template <int BM>
__device__ __forceinline__ W4Tile w4_find_tile(const W4Rows& rows, int64_t slot) {
  if (!rows.offsets) {
    const int64_t r0 = slot * BM;
    return W4Tile{0, r0, r0 + BM < rows.M ? r0 + BM : rows.M};
  }
  const int lane = threadIdx.x & 63;
  const int32_t M = (int32_t)rows.M;
  int32_t base = 0;
  for (int e0 = 0; e0 <= rows.experts; e0 += 64) {
    const int e = e0 + lane;
    int32_t a = M, b = M;
    if (e <= rows.experts) {
      a = rows.offsets[e];
      if (e < rows.experts) b = rows.offsets[e + 1];
    }
    a = a < 0 ? 0 : a > M ? M : a;
    b = b < a ? a : b > M ? M : b;
    int32_t incl = (b - a + BM - 1) / BM;
    const int32_t mine = incl;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t up = __shfl_up(incl, d);
      if (lane >= d) incl += up;
    }
    const int32_t lo = base + incl - mine;
    const uint64_t hit = __ballot(slot >= lo && slot < base + incl);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int32_t ra = __builtin_amdgcn_readlane(a, src);
      const int32_t rb = __builtin_amdgcn_readlane(b, src);
      const int32_t first = __builtin_amdgcn_readlane(lo, src);
      const int64_t r0 = ra + (slot - first) * BM;
      return W4Tile{e0 + src, r0, r0 + BM < rb ? r0 + BM : rb};
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return W4Tile{-1, 0, 0};
}

// The row of X that row r of the product reads; -1: none.
__device__ __forceinline__ int64_t w4_source_row(const W4Rows& rows, int64_t r) {
  if (!rows.map) return r;
  const int32_t m = rows.map[r];
  const int64_t x = m < 0 ? -1 : (int64_t)((uint32_t)m / (uint32_t)rows.map_div);
  return x < rows.x_rows ? x : -1;
}

// ---- operand fragments -----------------------------------------------------
// The MFMA operands of 8 consecutive row elements: as they are for bf16 and
// f16; an f32 value is cut into three bf16 whose sum it is exactly (8 + 8 + 8
// bits of its 24), so the product keeps f32 accuracy at three MFMAs.
// load_n: the first n elements, the rest zero; the pointer must be readable for
// one element even where n <= 0.
template <typename T>
struct XFrag;

template <>
struct XFrag<f16_t> {
  static constexpr int kPieces = 1;
  using vec = f16x8;
  u32x4 v;
  __device__ __forceinline__ void load(const f16_t* p) {
    v = *reinterpret_cast<const u32x4_any*>(p);
  }
  __device__ __forceinline__ void load_n(const f16_t* p, int n) { v = load_piece(p, n).v; }
  __device__ __forceinline__ void split(vec (&o)[1]) const {
    o[0] = __builtin_bit_cast(f16x8, v);
  }
};

template <>
struct XFrag<bf16_t> {
  static constexpr int kPieces = 1;
  using vec = bf16x8;
  u32x4 v;
  __device__ __forceinline__ void load(const bf16_t* p) {
    v = *reinterpret_cast<const u32x4_any*>(p);
  }
  __device__ __forceinline__ void load_n(const bf16_t* p, int n) { v = load_piece(p, n).v; }
  __device__ __forceinline__ void split(vec (&o)[1]) const {
    o[0] = __builtin_bit_cast(bf16x8, v);
  }
};

// upper halves of two words: (hi(a), hi(b)) as two bf16, a first
__device__ __forceinline__ uint32_t hi_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// x = h + m + l, each a bf16 (the upper half of the words returned).  The
// cuts truncate, so that h stays finite; an infinity or NaN is h alone (a
// NaN with its quiet bit set, which the cut could drop).
__device__ __forceinline__ void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const bool special = (u & 0x7f800000u) == 0x7f800000u;
  h = u & 0xffff0000u;
  const float r = special ? 0.0f : x - __builtin_bit_cast(float, h);
  if (x != x) h |= 0x00400000u;
  m = __builtin_bit_cast(uint32_t, r) & 0xffff0000u;
  l = __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, m));
}

template <>
struct XFrag<float> {
  static constexpr int kPieces = 3;
  using vec = bf16x8;
  u32x4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = reinterpret_cast<const u32x4_any*>(p)[0];
    v[1] = reinterpret_cast<const u32x4_any*>(p)[1];
  }
  __device__ __forceinline__ void load_n(const float* p, int n) {
    v[0] = load_piece(p, n).v;
    v[1] = load_piece(p + (n > 4 ? 4 : 0), n - 4).v;
  }
  // o[0] the smallest piece, o[2] the largest
  __device__ __forceinline__ void split(vec (&o)[3]) const {
    u32x4 h4, m4, l4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = v[i / 2][2 * (i % 2)], b = v[i / 2][2 * (i % 2) + 1];
      uint32_t ha, ma, la, hb, mb, lb;
      split3(__builtin_bit_cast(float, a), ha, ma, la);
      split3(__builtin_bit_cast(float, b), hb, mb, lb);
      h4[i] = hi_halves(ha, hb);
      m4[i] = hi_halves(ma, mb);
      l4[i] = hi_halves(la, lb);
    }
    o[0] = __builtin_bit_cast(bf16x8, l4);
    o[1] = __builtin_bit_cast(bf16x8, m4);
    o[2] = __builtin_bit_cast(bf16x8, h4);
  }
};

__device__ __forceinline__ f32x4 mfma32(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The low four bits of x, a signed integer q, as q/16 (exact).
__device__ __forceinline__ float nib_f32(uint32_t x) {
  return __builtin_amdgcn_cvt_off_f32_i4((int)x);
}

// The eight values of a blob word as q/16 in the rows' type, in K order:
// q/16 has at most four significant bits, so both types hold it exactly.
template <typename V>
__device__ __forceinline__ V w4_unpack(uint32_t w) {
  uint32_t h = w >> 4;
  // (kept as one shift: the compiler would shift out each high nibble instead
  // of selecting bytes inside the conversion)
  asm("" : "+v"(h));
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = nib_f32((w >> (8 * j)) & 0xffu);
    f[4 + j] = nib_f32((h >> (8 * j)) & 0xffu);
  }
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(V) == sizeof(f16x8) && __is_same(V, f16x8))
      o[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[2 * i], f[2 * i + 1]));
    else
      o[i] = hi_halves(__builtin_bit_cast(uint32_t, f[2 * i]),
                       __builtin_bit_cast(uint32_t, f[2 * i + 1]));
  }
  return __builtin_bit_cast(V, o);
}

// Clamp and store one output in any of the row types (a NaN passes the clamp).
__device__ __forceinline__ void w4_store(void* Y, int32_t dtype, int64_t at, float y) {
  if (dtype == QP_F32)
    static_cast<float*>(Y)[at] = y;
  else if (dtype == QP_BF16)
    static_cast<bf16_t*>(Y)[at] = from_f32<bf16_t>(y);
  else
    static_cast<f16_t*>(Y)[at] = from_f32<f16_t>(y);
}

// The first n of eight neighbouring outputs.
__device__ __forceinline__ void w4_store8(void* Y, int32_t dtype, int64_t at, const float (&y)[8],
                                          int n) {
  if (dtype == QP_F32) {
    float* p = static_cast<float*>(Y) + at;
    const float lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
    store_piece(p, lo, n);
    if (n > 4) store_piece(p + 4, hi, n - 4);
  } else if (dtype == QP_BF16) {
    store_piece(static_cast<bf16_t*>(Y) + at, y, n);
  } else {
    store_piece(static_cast<f16_t*>(Y) + at, y, n);
  }
}

struct W4Args {
  W4View w;
  W4Rows rows;
  const void* X;
  int64_t ldx;
  const float* bias;   // [experts][N] or null
  float lo, hi;
  void* Y;
  int32_t y_dtype;
  int64_t ldy;
};

// Orders a wave's LDS accesses before it and after it (a wave's own complete in
// order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- host side -------------------------------------------------------------
// The shapes of the kernels (16-row fragments, 16-channel tiles of a workgroup),
// see w4_choose.
enum W4Shape { kRows1x1, kRows1x2, kRows1x3, kRows1x4, kRows2x3, kRows2x4, kTile4x8, kTile8x8 };
qp_status run_w4_f32(const W4Args& a, int32_t format, W4Shape shape, hipStream_t stream);
qp_status run_w4_bf16(const W4Args& a, int32_t format, W4Shape shape, hipStream_t stream);
qp_status run_w4_f16(const W4Args& a, int32_t format, W4Shape shape, hipStream_t stream);

// the gradient's kernel for M rows, see qgemm_w4_kernel_name
void w4_dx_kernel_name(int64_t M, const qp_packed_info* w, int32_t dtype, int64_t experts,
                       char* name, size_t bytes);

W4View w4_view(const qp_packed_info* w, const void* packed, int64_t expert_stride);
qp_status w4_check_weights(const char* what, const qp_packed_info* w, const void* packed,
                           int64_t experts, int64_t expert_stride);
qp_status w4_check_float(const char* what, const char* name, const void* p, int32_t dtype,
                         int64_t ld, int64_t cols);

}  // namespace qp
