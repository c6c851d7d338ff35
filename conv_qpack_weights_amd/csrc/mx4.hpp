// mx4.hpp -- what the operators of microscaled 4-bit floating point share: the
// matrices' view, operands, conversions.
//
// A row is K values of four bits, e2m1 (sign, two exponent bits, one of
// mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte, the first in the low bits;
// every 32 of them (16 bytes) share a scale byte s, and stand for the value
// times 2^(s - 127) (s = 255: the block is NaN).  Sixteen bytes with one scale
// are what a lane holds of a scaled 4-bit MFMA operand, so the matrices are used
// as they lie in memory, row after row, weights and quantized rows alike.
//
// A value times its scale is a bf16 exactly (one bit of mantissa, 8 of exponent,
// subnormal ones included), which v_cvt_scalef32_pk_bf16_fp4 gives two of at a
// time: float rows are multiplied with the weights in bf16 MFMAs with no
// rounding but that of the f32 sums.
#pragma once

#include "dev_util.hpp"
#include "float_types.hpp"
#include "qp_internal.hpp"
#include "w4.hpp"

namespace qp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int64_t kMxMaxK = INT64_C(1) << 22;   // lane offsets within a tile in 32 bits
constexpr int64_t kMxMaxLd = INT64_C(1) << 23;

// Rows of the row type "MXFP4" in the kernels' templates.
struct mx4_t {};

struct MxMat {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ldc, lds;           // bytes between rows
  int64_t cstride, sstride;   // bytes between matrices (experts)
  int64_t rows, K;
  int64_t G;                  // blocks of a row
};

// ---- operands ----------------------------------------------------------------
// The f32 whose exponent bits are the scale byte: what the conversions take
// (they read the exponent alone: 0 stands for 2^-127, 255 for NaN).
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __builtin_bit_cast(float, s << 23);
}

// The eight values of a word of codes, as bf16.
__device__ __forceinline__ bf16x8 mx_unpack(uint32_t w, float scale) {
  u32x4 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(bf16x8, o);
}

// Whether a block's weights are f16 values, exactly: its scale one of 2^-23 .. 2^13
// (then 0.5 and 6 times it are), which the weights of layers have, or all its codes
// zeros under any scale but NaN's (the quantizer gives zeros the smallest).  The kernels
// ask for the scales alone at their steps; the tiles, which begin again where one is out
// of range, look at its codes before they do.
__device__ __forceinline__ bool mx_f16_scale(float scale) {
  return __builtin_bit_cast(uint32_t, scale) - (104u << 23) <= (36u << 23);
}
__device__ __forceinline__ bool mx_f16_block(u32x4 codes, float scale) {
  return mx_f16_scale(scale) || (((codes[0] | codes[1] | codes[2] | codes[3]) & 0x77777777u) == 0 &&
                                 __builtin_bit_cast(uint32_t, scale) < (255u << 23));
}
// The eight values of a word of codes as f16, where they are.
__device__ __forceinline__ f16x8 mx_unpack_f16(uint32_t w, float scale) {
  u32x4 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3));
  return __builtin_bit_cast(f16x8, o);
}

// d + a b^T over 128 K: lane l holds 32 values of row l%16 from 32 (l/16) on
// and their scale in the low byte of sa / sb.
__device__ __forceinline__ f32x4 mx_mfma16(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 d) {
  const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, d, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Eight elements of a float row as bf16 pieces whose sum they are exactly: one
// for bf16, two for f16 (8 + 3 of its 11 bits), three for f32; the smallest
// first.  The cuts truncate; an infinity or a NaN is the largest piece alone.
template <typename T>
struct MxFrag : XFrag<T> {};

template <>
struct MxFrag<f16_t> {
  static constexpr int kPieces = 2;
  using vec = bf16x8;
  u32x4 v;
  __device__ __forceinline__ void load(const f16_t* p) {
    v = *reinterpret_cast<const u32x4_any*>(p);
  }
  __device__ __forceinline__ void load_n(const f16_t* p, int n) { v = load_piece(p, n).v; }
  __device__ __forceinline__ void split(vec (&o)[2]) const {
    const f16x8 f = __builtin_bit_cast(f16x8, v);
    u32x4 h4, l4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2], l[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float x = (float)f[2 * i + j];
        const uint32_t u = __builtin_bit_cast(uint32_t, x);
        h[j] = u & 0xffff0000u;
        const float r = x - __builtin_bit_cast(float, h[j]);
        l[j] = (u & 0x7f800000u) == 0x7f800000u ? 0u : __builtin_bit_cast(uint32_t, r);
      }
      h4[i] = hi_halves(h[0], h[1]);
      l4[i] = hi_halves(l[0], l[1]);
    }
    o[0] = __builtin_bit_cast(bf16x8, l4);
    o[1] = __builtin_bit_cast(bf16x8, h4);
  }
};

// ---- arguments of the products -----------------------------------------------
struct MxArgs {
  MxMat w;
  W4Rows rows;
  const void* X;       // float rows
  int64_t ldx;
  MxMat a;             // or MXFP4 rows
  const float* bias;   // [experts][N] or null
  float lo, hi;
  void* Y;
  int32_t y_dtype;
  int64_t ldy;
};

// Workgroups go round the 8 XCDs in launch order: gives each XCD a run of
// neighbouring tiles, which share an L2.
__device__ __forceinline__ uint32_t xcd_run(uint32_t id, uint32_t n) {
  const uint32_t per = n / 8, rest = n % 8, x = id % 8;
  return x * per + (x < rest ? x : rest) + id / 8;
}

// ---- host side ---------------------------------------------------------------
// The shapes of the products' kernels, see mx_choose: rows x channels of a workgroup.
enum MxShape {
  kMxRows16x16,
  kMxRows16x32,
  kMxRows16x48,
  kMxRows16x64,
  kMxTile32x64,
  kMxTile32x128,
  kMxTile64x64,
  kMxTile128x128,
  kMxTile256x256
};

// What a shape takes at K = 4096, the only length it was measured at (the choice does
// not look at K): `first` microseconds for up to one workgroup a CU (256); `cold` for
// every further round of workgroups that bring weights of their own, `more` for one that
// finds its weights in the caches (further row tiles of the same matrix).  Rounds are
// whole ones for the few-row kernels, whose workgroups all wait for memory alike; the
// largest tile is one to a CU, its last round in halves where it is half empty.
struct MxCost {
  MxShape shape;
  int rows, channels;
  double first, cold, more;
  const char* name;
};
double mx_halved_rounds(double rounds);
const MxCost& mx_choose(const MxCost* shapes, int n, int64_t M, int64_t parts, int64_t N);
const MxCost& mx_a4w4_shape(int64_t M, int64_t parts, int64_t N);
const MxCost& mx_w4_shape(int32_t dtype, int64_t M, int64_t parts, int64_t N);
void mx_dx_kernel_name(const qp_mx4* w, int32_t dtype, int64_t M, char* name, size_t bytes);

// The tiles' direct loads take 32-bit offsets from a tile's first row (from row 0
// through a map): rows `row_bytes` apart, x_rows of them.
inline bool mx_tile_reaches(const W4Rows& rows, int64_t row_bytes) {
  constexpr int64_t kMost = (INT64_C(1) << 31) - 1;
  return row_bytes <= kMost / 256 && (!rows.map || rows.x_rows <= kMost / row_bytes);
}

// How many tiles of 16 rows the rows have, about: one of every expert that has any, or what
// all of them take.
inline int64_t mx_row_tiles(const MxArgs& a) {
  const int64_t tiles = ceil_div(a.rows.M, 16);
  const int64_t parts = !a.rows.offsets           ? 1
                        : a.rows.experts < a.rows.M ? (int64_t)a.rows.experts
                                                    : a.rows.M;
  return tiles > parts ? tiles : parts;
}

// Whether tiles of `tile` rows are about one a matrix, so that each reads its weights alone.
inline bool mx_read_once(const MxArgs& a, int64_t tile) {
  return a.rows.M <= tile * (a.rows.offsets ? a.rows.experts : 1);
}

MxMat mx_view(const qp_mx4* m);
qp_status mx_check(const char* what, const char* name, const qp_mx4* m);
qp_status run_mx_a4w4(const MxArgs& a, hipStream_t stream);
qp_status run_mx_f32(const MxArgs& a, hipStream_t stream);
qp_status run_mx_bf16(const MxArgs& a, hipStream_t stream);
qp_status run_mx_f16(const MxArgs& a, hipStream_t stream);

}  // namespace qp
