// mx4_quant.hip -- rows to MXFP4 and back.
//
// quantize: per block of 32, s = the biased exponent of the largest magnitude
// less 2 (kCeil: one more where that magnitude is above 6 2^(s-127)), at least
// 0; the codes are x 2^(127-s) rounded to the nearest e2m1 value, ties to the
// even code, 6 at most.  The largest magnitude is found on the bits, where
// infinities and NaN come out largest: their block gets s = 255 and zero codes.
// x 2^(127-s) is exact (or far below 0.25, a zero code), so each value is rounded
// once, by v_cvt_scalef32_pk_fp4_f32.
//
// Four lanes hold a block, eight elements each, so a wave reads 512 elements of a
// row in 16-byte pieces and writes 256 bytes of codes.  Bound by memory: 8192 x 4096
// bf16 to codes in 13.4 us (85 MB, 6.3 TB/s from what the caches still hold), back to f32
// in 24 (152 MB); 16 x 4096 2.7 us each, a launch's.
#include "mx4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

// The largest over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true);  // lanes 1 0 3 2
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);           // lanes 2 3 0 1
  return v > o ? v : o;
}

// Eight elements from p on, the first n of them (none for n <= 0; p readable for
// one element in any case), the rest zero.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&f)[8]) {
  constexpr int kPer = Piece<T>::kPer;
#pragma unroll
  for (int h = 0; h < 8 / kPer; ++h) {
    const Piece<T> v = load_piece(p + (n > h * kPer ? h * kPer : 0), n - h * kPer);
#pragma unroll
    for (int i = 0; i < kPer; ++i) f[h * kPer + i] = v.get(i);
  }
}

// `at` numbers the pieces of eight elements of row0, row0 + step, ...: a thread
// keeps its place in the row and goes down the rows.
template <typename T, bool kCeil>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* __restrict__ X, int64_t M,
                                                          int64_t K, int64_t ldx, uint32_t pieces,
                                                          int64_t step, uint8_t* __restrict__ codes,
                                                          int64_t ldc, uint8_t* __restrict__ scales,
                                                          int64_t lds) {
  const uint32_t at = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row0 = at / pieces, piece = at - row0 * pieces;
  const int64_t k = (int64_t)piece * 8;
  const int n = K - k > 8 ? 8 : K - k < 0 ? 0 : (int)(K - k);
  // (pieces is a multiple of 4: a block's four lanes are of one row and leave
  // together)
  for (int64_t m = row0; row0 < step && m < M; m += step) {
    float f[8];
    load8(X + m * ldx + (n > 0 ? k : 0), n, f);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __builtin_bit_cast(uint32_t, f[i]) & 0x7fffffffu;
      big = b > big ? b : big;
    }
    big = quad_max(big);
    const bool nan = big >= 0x7f800000u;
    int s = (int)(big >> 23) - 2 + (kCeil && (big & 0x7fffffu) > 0x400000u ? 1 : 0);
    s = s < 0 ? 0 : s;
    const float by = __builtin_bit_cast(float, (uint32_t)(254 - s) << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0] * by, f[1] * by, 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2] * by, f[3] * by, 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4] * by, f[5] * by, 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6] * by, f[7] * by, 1.0f, 3);
    *reinterpret_cast<uint32_t*>(codes + m * ldc + piece * 4) = nan ? 0u : c;
    if ((piece & 3) == 0) scales[m * lds + piece / 4] = (uint8_t)(nan ? 255 : s);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(MxMat a, uint32_t pieces, int64_t step,
                                                            T* __restrict__ Y, int64_t ldy) {
  const uint32_t at = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row0 = at / pieces, piece = at - row0 * pieces;
  const int64_t k = (int64_t)piece * 8;
  const int n = a.K - k > 8 ? 8 : (int)(a.K - k);
  for (int64_t m = row0; row0 < step && m < a.rows; m += step) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(a.codes + m * a.ldc + piece * 4);
    const float s = mx_scale(a.scales[m * a.lds + piece / 4]);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      f32x2 p;
      if (i == 0) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
      if (i == 2) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
      if (i == 4) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
      if (i == 6) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
      f[i] = p[0];
      f[i + 1] = p[1];
    }
    T* y = Y + m * ldy + k;
    if constexpr (sizeof(T) == 4) {
      const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
      store_piece(y, lo, n);
      if (n > 4) store_piece(y + 4, hi, n - 4);
    } else {
      store_piece(y, f, n);
    }
  }
}

// Rows at a time and workgroups: up to 2048 threads a CU, every one with a piece.
struct Grid {
  int64_t step;
  unsigned blocks;
};
Grid row_grid(int64_t M, int64_t pieces) {
  int64_t step = ceil_div(INT64_C(256) * 2048, pieces);
  if (step > M) step = M;
  return Grid{step, (unsigned)ceil_div(step * pieces, 256)};
}

template <typename T>
void quantize(const void* X, int64_t M, int64_t K, int64_t ldx, int32_t rule, uint8_t* codes,
              int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t stream) {
  const int64_t pieces = ceil_div(K, 32) * 4;
  const Grid g = row_grid(M, pieces);
  if (rule == QP_MX_CEIL)
    hipLaunchKernelGGL((mx_quantize_kernel<T, true>), dim3(g.blocks), dim3(256), 0, stream,
                       static_cast<const T*>(X), M, K, ldx, (uint32_t)pieces, g.step, codes, ldc,
                       scales, lds);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<T, false>), dim3(g.blocks), dim3(256), 0, stream,
                       static_cast<const T*>(X), M, K, ldx, (uint32_t)pieces, g.step, codes, ldc,
                       scales, lds);
}

template <typename T>
void dequantize(const MxMat& a, void* Y, int64_t ldy, hipStream_t stream) {
  const int64_t pieces = ceil_div(a.K, 8);
  const Grid g = row_grid(a.rows, pieces);
  hipLaunchKernelGGL((mx_dequantize_kernel<T>), dim3(g.blocks), dim3(256), 0, stream, a,
                     (uint32_t)pieces, g.step, static_cast<T*>(Y), ldy);
}

}  // namespace

MxMat mx_view(const qp_mx4* m) {
  return MxMat{m->codes,        m->scales,        m->ld_codes, m->ld_scales, m->codes_stride,
               m->scales_stride, m->rows, m->K,   ceil_div(m->K, 32)};
}

qp_status mx_check(const char* what, const char* name, const qp_mx4* m) {
  QP_REQUIRE(m, QP_EINVAL, "%s: %s is null", what, name);
  QP_REQUIRE(m->rows >= 0 && m->K > 0, QP_EINVAL, "%s: %s has %lld rows of K=%lld", what, name,
             (long long)m->rows, (long long)m->K);
  QP_REQUIRE(m->K <= kMxMaxK && m->rows <= kW4MaxRows, QP_EUNSUPPORTED,
             "%s: %s has more than 2^30 rows or K above 2^22", what, name);
  const int64_t G = ceil_div(m->K, 32);
  QP_REQUIRE(m->ld_codes >= 16 * G, QP_EINVAL,
             "%s: the codes' stride of %s is below 16 bytes a block",
             what, name);
  QP_REQUIRE(m->ld_scales >= round_up(G, 4), QP_EINVAL,
             "%s: the scales' stride of %s is below a row's blocks rounded up to 4", what, name);
  QP_REQUIRE(m->ld_codes <= kMxMaxLd && m->ld_scales <= kMxMaxLd, QP_EUNSUPPORTED,
             "%s: the rows of %s are more than 2^23 bytes apart", what, name);
  QP_REQUIRE(m->matrices >= 1, QP_EINVAL, "%s: %s needs at least one matrix", what, name);
  QP_REQUIRE(m->matrices <= 65536, QP_EUNSUPPORTED, "%s: %s has more than 65536 matrices", what,
             name);
  QP_REQUIRE(m->matrices == 1 || (m->codes_stride >= 0 && m->scales_stride >= 0), QP_EINVAL,
             "%s: a stride between the matrices of %s is negative", what, name);
  if (m->rows == 0) return QP_OK;
  QP_REQUIRE(m->codes && m->scales, QP_EINVAL, "%s: %s has null codes or scales", what, name);
  QP_REQUIRE((uintptr_t)m->codes % 16 == 0 && m->ld_codes % 16 == 0 &&
                 (m->matrices == 1 || m->codes_stride % 16 == 0),
             QP_EALIGN, "%s: the codes of %s must be at multiples of 16 bytes", what, name);
  QP_REQUIRE((uintptr_t)m->scales % 4 == 0 && m->ld_scales % 4 == 0 &&
                 (m->matrices == 1 || m->scales_stride % 4 == 0),
             QP_EALIGN, "%s: the scales of %s must be at multiples of 4 bytes", what, name);
  return QP_OK;
}

}  // namespace qp

extern "C" qp_status qquantize_rows_mx4(const void* X, int32_t dtype, int64_t M, int64_t K,
                                        int64_t ldx, int32_t rule, uint8_t* codes,
                                        int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                                        hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qquantize_rows_mx4";
  QP_REQUIRE(rule == QP_MX_FLOOR || rule == QP_MX_CEIL, QP_EINVAL,
             "%s: rule must be QP_MX_FLOOR or QP_MX_CEIL (got %d)", what, rule);
  const qp_mx4 out{codes, scales, M, K, ld_codes, ld_scales, 1, 0, 0};
  qp_status st = mx_check(what, "the result", &out);
  if (st) return st;
  if (M == 0) return QP_OK;
  if ((st = w4_check_float(what, "X", X, dtype, ldx, K))) return st;
  if (dtype == QP_F32)
    quantize<float>(X, M, K, ldx, rule, codes, ld_codes, scales, ld_scales, stream);
  else if (dtype == QP_BF16)
    quantize<bf16_t>(X, M, K, ldx, rule, codes, ld_codes, scales, ld_scales, stream);
  else
    quantize<f16_t>(X, M, K, ldx, rule, codes, ld_codes, scales, ld_scales, stream);
  return check_launch(what);
}

extern "C" qp_status qdequantize_rows_mx4(const qp_mx4* a, void* Y, int32_t y_dtype, int64_t ldy,
                                          hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qdequantize_rows_mx4";
  qp_status st = mx_check(what, "a", a);
  if (st) return st;
  QP_REQUIRE(a->matrices == 1, QP_EINVAL, "%s: one matrix at a time", what);
  if (a->rows == 0) return QP_OK;
  if ((st = w4_check_float(what, "Y", Y, y_dtype, ldy, a->K))) return st;
  const MxMat v = mx_view(a);
  if (y_dtype == QP_F32)
    dequantize<float>(v, Y, ldy, stream);
  else if (y_dtype == QP_BF16)
    dequantize<bf16_t>(v, Y, ldy, stream);
  else
    dequantize<f16_t>(v, Y, ldy, stream);
  return check_launch(what);
}
