// mx4.hip -- entry points of the products with MXFP4 weights: MXFP4 rows
// (qgemm_a4w4_mx*) and float rows (qgemm_w4_mx*), dense or grouped by expert.
#include "mx4.hpp"

namespace qp {
namespace {

qp_status check_common(const char* what, int64_t M, const qp_mx4* w, int64_t K, float lo, float hi) {
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= kW4MaxRows, QP_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  qp_status st = mx_check(what, "w", w);
  if (st) return st;
  QP_REQUIRE(w->rows > 0, QP_EINVAL, "%s: w has no rows", what);
  QP_REQUIRE(K == w->K, QP_EINVAL, "%s: the rows have K=%lld but the weights K=%lld", what,
             (long long)K, (long long)w->K);
  QP_REQUIRE(!(lo > hi) && lo == lo && hi == hi, QP_EINVAL,
             "%s: clamp bounds are NaN or reversed", what);
  return QP_OK;
}

qp_status check_map(const char* what, int64_t M, int64_t x_rows, const int32_t* rows,
                    int64_t row_div, const int32_t* offsets) {
  QP_REQUIRE(offsets, QP_EINVAL, "%s: offsets is null", what);
  QP_REQUIRE(rows || x_rows >= M, QP_EINVAL, "%s: %lld rows are given, fewer than M=%lld", what,
             (long long)x_rows, (long long)M);
  QP_REQUIRE(!rows || (row_div >= 1 && row_div <= INT32_MAX), QP_EINVAL, "%s: row_div must be >= 1",
             what);
  QP_REQUIRE(M == 0 || x_rows > 0, QP_EINVAL, "%s: there are no rows to read", what);
  return QP_OK;
}

qp_status run_float(const char* what, const MxArgs& a, int32_t dtype, hipStream_t stream) {
  qp_status st = w4_check_float(what, "X", a.X, dtype, a.ldx, a.w.K);
  if (st) return st;
  if ((st = w4_check_float(what, "Y", a.Y, a.y_dtype, a.ldy, a.w.rows))) return st;
  QP_REQUIRE(a.y_dtype == dtype || a.y_dtype == QP_F32, QP_EUNSUPPORTED,
             "%s: outputs are stored in the rows' type or in f32", what);
  if (dtype == QP_F32) return run_mx_f32(a, stream);
  if (dtype == QP_BF16) return run_mx_bf16(a, stream);
  return run_mx_f16(a, stream);
}

}  // namespace
}  // namespace qp

extern "C" qp_status qgemm_a4w4_mx(const qp_mx4* a, const qp_mx4* w, const float* bias,
                                   float clamp_lo, float clamp_hi, void* Y, int32_t y_dtype,
                                   int64_t ldy, hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_a4w4_mx";
  qp_status st = mx_check(what, "a", a);
  if (st) return st;
  if ((st = check_common(what, a->rows, w, a->K, clamp_lo, clamp_hi))) return st;
  QP_REQUIRE(a->matrices == 1 && w->matrices == 1, QP_EINVAL, "%s: one matrix of each", what);
  if (a->rows == 0) return QP_OK;
  if ((st = w4_check_float(what, "Y", Y, y_dtype, ldy, w->rows))) return st;
  MxArgs args{mx_view(w), W4Rows{nullptr, 1, a->rows, nullptr, 1, a->rows}, nullptr, 0, mx_view(a),
              bias, clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_mx_a4w4(args, stream);
}

extern "C" qp_status qgemm_a4w4_mx_experts(const qp_mx4* a, const int32_t* rows, int64_t row_div,
                                           int64_t M, const qp_mx4* w, const int32_t* offsets,
                                           const float* bias, float clamp_lo, float clamp_hi,
                                           void* Y, int32_t y_dtype, int64_t ldy,
                                           hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_a4w4_mx_experts";
  qp_status st = mx_check(what, "a", a);
  if (st) return st;
  if ((st = check_common(what, M, w, a->K, clamp_lo, clamp_hi))) return st;
  QP_REQUIRE(a->matrices == 1, QP_EINVAL, "%s: the rows are one matrix", what);
  if ((st = check_map(what, M, a->rows, rows, row_div, offsets))) return st;
  if (M == 0) return QP_OK;
  if ((st = w4_check_float(what, "Y", Y, y_dtype, ldy, w->rows))) return st;
  MxArgs args{mx_view(w),
              W4Rows{offsets, (int32_t)w->matrices, M, rows, rows ? row_div : 1, a->rows},
              nullptr, 0, mx_view(a), bias, clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_mx_a4w4(args, stream);
}

extern "C" qp_status qgemm_w4_mx(const void* X, int32_t dtype, int64_t M, int64_t K, int64_t ldx,
                                 const qp_mx4* w, const float* bias, float clamp_lo,
                                 float clamp_hi, void* Y, int32_t y_dtype, int64_t ldy,
                                 hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_mx";
  qp_status st = check_common(what, M, w, K, clamp_lo, clamp_hi);
  if (st) return st;
  QP_REQUIRE(w->matrices == 1, QP_EINVAL, "%s: one matrix of weights", what);
  if (M == 0) return QP_OK;
  MxArgs args{mx_view(w), W4Rows{nullptr, 1, M, nullptr, 1, M}, X, ldx, MxMat{}, bias, clamp_lo,
              clamp_hi, Y, y_dtype, ldy};
  return run_float(what, args, dtype, stream);
}

extern "C" qp_status qgemm_w4_mx_experts(const void* X, int32_t dtype, int64_t x_rows, int64_t K,
                                         int64_t ldx, const int32_t* rows, int64_t row_div,
                                         int64_t M, const qp_mx4* w, const int32_t* offsets,
                                         const float* bias, float clamp_lo, float clamp_hi,
                                         void* Y, int32_t y_dtype, int64_t ldy,
                                         hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_mx_experts";
  qp_status st = check_common(what, M, w, K, clamp_lo, clamp_hi);
  if (st) return st;
  QP_REQUIRE(x_rows >= 0, QP_EINVAL, "%s: a row count is negative", what);
  if ((st = check_map(what, M, x_rows, rows, row_div, offsets))) return st;
  if (M == 0) return QP_OK;
  MxArgs args{mx_view(w),
              W4Rows{offsets, (int32_t)w->matrices, M, rows, rows ? row_div : 1, x_rows},
              X, ldx, MxMat{}, bias, clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_float(what, args, dtype, stream);
}
