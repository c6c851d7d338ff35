// mx4.hip -- entry points of the products with MXFP4 weights: MXFP4 rows
// (qgemm_a4w4_mx*) and float rows (qgemm_w4_mx*), dense or grouped by expert.
#include <cstdio>

#include "mx4.hpp"

namespace qp {
namespace {

qp_status check_common(const char* what, int64_t M, const qp_mx4* w, int64_t K, float lo,
                       float hi) {
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

// The products of float rows.  Measured with bf16 rows, cold weights, all shapes on one card
// (those that are taken, on the present kernels: 16 x 4096 6.0 to 6.4 us, 64 x 4096 9.8, 16 x
// 11008 9.8, 64 x 11008 21.9, 1024 x 4096 39): 16 x 4096 rows of 16 / 32 / 48 / 64 channels 5.6,
// 6.2, 7.4, 8.2 us, tiles of 32 x 64 / 32 x 128 15.7, 17.1; 16 x 11008 15.7, 13.5, 10.3, 11.0,
// 18.2, 19.8; 64 x 4096 14.8, 10.1, 12.3, 8.3, 16.5, 17.5; 64 x 11008 47, 31, 28, 24.5, 22,
// 20.5; 64 tokens x 2 of 16 experts of 11008 (32 channels on) 152, 136, 107, 121, 112, 128 x 128
// tiles 161; 4096 tokens x 2 of 8 of them tiles of 128 / 256 rows 776, 717; 1024 x 4096 tiles of
// 32 x 64 / 128 / 256 rows 62, 42, 87; 8192 x 11008 1089, 667, 630.
constexpr MxCost kW4Shapes[] = {
    {kMxRows16x16, 16, 16, 5.6, 5.0, 3.1, "rows16x16"},
    {kMxRows16x32, 16, 32, 6.3, 7.2, 3.8, "rows16x32"},
    {kMxRows16x48, 16, 48, 7.4, 9.0, 5.0, "rows16x48"},
    {kMxRows16x64, 16, 64, 8.3, 8.8, 6.0, "rows16x64"},
    {kMxTile32x64, 32, 64, 15.7, 11.0, 6.5, "tile32x64"},
    {kMxTile32x128, 32, 128, 19.8, 20.0, 14.0, "tile32x128"},
    {kMxTile128x128, 128, 128, 34.0, 29.0, 29.0, "tile128x128"},
    {kMxTile256x256, 256, 256, 103.0, 100.0, 100.0, "tile256x256"},
};
// The same of f32 rows (64 tokens x 2 of 16 experts of 11008 x 4096 197, 1024 x 2 of 8 of 4096 x
// 4096 330): 16 x 4096 14.1, 14.8, 15.4, 16.6; 16 x 11008 38, 34, 19.6, 20.8; 64 x 11008 112,
// 84, 58, 52; 128 x 4096 78, 56, 40, 33; 128 x 128 tiles 512 x 4096 109, 1024 x 4096 115, 4096 x
// 4096 454.
constexpr MxCost kW4ShapesF32[] = {
    {kMxRows16x16, 16, 16, 14.1, 9.2, 9.2, "rows16x16"},
    {kMxRows16x32, 16, 32, 15.2, 13.5, 13.5, "rows16x32"},
    {kMxRows16x48, 16, 48, 16.0, 13.5, 13.5, "rows16x48"},
    {kMxRows16x64, 16, 64, 17.5, 16.0, 16.0, "rows16x64"},
    {kMxTile128x128, 128, 128, 111.0, 111.0, 111.0, "tile128x128"},
};

}  // namespace

// Rounds of tiles one to a CU, the last one in halves where it is half empty.
double mx_halved_rounds(double rounds) {
  const double whole = (double)(int64_t)rounds, last = rounds - whole;
  return rounds <= 1.0 || last == 0.0 ? rounds : whole + (last <= 0.5 ? 0.6 : 1.0);
}

const MxCost& mx_choose(const MxCost* shapes, int n, int64_t M, int64_t parts, int64_t N) {
  const double experts = (double)(parts < M ? parts : M);
  const double each = (double)M / experts;  // rows of an expert, if all were alike
  const MxCost* best = shapes;
  double least = 1e300;
  for (const MxCost* s = shapes; s < shapes + n; ++s) {
    // row tiles of an expert: its last one is half empty on average
    double tiles = (double)ceil_div(M, s->rows);
    if (experts > 1.0) {
      tiles = each / s->rows + 0.5;
      tiles = experts * (tiles > 1.0 ? tiles : 1.0);
    }
    const double groups = (double)ceil_div(N, s->channels) / 256.0;
    double rounds = tiles * groups, own = experts * groups;
    const bool tile = s->shape >= kMxTile32x64;
    // (experts of unlike sizes have more tiles than that)
    if (tile && experts > 1.0) rounds *= 1.1;
    if (!tile) {
      rounds = (double)(int64_t)(rounds + 255.0 / 256.0);
      own = (double)(int64_t)(own + 255.0 / 256.0);
    } else if (s->shape == kMxTile256x256) {
      rounds = mx_halved_rounds(rounds);
      own = mx_halved_rounds(own);
    }
    own = own < 1.0 ? 1.0 : own;
    const double cost = s->first + s->cold * (own - 1.0) +
                        s->more * (rounds > own ? rounds - own : 0.0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return *best;
}

const MxCost& mx_w4_shape(int32_t dtype, int64_t M, int64_t parts, int64_t N) {
  if (dtype == QP_F32)
    return mx_choose(kW4ShapesF32, sizeof(kW4ShapesF32) / sizeof(MxCost), M, parts, N);
  return mx_choose(kW4Shapes, sizeof(kW4Shapes) / sizeof(MxCost), M, parts, N);
}

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

extern "C" qp_status qgemm_mx_kernel_name(int32_t product, int64_t M, const qp_mx4* w,
                                          int32_t dtype, char* name, size_t bytes) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_mx_kernel_name";
  qp_status st = mx_check(what, "w", w);
  if (st) return st;
  QP_REQUIRE(M >= 1 && M <= kW4MaxRows && w->rows > 0, QP_EINVAL, "%s: needs a row and a channel",
             what);
  QP_REQUIRE(name && bytes >= 24, QP_EINVAL, "%s: needs room for 24 characters", what);
  QP_REQUIRE(product >= QP_MX_A4W4 && product <= QP_MX_W4_DX, QP_EINVAL, "%s: no product %d", what,
             product);
  QP_REQUIRE(product == QP_MX_A4W4 || dtype == QP_F32 || dtype == QP_BF16 || dtype == QP_F16,
             QP_EINVAL, "%s: rows must be QP_F32, QP_BF16 or QP_F16 (got %d)", what, dtype);
  if (product == QP_MX_W4_DX)
    mx_dx_kernel_name(w, dtype, M, name, bytes);
  else
    std::snprintf(name, bytes, "%s",
                  product == QP_MX_A4W4 ? mx_a4w4_shape(M, w->matrices, w->rows).name
                                        : mx_w4_shape(dtype, M, w->matrices, w->rows).name);
  return QP_OK;
}
