// w4.hip -- float rows times packed int4 weights with group scales, dense or
// grouped by expert:
//   y[r,n] = clamp(sum_g s[n,g] * P[r,n,g] (+ o[n,g] * S[r,g]) + bias[n], lo, hi)
//   P[r,n,g] = sum_{k in g} x[r,k] q[n,k],   S[r,g] = sum_{k in g} x[r,k]
// The rows stay in their own type (bf16, f16; f32 as three bf16 pieces) and q
// goes into the MFMA exactly, so the only roundings are those of the f32
// sums; the scales multiply the f32 group sums.  q enters as q/16 (what the
// 4-bit conversion gives); the factor 16 leaves exactly at the end.
#include <cstdio>

#include "w4.hpp"

namespace qp {
namespace {

// Which kernel: the one whose time the following estimate puts lowest.  A shape
// takes `first` microseconds for up to one workgroup a CU (256) and `more` for
// every further round of them, at K = 4096 (both grow with K, which changes no
// order).  Measured with bf16 rows, groups of 32, 4096 and 11008 channels, 1 to
// 1024 rows, four copies of the weights in turn: e.g. 16 x 11008 rows1x1 15.6,
// 1x2 13.1, 1x3 9.5, 1x4 10.4 us; 64 x 11008 48.6, 32.8, 26.2, 23.3 and rows2x3
// 24.4; 512 x 4096 rows2x4 52, tile4x8 45, tile8x8 61.  Over all shapes and rows
// swept, and over 8 and 16 experts, the best was at most a fifth faster than the
// one chosen.  (Same order for f32 rows, at twice the times.)
struct ShapeCost {
  W4Shape shape;
  int rows, tiles;   // 16-row fragments and 16-channel tiles of a workgroup
  double first, more;
};
constexpr ShapeCost kShapes[] = {
    {kRows1x1, 1, 1, 7.5, 4.1},   {kRows1x2, 1, 2, 8.4, 4.8},   {kRows1x3, 1, 3, 9.5, 5.6},
    {kRows1x4, 1, 4, 10.3, 6.5},  {kRows2x3, 2, 3, 13.2, 11.0}, {kRows2x4, 2, 4, 14.4, 12.1},
    {kTile4x8, 4, 8, 42.0, 21.7}, {kTile8x8, 8, 8, 59.0, 42.0},
};

const ShapeCost& w4_choose(int64_t M, int64_t parts, int64_t Npad) {
  const double experts = (double)(parts < M ? parts : M);
  const double each = (double)M / experts;  // rows of an expert, if all were alike
  const ShapeCost* best = kShapes;
  double least = 1e300;
  for (const ShapeCost& s : kShapes) {
    // row tiles of an expert: its last one is half empty on average
    double tiles = (double)ceil_div(M, 16 * s.rows);
    if (experts > 1.0) {
      tiles = each / (16 * s.rows) + 0.5;
      tiles = experts * (tiles > 1.0 ? tiles : 1.0);
    }
    const double groups = tiles * (double)ceil_div(Npad / 16, s.tiles);
    const double rounds = groups <= 256.0 ? 0.0 : (double)(int64_t)((groups + 255.0) / 256.0) - 1.0;
    const double cost = s.first + s.more * rounds;
    if (cost < least) {
      least = cost;
      best = &s;
    }
  }
  return *best;
}

qp_status run_w4(const W4Args& a, int32_t dtype, int32_t format, hipStream_t stream) {
  const W4Shape shape =
      w4_choose(a.rows.M, a.rows.offsets ? a.rows.experts : 1, a.w.Npad).shape;
  if (dtype == QP_F32) return run_w4_f32(a, format, shape, stream);
  if (dtype == QP_BF16) return run_w4_bf16(a, format, shape, stream);
  return run_w4_f16(a, format, shape, stream);
}

qp_status check_y(const char* what, const void* Y, int32_t dtype, int32_t y_dtype, int64_t ldy,
                  int64_t N) {
  qp_status st = w4_check_float(what, "Y", Y, y_dtype, ldy, N);
  if (st) return st;
  QP_REQUIRE(y_dtype == dtype || y_dtype == QP_F32, QP_EUNSUPPORTED,
             "%s: outputs are stored in the rows' type or in f32", what);
  return QP_OK;
}

}  // namespace

W4View w4_view(const qp_packed_info* w, const void* packed, int64_t expert_stride) {
  W4View v;
  v.blob = static_cast<const uint8_t*>(packed);
  v.expert_stride = expert_stride;
  v.data_off = w->data_off;
  v.scale_off = w->scale_off;
  v.offs_off = w->format == 4 ? w->zp_off : 0;
  v.N = w->N;
  v.Npad = w->Npad;
  v.K = w->K;
  v.nblk = w->Kpad / 128;
  v.G4 = ceil_div(w->Kpad / w->group, 4);
  v.group = (int32_t)w->group;
  return v;
}

qp_status w4_check_weights(const char* what, const qp_packed_info* w, const void* packed,
                           int64_t experts, int64_t expert_stride) {
  QP_REQUIRE(w && w->format >= 2 && w->format <= 4, QP_EINVAL,
             "%s: weights must be an int4 blob", what);
  // the kernels index the blob by these: hold a description made by hand to them too
  qp_packed_info g;
  qp_status st = blob_geometry(w->format, w->scheme, w->N, w->K, w->group, &g);
  if (st) return st;
  QP_REQUIRE(g.Npad == w->Npad && g.Kpad == w->Kpad && g.data_off == w->data_off &&
                 g.scale_off == w->scale_off && g.zp_off == w->zp_off &&
                 g.total_bytes == w->total_bytes,
             QP_EINVAL, "%s: the weights' description does not match their shape", what);
  QP_REQUIRE(packed, QP_EINVAL, "%s: the weights are null", what);
  QP_REQUIRE((uintptr_t)packed % 256 == 0, QP_EALIGN, "%s: the weights must be 256-byte aligned",
             what);
  QP_REQUIRE(experts >= 1, QP_EINVAL, "%s: needs at least one expert", what);
  QP_REQUIRE(experts <= 65536, QP_EUNSUPPORTED, "%s: more than 65536 experts", what);
  QP_REQUIRE(experts == 1 || (expert_stride >= w->total_bytes && expert_stride % 256 == 0),
             QP_EINVAL, "%s: the experts' blobs must be total_bytes or more apart, a multiple of 256",
             what);
  return QP_OK;
}

qp_status w4_check_float(const char* what, const char* name, const void* p, int32_t dtype,
                         int64_t ld, int64_t cols) {
  QP_REQUIRE(dtype == QP_F32 || dtype == QP_BF16 || dtype == QP_F16, QP_EINVAL,
             "%s: %s must be QP_F32, QP_BF16 or QP_F16 (got %d)", what, name, dtype);
  QP_REQUIRE(ld >= cols, QP_EINVAL, "%s: the stride of %s is below its %lld columns", what, name,
             (long long)cols);
  QP_REQUIRE(p, QP_EINVAL, "%s: %s is null", what, name);
  QP_REQUIRE((uintptr_t)p % elem_bytes(dtype) == 0, QP_EALIGN,
             "%s: %s is not aligned to its elements", what, name);
  return QP_OK;
}

}  // namespace qp

extern "C" qp_status qgemm_w4_blockwise(const void* X, int32_t dtype, int64_t M, int64_t K,
                                        int64_t ldx, const qp_packed_info* w,
                                        const void* packedW_dev, const float* bias, float clamp_lo,
                                        float clamp_hi, void* Y, int32_t y_dtype, int64_t ldy,
                                        hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_blockwise";
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= kW4MaxRows, QP_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  qp_status st = w4_check_weights(what, w, packedW_dev, 1, 0);
  if (st) return st;
  QP_REQUIRE(K == w->K, QP_EINVAL, "%s: the rows have K=%lld but the weights K=%lld", what,
             (long long)K, (long long)w->K);
  QP_REQUIRE(!(clamp_lo > clamp_hi) && clamp_lo == clamp_lo && clamp_hi == clamp_hi, QP_EINVAL,
             "%s: clamp bounds are NaN or reversed", what);
  if (M == 0) return QP_OK;
  if ((st = w4_check_float(what, "X", X, dtype, ldx, K))) return st;
  if ((st = check_y(what, Y, dtype, y_dtype, ldy, w->N))) return st;
  W4Args a{w4_view(w, packedW_dev, 0), W4Rows{nullptr, 1, M, nullptr, 1, M}, X, ldx, bias,
           clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_w4(a, dtype, w->format, stream);
}

extern "C" qp_status qgemm_w4_experts(const void* X, int32_t dtype, int64_t x_rows, int64_t K,
                                      int64_t ldx, const int32_t* rows, int64_t row_div, int64_t M,
                                      const qp_packed_info* w, const void* packedW_dev,
                                      int64_t expert_stride, int64_t experts,
                                      const int32_t* offsets, const float* bias, float clamp_lo,
                                      float clamp_hi, void* Y, int32_t y_dtype, int64_t ldy,
                                      hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_experts";
  QP_REQUIRE(M >= 0 && x_rows >= 0, QP_EINVAL, "%s: a row count is negative", what);
  QP_REQUIRE(M <= kW4MaxRows, QP_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  qp_status st = w4_check_weights(what, w, packedW_dev, experts, expert_stride);
  if (st) return st;
  QP_REQUIRE(K == w->K, QP_EINVAL, "%s: the rows have K=%lld but the weights K=%lld", what,
             (long long)K, (long long)w->K);
  QP_REQUIRE(!(clamp_lo > clamp_hi) && clamp_lo == clamp_lo && clamp_hi == clamp_hi, QP_EINVAL,
             "%s: clamp bounds are NaN or reversed", what);
  QP_REQUIRE(offsets, QP_EINVAL, "%s: offsets is null", what);
  QP_REQUIRE(rows || x_rows >= M, QP_EINVAL, "%s: X has %lld rows, fewer than M=%lld", what,
             (long long)x_rows, (long long)M);
  QP_REQUIRE(!rows || (row_div >= 1 && row_div <= INT32_MAX), QP_EINVAL, "%s: row_div must be >= 1",
             what);
  if (M == 0) return QP_OK;
  QP_REQUIRE(x_rows > 0, QP_EINVAL, "%s: X has no rows", what);
  if ((st = w4_check_float(what, "X", X, dtype, ldx, K))) return st;
  if ((st = check_y(what, Y, dtype, y_dtype, ldy, w->N))) return st;
  W4Args a{w4_view(w, packedW_dev, expert_stride),
           W4Rows{offsets, (int32_t)experts, M, rows, rows ? row_div : 1, x_rows},
           X, ldx, bias, clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_w4(a, dtype, w->format, stream);
}

extern "C" qp_status qgemm_w4_kernel_name(int64_t M, const qp_packed_info* w, int32_t dtype,
                                          int64_t experts, int32_t gradient, char* name,
                                          size_t bytes) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_kernel_name";
  QP_REQUIRE(w && w->format >= 2 && w->format <= 4, QP_EINVAL, "%s: weights must be an int4 blob",
             what);
  QP_REQUIRE(M >= 1 && M <= kW4MaxRows && experts >= 1 && w->N > 0 && w->K > 0, QP_EINVAL,
             "%s: needs a row and an expert", what);
  QP_REQUIRE(dtype == QP_F32 || dtype == QP_BF16 || dtype == QP_F16, QP_EINVAL,
             "%s: rows must be QP_F32, QP_BF16 or QP_F16 (got %d)", what, dtype);
  QP_REQUIRE(name && bytes >= 16, QP_EINVAL, "%s: needs room for 16 characters", what);
  if (gradient) {
    w4_dx_kernel_name(M, w, dtype, experts, name, bytes);
    return QP_OK;
  }
  const ShapeCost& s = w4_choose(M, experts, w->Npad);
  const bool tile = s.shape == kTile4x8 || s.shape == kTile8x8;
  // (f32 rows take the 64-row tile for either)
  std::snprintf(name, bytes, "%s%dx%d", tile ? "tile" : "rows",
                tile && dtype == QP_F32 ? 4 : s.rows, s.tiles);
  return QP_OK;
}
