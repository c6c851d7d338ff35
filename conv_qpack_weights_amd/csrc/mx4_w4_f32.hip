// mx4_w4_f32.hip -- the products' kernels for f32 rows times MXFP4 weights.
#include "mx4_w4_tile.hpp"

namespace qp {
qp_status run_mx_f32(const MxArgs& a, hipStream_t stream) {
  const MxShape shape =
      mx_w4_shape(QP_F32, a.rows.M, a.rows.offsets ? a.rows.experts : 1, a.w.rows).shape;
  // (LDS holds three pieces of 128 rows)
  if (shape == kMxTile128x128 && a.w.ldc < kMxMaxLd)
    return mx_launch_w4_tile<float, false, 128, 128, 2, 2, 2>(a, stream);
  return mx_run_rows<float>(a, shape, stream);
}
}  // namespace qp
