// mx4_w4_f32.hip -- the products' kernels for f32 rows times MXFP4 weights.
#include "mx4_w4_tile.hpp"

namespace qp {
qp_status run_mx_f32(const MxArgs& a, hipStream_t stream) {
  switch (mx_w4_shape(QP_F32, a.rows.M, a.rows.offsets ? a.rows.experts : 1, a.w.rows).shape) {
    case kMxRows16x16: return mx_launch_rows<float, 1, 8>(a, stream);
    case kMxRows16x32: return mx_launch_rows<float, 2, 8>(a, stream);
    case kMxRows16x48: return mx_launch_rows<float, 3, 8>(a, stream);
    case kMxRows16x64: break;
    default:
      // (LDS holds three pieces of 128 rows)
      if (a.w.ldc < kMxMaxLd && a.w.lds < kMxMaxLd)
        return mx_launch_w4_tile<float, false, 128, 128, 2, 2, 2>(a, stream);
  }
  return mx_launch_rows<float, 4, 8>(a, stream);
}
}  // namespace qp
