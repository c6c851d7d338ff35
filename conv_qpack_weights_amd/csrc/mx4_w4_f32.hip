// mx4_w4_f32.hip -- the products' kernels for f32 rows times MXFP4 weights.
#include "mx4_rows.hpp"

namespace qp {
qp_status run_mx_f32(const MxArgs& a, hipStream_t stream) {
  return mx_launch_rows<float, 1, 2, 8, 1>(a, stream);
}
}  // namespace qp
