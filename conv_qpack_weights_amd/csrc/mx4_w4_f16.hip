// mx4_w4_f16.hip -- the products' kernels for f16 rows times MXFP4 weights.
#include "mx4_rows.hpp"

namespace qp {
qp_status run_mx_f16(const MxArgs& a, hipStream_t stream) {
  return mx_launch_rows<f16_t, 1, 2, 8, 1>(a, stream);
}
}  // namespace qp
