// mx4_w4_bf16.hip -- the products' kernels for bf16 rows times MXFP4 weights.
#include "mx4_rows.hpp"

namespace qp {
qp_status run_mx_bf16(const MxArgs& a, hipStream_t stream) {
  return mx_launch_rows<bf16_t, 1, 2, 8, 1>(a, stream);
}
}  // namespace qp
