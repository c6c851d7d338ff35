// mx4_w4_f16.hip -- the products' kernels for f16 rows times MXFP4 weights.
#include "mx4_w4_tile.hpp"

namespace qp {
qp_status run_mx_f16(const MxArgs& a, hipStream_t stream) {
  return mx_run_16bit<f16_t>(a, stream);
}
}  // namespace qp
