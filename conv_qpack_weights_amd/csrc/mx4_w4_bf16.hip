// mx4_w4_bf16.hip -- the products' kernels for bf16 rows times MXFP4 weights.
#include "mx4_w4_tile.hpp"

namespace qp {
qp_status run_mx_bf16(const MxArgs& a, hipStream_t stream) {
  return mx_run_16bit<bf16_t>(a, stream);
}
}  // namespace qp
