// mx4_a4w4.hip -- MXFP4 rows times MXFP4 weights: both go into the scaled 4-bit
// MFMA as they are.
#include "mx4_rows.hpp"

namespace qp {
qp_status run_mx_a4w4(const MxArgs& a, hipStream_t stream) {
  return mx_launch_rows<mx4_t, 1, 2, 8, 1>(a, stream);
}
}  // namespace qp
