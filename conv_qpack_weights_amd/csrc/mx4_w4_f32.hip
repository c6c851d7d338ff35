// mx4_w4_f32.hip -- the products' kernels for f32 rows times MXFP4 weights.
#include <cstdlib>
#include "mx4_w4_tile.hpp"

namespace qp {
qp_status run_mx_f32(const MxArgs& a, hipStream_t stream) {
  const char* e = getenv("MXT");
  int t = e ? atoi(e) : 1;
  if (t == 1) return mx_launch_w4_tile<float, false, 128, 128, 2, 2, 2>(a, stream);
  if (t <= 7) return mx_launch_w4_tile<float, false, 64, 64, 1, 2, 2>(a, stream);
  return mx_launch_rows<float, 1, 2, 8, 1>(a, stream);
}
}  // namespace qp
