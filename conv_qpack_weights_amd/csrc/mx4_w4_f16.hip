// mx4_w4_f16.hip -- the products' kernels for f16 rows times MXFP4 weights.
#include <cstdlib>
#include "mx4_w4_tile.hpp"

namespace qp {
qp_status run_mx_f16(const MxArgs& a, hipStream_t stream) {
  const char* e = getenv("MXT");
  int t = e ? atoi(e) : 1;
  const bool al = ((uintptr_t)a.X % 4 == 0) && (a.ldx % 2 == 0);
  if (t == 1 && al) return mx_launch_w4_tile<f16_t, true, 256, 256, 2, 4, 2>(a, stream);
  if (t == 2 && al) return mx_launch_w4_tile<f16_t, true, 128, 128, 2, 2, 2>(a, stream);
  if (t == 4 && al) return mx_launch_w4_tile<f16_t, true, 128, 128, 2, 2, 4>(a, stream);
  if (t == 5 && al) return mx_launch_w4_tile<f16_t, true, 64, 128, 1, 4, 4>(a, stream);
  if (t == 6 && al) return mx_launch_w4_tile<f16_t, true, 64, 64, 1, 2, 4>(a, stream);
  if (t == 7 && al) return mx_launch_w4_tile<f16_t, true, 32, 64, 1, 2, 4>(a, stream);
  if (t <= 7) return mx_launch_w4_tile<f16_t, false, 128, 128, 2, 2, 2>(a, stream);
  return mx_launch_rows<f16_t, 1, 2, 8, 1>(a, stream);
}
}  // namespace qp
