// w4_f16.hip -- the weight-only int4 products' kernels for f16 rows.
#include "w4_kernels.hpp"

namespace qp {
qp_status run_w4_f16(const W4Args& a, int32_t format, W4Shape shape, hipStream_t stream) {
  return run_w4_type<f16_t>(a, format, shape, stream);
}
}  // namespace qp
