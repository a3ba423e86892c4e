// w4_f16.cu - moe_w4_linear for f16 (kernel in w4_body.cuh).
#include "w4_body.cuh"

namespace moe {
moe_status w4_f16(const W4Args& a, int format, cudaStream_t s) {
  return format == MOE_W4_U4 ? pick_w4<MOE_DT_F16, MOE_W4_U4>(a, s)
                             : pick_w4<MOE_DT_F16, MOE_W4_E2M1>(a, s);
}
}  // namespace moe
