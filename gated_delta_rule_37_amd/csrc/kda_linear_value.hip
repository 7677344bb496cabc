// Linear attention's gradient of the values and initial states: the reversed pass
// of (k, q, do) over the cotangent of the state.
#include "kda_linear_pass.h"

namespace kda {

void (*linear_value_kernel(int32_t KW, int32_t VW, bool fp32))(LinearParams) {
  return fp32 ? linear_kernel_of<3, 3, true, kOutput>(KW, VW) : linear_kernel_of<2, 2, true, kOutput>(KW, VW);
}

}  // namespace kda
