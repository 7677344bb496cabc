// Linear attention's gradient of the keys, with the rest of the gates': the
// reversed pass of (v, do, q) over the transposed cotangent of the state.
#include "kda_linear_pass.h"

namespace kda {

void (*linear_key_kernel(int32_t KW, int32_t VW, bool fp32))(LinearParams) {
  return fp32 ? linear_kernel_of<3, 3, true, kKey>(KW, VW) : linear_kernel_of<3, 2, true, kKey>(KW, VW);
}

}  // namespace kda
