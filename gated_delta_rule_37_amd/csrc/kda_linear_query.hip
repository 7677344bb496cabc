// Linear attention's gradient of the queries, with the gates' as the queries see
// it: the forward pass of (do, v, k) over the transposed state.
#include "kda_linear_pass.h"

namespace kda {

void (*linear_query_kernel(int32_t KW, int32_t VW, bool fp32))(LinearParams) {
  return fp32 ? linear_kernel_of<3, 3, false, kQuery>(KW, VW) : linear_kernel_of<3, 2, false, kQuery>(KW, VW);
}

}  // namespace kda
