// Linear attention's gradients in FP32: the passes of kda_linear_grad.hip with
// factors of 24 bits.
#include "kda_linear_pass.h"

namespace kda {

LinearGrad linear_grad_fp32(int32_t K, int32_t V) { return linear_grad_of<3>(K, V); }

}  // namespace kda
