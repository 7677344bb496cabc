// Linear attention's gradients in BF16: dq is the forward pass of (do, v, k) over the
// transposed state, dk the reversed pass of (v, do, q) over its cotangent, transposed,
// dv the reversed pass of (k, q, do).
#include "kda_linear_pass.h"

namespace kda {

LinearGrad linear_grad_bf16(int32_t K, int32_t V) { return linear_grad_of<2>(K, V); }

}  // namespace kda
