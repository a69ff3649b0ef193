// radamw_residual_grad_bf16.hip -- the gradient of the residual stream's
// norms for BF16 streams (radamw_residual_grad.h).
#include "radamw_residual_grad.h"

namespace radamw {

hipError_t residual_grad_bf16(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream) {
    return residual_grad_rows<G_BF16, G_BF16>(a, p, stream);
}

}  // namespace radamw
