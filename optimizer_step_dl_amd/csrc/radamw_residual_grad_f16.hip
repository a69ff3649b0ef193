// radamw_residual_grad_f16.hip -- the gradient of the residual stream's
// norms for FP16 streams (radamw_residual_grad.h).
#include "radamw_residual_grad.h"

namespace radamw {

hipError_t residual_grad_f16(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream) {
    return residual_grad_rows<G_F16, G_F16>(a, p, stream);
}

}  // namespace radamw
