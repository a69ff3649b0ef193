// radamw_residual_grad_f32.hip -- the gradient of the residual stream's norms
// for FP32 streams (radamw_residual_grad.h), compiled beside the other types.
#include "radamw_residual_grad.h"

namespace radamw {

hipError_t residual_grad_f32(const ResidualGradArgs &a, const ResidualPlan &p, int bdt, hipStream_t stream) {
    switch (bdt) {
    case G_F32: return residual_grad_rows<G_F32, G_F32>(a, p, stream);
    case G_F16: return residual_grad_rows<G_F32, G_F16>(a, p, stream);
    default: return residual_grad_rows<G_F32, G_BF16>(a, p, stream);
    }
}

}  // namespace radamw
