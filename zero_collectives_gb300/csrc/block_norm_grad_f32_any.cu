// block_norm_grad_f32_any.cu -- the gradient of the block norm over rows of any alignment
// of an fp32 stream.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

DPRED_NORM_GRAD_FORM(float, false, false);

}  // namespace layers
}  // namespace dpred
