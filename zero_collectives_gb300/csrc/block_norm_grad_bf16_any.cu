// block_norm_grad_bf16_any.cu -- the gradient of the block norm over rows of any alignment
// of a bf16 stream.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

DPRED_NORM_GRAD_FORM(__nv_bfloat16, false, false);

}  // namespace layers
}  // namespace dpred
