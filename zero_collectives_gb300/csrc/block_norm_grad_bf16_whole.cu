// block_norm_grad_bf16_whole.cu -- the gradient of the block norm over aligned rows
// of a bf16 stream.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

DPRED_NORM_GRAD_FORM(__nv_bfloat16, true, true);

}  // namespace layers
}  // namespace dpred
