// block_norm_grad_f32_whole.cu -- the gradient of the block norm over aligned rows
// of an fp32 stream.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

DPRED_NORM_GRAD_FORM(float, true, true);

}  // namespace layers
}  // namespace dpred
