// block_norm_grad_f32_part.cu -- the gradient of the block norm over aligned rows
// of an fp32 stream, with parts of the formula left out or a gate
// for every row.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

DPRED_NORM_GRAD_FORM(float, true, false);

}  // namespace layers
}  // namespace dpred
