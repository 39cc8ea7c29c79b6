// block_norm_grad_bf16_part.cu -- the gradient of the block norm over aligned rows
// of a bf16 stream, with parts of the formula left out or a gate
// for every row.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

DPRED_NORM_GRAD_FORM(__nv_bfloat16, true, false);

}  // namespace layers
}  // namespace dpred
