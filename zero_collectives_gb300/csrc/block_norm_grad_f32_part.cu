// block_norm_grad_f32_part.cu -- the gradient of the block norm over aligned rows of
// an fp32 stream, with parts of the formula left out or a gate for every row.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

template cudaError_t launch_ring<float, false>(const BackwardArgs&, const Rows&, const Grid&, int, cudaStream_t);

}  // namespace layers
}  // namespace dpred
