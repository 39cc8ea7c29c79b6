// block_norm_grad_f32_whole.cu -- the gradient of the block norm over aligned rows of
// an fp32 stream.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

template cudaError_t launch_ring<float, true>(const BackwardArgs&, const Rows&, const Grid&, int, cudaStream_t);

}  // namespace layers
}  // namespace dpred
