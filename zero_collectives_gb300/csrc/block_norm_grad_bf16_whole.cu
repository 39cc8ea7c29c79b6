// block_norm_grad_bf16_whole.cu -- the gradient of the block norm over aligned rows of
// a bf16 stream.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

template cudaError_t launch_ring<__nv_bfloat16, true>(const BackwardArgs&, const Rows&, const Grid&, int, cudaStream_t);

}  // namespace layers
}  // namespace dpred
