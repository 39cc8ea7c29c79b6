// block_norm_grad_bf16_part.cu -- the gradient of the block norm over aligned rows of
// a bf16 stream, with parts of the formula left out or a gate for every row.
#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {

template cudaError_t launch_ring<__nv_bfloat16, false>(const BackwardArgs&, const Rows&, const Grid&, int, cudaStream_t);

}  // namespace layers
}  // namespace dpred
