// linear_any.cu -- the tile kernel of the linear layers of KIND_LINEAR.
#include "gemm_host.cuh"

namespace dpred {
namespace gemm {

int linear_tiles_any(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s) {
    return tiles_of_kind<KIND_LINEAR>(p, sh, e, s);
}

}  // namespace gemm
}  // namespace dpred
