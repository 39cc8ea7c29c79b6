// linear_f32.cu -- the tile kernel of the linear layers of KIND_F32.
#include "gemm_host.cuh"

namespace dpred {
namespace gemm {

int linear_tiles_f32(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s) {
    return tiles_of_kind<KIND_F32>(p, sh, e, s);
}

}  // namespace gemm
}  // namespace dpred
