// gemm_host.cuh -- launch of a matrix product, included by the translation
// units that instantiate its kernels (one per family of epilogues).
#pragma once

#include "gemm.cuh"

namespace dpred {
namespace gemm {

struct Shape {
    int bn, split;
    int64_t tiles;
};

int make_map(const Operand& o, int batch, int box_rows, bool bf16, CUtensorMap* m);
bool tma_able(const void* p, int64_t rows, int64_t ld);
int64_t tiles_of(const Args& a, int bm, int bn);
Shape choose_shape(const Args& a);

template <int KIND, int BN>
int launch_split(const Plan& p, const Shape& sh, const typename EpiOf<KIND>::T& e, cudaStream_t s) {
    static bool attr[64] = {};
    auto kernel = split_kernel<KIND, BN>;
    cudaError_t err = ensure_smem_attr(kernel, split_smem<BN>(), attr);
    if (err != cudaSuccess) return cuda_error(err, "shared-memory limit of a matrix product");
    CUtensorMap ma = {}, mb = {};
    if (p.args.kblocks) {  // an empty reduction loads nothing
        int rc = make_map(p.a, p.args.batch, 128, p.args.bf16, &ma);
        if (rc != DPRED_OK) return rc;
        rc = make_map(p.b, p.args.batch, BN, p.args.bf16, &mb);
        if (rc != DPRED_OK) return rc;
    }
    Args g = p.args;
    g.tiles_m = (g.m + 127) / 128;
    g.tiles_n = (g.n + BN - 1) / BN;
    g.tiles_per_batch = (int)tiles_of(g, 128, BN);
    g.split = sh.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sh.tiles * sh.split));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = split_smem<BN>();
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)sh.split;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, g, e);
    return err == cudaSuccess ? DPRED_OK : cuda_error(err, "matrix product launch");
}

template <int KIND>
int run(const Plan& p, const typename EpiOf<KIND>::T& e, cudaStream_t s) {
    const Shape sh = choose_shape(p.args);
    if (sh.tiles * sh.split > 0x7FFFFFFF) return set_error(DPRED_E_SIZE, "a matrix product of too many tiles");
    switch (sh.bn) {
        case 32: return launch_split<KIND, 32>(p, sh, e, s);
        case 64: return launch_split<KIND, 64>(p, sh, e, s);
        default: return launch_split<KIND, 128>(p, sh, e, s);
    }
}

}  // namespace gemm
}  // namespace dpred
