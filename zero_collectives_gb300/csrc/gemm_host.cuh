// gemm_host.cuh -- launch of a matrix product, included by the translation
// units that instantiate its kernels (one per family of epilogues).
#pragma once

#include "gemm.cuh"

namespace dpred {
namespace gemm {

struct Shape {
    bool pairs;   // tile kernel (CTA pairs, 256 x bn tiles); else split kernel (128 x bn)
    int bn, split;
    int64_t tiles;
};

// CTA pairs that can be resident at once (all kernels of the family take a whole SM per CTA).
int resident_pairs(const void* kernel, int threads, int smem);

int make_map(const Operand& o, int batch, int box_rows, bool bf16, CUtensorMap* m);
// A row-major matrix as the streaming epilogue moves it: boxes of 32 rows x 128 bytes.
int make_box_map(const void* p, int64_t rows, int64_t cols, int64_t ld, bool fp32, CUtensorMap* m);
bool tma_able(const void* p, int64_t rows, int64_t ld);
int64_t tiles_of(const Args& a, int bm, int bn);
Shape choose_shape(const Args& a, bool fp32);
double estimate(const Args& a, bool fp32);  // time of the chosen shape, us
// Whether a split launch gives every CTA an SM of its own (eight-CTA clusters do not fit every SM of a GPC).
bool split_alone(double ctas, int split, int sms);

template <int KIND, int BN, bool DRAIN = false>
int launch_split(const Plan& p, const Shape& sh, const typename EpiOf<KIND>::Param& e, cudaStream_t s) {
    if constexpr (is_linear(KIND) && !DRAIN) {  // fp32 results of more parts than a CTA has accumulators
        if (p.fp32_result && (p.args.kblocks + sh.split - 1) / sh.split > kPromoteBlocks * (256 / BN))
            return launch_split<KIND, BN, true>(p, sh, e, s);
    }
    static bool attr[64] = {};
    auto kernel = split_kernel<KIND, BN, DRAIN>;
    cudaError_t err = ensure_smem_attr(kernel, split_smem<BN>(true), attr);
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
    const bool deep = split_alone((double)sh.tiles * sh.split, sh.split, sm_count());
    g.stages = split_stages<BN>(deep);
    g.regions = p.fp32_result ? 256 / BN : 1;
    if (g.row_sums) g.release = 1;  // formed by a launch of their own, right after this one
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sh.tiles * sh.split));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = split_smem<BN>(deep);
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

constexpr int kDirectBlocks = 8;

template <int KIND, int BN, bool PROMOTE>
int launch_tiles(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s) {
    static bool attr[64] = {};
    auto kernel = tile_kernel<KIND, BN, PROMOTE>;
    cudaError_t err = ensure_smem_attr(kernel, tile_smem<BN>(), attr);
    if (err != cudaSuccess) return cuda_error(err, "shared-memory limit of a matrix product");
    CUtensorMap ma = {}, mb = {};
    int rc = make_map(p.a, p.args.batch, 128, p.args.bf16, &ma);
    if (rc != DPRED_OK) return rc;
    rc = make_map(p.b, p.args.batch, BN / 2, p.args.bf16, &mb);
    if (rc != DPRED_OK) return rc;
    TileParams t = {};
    t.e = e;
    t.row_sum = p.row_sum;
    t.row_sum_add = p.row_sum_add;
    // what the streaming epilogue covers; block_epilogue does the rest
    t.stream = e.vec && (KIND == KIND_F32 ? !e.z && !e.res && !e.pre_out && !e.act : KIND != KIND_LINEAR && !(e.res && e.z));
    const int whole = e.out_f32 ? whole_columns<float>(p.args.n) : whole_columns<__nv_bfloat16>(p.args.n);
    t.stream = t.stream && whole > 0;
    if (t.stream) {
        rc = make_box_map(e.out, p.args.m, whole, e.o_ld, e.out_f32, &t.out);
        if (rc == DPRED_OK && e.pre_out) rc = make_box_map(e.pre_out, p.args.m, whole, e.p_ld, false, &t.pre);
        if (rc == DPRED_OK && (e.res || e.z))
            rc = e.z ? make_box_map(e.z, p.args.m, p.args.n, e.z_ld, false, &t.in)
                     : make_box_map(e.res, p.args.m, p.args.n, e.r_ld, false, &t.in);
        if (rc != DPRED_OK) return rc;
    }
    Args g = p.args;
    g.tiles_m = (g.m + 255) / 256;
    g.tiles_n = (g.n + BN - 1) / BN;
    g.tiles_per_batch = (int)tiles_of(g, 256, BN);
    g.split = 1;
    g.regions = 1;
    const int pairs = resident_pairs(reinterpret_cast<const void*>(kernel), kTileThreads, tile_smem<BN>());
    if (pairs < 1) return set_error(DPRED_E_CUDA, "no CTA pair fits on this device");
    // A plain result without a residual leaves straight from the registers where
    // the next tile's reduction is long enough to hide its partly filled lines:
    // 8192 x 8192 outputs of reductions of 256 / 512 / 1024 take 40 / 50 / 80 us
    // so and 33 / 52 / 85 us as boxes, whose copies queue with the operands'.  With
    // few tiles nothing hides it (4096 x 1024 x 1024: 11.1 us so, 10.5 as boxes).
    t.direct = KIND == KIND_PLAIN && t.stream && !e.res && p.args.kblocks >= kDirectBlocks && sh.tiles >= 4 * pairs &&
               e.o_ld % 16 == 0 && reinterpret_cast<uintptr_t>(e.out) % 32 == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (sh.tiles < pairs ? sh.tiles : pairs)));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tile_smem<BN>();
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, g, t);
    return err == cudaSuccess ? DPRED_OK : cuda_error(err, "matrix product launch");
}

template <int KIND>
int tiles_of_kind(const Plan& p, const Shape& sh, const typename EpiOf<KIND>::Param& e, cudaStream_t s) {
    constexpr bool kPromote = KIND == KIND_F32;
    return sh.bn == 256 ? launch_tiles<KIND, 256, kPromote>(p, sh, e, s) : launch_tiles<KIND, 128, kPromote>(p, sh, e, s);
}

// The tile kernels of the linear layers, one translation unit per kind.
int linear_tiles_any(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s);
int linear_tiles_plain(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s);
int linear_tiles_act(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s);
int linear_tiles_grad(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s);
int linear_tiles_f32(const Plan& p, const Shape& sh, const LinearEpi& e, cudaStream_t s);

template <int KIND>
int run_tiles(const Plan& p, const Shape& sh, const typename EpiOf<KIND>::Param& e, cudaStream_t s) {
    switch (linear_kind(e)) {
        case KIND_PLAIN: return linear_tiles_plain(p, sh, e, s);
        case KIND_ACT: return linear_tiles_act(p, sh, e, s);
        case KIND_GRAD: return linear_tiles_grad(p, sh, e, s);
        case KIND_F32: return linear_tiles_f32(p, sh, e, s);
        default: return linear_tiles_any(p, sh, e, s);
    }
}

template <int KIND>
int run(const Plan& p, const typename EpiOf<KIND>::Param& e, cudaStream_t s, bool* row_sums_formed = nullptr) {
    const Shape sh = choose_shape(p.args, p.fp32_result);
    if (row_sums_formed) *row_sums_formed = p.args.row_sums && sh.pairs;
    if (sh.tiles * sh.split > 0x7FFFFFFF) return set_error(DPRED_E_SIZE, "a matrix product of too many tiles");
    if constexpr (is_linear(KIND)) {
        if (sh.pairs) return run_tiles<KIND>(p, sh, e, s);
    }
    switch (sh.bn) {
        case 32: return launch_split<KIND, 32>(p, sh, e, s);
        case 64: return launch_split<KIND, 64>(p, sh, e, s);
        default: return launch_split<KIND, 128>(p, sh, e, s);
    }
}

}  // namespace gemm
}  // namespace dpred
