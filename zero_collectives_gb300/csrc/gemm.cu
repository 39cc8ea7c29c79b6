// gemm.cu -- host side of the matrix products: tensor maps, launch shapes.
#include "gemm_host.cuh"

#include <mutex>

namespace dpred {
namespace gemm {

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once through the runtime (the
// library does not link against the driver).
EncodeFn encoder() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

}  // namespace

int make_map(const Operand& o, int batch, int box_rows, bool bf16, CUtensorMap* m) {
    EncodeFn f = encoder();
    if (!f) return set_error(DPRED_E_CUDA, "the driver has no tensor-map encoder");
    const cuuint64_t ld = o.rows > 1 ? (cuuint64_t)o.ld : (cuuint64_t)((o.cols + 7) / 8 * 8);
    const cuuint64_t bs = batch > 1 ? (cuuint64_t)o.bstride : ld * (cuuint64_t)o.rows;
    cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)batch};
    cuuint64_t strides[2] = {ld * 2, bs * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)(o.reduce_rows ? mma::kBlockK : box_rows), 1};
    cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(o.p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(DPRED_E_CUDA, "tensor map of a %lld x %lld operand (stride %lld): driver error %d",
                         (long long)o.rows, (long long)o.cols, (long long)o.ld, (int)r);
    return DPRED_OK;
}

bool tma_able(const void* p, int64_t rows, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld % 8 == 0);
}

// Tiles that a product of this shape computes with bm x bn tiles.
int64_t tiles_of(const Args& a, int bm, int bn) {
    const int64_t tm = (a.m + bm - 1) / bm, tn = (a.n + bn - 1) / bn;
    if (!a.symmetric) return tm * tn;
    int64_t n = 0;
    for (int64_t t = 0; t < tm; ++t) n += tn - t * bm / bn;
    return n;
}

int resident_pairs(const void* kernel, int threads, int smem) {
    static std::mutex mu;
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(2 * sm_count()));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        cached[dev] = n < sm_count() / 2 ? n : sm_count() / 2;
    }
    return cached[dev];
}

Shape choose_shape(const Args& a) {
    Shape s;
    const int sms = sm_count();
    s.pairs = false;
    if (a.kblocks > 0 && a.m > 128) {
        const int64_t wide = tiles_of(a, 256, 256) * a.batch, narrow = tiles_of(a, 256, 128) * a.batch;
        if (narrow * 2 >= sms) {
            s.pairs = true;
            s.bn = wide * 2 >= sms && a.n > 128 ? 256 : 128;
            s.tiles = s.bn == 256 ? wide : narrow;
            s.split = 1;
            return s;
        }
    }
    s.bn = a.n <= 32 && !a.b_mn ? 32 : a.n <= 64 ? 64 : tiles_of(a, 128, 128) * a.batch >= sms ? 128 : 64;
    s.tiles = tiles_of(a, 128, s.bn) * a.batch;
    s.split = 1;
    // twice as many CTAs while the SMs are not filled once and every CTA keeps two reduction blocks
    while (s.split < 8 && s.tiles * s.split * 2 <= 2 * sms && a.kblocks >= s.split * 4) s.split *= 2;
    return s;
}

}  // namespace gemm
}  // namespace dpred
