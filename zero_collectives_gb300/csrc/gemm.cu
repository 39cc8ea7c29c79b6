// gemm.cu -- host side of the matrix products: tensor maps, launch shapes.
#include "gemm_host.cuh"

#include <cmath>
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

int make_box_map(const void* p, int64_t rows, int64_t cols, int64_t ld, bool fp32, CUtensorMap* m) {
    EncodeFn f = encoder();
    if (!f) return set_error(DPRED_E_CUDA, "the driver has no tensor-map encoder");
    const int esize = fp32 ? 4 : 2;
    const cuuint64_t row = rows > 1 ? (cuuint64_t)ld * esize : (cuuint64_t)((cols * esize + 15) / 16 * 16);
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
    cuuint64_t strides[2] = {row, row * (cuuint64_t)rows};
    cuuint32_t box[3] = {(cuuint32_t)(128 / esize), 32, 1};
    cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = f(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p),
                         dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(DPRED_E_CUDA, "tensor map of a %lld x %lld matrix (stride %lld): driver error %d", (long long)rows,
                         (long long)cols, (long long)ld, (int)r);
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

// The estimated time (us) of a product on one kernel.  The form is that of the
// kernels: a start, then waves of tiles, each reduction block costing what its
// copies and matrix instructions take and each tile its epilogue (which the
// tile kernel hides behind the next tile's reduction).  The constants were
// fitted to the timings of every kernel on 122 shapes from 1 to 16384 rows and
// 256 to 32768 columns (forward, dgrad, wgrad; bf16 and fp32 results); on those
// the choice by these estimates is 1.2% slower on average than the best kernel
// of each, 18% at most (1024 x 1024 x 1024: 9.0 us against 7.8).
static double split_time(const Args& a, int bn, int split, int sms) {
    const double start = bn == 32 ? 0.6 : bn == 64 ? 2.0 : 1.2;
    const double block = bn == 32 ? 0.23 : bn == 64 ? 0.289 : 0.375, epilogue = bn == 32 ? 2.26 : bn == 64 ? 2.44 : 5.1;
    const double ctas = (double)tiles_of(a, 128, bn) * a.batch * split;
    const double per_wave = split_alone(ctas, split, sms) ? sms : 2 * sms;
    double load = (ctas < 2 * sms ? ctas : 2 * sms) / sms;  // CTAs per SM, sharing its bandwidth and issue slots
    if (load < 1) load = 1;
    const double join = split == 1 ? 0.0 : split < 8 ? 1.85 : 2.9;
    return 0.6 + start + std::ceil(ctas / per_wave) * (a.kblocks / (double)split * block * std::pow(load, 0.23) + epilogue * load) + join;
}

static double tile_time(const Args& a, int bn, bool fp32, int pairs) {
    const double start = bn == 128 ? 3.6 : 2.9, block = bn == 128 ? 0.248 : 0.313;
    const double epilogue = (bn == 128 ? 1.6 : 2.42) * (fp32 ? 2.5 : 1.0), reduction = a.kblocks * block;
    const double waves = std::ceil((double)tiles_of(a, 256, bn) * a.batch / pairs);
    return start + (waves - 1) * (reduction > epilogue ? reduction : epilogue) + reduction + epilogue;
}

bool split_alone(double ctas, int split, int sms) { return ctas <= (split < 8 ? sms : sms * 5 / 8); }

static Shape choose(const Args& a, bool fp32, double& t) {
    const int sms = sm_count();
    // the launch that forms the row sums beside a split product: 3 us and A at 4.8 TB/s
    const double apart = a.row_sums ? 3.0 + (double)a.m * a.kblocks * mma::kBlockK * 2 / 4.8e6 : 0.0;
    Shape best = {};
    t = 1e30;
    for (int bn = 32; bn <= 128; bn *= 2) {
        if (bn == 32 && a.b_mn) continue;  // MN-major copies are 64 columns wide
        for (int split = 1; split <= 8 && (split == 1 || split <= a.kblocks); split *= 2) {
            const double u = split_time(a, bn, split, sms) + apart;
            if (u < t) {
                t = u;
                best = {false, bn, split, tiles_of(a, 128, bn) * a.batch};
            }
        }
    }
    if (a.kblocks > 0 && !a.split_only)
        for (int bn = 128; bn <= 256; bn *= 2) {
            const double u = tile_time(a, bn, fp32, sms / 2);
            if (u < t) {
                t = u;
                best = {true, bn, 1, tiles_of(a, 256, bn) * a.batch};
            }
        }
    return best;
}

Shape choose_shape(const Args& a, bool fp32) {
    double t;
    return choose(a, fp32, t);
}

double estimate(const Args& a, bool fp32) {
    double t;
    choose(a, fp32, t);
    return t;
}

}  // namespace gemm
}  // namespace dpred
