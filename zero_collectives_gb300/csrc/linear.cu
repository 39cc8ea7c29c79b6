// linear.cu -- the products of a linear layer: dpred_linear (forward),
// dpred_linear_dgrad and dpred_linear_wgrad (backward).
//
// These stand on either side of the gradient reduction: wgrad writes the bf16
// gradient that a bucket flush reads, or adds into the fp32 accumulator of the
// deferred reduction (MaxText PR #5099, section "What": the cotangent is added
// replica-locally), without a gradient array of its own in between.
#include "gemm_host.cuh"

namespace dpred {
namespace gemm {
namespace {

// ----------------------------------------------------------------- packing --
//
// The tensor-map loads need 16-byte aligned rows.  An operand without them is
// copied once into the workspace with its rows padded to 8 elements: 2 bytes
// read and 2 written per element, against 2 * (the other side) flops per
// element of the product.
struct PackJob {
    const uint16_t* src;
    uint16_t* dst;
    int64_t ld, rows, cols, ldd;
};

__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackJob first, const __grid_constant__ PackJob second,
                                                   int first_blocks) {
    const bool one = (int)blockIdx.x < first_blocks;
    const PackJob& j = one ? first : second;
    const int64_t block = one ? blockIdx.x : blockIdx.x - first_blocks;
    const int64_t blocks = one ? first_blocks : (int64_t)gridDim.x - first_blocks;
    const int64_t per = j.ldd / 8, total = j.rows * per, step = blocks * 256;
    mma::grid_launch_dependents();
    mma::grid_wait();
    for (int64_t v = block * 256 + threadIdx.x; v < total; v += step) {
        const int64_t r = v / per, c = (v - r * per) * 8;
        const uint16_t* p = j.src + r * j.ld + c;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = c + 2 * k < j.cols ? p[2 * k] : 0, hi = c + 2 * k + 1 < j.cols ? p[2 * k + 1] : 0;
            w[k] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4*>(j.dst + r * j.ldd + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }
size_t packed_bytes(int64_t rows, int64_t cols) { return ((size_t)rows * round8(cols) * 2 + 255) / 256 * 256; }

// Bytes of workspace that an operand takes: 0 when it can be loaded as it is.
size_t pack_need(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return tma_able(p, rows, ld) ? 0 : packed_bytes(rows, cols);
}

// Packs the operands that need it, in one launch.
int pack(Operand* const (&ops)[2], char* ws, cudaStream_t s) {
    PackJob jobs[2] = {};
    int64_t blocks[2] = {0, 0};
    const int64_t most = (int64_t)sm_count() * 16;
    for (int k = 0; k < 2; ++k) {
        Operand& o = *ops[k];
        if (tma_able(o.p, o.rows, o.ld)) continue;
        const int64_t ldd = round8(o.cols);
        jobs[k] = {static_cast<const uint16_t*>(o.p), reinterpret_cast<uint16_t*>(ws), o.ld, o.rows, o.cols, ldd};
        blocks[k] = (o.rows * (ldd / 8) + 255) / 256;
        if (blocks[k] > most) blocks[k] = most;
        o.p = ws;
        o.ld = ldd;
        ws += packed_bytes(o.rows, o.cols);
    }
    if (blocks[0] + blocks[1] == 0) return DPRED_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks[0] + blocks[1]));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pack_kernel, jobs[0], jobs[1], (int)blocks[0]);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "operand packing launch");
}

// ------------------------------------------------------------- bias gradient --
//
// db[j] = sum_i dy[i][j], where the product runs on the split kernel (the tile
// kernel sums dy from its own stages) or there is no product: bandwidth bound,
// each row read once.  A cluster of 8
// CTAs shares a strip of columns; every thread sums 8 columns of every
// ROWS-th row in fp32, the CTA adds its row groups and the cluster its 8 partial
// rows in rank order, so the sum has one fixed order.
// [16384, 4096] takes 28 us, 4.8 TB/s (a strip of 128 columns, half the CTAs:
// 48 us; twice the rows in flight: the same).
constexpr int kBiasCluster = 8, kBiasStrip = 64;

__global__ void __cluster_dims__(kBiasCluster, 1, 1) __launch_bounds__(256, 2)
    bias_grad_kernel(const __nv_bfloat16* __restrict__ dy, int64_t ld, int64_t m, int64_t n, float* __restrict__ db,
                     int accumulate, int vec) {
    constexpr int STRIP = kBiasStrip, kGroups = STRIP / 8, ROWS = 256 / kGroups, kUnroll = 8;
    __shared__ float part[ROWS][STRIP + 1];
    __shared__ float mine[STRIP];
    mma::grid_wait();
    const int rank = (int)mma::cluster_rank();
    const int64_t j0 = (int64_t)(blockIdx.x / kBiasCluster) * STRIP;
    const int cg = threadIdx.x % kGroups, rg = threadIdx.x / kGroups;
    const int64_t r0 = m * rank / kBiasCluster, r1 = m * (rank + 1) / kBiasCluster;
    const int64_t j = j0 + cg * 8;
    float sum[8] = {};
    if (vec && j + 8 <= n) {
        const __nv_bfloat16* p = dy + j;
        int64_t r = r0 + rg;
        for (; r + (kUnroll - 1) * ROWS < r1; r += kUnroll * ROWS) {
            uint4 q[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) q[u] = __ldcs(reinterpret_cast<const uint4*>(p + (r + ROWS * u) * ld));
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int c = 0; c < 8; ++c) sum[c] += bf16_of(q[u], c);
        }
        for (; r < r1; r += ROWS) {
            float f[8];
            load8_bf16(p + r * ld, f);
#pragma unroll
            for (int c = 0; c < 8; ++c) sum[c] += f[c];
        }
    } else {
        for (int64_t r = r0 + rg; r < r1; r += ROWS)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (j + c < n) sum[c] += load_bf16(dy + r * ld + j + c);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) part[rg][cg * 8 + c] = sum[c];
    __syncthreads();
    if (threadIdx.x < STRIP) {
        float t = 0.0f;
        for (int k = 0; k < ROWS; ++k) t += part[k][threadIdx.x];
        mine[threadIdx.x] = t;
    }
    mma::cluster_sync();
    if (rank == 0 && threadIdx.x < STRIP && j0 + threadIdx.x < n) {
        float t = 0.0f;
        for (int p = 0; p < kBiasCluster; ++p)
            t += mma::ld_cluster(mma::map_rank(tma::smem_addr(&mine[threadIdx.x]), p));
        float* o = db + j0 + threadIdx.x;
        *o = accumulate ? *o + t : t;
    }
    mma::cluster_sync();
}

cudaError_t launch_bias_grad(const void* dy, int64_t ld, int64_t m, int64_t n, float* db, int accumulate, int vec, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n + kBiasStrip - 1) / kBiasStrip * kBiasCluster));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bias_grad_kernel, static_cast<const __nv_bfloat16*>(dy), ld, m, n, db, accumulate, vec);
}

// --------------------------------------------------------------- validation --

struct Mat {
    const void* p;
    int64_t rows, cols, ld;
    int esize;
    const char* name;
};

int check_matrix(const Mat& a) {
    if (a.rows == 0 || a.cols == 0) return DPRED_OK;
    if (!a.p) return set_error(DPRED_E_INVAL, "%s is null", a.name);
    if (reinterpret_cast<uintptr_t>(a.p) % a.esize) return set_error(DPRED_E_ALIGN, "%s is not aligned to its element size", a.name);
    if (a.rows > 1 && a.ld < a.cols)
        return set_error(DPRED_E_SIZE, "%s: row stride %lld is less than its %lld columns", a.name, (long long)a.ld,
                         (long long)a.cols);
    return DPRED_OK;
}

int check_sizes(int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || k < 0) return set_error(DPRED_E_INVAL, "a negative size (%lld, %lld, %lld)", (long long)m, (long long)n, (long long)k);
    if (m > 0x3FFFFFFF || n > 0x3FFFFFFF || k > 0x3FFFFFFF)
        return set_error(DPRED_E_SIZE, "a size above 2^30 - 1 (%lld, %lld, %lld)", (long long)m, (long long)n, (long long)k);
    return DPRED_OK;
}

bool dtype_ok(int dt) { return dt == DPRED_BF16 || dt == DPRED_F32; }

// A call of at most this many tokens puts the features on the 128 lanes and
// the tokens on the column side.
constexpr int64_t kFewTokens = 64;

// Rows whose 8-column groups are 16-byte aligned.
bool aligned_rows(const void* p, int64_t rows, int64_t ld, int esize) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * esize % 16 == 0);
}

int launch(Operand a, Operand b, int64_t red, const LinearEpi& e, void* workspace, size_t workspace_bytes, size_t need,
           cudaStream_t s, float* row_sum = nullptr, int row_sum_add = 0,
           bool* row_sum_formed = nullptr) {
    if (need > workspace_bytes || (need && !workspace))
        return set_error(DPRED_E_SIZE, "workspace of %zu bytes, %zu needed (operands whose rows are not 16-byte aligned)",
                         workspace_bytes, need);
    if (need && reinterpret_cast<uintptr_t>(workspace) % 16)
        return set_error(DPRED_E_ALIGN, "workspace is not 16-byte aligned");
    Plan p = {};
    p.args.err = device_error_word();
    if (red > 0) {
        Operand* const both[2] = {&a, &b};
        const int rc = pack(both, static_cast<char*>(workspace), s);
        if (rc != DPRED_OK) return rc;
    }
    p.a = a;
    p.b = b;
    p.args.m = (int)(a.reduce_rows ? a.cols : a.rows);
    p.args.n = (int)(b.reduce_rows ? b.cols : b.rows);
    p.args.kblocks = (int)((red + mma::kBlockK - 1) / mma::kBlockK);
    p.args.batch = 1;
    p.args.a_mn = a.reduce_rows;
    p.args.b_mn = b.reduce_rows;
    p.args.bf16 = 1;
    p.args.split_only = e.swapped;
    p.fp32_result = e.out_f32;
    p.args.row_sums = row_sum != nullptr;
    p.row_sum = row_sum;
    p.row_sum_add = row_sum_add;
    return run<KIND_LINEAR>(p, e, s, row_sum_formed);
}

}  // namespace
}  // namespace gemm
}  // namespace dpred

using namespace dpred;
using namespace dpred::gemm;

extern "C" size_t dpred_linear_workspace_bytes(const void* a, int64_t a_rows, int64_t a_cols, int64_t lda, const void* b,
                                               int64_t b_rows, int64_t b_cols, int64_t ldb) {
    if (a_rows <= 0 || a_cols <= 0 || b_rows <= 0 || b_cols <= 0) return 0;
    return pack_need(a, a_rows, a_cols, lda) + pack_need(b, b_rows, b_cols, ldb);
}

extern "C" int dpred_linear(int64_t m, int64_t n, int64_t k, const void* x, int64_t ldx, const void* w, int64_t ldw,
                            int32_t bias_dtype, const void* bias, int32_t act, const void* residual, int64_t ldr,
                            void* preact, int64_t ldp, int32_t out_dtype, void* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, void* stream) {
    int rc = check_sizes(m, n, k);
    if (rc != DPRED_OK) return rc;
    if (act < ACT_NONE || act > ACT_SILU) return set_error(DPRED_E_INVAL, "unknown activation %d", act);
    if (!dtype_ok(out_dtype)) return set_error(DPRED_E_INVAL, "unknown output type %d", out_dtype);
    if (bias && !dtype_ok(bias_dtype)) return set_error(DPRED_E_INVAL, "unknown bias type %d", bias_dtype);
    const int osize = out_dtype == DPRED_F32 ? 4 : 2, bsize = bias_dtype == DPRED_F32 ? 4 : 2;
    const Mat mats[] = {{x, m, k, ldx, 2, "x"}, {w, n, k, ldw, 2, "w"}, {y, m, n, ldy, osize, "y"}};
    for (const Mat& a : mats)
        if ((rc = check_matrix(a)) != DPRED_OK) return rc;
    if (residual && (rc = check_matrix({residual, m, n, ldr, 2, "residual"})) != DPRED_OK) return rc;
    if (preact && (rc = check_matrix({preact, m, n, ldp, 2, "preact"})) != DPRED_OK) return rc;
    if (bias && reinterpret_cast<uintptr_t>(bias) % bsize) return set_error(DPRED_E_ALIGN, "bias is not aligned to its element size");
    if (m == 0 || n == 0) return DPRED_OK;
    const bool few = m <= kFewTokens;
    LinearEpi e = {};
    e.out = y;
    e.bias = bias;
    e.res = static_cast<const __nv_bfloat16*>(residual);
    e.pre_out = static_cast<__nv_bfloat16*>(preact);
    e.out_f32 = out_dtype == DPRED_F32;
    e.bias_f32 = bias_dtype == DPRED_F32;
    e.act = act;
    e.swapped = few;
    e.o_ld = ldy;
    e.r_ld = ldr;
    e.p_ld = ldp;
    e.vec = aligned_rows(y, m, ldy, osize) && (!residual || aligned_rows(residual, m, ldr, 2)) &&
            (!preact || aligned_rows(preact, m, ldp, 2)) && reinterpret_cast<uintptr_t>(bias) % 16 == 0;
    const Operand tokens = {x, m, k, ldx, 0, false}, weight = {w, n, k, ldw, 0, false};
    const size_t need = k > 0 ? dpred_linear_workspace_bytes(x, m, k, ldx, w, n, k, ldw) : 0;
    return launch(few ? weight : tokens, few ? tokens : weight, k, e, workspace, workspace_bytes, need,
                  static_cast<cudaStream_t>(stream));
}

extern "C" int dpred_linear_dgrad(int64_t m, int64_t n, int64_t k, const void* dy, int64_t lddy, const void* w,
                                  int64_t ldw, int32_t act, const void* preact, int64_t ldp, const void* residual,
                                  int64_t ldr, int32_t out_dtype, void* dx, int64_t lddx, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    int rc = check_sizes(m, n, k);
    if (rc != DPRED_OK) return rc;
    if (act < ACT_NONE || act > ACT_SILU) return set_error(DPRED_E_INVAL, "unknown activation %d", act);
    if (!dtype_ok(out_dtype)) return set_error(DPRED_E_INVAL, "unknown output type %d", out_dtype);
    if (act != ACT_NONE && !preact && m && k) return set_error(DPRED_E_INVAL, "an activation's gradient needs preact");
    const int osize = out_dtype == DPRED_F32 ? 4 : 2;
    const Mat mats[] = {{dy, m, n, lddy, 2, "dy"}, {w, n, k, ldw, 2, "w"}, {dx, m, k, lddx, osize, "dx"}};
    for (const Mat& a : mats)
        if ((rc = check_matrix(a)) != DPRED_OK) return rc;
    if (residual && (rc = check_matrix({residual, m, k, ldr, 2, "residual"})) != DPRED_OK) return rc;
    if (act != ACT_NONE && (rc = check_matrix({preact, m, k, ldp, 2, "preact"})) != DPRED_OK) return rc;
    if (m == 0 || k == 0) return DPRED_OK;
    const bool few = m <= kFewTokens;
    LinearEpi e = {};
    e.out = dx;
    e.res = static_cast<const __nv_bfloat16*>(residual);
    e.z = act != ACT_NONE ? static_cast<const __nv_bfloat16*>(preact) : nullptr;
    e.out_f32 = out_dtype == DPRED_F32;
    e.act = act;
    e.swapped = few;
    e.o_ld = lddx;
    e.r_ld = ldr;
    e.z_ld = ldp;
    e.vec = aligned_rows(dx, m, lddx, osize) && (!residual || aligned_rows(residual, m, ldr, 2)) &&
            (!e.z || aligned_rows(preact, m, ldp, 2));
    const Operand tokens = {dy, m, n, lddy, 0, false}, weight = {w, n, k, ldw, 0, true};
    const size_t need = n > 0 ? dpred_linear_workspace_bytes(dy, m, n, lddy, w, n, k, ldw) : 0;
    return launch(few ? weight : tokens, few ? tokens : weight, n, e, workspace, workspace_bytes, need,
                  static_cast<cudaStream_t>(stream));
}

extern "C" int dpred_linear_wgrad(int64_t m, int64_t n, int64_t k, const void* dy, int64_t lddy, const void* x,
                                  int64_t ldx, int32_t accumulate, int32_t out_dtype, void* dw, int64_t lddw,
                                  float* bias_grad, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_sizes(m, n, k);
    if (rc != DPRED_OK) return rc;
    if (!dtype_ok(out_dtype)) return set_error(DPRED_E_INVAL, "unknown output type %d", out_dtype);
    const int osize = out_dtype == DPRED_F32 ? 4 : 2;
    const Mat mats[] = {{dy, m, n, lddy, 2, "dy"}, {x, m, k, ldx, 2, "x"}, {dw, n, k, lddw, osize, "dw"}};
    for (const Mat& a : mats)
        if ((rc = check_matrix(a)) != DPRED_OK) return rc;
    if (bias_grad && reinterpret_cast<uintptr_t>(bias_grad) % 4) return set_error(DPRED_E_ALIGN, "bias_grad is not aligned to 4 bytes");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Operand a = {dy, m, n, lddy, 0, true}, b = {x, m, k, ldx, 0, true};
    bool formed = false;  // the product's kernel has formed the bias gradient
    if (n > 0 && k > 0) {
        LinearEpi e = {};
        e.out = dw;
        e.out_f32 = out_dtype == DPRED_F32;
        e.accumulate = accumulate != 0;
        e.o_ld = lddw;
        e.vec = aligned_rows(dw, n, lddw, osize);
        const size_t need = m > 0 ? dpred_linear_workspace_bytes(dy, m, n, lddy, x, m, k, ldx) : 0;
        if ((rc = launch(a, b, m, e, workspace, workspace_bytes, need, s, bias_grad, accumulate != 0, &formed)) != DPRED_OK) return rc;
    }
    if (bias_grad && n > 0 && !formed) {
        const int vec = aligned_rows(dy, m, lddy, 2);
        const cudaError_t e = launch_bias_grad(dy, lddy, m, n, bias_grad, accumulate != 0, vec, s);
        if (e != cudaSuccess) return cuda_error(e, "bias gradient launch");
    }
    return DPRED_OK;
}
