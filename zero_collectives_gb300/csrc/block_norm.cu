// block_norm.cu -- what stands between two blocks of a residual stream:
// dpred_block_norm.
//
//     N(a, w) = w a / sqrt(mean(a^2) + eps)
//     u = N(y, post)   (y without post);  r = s x + gate u;  h = N(r, pre)
//
// One pass: a row lies in the registers of `lanes` threads from its load to its
// store.  Statistics, r and u are fp32; r and h are each rounded once, so h is
// the norm of the unrounded r.  Bandwidth bound: x and y are read, r and h
// written once.
#include <algorithm>

#include "block_norm.cuh"

namespace dpred {
namespace layers {
namespace {

struct ForwardArgs {
    const void* x;
    const __nv_bfloat16* y;
    Weight post, gate, pre;
    void* r;
    __nv_bfloat16* h;
    int64_t ldx, ldy, ldr, ldh, m, per_gate;  // per_gate: rows of a gate row
    int32_t d;
    float scale, eps;
};

template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(512) forward_kernel(const __grid_constant__ ForwardArgs a, int lanes) {
    mma::grid_wait();
    const int id = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = blockDim.x / lanes;
    RowSum sum(lanes, group);
    const float inv_d = 1.0f / (float)a.d;
    for (int64_t row = (int64_t)blockIdx.x * groups + group; row < a.m; row += (int64_t)gridDim.x * groups) {
        Cols<T, VEC> x[VPT];
        Cols<__nv_bfloat16, VEC> y[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) x[v].load(static_cast<const T*>(a.x) + row * a.ldx, first<VEC>(v, id, lanes), lanes, a.d);
        float r[VPT][8];
        if (a.y) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) y[v].load(a.y + row * a.ldy, first<VEC>(v, id, lanes), lanes, a.d);
            float iy = 1.0f;
            if (a.post.p) {
                float s[1] = {};
#pragma unroll
                for (int v = 0; v < VPT; ++v)
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[0] = fmaf(y[v][k], y[v][k], s[0]);
                sum(s);
                iy = rsqrtf(fmaf(s[0], inv_d, a.eps));
            }
            const int64_t gate_row = a.per_gate == a.m ? 0 : a.per_gate == 1 ? row : row / a.per_gate;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
                float w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) r[v][k] = y[v][k] * iy;
                if (a.post.p) {
                    a.post.load<VEC>(0, c0, lanes, a.d, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) r[v][k] *= w[k];
                }
                if (a.gate.p) {
                    a.gate.load<VEC>(gate_row, c0, lanes, a.d, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) r[v][k] *= w[k];
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) r[v][k] = fmaf(a.scale, x[v][k], r[v][k]);
                store_cols<VEC>(static_cast<T*>(a.r) + row * a.ldr, c0, lanes, a.d, r[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int k = 0; k < 8; ++k) r[v][k] = x[v][k];
        }
        if (a.pre.p) {
            float s[1] = {};
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[0] = fmaf(r[v][k], r[v][k], s[0]);
            sum(s);
            const float ir = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
                float w[8];
                a.pre.load<VEC>(0, c0, lanes, a.d, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] *= r[v][k] * ir;
                store_cols<VEC>(a.h + row * a.ldh, c0, lanes, a.d, w);
            }
        }
    }
}

template <typename T, bool VEC>
cudaError_t launch_forward(const ForwardArgs& a, cudaStream_t s) {
    const RowShape q = shape_of(a.d);
    const int64_t groups = q.threads / q.lanes, blocks = (a.m + groups - 1) / groups;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, 0x7FFFFFFF));
    if (q.vecs == 1) return launch(forward_kernel<T, VEC, 1>, grid, q.threads, 0, s, a, q.lanes);
    if (q.vecs == 2) return launch(forward_kernel<T, VEC, 2>, grid, q.threads, 0, s, a, q.lanes);
    return launch(forward_kernel<T, VEC, 4>, grid, q.threads, 0, s, a, q.lanes);
}

}  // namespace
}  // namespace layers
}  // namespace dpred

using namespace dpred;
using namespace dpred::layers;

extern "C" int dpred_block_norm(int64_t m, int64_t d, int32_t r_dtype, const void* x, int64_t ldx, const void* y, int64_t ldy,
                                int32_t post_dtype, const void* post, int32_t gate_dtype, const void* gate, int64_t gate_rows, float scale,
                                int32_t pre_dtype, const void* pre, float eps, void* r, int64_t ldr, void* h, int64_t ldh, void* stream) {
    const NormShape n = {m, d, r_dtype, y, post_dtype, post, gate_dtype, gate, gate_rows, scale, pre_dtype, pre, eps};
    int rc = check_norm(n);
    if (rc != DPRED_OK) return rc;
    if (m == 0 || d == 0) return DPRED_OK;
    const int es = esize(r_dtype);
    if ((rc = check_matrix(x, m, d, ldx, es, "x")) != DPRED_OK || (y && (rc = check_matrix(y, m, d, ldy, 2, "y")) != DPRED_OK) ||
        (y && (rc = check_matrix(r, m, d, ldr, es, "r")) != DPRED_OK) || (pre && (rc = check_matrix(h, m, d, ldh, 2, "h")) != DPRED_OK))
        return rc;
    ForwardArgs a = {};
    a.x = x;
    a.y = static_cast<const __nv_bfloat16*>(y);
    a.post = {post, post_dtype == DPRED_F32, d};
    a.gate = {gate, gate_dtype == DPRED_F32, d};
    a.pre = {pre, pre_dtype == DPRED_F32, d};
    a.r = r;
    a.h = static_cast<__nv_bfloat16*>(h);
    a.ldx = ldx;
    a.ldy = ldy;
    a.ldr = ldr;
    a.ldh = ldh;
    a.m = m;
    a.per_gate = gate ? m / gate_rows : m;
    a.d = (int32_t)d;
    a.scale = scale;
    a.eps = eps;
    const bool vec = weights_aligned(n) && aligned_rows(x, m, ldx, es) && (!y || (aligned_rows(y, m, ldy, 2) && aligned_rows(r, m, ldr, es))) &&
                     (!pre || aligned_rows(h, m, ldh, 2));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = r_dtype == DPRED_F32 ? (vec ? launch_forward<float, true>(a, s) : launch_forward<float, false>(a, s))
                                               : (vec ? launch_forward<__nv_bfloat16, true>(a, s) : launch_forward<__nv_bfloat16, false>(a, s));
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "block norm launch");
}
