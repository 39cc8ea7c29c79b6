// block_norm_grad.cu -- the gradient of the block norm: dpred_block_norm_grad.
//
// With n_r = r / sqrt(mean(r^2) + eps), i_r the reciprocal of that root, and n_y,
// i_y for y (y itself and 1 without post):
//
//     v  = dh pre,            g  = dr + i_r (v - n_r mean(v n_r))
//     dx = s g,               dpre  = sum of dh n_r over the rows
//     u  = n_y post,          dgate = sum of g u over the rows of a gate row
//     e  = g gate,            dpost = sum of e n_y over the rows
//     w  = e post,            dy = i_y (w - n_y mean(w n_y))
//
// One pass: the roots are formed again from r and y, which are read anyway, in
// the same sums over the row as the means (r^2, v r and y^2 at once, then w y),
// so the forward pass keeps nothing.  Sums over rows stay in registers while a
// block walks its rows, meet in shared memory, and leave one partial row per
// block; a second launch adds those in block order.  All of it is fp32; dx, dy
// and the weight gradients are each rounded once.
//
// Bandwidth bound: r, y, dr and dh are read, dx and dy written once.
#include <algorithm>

#include "block_norm.cuh"

namespace dpred {
namespace layers {
namespace {

// A weight gradient: where it goes and how.
struct Target {
    void* p;
    int64_t ld;
    int32_t f32, add;
#ifdef __CUDACC__
    __device__ __forceinline__ void put(int64_t row, int c, float v) const {
        if (f32) {
            float* o = static_cast<float*>(p) + row * ld + c;
            *o = add ? *o + v : v;
        } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p) + row * ld + c;
            store1(o, add ? load1(o) + v : v);
        }
    }
#endif
};

struct BackwardArgs {
    const void* r;
    const void* dr;           // null: 0
    const __nv_bfloat16* dh;  // null: no norm above
    const __nv_bfloat16* y;   // null: no block below
    Weight post, gate, pre;
    void* dx;
    __nv_bfloat16* dy;
    Target dpost, dgate, dpre;  // p null: not wanted
    float* partial;             // rows of d: dpost and dpre of each block, dgate of each unit
    int64_t ldr, lddr, lddh, ldy, lddx, lddy;
    int64_t sections;  // consecutive rows that share a gate row (the whole when each row has its own)
    int64_t per;       // rows of a section
    int32_t parts;     // units of a section
    int32_t each;      // every row has a gate row of its own
    int32_t d;
    int32_t release;   // another launch of the call follows
    float scale, eps;
};

constexpr int kCombine = 2048;  // columns of a block's row groups where there are several: 256 threads of 8

// Adds the threads' sums of a column over the block's row groups, in order.
template <bool VEC, int VPT, typename F>
__device__ __forceinline__ void combine(float (&s)[VPT][8], int id, int group, int groups, int lanes, int d, float* buf, F put) {
    if (groups == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = column<VEC>(first<VEC>(v, id, lanes), lanes, k);
                if (c < d) put(c, s[v][k]);
            }
        return;
    }
    // several groups hold a row in one vector a thread
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) buf[(group * 8 + k) * lanes + id] = s[0][k];
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * lanes; i += blockDim.x) {
        const int k = i / lanes, t = i % lanes, c = column<VEC>(first<VEC>(0, t, lanes), lanes, k);
        if (c >= d) continue;
        float v = 0.0f;
        for (int g = 0; g < groups; ++g) v += buf[(g * 8 + k) * lanes + t];
        put(c, v);
    }
}

template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(512) backward_kernel(const __grid_constant__ BackwardArgs a, int lanes) {
    __shared__ float buf[kCombine];
    if (a.release) mma::grid_launch_dependents();
    mma::grid_wait();
    const int id = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = blockDim.x / lanes;
    RowSum sum(lanes, group);
    const float inv_d = 1.0f / (float)a.d;
    float dpost[VPT][8] = {}, dpre[VPT][8] = {};
    const int64_t units = a.sections * a.parts;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t section = unit / a.parts, part = unit - section * a.parts;
        const int64_t row0 = section * a.per + a.per * part / a.parts, row1 = section * a.per + a.per * (part + 1) / a.parts;
        float dgate[VPT][8] = {};
        for (int64_t row = row0 + group; row < row1; row += groups) {
            Cols<T, VEC> r[VPT], dr[VPT];
            Cols<__nv_bfloat16, VEC> dh[VPT], y[VPT];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
                if (a.dh) {
                    r[v].load(static_cast<const T*>(a.r) + row * a.ldr, c0, lanes, a.d);
                    dh[v].load(a.dh + row * a.lddh, c0, lanes, a.d);
                }
                if (a.y) y[v].load(a.y + row * a.ldy, c0, lanes, a.d);
                if (a.dr) dr[v].load(static_cast<const T*>(a.dr) + row * a.lddr, c0, lanes, a.d);
            }
            float s[3] = {};  // r^2, dh pre r, y^2
            float w[8];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (a.dh) {
                    a.pre.load<VEC>(0, first<VEC>(v, id, lanes), lanes, a.d, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        s[0] = fmaf(r[v][k], r[v][k], s[0]);
                        s[1] = fmaf(dh[v][k] * w[k], r[v][k], s[1]);
                    }
                }
                if (a.post.p)
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[2] = fmaf(y[v][k], y[v][k], s[2]);
            }
            if (a.dh || a.post.p) sum(s);
            const float ir = rsqrtf(fmaf(s[0], inv_d, a.eps)), iy = a.post.p ? rsqrtf(fmaf(s[2], inv_d, a.eps)) : 1.0f;
            const float mean_r = s[1] * inv_d * ir;  // of v n_r
            float q[1] = {};                         // w y
            float g[VPT][8];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
#pragma unroll
                for (int k = 0; k < 8; ++k) g[v][k] = a.dr ? dr[v][k] : 0.0f;
                if (a.dh) {
                    a.pre.load<VEC>(0, c0, lanes, a.d, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float n = r[v][k] * ir;
                        g[v][k] = fmaf(ir, fmaf(-n, mean_r, dh[v][k] * w[k]), g[v][k]);
                        dpre[v][k] = fmaf(dh[v][k], n, dpre[v][k]);
                    }
                }
                float o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = a.scale * g[v][k];
                store_cols<VEC>(static_cast<T*>(a.dx) + row * a.lddx, c0, lanes, a.d, o);
                if (!a.y) continue;
                float post[8];
                if (a.post.p) a.post.load<VEC>(0, c0, lanes, a.d, post);
                if (a.gate.p) {
                    a.gate.load<VEC>(a.each ? row : section, c0, lanes, a.d, w);
                    if (a.dgate.p) {
                        float u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] = a.post.p ? y[v][k] * iy * post[k] : y[v][k];
                        if (a.each) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int c = column<VEC>(c0, lanes, k);
                                if (c < a.d) a.dgate.put(row, c, g[v][k] * u[k]);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k) dgate[v][k] = fmaf(g[v][k], u[k], dgate[v][k]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[v][k] *= w[k];
                }
                if (a.post.p) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        dpost[v][k] = fmaf(g[v][k], y[v][k] * iy, dpost[v][k]);
                        g[v][k] *= post[k];
                        q[0] = fmaf(g[v][k], y[v][k], q[0]);
                    }
                }
            }
            if (!a.y) continue;
            if (a.post.p) sum(q);
            const float mean_y = q[0] * inv_d * iy;  // of w n_y
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (a.post.p)
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[v][k] = iy * fmaf(-(y[v][k] * iy), mean_y, g[v][k]);
                store_cols<VEC>(a.dy + row * a.lddy, first<VEC>(v, id, lanes), lanes, a.d, g[v]);
            }
        }
        if (a.dgate.p && !a.each)
            combine<VEC>(dgate, id, group, groups, lanes, a.d, buf, [&](int c, float v) {
                if (a.parts == 1)
                    a.dgate.put(section, c, v);
                else
                    a.partial[(2 * (int64_t)gridDim.x + unit) * a.d + c] = v;
            });
    }
    if (a.dpost.p)
        combine<VEC>(dpost, id, group, groups, lanes, a.d, buf, [&](int c, float v) {
            if (gridDim.x == 1)
                a.dpost.put(0, c, v);
            else
                a.partial[(int64_t)blockIdx.x * a.d + c] = v;
        });
    if (a.dpre.p)
        combine<VEC>(dpre, id, group, groups, lanes, a.d, buf, [&](int c, float v) {
            if (gridDim.x == 1)
                a.dpre.put(0, c, v);
            else
                a.partial[((int64_t)gridDim.x + blockIdx.x) * a.d + c] = v;
        });
}

// Adds the partial rows of one weight gradient: 32 columns a block, 32 shares of
// the rows, added in order.
struct Job {
    const float* src;
    int64_t rows;
    Target to;
};
struct FinishArgs {
    Job dpost, dpre, dgate;  // in this order, gate rows last
    int32_t d;
};

__global__ void __launch_bounds__(1024) finish_kernel(const __grid_constant__ FinishArgs a) {
    __shared__ float part[32][33];
    mma::grid_wait();
    int at = blockIdx.y;
    int64_t out_row = 0;
    const Job* j = &a.dpost;
    if (!a.dpost.to.p || at > 0) {
        at -= a.dpost.to.p != nullptr;
        j = &a.dpre;
        if (!a.dpre.to.p || at > 0) {
            out_row = at - (a.dpre.to.p != nullptr);
            j = &a.dgate;
        }
    }
    const float* src = j->src + out_row * j->rows * a.d;
    const int lane = threadIdx.x % 32, share = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const int64_t r0 = j->rows * share / 32, r1 = j->rows * (share + 1) / 32;
    float v = 0.0f;
    if (c < a.d) {
#pragma unroll 8
        for (int64_t r = r0; r < r1; ++r) v += src[r * a.d + c];
    }
    part[share][lane] = v;
    __syncthreads();
    if (share || c >= a.d) return;
    v = 0.0f;
    for (int w = 0; w < 32; ++w) v += part[w][lane];
    j->to.put(out_row, c, v);
}

// --------------------------------------------------------------------- host --

constexpr int kBlocksPerSm = 2;

struct Grid {
    RowShape q;
    int64_t sections, per, blocks;
    int32_t parts;
};

// Sections are cut into as many units as there are resident blocks, or dealt
// out whole where there are more of them.
Grid grid_of(int64_t m, int64_t d, int64_t gate_rows) {
    Grid g;
    g.q = shape_of(d);
    g.sections = gate_rows <= 1 || gate_rows == m ? 1 : gate_rows;
    g.per = m / g.sections;
    const int64_t groups = g.q.threads / g.q.lanes, most = (int64_t)kBlocksPerSm * sm_count();
    const int64_t parts = std::min((g.per + groups - 1) / groups, std::max<int64_t>(1, most / g.sections));
    g.parts = (int32_t)std::max<int64_t>(1, parts);
    g.blocks = std::min(most, g.sections * g.parts);
    return g;
}

size_t partial_bytes(const Grid& g, int64_t d) { return (size_t)((2 * g.blocks + (g.parts > 1 ? g.sections * g.parts : 0)) * d) * 4; }

template <typename T, bool VEC>
cudaError_t launch_backward(const BackwardArgs& a, const Grid& g, cudaStream_t s) {
    const dim3 grid((unsigned)g.blocks);
    if (g.q.vecs == 1) return launch(backward_kernel<T, VEC, 1>, grid, g.q.threads, 0, s, a, g.q.lanes);
    if (g.q.vecs == 2) return launch(backward_kernel<T, VEC, 2>, grid, g.q.threads, 0, s, a, g.q.lanes);
    return launch(backward_kernel<T, VEC, 4>, grid, g.q.threads, 0, s, a, g.q.lanes);
}

}  // namespace
}  // namespace layers
}  // namespace dpred

using namespace dpred;
using namespace dpred::layers;

extern "C" size_t dpred_block_norm_grad_workspace_bytes(int64_t m, int64_t d, int64_t gate_rows) {
    if (m <= 0 || d <= 0 || d > kMaxWidth || gate_rows < 0 || (gate_rows > 0 && m % gate_rows)) return 0;
    return partial_bytes(grid_of(m, d, gate_rows), d);
}

extern "C" int dpred_block_norm_grad(int64_t m, int64_t d, int32_t r_dtype, const void* r, int64_t ldr, const void* dr, int64_t lddr,
                                     const void* dh, int64_t lddh, const void* y, int64_t ldy, int32_t post_dtype, const void* post,
                                     int32_t gate_dtype, const void* gate, int64_t gate_rows, float scale, int32_t pre_dtype, const void* pre,
                                     float eps, void* dx, int64_t lddx, void* dy, int64_t lddy, int32_t grad_dtype, void* post_grad,
                                     void* gate_grad, void* pre_grad, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    const NormShape n = {m, d, r_dtype, y, post_dtype, post, gate_dtype, gate, gate_rows, scale, pre_dtype, pre, eps};
    int rc = check_norm(n);
    if (rc != DPRED_OK) return rc;
    if ((rc = check_dtype(grad_dtype, "the weight gradients")) != DPRED_OK) return rc;
    if ((post_grad && !post) || (gate_grad && !gate) || (pre_grad && !pre)) return set_error(DPRED_E_INVAL, "a gradient of a weight that is not given");
    const int gs = esize(grad_dtype), es = esize(r_dtype);
    for (const void* p : {post_grad, gate_grad, pre_grad})
        if (reinterpret_cast<uintptr_t>(p) % gs) return set_error(DPRED_E_ALIGN, "a weight gradient is not aligned to its element size");
    if (d == 0) return DPRED_OK;
    if ((pre && (rc = check_matrix(r, m, d, ldr, es, "r")) != DPRED_OK) || (pre && (rc = check_matrix(dh, m, d, lddh, 2, "dh")) != DPRED_OK) ||
        (dr && (rc = check_matrix(dr, m, d, lddr, es, "dr")) != DPRED_OK) || (rc = check_matrix(dx, m, d, lddx, es, "dx")) != DPRED_OK ||
        (y && (rc = check_matrix(y, m, d, ldy, 2, "y")) != DPRED_OK) || (y && (rc = check_matrix(dy, m, d, lddy, 2, "dy")) != DPRED_OK))
        return rc;
    if (m > 0 && !dr && !pre) return set_error(DPRED_E_INVAL, "neither dr nor pre: no gradient comes in");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (m == 0) {  // sums of no rows
        if (accumulate) return DPRED_OK;
        struct { void* p; int64_t n; } const outs[] = {{post_grad, d}, {pre_grad, d}, {gate_grad, std::max<int64_t>(gate_rows, 0) * d}};
        for (const auto& o : outs) {
            const cudaError_t e = o.p && o.n ? cudaMemsetAsync(o.p, 0, (size_t)o.n * gs, s) : cudaSuccess;
            if (e != cudaSuccess) return cuda_error(e, "block norm gradient of no rows");
        }
        return DPRED_OK;
    }
    const Grid g = grid_of(m, d, gate ? gate_rows : 0);
    const bool each = gate && gate_rows == m && m > 1;
    const bool gate_sums = gate_grad && !each;
    if ((post_grad || pre_grad || gate_sums) && (rc = check_workspace(workspace, workspace_bytes, partial_bytes(g, d))) != DPRED_OK) return rc;
    BackwardArgs a = {};
    a.r = r;
    a.dr = dr;
    a.dh = pre ? static_cast<const __nv_bfloat16*>(dh) : nullptr;
    a.y = static_cast<const __nv_bfloat16*>(y);
    a.post = {post, post_dtype == DPRED_F32, d};
    a.gate = {gate, gate_dtype == DPRED_F32, d};
    a.pre = {pre, pre_dtype == DPRED_F32, d};
    a.dx = dx;
    a.dy = static_cast<__nv_bfloat16*>(dy);
    const int32_t f32 = grad_dtype == DPRED_F32, add = accumulate != 0;
    a.dpost = {post_grad, d, f32, add};
    a.dgate = {gate_grad, d, f32, add};
    a.dpre = {pre_grad, d, f32, add};
    a.partial = static_cast<float*>(workspace);
    a.ldr = ldr;
    a.lddr = lddr;
    a.lddh = lddh;
    a.ldy = ldy;
    a.lddx = lddx;
    a.lddy = lddy;
    a.sections = g.sections;
    a.per = g.per;
    a.parts = g.parts;
    a.each = each;
    a.d = (int32_t)d;
    a.scale = scale;
    a.eps = eps;
    const bool vec = weights_aligned(n) && (!pre || (aligned_rows(r, m, ldr, es) && aligned_rows(dh, m, lddh, 2))) && (!dr || aligned_rows(dr, m, lddr, es)) &&
                     aligned_rows(dx, m, lddx, es) && (!y || (aligned_rows(y, m, ldy, 2) && aligned_rows(dy, m, lddy, 2)));
    FinishArgs f = {};
    f.d = (int32_t)d;
    if (g.blocks > 1) {
        if (post_grad) f.dpost = {a.partial, g.blocks, a.dpost};
        if (pre_grad) f.dpre = {a.partial + g.blocks * d, g.blocks, a.dpre};
    }
    if (gate_sums && g.parts > 1) f.dgate = {a.partial + 2 * g.blocks * d, g.parts, a.dgate};
    const int64_t jobs = (f.dpost.to.p != nullptr) + (f.dpre.to.p != nullptr) + (f.dgate.to.p ? g.sections : 0);
    a.release = jobs > 0;
    cudaError_t e = r_dtype == DPRED_F32 ? (vec ? launch_backward<float, true>(a, g, s) : launch_backward<float, false>(a, g, s))
                                         : (vec ? launch_backward<__nv_bfloat16, true>(a, g, s) : launch_backward<__nv_bfloat16, false>(a, g, s));
    if (e != cudaSuccess) return cuda_error(e, "block norm gradient launch");
    if (jobs == 0) return DPRED_OK;
    e = launch(finish_kernel, dim3((unsigned)((d + 31) / 32), (unsigned)jobs), 1024, 0, s, f);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "block norm gradient launch");
}
