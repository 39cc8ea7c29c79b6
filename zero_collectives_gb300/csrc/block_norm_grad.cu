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

#include "block_norm_grad.cuh"

namespace dpred {
namespace layers {
namespace {

// Adds the partial rows of one weight gradient: 32 columns a block, 16 shares of
// the rows, added in order.
constexpr int kShares = 16;
struct Job {
    const float* src;
    int64_t rows;
    Target to;
};
struct FinishArgs {
    Job dpost, dpre, dgate;  // in this order, gate rows last
    int32_t d;
};

__global__ void __launch_bounds__(kShares * 32) finish_kernel(const __grid_constant__ FinishArgs a) {
    __shared__ float part[kShares][32];
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
    const int64_t r0 = j->rows * share / kShares, r1 = j->rows * (share + 1) / kShares;
    float v = 0.0f;
    if (c < a.d) {
#pragma unroll 8
        for (int64_t r = r0; r < r1; ++r) v += src[r * a.d + c];
    }
    part[share][lane] = v;
    __syncthreads();
    if (share || c >= a.d) return;
    v = 0.0f;
    for (int w = 0; w < kShares; ++w) v += part[w][lane];
    j->to.put(out_row, c, v);
}

// --------------------------------------------------------------------- host --

// Sections are cut into as many units as there are blocks (one to an SM), or dealt
// out whole where there are more of them.
Grid grid_of(int64_t m, int64_t d, int64_t gate_rows, bool vec) {
    Grid g;
    g.q = shape_of(d, vec ? 2 : 1);
    g.sections = gate_rows <= 1 || gate_rows == m ? 1 : gate_rows;
    g.per = m / g.sections;
    g.groups = std::max(1, kThreads / g.q.lanes);
    const int64_t most = sm_count(), parts = std::min((g.per + g.groups - 1) / g.groups, std::max<int64_t>(1, most / g.sections));
    g.parts = (int32_t)std::max<int64_t>(1, parts);
    g.blocks = std::min(most, g.sections * g.parts);
    return g;
}

size_t partial_bytes(const Grid& g, int64_t d) { return (size_t)((2 * g.blocks + (g.parts > 1 ? g.sections * g.parts : 0)) * d) * 4; }

template <typename T>
cudaError_t launch_backward(const BackwardArgs& a, int64_t m, const Grid& g, bool vec, cudaStream_t s) {
    Rows in = {};
    const int es = (int)sizeof(T), gs = a.gate.f32 ? 4 : 2;
    const struct { const void* p; int64_t ld; int es; } parts[kSegments] = {
        {a.dh ? a.r : nullptr, a.ldr, es}, {a.dr, a.lddr, es}, {a.dh, a.lddh, 2}, {a.y, a.ldy, 2}, {a.each ? a.gate.p : nullptr, a.gate.ld, gs}};
    for (int k = 0; k < kSegments; ++k)
        if (parts[k].p) in.add(k, vec, parts[k].p, m, parts[k].ld, a.d, parts[k].es);
    const int room = kRoom - 4 * staged_space(g.q.lanes, g.q.vecs, g.groups);
    if (in.seg[4].p && in.slot() + kBarrierBytes > room) in.drop(4);  // the gate of the widest rows is read in place
    in.slot_bytes = in.slot();
    in.err = device_error_word();
    const int groups = std::max(1, ring_groups(g.q, in.slot_bytes, room, g.groups * g.q.lanes));  // the widest rows have a single slot
    in.stages = ring_stages(groups, in.slot_bytes, room);
    const bool whole = a.dr && a.dh && a.y && a.post.p && !a.each;
    if (!vec) return launch_rows<T, false, false>(a, in, g, groups, s);
    return whole ? launch_rows<T, true, true>(a, in, g, groups, s) : launch_rows<T, true, false>(a, in, g, groups, s);
}

}  // namespace
}  // namespace layers
}  // namespace dpred

using namespace dpred;
using namespace dpred::layers;

extern "C" size_t dpred_block_norm_grad_workspace_bytes(int64_t m, int64_t d, int64_t gate_rows) {
    if (m <= 0 || d <= 0 || d > kMaxWidth || gate_rows < 0 || (gate_rows > 0 && m % gate_rows)) return 0;
    return std::max(partial_bytes(grid_of(m, d, gate_rows, true), d), partial_bytes(grid_of(m, d, gate_rows, false), d));
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
    const bool each = gate && gate_rows == m && m > 1;
    const bool vec = weights_aligned(n) && (!pre || (aligned_rows(r, m, ldr, es) && aligned_rows(dh, m, lddh, 2))) &&
                     (!dr || aligned_rows(dr, m, lddr, es)) && aligned_rows(dx, m, lddx, es) &&
                     (!each || reinterpret_cast<uintptr_t>(gate_grad) % 16 == 0) &&
                     (!y || (aligned_rows(y, m, ldy, 2) && aligned_rows(dy, m, lddy, 2)));
    const Grid g = grid_of(m, d, gate ? gate_rows : 0, vec);
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
    FinishArgs f = {};
    f.d = (int32_t)d;
    if (post_grad && g.sections * g.parts > 1) f.dpost = {a.partial, g.blocks, a.dpost};
    if (pre_grad && g.blocks > 1) f.dpre = {a.partial + g.blocks * d, g.blocks, a.dpre};
    if (gate_sums && g.parts > 1) f.dgate = {a.partial + 2 * g.blocks * d, g.parts, a.dgate};
    const int64_t jobs = (f.dpost.to.p != nullptr) + (f.dpre.to.p != nullptr) + (f.dgate.to.p ? g.sections : 0);
    a.release = jobs > 0;
    cudaError_t e = r_dtype == DPRED_F32 ? launch_backward<float>(a, m, g, vec, s) : launch_backward<__nv_bfloat16>(a, m, g, vec, s);
    if (e != cudaSuccess) return cuda_error(e, "block norm gradient launch");
    if (jobs == 0) return DPRED_OK;
    e = launch(finish_kernel, dim3((unsigned)((d + 31) / 32), (unsigned)jobs), kShares * 32, 0, s, f);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "block norm gradient launch");
}
