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

// Few rows: a row group loads its row itself, up to 8 columns a thread where they
// are enough.
template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(512) forward_kernel(const __grid_constant__ ForwardArgs a, int lanes) {
    mma::grid_wait();
    const int id = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = blockDim.x / lanes;
    RowSum sum(lanes, group);
    // only 512 threads have several vectors each
    const float share = VPT > 1 ? 1.0f / 512 : share_of(lanes), inv_d = mean_of(lanes, a.d);
    for (int64_t row = (int64_t)blockIdx.x * groups + group; row < a.m; row += (int64_t)gridDim.x * groups) {
        Cols<T, VEC> x[VPT];
        Cols<__nv_bfloat16, VEC> y[VPT];
        F8 gate, pre;
        const int64_t gate_row = a.per_gate == a.m ? 0 : a.per_gate == 1 ? row : (uint32_t)row / (uint32_t)a.per_gate;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c0 = first<VEC>(v, id, lanes);
            if (a.y) y[v].load(a.y + row * a.ldy, c0, lanes, a.d);
            x[v].load(static_cast<const T*>(a.x) + row * a.ldx, c0, lanes, a.d);
            if (VPT == 1 && a.gate.p) gate = a.gate.load<VEC>(gate_row, c0, lanes, a.d);
            if (VPT == 1 && a.post.p) {
                const F8 post = a.post.load<VEC>(0, c0, lanes, a.d);
                gate = a.gate.p ? post * gate : post;
            }
            if (VPT == 1 && a.pre.p) pre = a.pre.load<VEC>(0, c0, lanes, a.d);
        }
        F8 r[VPT];
        if (a.y) {
            float iy = 1.0f;
            if (a.post.p) {
                float2 t = {};
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const F8 f = widen(y[v]);
                    t = dot8(f, f, t);
                }
                float s[1] = {(t.x + t.y) * share};
                sum(s);
                iy = rsqrtf(fmaf(s[0], inv_d, a.eps));
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
                F8 u = widen(y[v]) * splat(iy);
                if (VPT == 1) {
                    if (a.post.p || a.gate.p) u = u * gate;
                } else {
                    if (a.post.p) u = u * a.post.load<VEC>(0, c0, lanes, a.d);
                    if (a.gate.p) u = u * a.gate.load<VEC>(gate_row, c0, lanes, a.d);
                }
                r[v] = fma8(splat(a.scale), widen(x[v]), u);
                store_cols<VEC>(static_cast<T*>(a.r) + row * a.ldr, c0, lanes, a.d, r[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v) r[v] = widen(x[v]);
        }
        if (!a.pre.p) continue;
        float2 t = {};
#pragma unroll
        for (int v = 0; v < VPT; ++v) t = dot8(r[v], r[v], t);
        float s[1] = {(t.x + t.y) * share};
        sum(s);
        const float ir = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c0 = first<VEC>(v, id, lanes);
            if (VPT > 1) pre = a.pre.load<VEC>(0, c0, lanes, a.d);
            store_cols<VEC>(a.h + row * a.ldh, c0, lanes, a.d, r[v] * splat(ir) * pre);
        }
    }
}

// Many rows: a block for each SM has a stretch of them, and they come through a ring of
// bulk copies while rows before them are worked on.  The weights lie in shared memory,
// post and a gate that all rows share as one product.  What bounds it next to HBM is
// issue: LANES known to the compiler turns addresses into immediates, and WHOLE (y, post
// and pre are there, and all rows share a gate) spares the loop its tests.  16384 x 1024,
// bf16: 24.6 us, floor 20.0; 43196 x 777, rows of no alignment: 62 us, floor 40.
template <typename T, bool VEC, int VPT, int LANES, bool WHOLE>
__global__ void __launch_bounds__(512, 1) ring_forward_kernel(const __grid_constant__ ForwardArgs a, const __grid_constant__ Rows in) {
    extern __shared__ __align__(128) char smem[];
    constexpr int lanes = LANES;
    const bool has_y = WHOLE || a.y, has_post = WHOLE || a.post.p, has_pre = WHOLE || a.pre.p, own_gate = !WHOLE && in.seg[2].p;
    const int id = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = blockDim.x / lanes;
    const int64_t row0 = a.m * blockIdx.x / gridDim.x + group, row1 = a.m * (blockIdx.x + 1) / gridDim.x;
    Ring<VEC> ring(in, smem, group);
    ring.start(id);
    mma::grid_wait();
    int64_t ahead = row0;
    auto request = [&]() {
        if (id == 0 && ahead < row1) ring.request(in.seg, ahead);
        ahead += groups;
    };
    for (int k = 0; k < in.stages; ++k) request();
    float* weights = reinterpret_cast<float*>(smem + kBarrierBytes + groups * in.stages * in.slot_bytes);
    const Staged<VEC, VPT> post = {weights, lanes}, pre = {weights + staged_floats(lanes, VPT), lanes};
    fill<VEC, VPT>(lanes, a.d, [&](int c, bool in_row, int at) {
        const float w = has_pre && in_row ? a.pre.at(0, c) : 0.0f, p = has_y && in_row ? a.post.at(0, c) : 0.0f,
                    q = has_y && in_row && !own_gate ? a.gate.at(0, c) : 1.0f;
        if (has_pre) pre.at[at] = w;
        if (has_y) post.at[at] = p * q;
    });
    __syncthreads();
    RowSum sum(lanes, group);
    const float share = share_of(lanes), inv_d = mean_of(lanes, a.d);
    const F8 scale = splat(a.scale);
    for (int64_t row = row0; row < row1; row += groups) {
        const char* slot = ring.take();
        const T* in_x = ring.in(slot, in.seg[0], static_cast<const T*>(a.x) + row * a.ldx);
        F8 r[VPT];
        if (has_y) {
            Cols<__nv_bfloat16, VEC> y[VPT];
            const __nv_bfloat16* in_y = ring.in(slot, in.seg[1], a.y + row * a.ldy);
            float iy = 1.0f;
            float2 t = {};
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                y[v].load(in_y, first<VEC>(v, id, lanes), lanes, a.d);
                const F8 f = widen(y[v]);
                t = dot8(f, f, t);
            }
            if (has_post) {
                float s[1] = {(t.x + t.y) * share};
                sum(s);
                iy = rsqrtf(fmaf(s[0], inv_d, a.eps));
            }
            T* out = static_cast<T*>(a.r) + row * a.ldr;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
                F8 u = widen(y[v]) * splat(iy) * post.get(v, id);
                Cols<T, VEC> x;
                x.load(in_x, c0, lanes, a.d);
                if (own_gate) {
                    const char* p = in.seg[2].p + (in.seg[2].div == 1 ? row : row / in.seg[2].div) * in.seg[2].pitch;
                    const Weight g = {slot + in.seg[2].at + (VEC ? 0 : reinterpret_cast<uintptr_t>(p) % 16), a.gate.f32, 0};
                    u = u * g.load<VEC>(0, c0, lanes, a.d);
                }
                r[v] = fma8(scale, widen(x), u);
                store_cols<VEC>(out, c0, lanes, a.d, r[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                Cols<T, VEC> x;
                x.load(in_x, first<VEC>(v, id, lanes), lanes, a.d);
                r[v] = widen(x);
            }
        }
        float s[1] = {};
        if (has_pre) {
            float2 t = {};
#pragma unroll
            for (int v = 0; v < VPT; ++v) t = dot8(r[v], r[v], t);
            s[0] = (t.x + t.y) * share;
            sum(s);
        }
        // the row is in registers: its slot takes another
        if (lanes == 32 || !has_pre) group_sync(group, lanes);
        request();
        if (!has_pre) continue;
        const F8 ir = splat(rsqrtf(fmaf(s[0], inv_d, a.eps)));
        __nv_bfloat16* out = a.h + row * a.ldh;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c0 = first<VEC>(v, id, lanes);
            store_cols<VEC>(out, c0, lanes, a.d, r[v] * ir * pre.get(v, id));
        }
    }
}

template <typename T, bool VEC, int VPT, int LANES, bool WHOLE>
cudaError_t launch_ring(const ForwardArgs& a, const Rows& in, int groups, cudaStream_t s) {
    static bool done[64];
    const cudaError_t e = ensure_smem_attr(ring_forward_kernel<T, VEC, VPT, LANES, WHOLE>, kRoom, done);
    if (e != cudaSuccess) return e;
    const size_t smem = kBarrierBytes + (size_t)groups * in.stages * in.slot_bytes + 2 * 4 * staged_floats(LANES, VPT);
    return launch(ring_forward_kernel<T, VEC, VPT, LANES, WHOLE>, dim3((unsigned)sm_count()), groups * LANES, smem, s, a, in);
}

template <typename T, bool VEC, bool WHOLE>
cudaError_t launch_ring(const ForwardArgs& a, const RowShape& q, const Rows& in, int groups, cudaStream_t s) {
    if (q.vecs == 1) return launch_ring<T, VEC, 1, 32, WHOLE>(a, in, groups, s);
    if (q.vecs == 2) return launch_ring<T, VEC, 2, 32, WHOLE>(a, in, groups, s);
    if (q.lanes == 32) return launch_ring<T, VEC, 4, 32, WHOLE>(a, in, groups, s);
    if (q.lanes == 64) return launch_ring<T, VEC, 4, 64, WHOLE>(a, in, groups, s);
    if (q.lanes == 128) return launch_ring<T, VEC, 4, 128, WHOLE>(a, in, groups, s);
    if (q.lanes == 256) return launch_ring<T, VEC, 4, 256, WHOLE>(a, in, groups, s);
    return launch_ring<T, VEC, 4, 512, WHOLE>(a, in, groups, s);
}

template <typename T, bool VEC, int VPT>
cudaError_t launch_kernel(const ForwardArgs& a, const RowShape& q, cudaStream_t s) {
    const int64_t groups = q.threads / q.lanes;
    return launch(forward_kernel<T, VEC, VPT>, dim3((unsigned)((a.m + groups - 1) / groups)), q.threads, 0, s, a, q.lanes);
}

template <typename T, bool VEC>
cudaError_t launch_forward(const ForwardArgs& a, cudaStream_t s) {
    {
        const RowShape q = shape_of(a.d, 4);
        Rows in = {};
        in.add(0, VEC, a.x, a.m, a.ldx, a.d, sizeof(T));
        if (a.y) in.add(1, VEC, a.y, a.m, a.ldy, a.d, 2);
        if (a.gate.p && a.per_gate != a.m) in.add(2, VEC, a.gate.p, a.m, a.gate.ld, a.d, a.gate.f32 ? 4 : 2, a.per_gate);
        in.slot_bytes = in.slot();
        in.err = device_error_word();
        const int room = kRoom - 2 * 4 * staged_floats(q.lanes, q.vecs), groups = ring_groups(q, in.slot_bytes, room, 512);
        // A ring is worth its start where a row group has several rows.  Device time by
        // rows in registers / through rings, bf16 stream: 1216 x 1024 3.6 / 3.9 us, 4864
        // 13.3 / 10.3, 7296 18.6 / 13.4; 3648 x 256 2.8 / 4.4, 7296 5.0 / 5.4, 14592
        // 8.5 / 8.6; 4096 columns: 300 rows 4.0 / 5.1, 1216 15.2 / 13.2, 1800 21.9 / 16.2.
        // Rows of any alignment gain earlier: 1216 x 777 8.0 / 5.6, 4864 32 / 9.9.
        if (groups > 0 && a.m > 2 * (int64_t)groups * sm_count()) {
            in.stages = ring_stages(groups, in.slot_bytes, room);
            if (VEC && a.y && a.post.p && a.pre.p && !in.seg[2].p) return launch_ring<T, VEC, VEC>(a, q, in, groups, s);
            return launch_ring<T, VEC, false>(a, q, in, groups, s);
        }
    }
    const RowShape q = shape_of(a.d, 1);
    if (q.vecs == 1) return launch_kernel<T, VEC, 1>(a, q, s);
    if (q.vecs == 2) return launch_kernel<T, VEC, 2>(a, q, s);
    return launch_kernel<T, VEC, 4>(a, q, s);
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
