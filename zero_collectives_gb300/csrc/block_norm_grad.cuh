// block_norm_grad.cuh -- the kernel of dpred_block_norm_grad (block_norm_grad.cu),
// shared by the units that hold its forms.
#pragma once

#include "block_norm.cuh"

namespace dpred {
namespace layers {

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
    template <bool VEC>
    __device__ __forceinline__ void put8(int64_t row, int c0, int step, int d, const F8& v) const {
        if (f32)
            put8<VEC>(static_cast<float*>(p) + row * ld, c0, step, d, v);
        else
            put8<VEC>(static_cast<__nv_bfloat16*>(p) + row * ld, c0, step, d, v);
    }
    template <bool VEC, typename T>
    __device__ __forceinline__ void put8(T* o, int c0, int step, int d, F8 v) const {
        if (add) {
            Cols<T, VEC> old;
            old.load(o, c0, step, d);
            const F8 f = widen(old);
#pragma unroll
            for (int i = 0; i < 4; ++i) v.p[i] = make_float2(v.p[i].x + f.p[i].x, v.p[i].y + f.p[i].y);
        }
        store_cols<VEC>(o, c0, step, d, v);
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

// Adds the threads' sums of a column over the block's row groups, in order; put
// gets each column's, always in the same thread.
template <bool VEC, int VPT, typename F>
__device__ __forceinline__ void combine(const F8 (&s)[VPT], int id, int group, int groups, int lanes, int d, float* buf, F put) {
    if (groups == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = column<VEC>(first<VEC>(v, id, lanes), lanes, k);
                if (c < d) put(c, s[v].get(k));
            }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) buf[((group * VPT + v) * 8 + k) * lanes + id] = s[v].get(k);
    __syncthreads();
    for (int i = threadIdx.x; i < VPT * 8 * lanes; i += blockDim.x) {
        const int v = i / (8 * lanes), k = i / lanes % 8, t = i % lanes, c = column<VEC>(first<VEC>(v, t, lanes), lanes, k);
        if (c >= d) continue;
        float x = 0.0f;
        for (int g = 0; g < groups; ++g) x += buf[g * VPT * 8 * lanes + i];
        put(c, x);
    }
}

// Threads of a block: three warps a scheduler, which leaves a thread 168 registers;
// 512 where a row takes as many.
constexpr int kThreads = 384;

// The rows of a row group: every groups-th of its block's units, in turn.
struct Walk {
    int64_t unit, row = 0, end = 0;
    __device__ __forceinline__ explicit Walk(const BackwardArgs& a, int group) : unit(blockIdx.x) { enter(a, group); }
    __device__ __forceinline__ void enter(const BackwardArgs& a, int group) {
        const int64_t section = unit / a.parts, part = unit - section * a.parts;
        row = section * a.per + a.per * part / a.parts + group;
        end = section * a.per + a.per * (part + 1) / a.parts;
    }
    // Whether there is a row; moves on to the next unit that has one.
    __device__ __forceinline__ bool any(const BackwardArgs& a, int group) {
        while (row >= end) {
            unit += gridDim.x;
            if (unit >= a.sections * a.parts) return false;
            enter(a, group);
        }
        return true;
    }
};

// Rows come through a ring of bulk copies while rows before them are worked on;
// without it a row's loads and its two sums follow one another, and the few row
// groups that an SM holds cannot hide that (16384 x 1024 took 74 us).  A row that
// fills the only slot is asked for when the one before it is done.
// VEC: aligned rows, 8 columns next to each other a thread; otherwise every
// LANES-th, read from the slots and stored element by element, with one thread working
// out where the copies of a row begin and end (43196 x 777, bf16: 284 us, floor 60;
// 16384 x 1024 in the aligned form 44 us, floor 30).  Rows of more than 8192 columns
// come one at a time for each SM and are read three times from shared memory
// (2730 x 12288, bf16: 160 us, floor 60).
//
// Where rows share a gate row, sum of g n_y over them gives both gradients:
// dgate = post times it, dpost = gate times it, which is added per unit.
//
// What bounds it next to HBM is issue: LANES known to the compiler turns addresses
// into immediates, and WHOLE (dr, dh, y and post are there, and no gate row per
// row: what a step has in the middle of the model) spares the loop its tests.
template <typename T, bool VEC, int VPT, int LANES, bool WHOLE>
__global__ void __launch_bounds__(LANES == 512 ? 512 : kThreads, 1)
    backward_kernel(const __grid_constant__ BackwardArgs a, const __grid_constant__ Rows in) {
    extern __shared__ __align__(128) char smem[];
    if (a.release) mma::grid_launch_dependents();
    constexpr int lanes = LANES;
    const int id = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = blockDim.x / lanes;
    const bool has_dr = WHOLE || a.dr, has_dh = WHOLE || a.dh, has_y = WHOLE || a.y, has_post = WHOLE || a.post.p, each = !WHOLE && a.each;
    Ring<VEC> ring(in, smem, group);
    ring.start(id);
    mma::grid_wait();
    Walk ahead(a, group);
    bool more = id == 0 && ahead.any(a, group);
    auto request = [&]() {
        if (!more) return;
        ring.request(in.seg, ahead.row);
        ahead.row += groups;
        more = ahead.any(a, group);
    };
    for (int k = 0; k < in.stages; ++k) request();

    float* weights = reinterpret_cast<float*>(smem + kBarrierBytes + groups * in.stages * in.slot_bytes);
    constexpr bool kStaged = VPT <= 2;  // the weights of wider rows would take the room of their slots
    const int width = kStaged ? staged_floats(lanes, VPT) : 0;
    const Staged<VEC, VPT> post = {weights, lanes}, pre = {weights + width, lanes};  // post: with the unit's gate
    float* buf = weights + 2 * width;
    RowSum sum(lanes, group);
    const float share = share_of(lanes), inv_d = mean_of(lanes, a.d);
    const F8 zero = splat(0.0f), scale = splat(a.scale);
    F8 dpre[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) dpre[v] = zero;
    const bool early = VPT <= 2 && !each;  // nothing is read from a slot after the first sum over the row
    bool begun = false;
    const int64_t units = a.sections * a.parts;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t section = unit / a.parts, part = unit - section * a.parts;
        const int64_t row0 = section * a.per + a.per * part / a.parts, row1 = section * a.per + a.per * (part + 1) / a.parts;
        auto pre8 = [&](int v) { return kStaged ? pre.get(v, id) : a.pre.load<VEC>(0, first<VEC>(v, id, lanes), lanes, a.d); };
        auto post8 = [&](int v) {
            if (kStaged) return post.get(v, id);
            const int c0 = first<VEC>(v, id, lanes);
            F8 w = a.post.p ? a.post.load<VEC>(0, c0, lanes, a.d) : splat(1.0f);
            if (a.gate.p && !each) w = w * a.gate.load<VEC>(section, c0, lanes, a.d);
            return w;
        };
        if (kStaged && (unit == blockIdx.x || a.sections > 1)) {
            const bool begin = unit == blockIdx.x;
            if (!begin) __syncthreads();
            fill<VEC, VPT>(lanes, a.d, [&](int c, bool in_row, int at) {
                const float w = has_dh && begin && in_row ? a.pre.at(0, c) : 0.0f, p = has_y && in_row ? a.post.at(0, c) : 0.0f,
                            q = has_y && in_row && !each ? a.gate.at(section, c) : 1.0f;
                if (has_dh && begin) pre.at[at] = w;
                if (has_y) post.at[at] = p * q;
            });
            __syncthreads();
        }
        F8 dyn[VPT];  // sums of g n_y (times the gate where every row has its own)
#pragma unroll
        for (int v = 0; v < VPT; ++v) dyn[v] = zero;
        for (int64_t row = row0 + group; row < row1; row += groups) {
            const char* slot = ring.take();
            const T* in_r = ring.in(slot, in.seg[0], static_cast<const T*>(a.r) + row * a.ldr);
            const T* in_dr = ring.in(slot, in.seg[1], static_cast<const T*>(a.dr) + row * a.lddr);
            const __nv_bfloat16* in_dh = ring.in(slot, in.seg[2], a.dh + row * a.lddh);
            const __nv_bfloat16* in_y = ring.in(slot, in.seg[3], a.y + row * a.ldy);
            Cols<T, VEC> r;
            Cols<__nv_bfloat16, VEC> dh, y;
            // rows of up to two vectors a thread stay in registers, longer ones are read again
            constexpr int kHeld = VPT <= 2 ? VPT : 1;
            F8 r8[kHeld], dh8[kHeld], y8[kHeld];
            Cols<T, VEC> dr[kHeld];
            auto fetch = [&](int h, int c0) {
                if (has_dr) dr[h].load(in_dr, c0, lanes, a.d);
                if (has_dh) {
                    r.load(in_r, c0, lanes, a.d);
                    dh.load(in_dh, c0, lanes, a.d);
                    r8[h] = widen(r);
                    dh8[h] = widen(dh);
                }
                if (has_y) {
                    y.load(in_y, c0, lanes, a.d);
                    y8[h] = widen(y);
                }
            };
            float2 rr = {}, vr = {}, yy = {};  // r^2, v r, y^2
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int h = v % kHeld;
                fetch(h, first<VEC>(v, id, lanes));
                if (has_dh) {
                    rr = dot8(r8[h], r8[h], rr);
                    vr = dot8(dh8[h] * pre8(v), r8[h], vr);
                }
                if (has_post) yy = dot8(y8[h], y8[h], yy);
            }
            float s[3] = {(rr.x + rr.y) * share, (vr.x + vr.y) * share, (yy.x + yy.y) * share};
            if (has_dh || has_post) sum(s);
            {
                if (lanes == 32 || !(has_dh || has_post)) group_sync(group, lanes);
                // the row is in registers: its slot takes another; or everyone has left the row before
                if (early || (begun && in.stages > 1)) request();
                begun = true;
            }
            const float ir = rsqrtf(fmaf(s[0], inv_d, a.eps)), iy = has_post ? rsqrtf(fmaf(s[2], inv_d, a.eps)) : 1.0f;
            const F8 ir8 = splat(ir), iy8 = splat(iy), mean_r = splat(-(s[1] * inv_d * ir));  // minus the mean of v n_r
            float2 wn = {};                                                                    // w n_y
            F8 g[VPT];
            T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes), h = v % kHeld;
                if (VPT > kHeld) fetch(h, c0);
                g[v] = zero;
                if (has_dr) g[v] = widen(dr[h]);
                if (has_dh) {
                    const F8 n = r8[h] * ir8;
                    g[v] = fma8(ir8, fma8(n, mean_r, dh8[h] * pre8(v)), g[v]);
                    dpre[v] = fma8(dh8[h], n, dpre[v]);
                }
                // a gate row that is read in place, before outputs that may lie over it are written
                F8 gate;
                const bool in_place = VPT > 2 && each && !in.seg[4].p;
                if (in_place) gate = a.gate.load<VEC>(row, c0, lanes, a.d);
                store_cols<VEC>(dx, c0, lanes, a.d, scale * g[v]);
                if (!has_y) continue;
                const F8 n = y8[h] * iy8, w8 = post8(v);
                if (each) {
                    if (a.dgate.p) a.dgate.put8<VEC>(row, c0, lanes, a.d, g[v] * n * w8);
                    if (!in_place) {
                        const char* p = in.seg[4].p + row * in.seg[4].pitch;
                        const Weight w = {slot + in.seg[4].at + (VEC ? 0 : reinterpret_cast<uintptr_t>(p) % 16), a.gate.f32, 0};
                        gate = w.load<VEC>(0, c0, lanes, a.d);
                    }
                    g[v] = g[v] * gate;
                }
                dyn[v] = fma8(g[v], n, dyn[v]);
                g[v] = g[v] * w8;
                wn = dot8(g[v], n, wn);
                if (VPT == kHeld) y8[h] = n;
            }
            if (!early && in.stages == 1 && !has_post) {  // nothing more is read
                group_sync(group, lanes);
                request();
            }
            if (!has_y) continue;
            __nv_bfloat16* dy = a.dy + row * a.lddy;
            float q[1] = {(wn.x + wn.y) * share};
            if (has_post) sum(q);
            const F8 mean_y = splat(has_post ? -(q[0] * inv_d) : 0.0f);  // minus the mean of w n_y
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c0 = first<VEC>(v, id, lanes);
                if (VPT > kHeld) {
                    y.load(in_y, c0, lanes, a.d);
                    y8[0] = widen(y) * iy8;
                }
                if (has_post) g[v] = iy8 * fma8(y8[v % kHeld], mean_y, g[v]);
                store_cols<VEC>(dy, c0, lanes, a.d, g[v]);
            }
            if (!early && in.stages == 1 && has_post) {
                group_sync(group, lanes);
                request();
            }
        }
        if (a.dpost.p || (a.dgate.p && !a.each))
            combine<VEC>(dyn, id, group, groups, lanes, a.d, buf, [&](int c, float v) {
                if (a.dgate.p && !a.each) {
                    const float x = v * a.post.at(0, c);
                    if (a.parts == 1)
                        a.dgate.put(section, c, x);
                    else
                        a.partial[(2 * (int64_t)gridDim.x + unit) * a.d + c] = x;
                }
                if (a.dpost.p) {
                    const float x = a.each ? v : v * a.gate.at(section, c);
                    float* p = a.partial + (int64_t)blockIdx.x * a.d + c;
                    if (units == 1)
                        a.dpost.put(0, c, x);
                    else
                        *p = unit == blockIdx.x ? x : *p + x;
                }
            });
    }
    if (a.dpre.p)
        combine<VEC>(dpre, id, group, groups, lanes, a.d, buf, [&](int c, float v) {
            if (gridDim.x == 1)
                a.dpre.put(0, c, v);
            else
                a.partial[((int64_t)gridDim.x + blockIdx.x) * a.d + c] = v;
        });
}

struct Grid {
    RowShape q;
    int64_t sections, per, blocks;
    int32_t parts, groups;
};

// Floats of the weights and of combine().
inline int staged_space(int lanes, int vecs, int groups) { return vecs <= 2 ? staged_floats(lanes, vecs) * (2 + (groups > 1 ? groups : 0)) : 0; }

template <typename T, bool VEC, int VPT, int LANES, bool WHOLE>
cudaError_t launch_kernel(const BackwardArgs& a, const Rows& in, const Grid& g, int groups, cudaStream_t s) {
    static bool done[64];
    const cudaError_t e = ensure_smem_attr(backward_kernel<T, VEC, VPT, LANES, WHOLE>, kRoom, done);
    if (e != cudaSuccess) return e;
    const size_t smem = kBarrierBytes + (size_t)groups * in.stages * in.slot_bytes + 4 * (int)staged_space(g.q.lanes, VPT, groups);
    return launch(backward_kernel<T, VEC, VPT, LANES, WHOLE>, dim3((unsigned)g.blocks), groups * g.q.lanes, smem, s, a, in);
}

// Each form has units of its own: aligned rows, and rows of any alignment.
template <typename T, bool VEC, bool WHOLE>
cudaError_t launch_rows(const BackwardArgs& a, const Rows& in, const Grid& g, int groups, cudaStream_t s) {
    if constexpr (!VEC) {  // one vector a thread as far as 512 threads reach
        if (g.q.vecs == 1 && g.q.lanes == 64) return launch_kernel<T, VEC, 1, 64, WHOLE>(a, in, g, groups, s);
        if (g.q.vecs == 1 && g.q.lanes == 128) return launch_kernel<T, VEC, 1, 128, WHOLE>(a, in, g, groups, s);
        if (g.q.vecs == 1 && g.q.lanes == 256) return launch_kernel<T, VEC, 1, 256, WHOLE>(a, in, g, groups, s);
        if (g.q.vecs == 1 && g.q.lanes == 512) return launch_kernel<T, VEC, 1, 512, WHOLE>(a, in, g, groups, s);
        if (g.q.vecs == 2) return launch_kernel<T, VEC, 2, 512, WHOLE>(a, in, g, groups, s);
        if (g.q.vecs == 4) return launch_kernel<T, VEC, 4, 512, WHOLE>(a, in, g, groups, s);
        return launch_kernel<T, VEC, 1, 32, WHOLE>(a, in, g, groups, s);
    } else {
        if (g.q.vecs == 1) return launch_kernel<T, VEC, 1, 32, WHOLE>(a, in, g, groups, s);
        if (g.q.vecs == 4) return launch_kernel<T, VEC, 4, 512, WHOLE>(a, in, g, groups, s);
        if (g.q.lanes == 32) return launch_kernel<T, VEC, 2, 32, WHOLE>(a, in, g, groups, s);
        if (g.q.lanes == 64) return launch_kernel<T, VEC, 2, 64, WHOLE>(a, in, g, groups, s);
        if (g.q.lanes == 128) return launch_kernel<T, VEC, 2, 128, WHOLE>(a, in, g, groups, s);
        if (g.q.lanes == 256) return launch_kernel<T, VEC, 2, 256, WHOLE>(a, in, g, groups, s);
        return launch_kernel<T, VEC, 2, 512, WHOLE>(a, in, g, groups, s);
    }
}

#define DPRED_NORM_GRAD_FORM(T, VEC, WHOLE) \
    template cudaError_t launch_rows<T, VEC, WHOLE>(const BackwardArgs&, const Rows&, const Grid&, int, cudaStream_t)
extern DPRED_NORM_GRAD_FORM(__nv_bfloat16, true, true);
extern DPRED_NORM_GRAD_FORM(__nv_bfloat16, true, false);
extern DPRED_NORM_GRAD_FORM(__nv_bfloat16, false, false);
extern DPRED_NORM_GRAD_FORM(float, true, true);
extern DPRED_NORM_GRAD_FORM(float, true, false);
extern DPRED_NORM_GRAD_FORM(float, false, false);

}  // namespace layers
}  // namespace dpred
