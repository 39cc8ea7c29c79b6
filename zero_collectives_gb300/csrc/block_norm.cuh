// block_norm.cuh -- what the block norm and its gradient share: how threads
// cover rows, sums over a row, weights, argument checks.
#pragma once

#include <algorithm>

#include "layers.cuh"

namespace dpred {
namespace layers {

constexpr int kMaxWidth = 16384;

// `lanes` threads (a power of two, whole warps) hold a row, 8 * vecs columns each.
struct RowShape {
    int lanes, vecs, threads;
};
inline RowShape shape_of(int64_t d) {
    RowShape q;
    q.lanes = 32;
    while (q.lanes < 512 && q.lanes * 8 < d) q.lanes *= 2;
    q.vecs = d <= 4096 ? 1 : d <= 8192 ? 2 : 4;
    q.threads = std::max(q.lanes, 256);
    return q;
}

#ifdef __CUDACC__

// A thread's first column of its v-th group of 8.
template <bool VEC>
__device__ __forceinline__ int first(int v, int id, int lanes) {
    return v * 8 * lanes + (VEC ? 8 * id : id);
}

// Sums over the threads of a row, the same in all of them.  A row of several
// warps has a barrier of its own; one per sum is enough, since sums in turn use
// two places: whoever writes to one again has passed the barrier in between,
// and so has everyone who read it.
struct RowSum {
    int lanes, group, turn = 0;
    __device__ __forceinline__ RowSum(int lanes, int group) : lanes(lanes), group(group) {}

    template <int N>
    __device__ __forceinline__ void operator()(float (&s)[N]) {
        __shared__ float warps[2][16][4];
        static_assert(N <= 4, "sums at once");
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int o = 16; o; o >>= 1) s[n] += __shfl_xor_sync(0xFFFFFFFFu, s[n], o);
        if (lanes == 32) return;
        const int warp = threadIdx.x / 32, first_warp = group * (lanes / 32);
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) warps[turn][warp][n] = s[n];
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
#pragma unroll
        for (int n = 0; n < N; ++n) s[n] = 0.0f;
        for (int w = 0; w < lanes / 32; ++w)
#pragma unroll
            for (int n = 0; n < N; ++n) s[n] += warps[turn][first_warp + w][n];
        turn ^= 1;
    }
};

#endif  // __CUDACC__

// A weight vector, or gate rows, of either type; p is null where there is none.
struct Weight {
    const void* p;
    int32_t f32;
    int64_t ld;
#ifdef __CUDACC__
    template <bool VEC>
    __device__ __forceinline__ void load(int64_t row, int c0, int step, int d, float (&f)[8]) const {
        if (f32) {
            Cols<float, VEC> q;
            q.load(static_cast<const float*>(p) + row * ld, c0, step, d);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = q[k];
        } else {
            Cols<__nv_bfloat16, VEC> q;
            q.load(static_cast<const __nv_bfloat16*>(p) + row * ld, c0, step, d);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = q[k];
        }
    }
#endif
};

// The arguments that both directions have.
struct NormShape {
    int64_t m, d;
    int32_t r_dtype;
    const void* y;
    int32_t post_dtype;
    const void* post;
    int32_t gate_dtype;
    const void* gate;
    int64_t gate_rows;
    float scale;
    int32_t pre_dtype;
    const void* pre;
    float eps;
};

inline int check_norm(const NormShape& n) {
    int rc;
    if (n.m < 0 || n.d < 0) return set_error(DPRED_E_INVAL, "a negative size (%lld x %lld)", (long long)n.m, (long long)n.d);
    if (n.m > 0x7FFFFFFF || n.d > kMaxWidth)
        return set_error(DPRED_E_SIZE, "%lld rows of %lld: at most 2^31 - 1 of %d", (long long)n.m, (long long)n.d, kMaxWidth);
    if ((rc = check_dtype(n.r_dtype, "the residual stream")) != DPRED_OK) return rc;
    if (!(n.eps >= 0.0f) || !std::isfinite(n.eps)) return set_error(DPRED_E_INVAL, "eps must be finite and not negative");
    if (!std::isfinite(n.scale)) return set_error(DPRED_E_INVAL, "scale is not finite");
    const bool some = n.m > 0 && n.d > 0;  // empty matrices have no address
    if (some && !n.y && !n.pre) return set_error(DPRED_E_INVAL, "neither y nor pre: nothing to do");
    if (some && !n.y && (n.post || n.gate)) return set_error(DPRED_E_INVAL, "post and gate need y");
    if (some && !n.y && n.scale != 1.0f) return set_error(DPRED_E_INVAL, "without y, r is x: scale must be 1");
    const struct { const void* p; int32_t dt; const char* name; } w[] = {{n.post, n.post_dtype, "post"}, {n.gate, n.gate_dtype, "gate"}, {n.pre, n.pre_dtype, "pre"}};
    for (const auto& x : w) {
        if (!x.p) continue;
        if ((rc = check_dtype(x.dt, x.name)) != DPRED_OK) return rc;
        if (reinterpret_cast<uintptr_t>(x.p) % esize(x.dt)) return set_error(DPRED_E_ALIGN, "%s is not aligned to its element size", x.name);
    }
    if (n.gate && n.m > 0 && (n.gate_rows < 1 || n.m % n.gate_rows))
        return set_error(DPRED_E_SIZE, "%lld rows cannot be shared evenly by %lld gate rows", (long long)n.m, (long long)n.gate_rows);
    return DPRED_OK;
}

// Rows whose groups of 8 columns can be loaded at once.
inline bool weights_aligned(const NormShape& n) {
    for (const void* p : {n.post, n.gate, n.pre})
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    return n.d % 8 == 0;
}

}  // namespace layers
}  // namespace dpred
