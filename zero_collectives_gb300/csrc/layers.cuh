// layers.cuh -- what the bandwidth-bound operators of a training step share:
// element access in groups of 8, argument checks and launches.
#pragma once

#include <cmath>
#include <exception>

#include "common.cuh"
#include "mma.cuh"

namespace dpred {
namespace layers {

#ifdef __CUDACC__

// One element of either type.
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Eight consecutive elements, 16-byte aligned, as they lie in registers:
// loads are issued first and widened when they are used.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ float operator[](int c) const {
        const uint32_t w = c < 2 ? q.x : c < 4 ? q.y : c < 6 ? q.z : q.w;
        return c & 1 ? bf16_hi(w) : bf16_lo(w);
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ float operator[](int c) const {
        const float4& v = c < 4 ? a : b;
        return (c & 3) == 0 ? v.x : (c & 3) == 1 ? v.y : (c & 3) == 2 ? v.z : v.w;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// What a thread has of a row: 8 columns next to each other, c0 to c0 + 7
// (VEC: 16-byte aligned rows whose width is a multiple of 8), or every step-th
// from c0 on, so that scalar accesses of neighbouring threads meet in a line.
// Columns from d on read as 0 and are not written.
template <bool VEC>
__device__ __forceinline__ int column(int c0, int step, int k) {
    return VEC ? c0 + k : c0 + step * k;
}

template <typename T, bool VEC>
struct Cols;
template <typename T>
struct Cols<T, true> {
    Eight<T> q;
    __device__ __forceinline__ void load(const T* p, int c0, int, int d) {
        if (c0 < d)
            q.load(p + c0);
        else
            q = {};
    }
    __device__ __forceinline__ float operator[](int k) const { return q[k]; }
};
template <typename T>
struct Cols<T, false> {
    float f[8];
    __device__ __forceinline__ void load(const T* p, int c0, int step, int d) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = c0 + step * k < d ? load1(p + c0 + step * k) : 0.0f;
    }
    __device__ __forceinline__ float operator[](int k) const { return f[k]; }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_cols(T* p, int c0, int step, int d, const float (&f)[8]) {
    if constexpr (VEC) {
        if (c0 < d) store8(p + c0, f);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c0 + step * k < d) store1(p + c0 + step * k, f[k]);
    }
}

// Eight values in fp32, as four pairs: one instruction works on a pair (each half
// rounded as by itself), which is what keeps the norms from being bound by issue.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}

struct F8 {
    float2 p[4];
    __device__ __forceinline__ float get(int k) const { return k & 1 ? p[k / 2].y : p[k / 2].x; }
};
__device__ __forceinline__ F8 splat(float v) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = make_float2(v, v);
    return f;
}
__device__ __forceinline__ F8 operator*(const F8& a, const F8& b) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = mul2(a.p[i], b.p[i]);
    return f;
}
__device__ __forceinline__ F8 fma8(const F8& a, const F8& b, const F8& c) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = fma2(a.p[i], b.p[i], c.p[i]);
    return f;
}
// s + a . b, by halves.
__device__ __forceinline__ float2 dot8(const F8& a, const F8& b, float2 s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(a.p[i], b.p[i], s);
    return s;
}
template <typename C>
__device__ __forceinline__ F8 widen(const C& c) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = make_float2(c[2 * i], c[2 * i + 1]);
    return f;
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_cols(T* p, int c0, int step, int d, const F8& f) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f.get(k);
    store_cols<VEC>(p, c0, step, d, v);
}

#endif  // __CUDACC__

// -------------------------------------------------------------------- host --

inline int esize(int dtype) { return dtype == DPRED_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == DPRED_BF16 || dtype == DPRED_F32; }

inline int check_dtype(int dtype, const char* name) {
    return dtype_ok(dtype) ? DPRED_OK : set_error(DPRED_E_INVAL, "unknown type %d of %s", dtype, name);
}

inline int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int es, const char* name) {
    if (rows == 0 || cols == 0) return DPRED_OK;
    if (!p) return set_error(DPRED_E_INVAL, "%s is null", name);
    if (reinterpret_cast<uintptr_t>(p) % es) return set_error(DPRED_E_ALIGN, "%s is not aligned to its element size", name);
    if (rows > 1 && ld < cols)
        return set_error(DPRED_E_SIZE, "%s: row stride %lld is less than its %lld columns", name, (long long)ld, (long long)cols);
    return DPRED_OK;
}

inline int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need > bytes || (need && !workspace)) return set_error(DPRED_E_SIZE, "workspace of %zu bytes, %zu needed", bytes, need);
    if (need && reinterpret_cast<uintptr_t>(workspace) % 256) return set_error(DPRED_E_ALIGN, "workspace is not 256-byte aligned");
    return DPRED_OK;
}

// Rows whose groups of 8 elements are 16-byte aligned.
inline bool aligned_rows(const void* p, int64_t rows, int64_t ld, int es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * es % 16 == 0);
}

// Launches overlap the end of the one before: every kernel waits for it
// (grid_wait) before it touches memory, and only one that another of the same
// call follows lets the next one start early.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename F>
int guarded(F f) {  // no C++ exception leaves a C entry point
    try {
        return f();
    } catch (const std::exception& e) {
        return set_error(DPRED_E_INVAL, "host failure: %s", e.what());
    }
}

}  // namespace layers
}  // namespace dpred
