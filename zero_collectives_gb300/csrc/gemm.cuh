// gemm.cuh -- the matrix products behind the linear-layer and Newton-Schulz
// entry points: D[i][j] = epilogue(sum_k A[i][k] B[j][k]), 16-bit operands,
// fp32 accumulators in tensor memory (tcgen05), epilogue in registers.
//
// The side called A (rows i) always lies on the 128 tensor-memory lanes, so an
// epilogue thread owns one row and a run of columns.  Either operand may be
// K-major or MN-major in memory; D may be written along either index (the
// caller puts the few tokens of a short call on the column side and the many
// features on the lanes, and the output's strides say so).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "mma.cuh"

namespace dpred {
namespace gemm {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

// What the epilogue computes from an accumulator t = D[i][j].
enum Kind : int {
    KIND_LINEAR = 0,  // linear layers: bias, activation or its gradient, residual, accumulation
    KIND_GRAM = 1,    // Newton-Schulz: off-diagonal of X X^T in fp16, its diagonal in fp32
    KIND_POLY = 2,    // Newton-Schulz: off-diagonal of b A + c A^2 in fp16, a + its diagonal in fp32
    KIND_APPLY = 3,   // Newton-Schulz: the next X, as two terms
    KIND_FINAL = 4,   // Newton-Schulz: the last X, stored or applied to a weight
    // The tile kernel's linear layers, by what their epilogue can contain (its
    // code then holds nothing else; chosen by linear_kind()):
    KIND_PLAIN = 5,   // bf16 result, bias and residual at most
    KIND_ACT = 6,     // bf16 result, forward activation and stored pre-activation
    KIND_GRAD = 7,    // bf16 result, activation's gradient
    KIND_F32 = 8,     // fp32 result: everything
    KIND_MUL = 9,     // Newton-Schulz: product of two polynomials of one A, split as A is
};
__host__ __device__ constexpr bool is_linear(int kind) { return kind == KIND_LINEAR || (kind >= KIND_PLAIN && kind <= KIND_F32); }

// A linear layer's epilogue.  In order: t += bias; pre_out = t; t = act(t);
// t += residual; t *= act'(z); t += what the output holds; out = t.  All
// matrices are row-major with unit column stride.
struct LinearEpi {
    void* out;
    const void* bias;
    const __nv_bfloat16* res;
    __nv_bfloat16* pre_out;
    const __nv_bfloat16* z;
    int64_t o_ld, r_ld, p_ld, z_ld;
    int out_f32, bias_f32, act, accumulate;
    int swapped;  // the product computes the output's transpose: its rows (i) are the output's columns
    int vec;      // every matrix present has 16-byte aligned rows, the bias too
};

// The same for the tile kernel, with the maps of the matrices that its
// streaming epilogue moves (boxes of 32 rows x 128 bytes): the output, the
// stored pre-activation, and the residual or the pre-activation that is read.
struct TileParams {
    LinearEpi e;
    int stream;
    int direct;        // KIND_PLAIN, stream: whole chunks of the output leave by 32-byte stores from the registers
    float* row_sum;    // sums of A's rows over the reduction (a bias gradient), null: not wanted
    int row_sum_add;   // added to what is there
    CUtensorMap out, pre, in;
};
// The kinds a weight gradient takes, whose tile kernels can sum A's rows as well.
__host__ __device__ constexpr bool sums_rows(int kind) { return kind == KIND_LINEAR || kind == KIND_PLAIN || kind == KIND_F32; }

// One matrix of a Newton-Schulz batch as its last product writes it.
struct FinalOut {
    void* p;
    int64_t ld;
    float step;       // multiplies the orthogonalised value (negative: subtracted from the weight)
    int vec;          // 16-byte aligned rows
    int transposed;   // stored with rows and columns exchanged
};
constexpr int kMaxBatch = 64;  // matrices per Newton-Schulz launch (their output table travels in the launch)

struct NsEpi {
    __half* gram;      // [batch, r, ldr] off-diagonal of A (in for POLY, out for GRAM) or of a product (MUL, out)
    __half* poly;      // [batch, r, ldr] off-diagonal of the polynomial (out for POLY)
    float* gram_diag;  // [batch, ldr]
    float* coef;       // [batch, ldr] diagonal of a + b A + c A^2 (out for POLY, in for APPLY, FINAL)
    const __half *m1, *m2;  // MUL: the factors' off-diagonals
    const float *d1, *d2;   // and their diagonals
    const __half* hi_in;  // [batch, r, ldc] X's leading term, the products' operand
    __half* hi;           // the next X's
    uint8_t* lo;          // [batch, r, ldc] X's trailing term, updated in place (every element by the thread that reads it)
    int64_t ldr, ldc;
    float alpha;       // GRAM: multiplies the accumulator
    float a, b, c;     // the polynomial's coefficients
    float keep;        // FINAL: factor of the old weight (0: store)
    int out_f32;       // FINAL
    const FinalOut* out;  // FINAL: one entry per matrix of the batch
};

// The same as it travels in a launch, with its table.
struct NsParams {
    NsEpi e;
    FinalOut table[kMaxBatch];
};
__device__ __forceinline__ NsEpi epilogue_of(const NsParams& p) {
    NsEpi e = p.e;
    e.out = p.table;
    return e;
}
__device__ __forceinline__ const LinearEpi& epilogue_of(const LinearEpi& e) { return e; }

struct Args {
    int m, n;            // rows of A, rows of B
    int kblocks;         // reduction blocks of kBlockK
    int batch;
    int tiles_m, tiles_n, tiles_per_batch;
    int symmetric;       // only elements i <= j are needed (the epilogue mirrors them)
    int a_mn, b_mn;      // operand majors
    int split_only;    // split kernel only (a swapped epilogue, a Newton-Schulz product)
    int row_sums;      // the sums of A's rows are wanted too: the tile kernel forms them, else a launch of its own
    int split;           // CTAs of a cluster that share the reduction
    int stages;          // split kernel: pipeline stages
    int regions;         // split kernel: accumulators that share a CTA's part of the reduction
    int bf16;
    int release;         // a later launch of the same call follows (see grid_launch_dependents)
    int* err;
};

template <int KIND>
struct EpiOf {
    using T = std::conditional_t<is_linear(KIND), LinearEpi, NsEpi>;      // as the epilogue sees it
    using Param = std::conditional_t<is_linear(KIND), LinearEpi, NsParams>;  // as the launch carries it
};

// The tile kernel's kind for a linear layer's options.
inline int linear_kind(const LinearEpi& e) {
    if (e.out_f32) return KIND_F32;
    if (e.accumulate || (e.z && e.pre_out)) return KIND_LINEAR;
    if (e.z) return KIND_GRAD;
    return e.act || e.pre_out ? KIND_ACT : KIND_PLAIN;
}

// Factor that brings U to X = scale U / (|U| + eps), from the sum of U's squares.
// A zero matrix stays zero with eps = 0 too; a NaN in the sum stays one.
__device__ __forceinline__ float norm_factor(float scale, float squares, float eps) {
    return squares == 0.0f ? 0.0f : scale / (sqrtf(squares) + eps);
}

// ------------------------------------------------------------- activations --

// The logistic function of -x / log2(e), 1 / (1 + 2^x), from the hardware's
// approximate exponential and reciprocal (about 2^-22 relative each, far below
// the bf16 rounding of what is stored).
__device__ __forceinline__ float logistic2(float x) {
    float t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// gelu is the tanh form: 0.5 z (1 + tanh(u)) = z * logistic(2 u), u = sqrt(2/pi) (z + 0.044715 z^3).
constexpr float kGeluQ = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

// A NaN stays one, in the activations and their gradients.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == ACT_RELU) return z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == ACT_GELU) return z * logistic2(z * fmaf(-kLog2e * kGeluQ * kGeluC, z * z, -kLog2e * kGeluQ));
    if constexpr (ACT == ACT_SILU) return z * logistic2(-kLog2e * z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == ACT_GELU) {
        // beyond |z| = 1000 the logistic is 0 or 1 exactly; the clamp keeps z^2 finite there
        const float z2 = fminf(z * z, 1e6f);
        const float p = logistic2(z * fmaf(-kLog2e * kGeluQ * kGeluC, z2, -kLog2e * kGeluQ));
        return fmaf(z * p * (1.0f - p), fmaf(3.0f * kGeluC * kGeluQ, z2, kGeluQ), p);
    }
    if constexpr (ACT == ACT_SILU) {
        const float p = logistic2(-kLog2e * z);
        return fmaf(z * p, 1.0f - p, p);
    }
    return 1.0f;
}

__device__ __forceinline__ float activate(float z, int act) {
    return act == ACT_RELU ? activate<ACT_RELU>(z) : act == ACT_GELU ? activate<ACT_GELU>(z) : act == ACT_SILU ? activate<ACT_SILU>(z) : z;
}

__device__ __forceinline__ float activate_grad(float z, int act) {
    return act == ACT_RELU ? activate_grad<ACT_RELU>(z) : act == ACT_GELU ? activate_grad<ACT_GELU>(z) : act == ACT_SILU ? activate_grad<ACT_SILU>(z) : 1.0f;
}

// ---------------------------------------------------------------- epilogue --

__device__ __forceinline__ float load_bf16(const __nv_bfloat16* p) { return bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p)); }

__device__ __forceinline__ void load8_bf16(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    f[0] = bf16_lo(q.x); f[1] = bf16_hi(q.x); f[2] = bf16_lo(q.y); f[3] = bf16_hi(q.y);
    f[4] = bf16_lo(q.z); f[5] = bf16_hi(q.z); f[6] = bf16_lo(q.w); f[7] = bf16_hi(q.w);
}

// Element c of eight packed bf16 values.
__device__ __forceinline__ float bf16_of(const uint4& q, int c) {
    const uint32_t w = c < 2 ? q.x : c < 4 ? q.y : c < 6 ? q.z : q.w;
    return c & 1 ? bf16_hi(w) : bf16_lo(w);
}

__device__ __forceinline__ void half8(const uint4& q, float (&f)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        f[2 * k] = t.x;
        f[2 * k + 1] = t.y;
    }
}

__device__ __forceinline__ void store8_bf16(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                              pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void load8_f32(const float* p, float (&f)[8]) {
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w; f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
}

__device__ __forceinline__ void store8_f32(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

// X as two terms: the leading one in fp16 (what the matrix instructions read),
// the rest, times 2^12, in fp8 (e4m3).  Together about 15 significant bits in 3
// bytes: the products round X to 11 anyway, and the passes over X are bound by
// its bytes (with the rest in fp32, 6 matrices of 1024 x 4096 took 29% longer).
// What the rest's type costs, from an emulation of every rounding in 64 bits, five
// steps on 512 x 512: 1.5e-3 without it, 5.27e-4 with it in fp8, 5.23e-4 in fp16,
// 5.24e-4 in fp32 (512 x 2048 in double steps: 8.99e-4, 9.01e-4, 9.00e-4): the
// products' own operands, which are fp16 in all of them, decide the error.
constexpr float kLoScale = 4096.0f;

__device__ __forceinline__ void split8(const float (&t)[8], uint4& hi, uint2& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 p = __floats2half2_rn(t[2 * k], t[2 * k + 1]);
        const float2 f = __half22float2(p);
        h[k] = *reinterpret_cast<const uint32_t*>(&p);
        l[k] = __nv_cvt_float2_to_fp8x2(make_float2((t[2 * k] - f.x) * kLoScale, (t[2 * k + 1] - f.y) * kLoScale), __NV_SATFINITE,
                                        __NV_E4M3);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

__device__ __forceinline__ void join8(const uint4& hi, const uint2& lo, float (&x)[8]) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x & 0xFFFF, lo.x >> 16, lo.y & 0xFFFF, lo.y >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)l[k], __NV_E4M3);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[k])), q = __half22float2(__half2(r));
        x[2 * k] = fmaf(q.x, 1.0f / kLoScale, p.x);
        x[2 * k + 1] = fmaf(q.y, 1.0f / kLoScale, p.y);
    }
}

__device__ __forceinline__ void store8_half(__half* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

// Eight consecutive columns of one output row of a linear layer, one by one
// (`cols` columns; those past it are skipped): rows without 16-byte alignment
// and blocks on the right edge.
__device__ __forceinline__ void linear_row(const LinearEpi& e, int cols, int64_t row, int j0, float (&t)[8]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int j = j0 + c;
        if (j >= cols) break;
        float x = t[c];
        if (e.bias)
            x += e.bias_f32 ? static_cast<const float*>(e.bias)[j] : load_bf16(static_cast<const __nv_bfloat16*>(e.bias) + j);
        if (e.pre_out) e.pre_out[row * e.p_ld + j] = __float2bfloat16_rn(x);
        if (!e.z) x = activate(x, e.act);
        if (e.res) x += load_bf16(e.res + row * e.r_ld + j);
        if (e.z) x *= activate_grad(load_bf16(e.z + row * e.z_ld + j), e.act);
        if (e.out_f32) {
            float* o = static_cast<float*>(e.out) + row * e.o_ld + j;
            *o = e.accumulate ? *o + x : x;
        } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + row * e.o_ld + j;
            *o = __float2bfloat16_rn(e.accumulate ? load_bf16(o) + x : x);
        }
    }
}

// N rows (row + 8 s) of eight consecutive columns, all inside the matrix's
// columns and 16-byte aligned; rows past the end are skipped.  One test of each
// option for the whole block: tested row by row they took four times as long
// as the arithmetic.
template <int KIND, int N>
__device__ __forceinline__ void linear_rows(const LinearEpi& e, int rows, int row, int j0, float (&t)[N][8]) {
    // what this kind can contain
    constexpr bool kAll = KIND == KIND_LINEAR || KIND == KIND_F32;
    const bool pre_out = (kAll || KIND == KIND_ACT) && e.pre_out, grad = (kAll && e.z) || KIND == KIND_GRAD;
    const bool f32 = KIND == KIND_F32 || (KIND == KIND_LINEAR && e.out_f32), accumulate = kAll && e.accumulate;
    const bool act = (kAll || KIND == KIND_ACT) && !grad;
    bool in[N];
#pragma unroll
    for (int s = 0; s < N; ++s) in[s] = row + 8 * s < rows;
    if (e.bias) {
        float b[8];
        if (e.bias_f32)
            load8_f32(static_cast<const float*>(e.bias) + j0, b);
        else
            load8_bf16(static_cast<const __nv_bfloat16*>(e.bias) + j0, b);
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int c = 0; c < 8; ++c) t[s][c] += b[c];
    }
    if (pre_out) {
#pragma unroll
        for (int s = 0; s < N; ++s)
            if (in[s]) store8_bf16(e.pre_out + (int64_t)(row + 8 * s) * e.p_ld + j0, t[s]);
    }
#define DPRED_EACH(expr)                                   \
    _Pragma("unroll") for (int s = 0; s < N; ++s)          \
        _Pragma("unroll") for (int c = 0; c < 8; ++c) expr
    uint4 q[N];
    if (grad) {
#pragma unroll
        for (int s = 0; s < N; ++s)
            q[s] = in[s] ? *reinterpret_cast<const uint4*>(e.z + (int64_t)(row + 8 * s) * e.z_ld + j0) : make_uint4(0, 0, 0, 0);
    } else if (act && e.act == ACT_GELU) {
        DPRED_EACH(t[s][c] = activate<ACT_GELU>(t[s][c]);)
    } else if (act && e.act == ACT_SILU) {
        DPRED_EACH(t[s][c] = activate<ACT_SILU>(t[s][c]);)
    } else if (act && e.act == ACT_RELU) {
        DPRED_EACH(t[s][c] = activate<ACT_RELU>(t[s][c]);)
    }
    if (e.res) {
        uint4 p[N];
#pragma unroll
        for (int s = 0; s < N; ++s)
            p[s] = in[s] ? *reinterpret_cast<const uint4*>(e.res + (int64_t)(row + 8 * s) * e.r_ld + j0) : make_uint4(0, 0, 0, 0);
        DPRED_EACH(t[s][c] += bf16_of(p[s], c);)
    }
    if (grad) {
        if (e.act == ACT_GELU) {
            DPRED_EACH(t[s][c] *= activate_grad<ACT_GELU>(bf16_of(q[s], c));)
        } else if (e.act == ACT_SILU) {
            DPRED_EACH(t[s][c] *= activate_grad<ACT_SILU>(bf16_of(q[s], c));)
        } else {
            DPRED_EACH(t[s][c] *= activate_grad<ACT_RELU>(bf16_of(q[s], c));)
        }
    }
    if (f32) {
        float* o = static_cast<float*>(e.out) + (int64_t)row * e.o_ld + j0;
        if (accumulate) {
            float4 u[N], v[N];
#pragma unroll
            for (int s = 0; s < N; ++s)
                if (in[s]) {
                    u[s] = *reinterpret_cast<const float4*>(o + 8 * s * e.o_ld);
                    v[s] = *reinterpret_cast<const float4*>(o + 8 * s * e.o_ld + 4);
                }
#pragma unroll
            for (int s = 0; s < N; ++s) {
                t[s][0] += u[s].x; t[s][1] += u[s].y; t[s][2] += u[s].z; t[s][3] += u[s].w;
                t[s][4] += v[s].x; t[s][5] += v[s].y; t[s][6] += v[s].z; t[s][7] += v[s].w;
            }
        }
#pragma unroll
        for (int s = 0; s < N; ++s)
            if (in[s]) store8_f32(o + 8 * s * e.o_ld, t[s]);
    } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + (int64_t)row * e.o_ld + j0;
        if (accumulate) {
            uint4 p[N];
#pragma unroll
            for (int s = 0; s < N; ++s)
                p[s] = in[s] ? *reinterpret_cast<const uint4*>(o + 8 * s * e.o_ld) : make_uint4(0, 0, 0, 0);
            DPRED_EACH(t[s][c] += bf16_of(p[s], c);)
        }
#pragma unroll
        for (int s = 0; s < N; ++s)
            if (in[s]) store8_bf16(o + 8 * s * e.o_ld, t[s]);
    }
}

// A Newton-Schulz result: N rows (row + 8 s) of eight consecutive columns.
template <int N>
__device__ __forceinline__ void final_rows(const NsEpi& e, const FinalOut& f, int rows, int cols, int row, int j0,
                                           const float (&t)[N][8]) {
    if (f.vec && j0 + 8 <= cols) {
        if (e.out_f32) {
            float* p = static_cast<float*>(f.p) + (int64_t)row * f.ld + j0;
#pragma unroll
            for (int s0 = 0; s0 < N; s0 += 2) {
                float w[2][8] = {};
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (e.keep != 0.0f && row + 8 * (s0 + s) < rows) load8_f32(p + 8 * (s0 + s) * f.ld, w[s]);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) w[s][c] = fmaf(e.keep, w[s][c], t[s0 + s][c] * f.step);
                    if (row + 8 * (s0 + s) < rows) store8_f32(p + 8 * (s0 + s) * f.ld, w[s]);
                }
            }
        } else {
            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(f.p) + (int64_t)row * f.ld + j0;
            uint4 q[N];
#pragma unroll
            for (int s = 0; s < N; ++s)
                q[s] = e.keep != 0.0f && row + 8 * s < rows ? *reinterpret_cast<const uint4*>(p + 8 * s * f.ld)
                                                            : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int s = 0; s < N; ++s) {
                float x[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) x[c] = fmaf(e.keep, bf16_of(q[s], c), t[s][c] * f.step);
                if (row + 8 * s < rows) store8_bf16(p + 8 * s * f.ld, x);
            }
        }
        return;
    }
#pragma unroll
    for (int s = 0; s < N; ++s) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (row + 8 * s >= rows || j0 + c >= cols) continue;
            const int64_t o = (int64_t)(row + 8 * s) * f.ld + j0 + c;
            const float x = t[s][c] * f.step;
            if (e.out_f32) {
                float* p = static_cast<float*>(f.p) + o;
                *p = e.keep != 0.0f ? fmaf(e.keep, *p, x) : x;
            } else {
                __nv_bfloat16* p = static_cast<__nv_bfloat16*>(f.p) + o;
                *p = __float2bfloat16_rn(e.keep != 0.0f ? fmaf(e.keep, load_bf16(p), x) : x);
            }
        }
    }
}

// ------------------------------------------------------------ staged blocks --
//
// The tensor-memory load gives a thread one row; global memory wants a warp to
// touch few rows at a time (written straight from those registers, a bf16
// result of 256 columns a row took twice the time of its product).  So a warp
// passes its accumulators through a 32 x 32 fp32 block of shared memory, 16-byte
// pieces exchanged within a row by its number so that every access is free of
// bank conflicts, and reads it back eight columns of a row (or eight rows of a
// column, for a transposed result) at a time.
constexpr uint32_t kBlockBytes = 32 * 32 * 4;

__device__ __forceinline__ uint32_t piece(uint32_t block, int r, int c4) { return block + r * 128 + ((c4 ^ (r & 7)) << 4); }

__device__ __forceinline__ void sts4(uint32_t a, float x, float y, float z, float w) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

__device__ __forceinline__ void lds4(uint32_t a, float* v) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(a)
                 : "memory");
}

__device__ __forceinline__ float lds1(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Row `lane` of the block.
__device__ __forceinline__ void block_put_row(uint32_t block, int lane, const float (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) sts4(piece(block, lane, c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

// Columns 8 c8 .. 8 c8 + 7 of row r.
__device__ __forceinline__ void block_get(uint32_t block, int r, int c8, float (&t)[8]) {
    lds4(piece(block, r, 2 * c8), t);
    lds4(piece(block, r, 2 * c8 + 1), t + 4);
}

__device__ __forceinline__ void block_put(uint32_t block, int r, int c8, const float (&t)[8]) {
    sts4(piece(block, r, 2 * c8), t[0], t[1], t[2], t[3]);
    sts4(piece(block, r, 2 * c8 + 1), t[4], t[5], t[6], t[7]);
}

// Rows 8 r8 .. 8 r8 + 7 of column c.
__device__ __forceinline__ void block_get_column(uint32_t block, int r8, int c, float (&t)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = lds1(piece(block, 8 * r8 + k, c / 4) + (c % 4) * 4);
}

// One step (8 rows, or 8 columns of a transposed result) of a linear layer's
// block, or all four of them.
template <int KIND, int N>
__device__ __forceinline__ void linear_steps(const LinearEpi& e, const Args& g, int step, int lane, int i0, int j0,
                                             float (&t)[N][8]) {
    const bool swapped = KIND == KIND_LINEAR && e.swapped;  // only the split kernel's calls are
    const int rows = swapped ? g.n : g.m, cols = swapped ? g.m : g.n;
    const int row = (swapped ? j0 : i0) + step * 8 + lane / 4, c0 = swapped ? i0 : j0, c = c0 + lane % 4 * 8;
    if (e.vec && c0 + 32 <= cols) {
        linear_rows<KIND, N>(e, rows, row, c, t);
    } else {
#pragma unroll 1
        for (int s = 0; s < N; ++s) {
            float u[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) u[x] = t[0][x];
#pragma unroll
            for (int y = 1; y < N; ++y)
                if (s == y) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) u[x] = t[y][x];
                }
            if (row + 8 * s < rows && c < cols) linear_row(e, cols, row + 8 * s, c, u);
        }
    }
}

// What a Newton-Schulz block's epilogue reads from global memory, loaded ahead
// of the block's accumulators (their latency, about 1000 cycles, would otherwise
// come on top of every block), and past the first-level cache: in the chained
// kernel other SMs wrote it earlier in the same launch.
template <int KIND>
struct Ahead {};
template <>
struct Ahead<KIND_POLY> {
    uint4 q[4];
    float di[4], dj[8];
};
template <>
struct Ahead<KIND_MUL> {
    uint4 p[4], q[4];
    float di[4], dj[8];
};
template <>
struct Ahead<KIND_APPLY> {
    uint4 h[4];
    uint2 l[4];
    float k[4];
};
template <>
struct Ahead<KIND_FINAL> : Ahead<KIND_APPLY> {};

template <int KIND>
__device__ __forceinline__ void load_ahead(const typename EpiOf<KIND>::T& e, const Args& g, int batch, int i0, int j0,
                                           int lane, Ahead<KIND>& a) {
    const int i = i0 + lane / 4, j = j0 + lane % 4 * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (KIND == KIND_POLY) {
        const float* diag = e.gram_diag + (int64_t)batch * e.ldr;
        const __half* p = e.gram + ((int64_t)batch * g.m + i) * e.ldr + j;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = i + 8 * s < g.m && j < g.n;
            a.q[s] = in ? __ldcg(reinterpret_cast<const uint4*>(p + 8 * s * e.ldr)) : zero;
            a.di[s] = in ? __ldcg(diag + i + 8 * s) : 0.0f;
        }
        if (j < g.n) {  // rows and diagonals are padded to 8 elements
            const float4 x = __ldcg(reinterpret_cast<const float4*>(diag + j)), y = __ldcg(reinterpret_cast<const float4*>(diag + j + 4));
            a.dj[0] = x.x; a.dj[1] = x.y; a.dj[2] = x.z; a.dj[3] = x.w; a.dj[4] = y.x; a.dj[5] = y.y; a.dj[6] = y.z; a.dj[7] = y.w;
        }
    } else if constexpr (KIND == KIND_MUL) {
        const int64_t at = ((int64_t)batch * g.m + i) * e.ldr + j;
        const float* d1 = e.d1 + (int64_t)batch * e.ldr;
        const float* d2 = e.d2 + (int64_t)batch * e.ldr;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = i + 8 * s < g.m && j < g.n;
            a.p[s] = in ? __ldcg(reinterpret_cast<const uint4*>(e.m1 + at + 8 * s * e.ldr)) : zero;
            a.q[s] = in ? __ldcg(reinterpret_cast<const uint4*>(e.m2 + at + 8 * s * e.ldr)) : zero;
            a.di[s] = in ? __ldcg(d1 + i + 8 * s) : 0.0f;
        }
        if (j < g.n) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(d2 + j)), y = __ldcg(reinterpret_cast<const float4*>(d2 + j + 4));
            a.dj[0] = x.x; a.dj[1] = x.y; a.dj[2] = x.z; a.dj[3] = x.w; a.dj[4] = y.x; a.dj[5] = y.y; a.dj[6] = y.z; a.dj[7] = y.w;
        }
    } else if constexpr (KIND == KIND_APPLY || KIND == KIND_FINAL) {
        const int64_t at = ((int64_t)batch * g.m + i) * e.ldc + j;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = i + 8 * s < g.m && j < g.n;
            a.h[s] = in ? __ldcg(reinterpret_cast<const uint4*>(e.hi_in + at + 8 * s * e.ldc)) : zero;
            a.l[s] = in ? __ldcg(reinterpret_cast<const uint2*>(e.lo + at + 8 * s * e.ldc)) : make_uint2(0, 0);
            a.k[s] = in ? __ldcg(e.coef + (int64_t)batch * e.ldr + i + 8 * s) : 0.0f;
        }
    }
}

// Takes t[k] out of t (0 stays in its place; 0 where k is not 0..7), without a branch per element.
__device__ __forceinline__ float take(float (&t)[8], int k) {
    float d = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        d = c == k ? t[c] : d;
        t[c] = c == k ? 0.0f : t[c];
    }
    return d;
}

// The epilogue of a 32 x 32 block at (i0, j0), staged in shared memory by this
// warp.  mirror: the block lies off the diagonal square of its tile row, so
// the symmetric counterpart is written as well.
template <int KIND>
__device__ __forceinline__ void block_epilogue(const typename EpiOf<KIND>::T& e, const Args& g, int batch, int i0, int j0,
                                               uint32_t block, int lane, bool mirror, const Ahead<KIND>& a) {
    const int major = lane / 4, minor = lane % 4;
    if constexpr (is_linear(KIND)) {
        // fp32 results: two steps at a time, next to the accumulators in registers
        constexpr int kSteps = KIND == KIND_F32 ? 2 : 4;
#pragma unroll
        for (int s0 = 0; s0 < 4; s0 += kSteps) {
            float t[kSteps][8];
            if (KIND == KIND_LINEAR && e.swapped) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) block_get_column(block, minor, (s0 + s) * 8 + major, t[s]);
            } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) block_get(block, (s0 + s) * 8 + major, minor, t[s]);
            }
            linear_steps<KIND, kSteps>(e, g, s0, lane, i0, j0, t);
        }
        return;
    } else {
        float t[4][8];
        const int i = i0 + major, j = j0 + minor * 8;  // step s: row i + 8 s
        bool in[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            in[s] = i + 8 * s < g.m && j < g.n;
            block_get(block, s * 8 + major, minor, t[s]);
        }
        bool again = false;  // a second, transposed pass over the block
        if constexpr (KIND == KIND_GRAM || KIND == KIND_POLY) again = mirror;
        if constexpr (KIND == KIND_FINAL) again = e.out[batch].transposed;
        const bool diagonal = i0 < j0 + 32 && j0 < i0 + 32;
        if constexpr (KIND == KIND_GRAM) {
            __half* d = e.gram + ((int64_t)batch * g.m + i) * e.ldr + j;  // rows are padded to 8 columns
            if (diagonal) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float x = take(t[s], i + 8 * s - j);
                    if (in[s] && (unsigned)(i + 8 * s - j) < 8u) e.gram_diag[(int64_t)batch * e.ldr + i + 8 * s] = x * e.alpha;
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int c = 0; c < 8; ++c) t[s][c] *= e.alpha;
                if (in[s]) store8_half(d + 8 * s * e.ldr, t[s]);
            }
        } else if constexpr (KIND == KIND_POLY) {
            // With A = D + E (D diagonal, E the stored off-diagonal):
            //   A^2 = D^2 + D E + E D + E^2, so off the diagonal
            //   (b A + c A^2)_ij = (b + c (d_i + d_j)) E_ij + c (E^2)_ij
            // and on it b d_i + c d_i^2 + c (E^2)_ii.
            __half* d = e.poly + ((int64_t)batch * g.m + i) * e.ldr + j;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float x[8];
                half8(a.q[s], x);
                const float base = fmaf(e.c, a.di[s], e.b);
                if (diagonal) {  // the stored diagonal of E is 0, so the result's is too
                    const float sq = take(t[s], i + 8 * s - j);
                    if (in[s] && (unsigned)(i + 8 * s - j) < 8u)
                        e.coef[(int64_t)batch * e.ldr + i + 8 * s] = e.a + fmaf(e.c, fmaf(a.di[s], a.di[s], sq), e.b * a.di[s]);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) t[s][c] = fmaf(fmaf(e.c, a.dj[c], base), x[c], e.c * t[s][c]);
                if (in[s]) store8_half(d + 8 * s * e.ldr, t[s]);
            }
        } else if constexpr (KIND == KIND_MUL) {
            // (D1 + E1)(D2 + E2) = D1 D2 + D1 E2 + E1 D2 + E1 E2; symmetric, since the factors commute.
            __half* d = e.gram + ((int64_t)batch * g.m + i) * e.ldr + j;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float x[8], y[8];
                half8(a.p[s], x);
                half8(a.q[s], y);
                if (diagonal) {  // both factors' stored diagonals are 0, so the result's is too
                    const int k = i + 8 * s - j;
                    const float sq = take(t[s], k);
                    float dk = 0.0f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) dk = c == k ? a.dj[c] : dk;
                    if (in[s] && (unsigned)k < 8u) e.gram_diag[(int64_t)batch * e.ldr + i + 8 * s] = fmaf(a.di[s], dk, sq);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) t[s][c] = fmaf(a.di[s], y[c], fmaf(x[c], a.dj[c], t[s][c]));
                if (in[s]) store8_half(d + 8 * s * e.ldr, t[s]);
            }
        } else {
            // X' = (a + diagonal) X + E X: the large part of the polynomial is its
            // diagonal, which multiplies both terms of X.
            const int64_t at = ((int64_t)batch * g.m + i) * e.ldc + j;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float x[8];
                join8(a.h[s], a.l[s], x);
#pragma unroll
                for (int c = 0; c < 8; ++c) t[s][c] = fmaf(a.k[s], x[c], t[s][c]);
                if constexpr (KIND == KIND_APPLY) {
                    uint4 h;
                    uint2 l;
                    split8(t[s], h, l);
                    if (in[s]) {
                        *reinterpret_cast<uint4*>(e.hi + at + 8 * s * e.ldc) = h;
                        *reinterpret_cast<uint2*>(e.lo + at + 8 * s * e.ldc) = l;
                    }
                }
            }
            if constexpr (KIND == KIND_FINAL) {
                if (!again && j < g.n) final_rows<4>(e, e.out[batch], g.m, g.n, i, j, t);
            }
        }
        if (again) {
#pragma unroll
            for (int s = 0; s < 4; ++s) block_put(block, s * 8 + major, minor, t[s]);
            __syncwarp();
            const int col = j0 + major, row = i0 + minor * 8;  // step s: column col + 8 s, rows row .. row + 7
#pragma unroll
            for (int s = 0; s < 4; ++s) block_get_column(block, minor, s * 8 + major, t[s]);
            if constexpr (KIND == KIND_FINAL) {
                if (row < g.m) final_rows<4>(e, e.out[batch], g.n, g.m, col, row, t);
            } else if constexpr (KIND == KIND_GRAM || KIND == KIND_POLY) {
                __half* d = (KIND == KIND_GRAM ? e.gram : e.poly) + ((int64_t)batch * g.m + col) * e.ldr + row;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (col + 8 * s < g.n && row < g.m) store8_half(d + 8 * s * e.ldr, t[s]);
            }
        }
    }
}

// The tile of index t inside one batch entry.  In symmetric mode tile row tm
// starts at the first tile column that reaches its diagonal.
__device__ __forceinline__ void tile_at(const Args& g, int t, int bm, int bn, int& tm, int& tn) {
    if (!g.symmetric) {  // groups of 16 tile rows, so that tiles in flight share operands in L2
        const int group = t / (16 * g.tiles_n), rows = min(16, g.tiles_m - group * 16), in = t - group * 16 * g.tiles_n;
        tm = group * 16 + in % rows;
        tn = in / rows;
        return;
    }
    tm = 0;
    for (;;) {
        const int first = tm * bm / bn, count = g.tiles_n - first;
        if (t < count || tm + 1 >= g.tiles_m) {
            tn = first + t;
            return;
        }
        t -= count;
        ++tm;
    }
}

// ------------------------------------------------------------ split kernel --
//
// One 128 x BN tile per cluster of `split` CTAs; each CTA reduces its share of
// the K blocks with a TMA-fed pipeline (one producer thread, one issuing
// thread), and the cluster adds the partial tiles through distributed shared
// memory in rank order, so a result never depends on timing.  This is the
// kernel of the calls with few tiles: a short call spreads its weight reads
// over up to 8 times as many SMs.
//
// fp32 results (regions = 256 / BN) give each part of a CTA's reduction its own
// accumulator in tensor memory, added in fp32 registers: the tensor
// cores' accumulators truncate, about 1.9e-8 of the sum per 16-element step.
// A part is at most kPromoteBlocks blocks (512 elements, 6e-7).  Where there are
// no more parts than accumulators they are added at the end; a longer reduction
// (DRAIN: a kernel of its own, its code costs short calls 0.3 us) goes round the accumulators, and the epilogue warps empty one while the
// issuing thread fills the next (reduction of 98304 into 1024 x 2048: 2.8e-5 off
// and 341 us from two accumulators, 5.0e-7 and 344 us so; of 1048576 into
// 256 x 256: 3.8e-5 and 533 us, 5.6e-7 and 533 us).  The sums take up to 128 registers
// a thread, hence the bound on registers for BN = 128: two CTAs still share an SM.
//
// Stages: a copy takes about 1500 cycles from its issue until its stage is free
// again, so a CTA that has an SM to itself takes all the shared memory (`deep`:
// a reduction of 640 elements at BN = 32 is in flight at once); launches of
// more CTAs than SMs use half of it and run two CTAs per SM.

constexpr int kPromoteBlocks = 8;
constexpr int kSplitThreads = 192;  // producer warp, issuing warp, four epilogue warps
constexpr int kMaxStages = 10;

template <int BN>
__host__ __device__ constexpr int split_stage_bytes() {
    return 128 * 128 + BN * 128;
}
template <int BN>
__host__ __device__ constexpr int split_stages(bool deep) {
    return (BN == 32 ? 5 : BN == 64 ? 4 : 3) * (deep ? 2 : 1);
}
template <int BN>
__host__ __device__ constexpr int split_smem(bool deep) {  // stages + alignment; barriers are static
    return split_stages<BN>(deep) * split_stage_bytes<BN>() + 1024;
}

// 32 columns of one row, added over a CTA's accumulators.
template <int BN>
__device__ __forceinline__ void read_regions(uint32_t addr, int regions, float (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = 0.0f;
    for (int r = 0; r < regions; ++r) {
        float w[32];
        mma::tmem_ld32(addr + r * BN, w);
        mma::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] += w[c];
    }
}

// Element pieces of a block added over the cluster's partial tiles, in rank order.
__device__ __forceinline__ void cluster_get(uint32_t at, int split, float* t) {
    t[0] = t[1] = t[2] = t[3] = 0.0f;
    for (int p = 0; p < split; ++p) {
        float v[4];
        mma::ld_cluster4(mma::map_rank(at, p), v);
#pragma unroll
        for (int x = 0; x < 4; ++x) t[x] += v[x];
    }
}

template <int KIND, int BN, bool DRAIN>
__global__ void __launch_bounds__(kSplitThreads, DRAIN && BN == 128 ? 2 : 0)
    split_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const __grid_constant__ Args g, const __grid_constant__ typename EpiOf<KIND>::Param ep) {
    using namespace mma;
    const auto& e = epilogue_of(ep);
    const int S = g.stages;
    constexpr uint32_t kA = 128 * 128, kStage = kA + BN * 128;
    constexpr uint32_t kCols = 256;  // two CTAs per SM together allocate all 512
    extern __shared__ uint8_t raw[];
    constexpr int R = 256 / BN;  // accumulators
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], filled[R], drained[R], done;
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = g.split > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / g.split;
    const int batch = tile / g.tiles_per_batch;
    int tm, tn;
    tile_at(g, tile - batch * g.tiles_per_batch, 128, BN, tm, tn);
    const int kb0 = (int)((int64_t)g.kblocks * rank / g.split), kb1 = (int)((int64_t)g.kblocks * (rank + 1) / g.split);
    const int nkb = kb1 - kb0;
    // parts of the reduction: one, or (fp32 results) one per accumulator, or (DRAIN) more
    const int regions = min(g.regions, nkb);
    const int parts = DRAIN ? max(regions, (nkb + kPromoteBlocks - 1) / kPromoteBlocks) : regions;
    const bool mirror = g.symmetric && tn * BN >= (tm + 1) * 128;

    if (threadIdx.x == 0) {
        if (g.kblocks) {
            prefetch_map(&ma);
            prefetch_map(&mb);
        }
        for (int s = 0; s < S; ++s) {
            tma::mbar_init(&full[s], 1);
            tma::mbar_init(&empty[s], 1);
        }
        if (DRAIN)
            for (int r = 0; r < R; ++r) {
                tma::mbar_init(&filled[r], 1);
                tma::mbar_init(&drained[r], 4);  // the epilogue warps
            }
        tma::mbar_init(&done, 1);
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<1>(tma::smem_addr(&tmem_slot), kCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    if (g.release) grid_launch_dependents();
    grid_wait();

    bool ok = true;
    if (warp == 0) {
        if (elect_one()) {
            int issued = 0, s = 0, round = 0;
            for (int it = 0; it < nkb; ++it) {
                if (round && !tma::mbar_wait(&empty[s], (round - 1) & 1)) {
                    record_device_error(g.err, DPRED_E_TIMEOUT);
                    ok = false;
                    break;
                }
                const uint32_t a = base + s * kStage, b = a + kA, bar = tma::smem_addr(&full[s]);
                tma::mbar_arrive_expect_tx(&full[s], kStage);
                const int k0 = (kb0 + it) * kBlockK;
                if (g.a_mn) {
                    load_box(a, &ma, bar, tm * 128, k0, batch);
                    load_box(a + 8192, &ma, bar, tm * 128 + 64, k0, batch);
                } else {
                    load_box(a, &ma, bar, k0, tm * 128, batch);
                }
                if (g.b_mn) {
                    // boxes are 64 wide; a narrower tile still loads (and counts) whole 64-wide boxes only
                    // where BN is a multiple of 64, and the host keeps BN = 32 for K-major B
                    for (int c = 0; c < BN / 64; ++c) load_box(b + c * 8192, &mb, bar, tn * BN + c * 64, k0, batch);
                } else {
                    load_box(b, &mb, bar, k0, tn * BN, batch);
                }
                ++issued;
                if (++s == S) {
                    s = 0;
                    ++round;
                }
            }
            if (!ok)  // let the copies in flight land before the CTA can leave
                for (int it = issued > S ? issued - S : 0; it < issued; ++it) tma::mbar_wait(&full[it % S], (it / S) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint64_t da0 = operand_desc(base, g.a_mn), db0 = operand_desc(base + kA, g.b_mn);
            const uint32_t sa = g.a_mn ? 128 : 2, sb = g.b_mn ? 128 : 2;  // 16 reduction elements, in 16-byte units
            const uint32_t idesc = instr_desc(128, BN, g.bf16, g.a_mn, g.b_mn);
            int part = 0, region = 0, s = 0, round = 0;
            for (int it = 0, next = parts > 1 ? nkb / parts : nkb; it < nkb; ++it) {
                bool first = it == 0;
                if (it >= next) {
                    if (DRAIN) commit<1>(tma::smem_addr(&filled[region]));
                    ++part;
                    region = part % R;
                    next = DRAIN ? (int)((int64_t)nkb * (part + 1) / parts) : nkb * (part + 1) / parts;
                    first = true;
                    if (DRAIN && part >= R && !tma::mbar_wait(&drained[region], (part / R - 1) & 1)) {
                        record_device_error(g.err, DPRED_E_TIMEOUT);
                        ok = false;
                        break;
                    }
                }
                if (!tma::mbar_wait(&full[s], round & 1)) {
                    record_device_error(g.err, DPRED_E_TIMEOUT);
                    ok = false;
                    break;
                }
                fence_after();
                const uint64_t da = da0 + s * (kStage >> 4), db = db0 + s * (kStage >> 4);
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k)
                    issue<1>(tmem + region * BN, da + k * sa, db + k * sb, idesc, !first || k != 0);
                commit<1>(tma::smem_addr(&empty[s]));
                if (++s == S) {
                    s = 0;
                    ++round;
                }
            }
            if (ok && nkb) commit<1>(tma::smem_addr(DRAIN ? &filled[region] : &done));
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // tensor-memory lanes 32 q .. 32 q + 31 belong to this warp
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        float sum[DRAIN ? BN / 32 : 1][32];
        if constexpr (DRAIN) {
#pragma unroll
            for (int c = 0; c < BN / 32; ++c)
#pragma unroll
                for (int x = 0; x < 32; ++x) sum[c][x] = 0.0f;
            for (int part = 0; part < parts; ++part) {
                const int r = part % R;
                ok = __all_sync(0xFFFFFFFFu, tma::mbar_wait(&filled[r], (part / R) & 1));
                if (!ok) break;
                fence_after();
#pragma unroll
                for (int c = 0; c < BN / 16; ++c) {  // 16 columns: the sums take most of the registers
                    float v[16];
                    tmem_ld16(lanes + r * BN + c * 16, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 16; ++x) sum[c / 2][c % 2 * 16 + x] += v[x];
                }
                fence_before();
                __syncwarp();
                if (lane == 0) tma::mbar_arrive(&drained[r]);
            }
            if (!ok) record_device_error(g.err, DPRED_E_TIMEOUT);
        } else if (nkb && !tma::mbar_wait(&done, 0)) {
            record_device_error(g.err, DPRED_E_TIMEOUT);
            ok = false;
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        fence_after();
        // accumulators to the blocks of this warp's rows, 32 columns each (the
        // pipeline's stages are free: every load was consumed)
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 32) {
            float v[32];
            __syncwarp();
            if constexpr (DRAIN) {
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = sum[c0 / 32][x];
            } else {
                read_regions<BN>(lanes + c0, ok ? regions : 0, v);
            }
            const uint32_t block = base + (c0 / 32 * 4 + q) * kBlockBytes;
            block_put_row(block, lane, v);
            if (!DRAIN && g.split == 1) {
                __syncwarp();
                Ahead<KIND> ahead;
                load_ahead<KIND>(e, g, batch, tm * 128 + q * 32, tn * BN + c0, lane, ahead);
                if (ok) block_epilogue<KIND>(e, g, batch, tm * 128 + q * 32, tn * BN + c0, block, lane, mirror, ahead);
            }
        }
        if (DRAIN && g.split == 1 && ok) {  // after all of them: the sums and an epilogue together take too many registers
            __syncwarp();
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 32)
                block_epilogue<KIND>(e, g, batch, tm * 128 + q * 32, tn * BN + c0, base + (c0 / 32 * 4 + q) * kBlockBytes, lane, mirror,
                                     Ahead<KIND>());
        }
        fence_before();
    }
    if (g.split > 1) {
        cluster_sync();
        if (warp >= 2) {
            // the tile's blocks (their steps, for a linear layer) spread over the cluster's epilogue warps
            constexpr int kSteps = KIND == KIND_LINEAR ? 4 : 1;
            ok = __all_sync(0xFFFFFFFFu, ok);
            const int major = lane / 4, minor = lane % 4;
            for (int u = rank * 4 + (warp & 3); u < BN / 8 * kSteps && ok; u += 4 * g.split) {
                const int id = u / kSteps, q = id & 3, c0 = id / 4 * 32;
                const uint32_t block = base + id * kBlockBytes;
                const int i0 = tm * 128 + q * 32, j0 = tn * BN + c0;
                float t[1][8];
                if constexpr (KIND == KIND_LINEAR) {
                    const int step = u % 4;
                    if (e.swapped) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) t[0][k] = 0.0f;
                        for (int p = 0; p < g.split; ++p) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                t[0][k] += ld_cluster(map_rank(piece(block, 8 * minor + k, (step * 8 + major) / 4) + major % 4 * 4, p));
                        }
                    } else {
                        const int r = step * 8 + major;
                        cluster_get(piece(block, r, 2 * minor), g.split, t[0]);
                        cluster_get(piece(block, r, 2 * minor + 1), g.split, t[0] + 4);
                    }
                    linear_steps<KIND, 1>(e, g, step, lane, i0, j0, t);
                } else {
                    // into a block of this CTA's own, past the partial tile
                    const uint32_t mine = base + (BN / 8 + (warp & 3)) * kBlockBytes;
                    Ahead<KIND> ahead;
                    load_ahead<KIND>(e, g, batch, i0, j0, lane, ahead);
                    __syncwarp();
#pragma unroll
                    for (int step = 0; step < 4; ++step) {
                        const int r = step * 8 + major;
                        cluster_get(piece(block, r, 2 * minor), g.split, t[0]);
                        cluster_get(piece(block, r, 2 * minor + 1), g.split, t[0] + 4);
                        block_put(mine, r, minor, t[0]);
                    }
                    __syncwarp();
                    block_epilogue<KIND>(e, g, batch, i0, j0, mine, lane, mirror, ahead);
                }
            }
        }
        cluster_sync();  // no CTA leaves while another may still read its partial tile
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        fence_after();
        tmem_free<1>(tmem, kCols);
    }
}

// ------------------------------------------------------------- tile kernel --
//
// The kernel of the calls with many tiles: persistent CTA pairs, one
// 256 x BN tile per pair and step.  The pair's tcgen05.mma (cta_group::2)
// reads A rows 0..127 and B rows 0..BN/2-1 from the even CTA's shared memory and
// the other halves from the odd one's, so every operand byte is staged once
// per pair.  Accumulators are double-buffered in tensor memory: eight epilogue
// warps drain one while the issuing thread fills the other.
//
// PROMOTE (fp32 results): the tensor cores' accumulators truncate, which costs
// about 1.9e-8 of the sum per 16-element step (measured: 1.9e-5 after 16384
// elements).  Here an accumulator takes kPromoteBlocks reduction blocks (512
// elements, 6e-7) and the epilogue threads add it to fp32 registers.

// Twelve warps: producer, issuer, two that sum A's rows, eight of the epilogue.
//
// Row sums (the bias gradient beside a weight gradient, whose A is dy): the two
// warps read each stage of A, one 64-row box each, in the tiles of the first
// tile column; a stage is free once they have arrived as well.  A lane adds 8
// rows of A over 16 reduction elements a stage and the stage's sums to its
// total, so a sum has one fixed order.  Only the even CTA sees the copies land
// (its barrier counts both CTAs' bytes), and its warps read beside the matrix
// instructions.  The odd one's wait for a commit of the stage's products, which
// arrives in both CTAs on a barrier of its own: those products were issued by
// the thread that saw the bytes land, and have read them.  That holds a stage a
// little longer and costs nothing measurable.  (Passing the even CTA's
// observation on by an arrival of its own needs a releasing one, which took
// longer than the stage's products: 250 us for the call below.  A fence over
// all proxies before the reads, instead of the one over this CTA's shared
// memory: 205 us.  A second wait in the producer, instead of the second commit:
// 3-5% on short products without row sums.)
// Unpacked to fp32 and added, the sums took 830 cycles a stage against the
// products' 600; with adds that take the bf16 half as it is they keep up:
// [16384, 4096] x [16384, 1024] into fp32, cache flushed, 84-88 us and 98 with
// the row sums (in a launch of their own they add 28).
constexpr int kTileThreads = 384;
constexpr int kEpilogueWarp0 = 4;

//
// Streaming epilogue (16-byte aligned matrices).  A warp owns 32 rows; a thread
// computes one row, 32 columns at a time, straight from the tensor-memory load,
// and packs it into a 32-row x 128-byte box of shared memory (128-byte swizzle:
// no bank conflicts), which one bulk tensor copy writes; the copies' bounds
// checks take care of ragged edges but for a last part of 16 bytes (box_tail).  What is read per element (residual, stored
// pre-activation) comes in as a box the same way, requested before the
// accumulator is waited for.  fp32 accumulation is a bulk copy that adds.
// Against writing global memory from the registers by way of an fp32 block
// (block_epilogue, which remains for unaligned matrices), a plain tile's
// epilogue went from 7,000 cycles to 2,800.  Beyond a reduction of about 1024
// (9,500 cycles) the tile is bound by its operands: 512 KB a CTA at the 64 bytes
// a cycle that reach an SM, which the output and what the epilogue reads share.

//
// One box per warp: the reduction's pipeline needs the rest of the shared
// memory more (8192 x 8192 x 1024 with relu: 4 stages and three boxes 92 us,
// 6 stages and one box 84 us).

template <int BN>
__host__ __device__ constexpr int tile_stages() {
    return BN == 256 ? 6 : 8;
}
constexpr uint32_t kBoxBytes = 32 * 128;
static_assert(kBoxBytes == kBlockBytes, "a warp's box and its block share memory");
template <int BN>
__host__ __device__ constexpr int tile_smem() {
    return tile_stages<BN>() * (128 * 128 + BN / 2 * 128) + 8 * (int)kBoxBytes + 1024;
}

#define DPRED_EACH32(expr) _Pragma("unroll") for (int x = 0; x < 32; ++x) expr

// The bias of 32 columns from j on (`cols` in all), every lane the same ones.
// Loaded before the accumulators are waited for, without a test per column: read
// where it is added, it cost as much as the gelu.
__device__ __forceinline__ void load_bias(const LinearEpi& e, int cols, int j, float (&b)[32]) {
    if (!e.bias) {
        DPRED_EACH32(b[x] = 0.0f;)
    } else if (j + 32 <= cols && !e.bias_f32) {
        uint4 q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.bias) + j + 8 * k);
        DPRED_EACH32(b[x] = bf16_of(q[x / 8], x % 8);)
    } else if (j + 32 <= cols) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(e.bias) + j + 4 * k);
            b[4 * k] = q.x; b[4 * k + 1] = q.y; b[4 * k + 2] = q.z; b[4 * k + 3] = q.w;
        }
    } else {  // clamped to the last column: what lies past it is never stored
        DPRED_EACH32(b[x] = e.bias_f32 ? static_cast<const float*>(e.bias)[min(j + x, cols - 1)]
                                       : load_bf16(static_cast<const __nv_bfloat16*>(e.bias) + min(j + x, cols - 1));)
    }
}

// 32 bf16 columns (half h of the 64 in a box) of row `lane`.
__device__ __forceinline__ void box_put(uint32_t box, int lane, int h, const float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t w0 = pack_bf16x2(v[8 * q], v[8 * q + 1]), w1 = pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                       w2 = pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), w3 = pack_bf16x2(v[8 * q + 6], v[8 * q + 7]);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(piece(box, lane, 4 * h + q)), "r"(w0), "r"(w1), "r"(w2),
                     "r"(w3)
                     : "memory");
    }
}

// 16 bf16 columns, 32-byte aligned.
__device__ __forceinline__ void store16_bf16(__nv_bfloat16* p, const float* v) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ uint4 box_get(uint32_t box, int lane, int c) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "r"(piece(box, lane, c))
                 : "memory");
    return q;
}

// A bulk tensor copy writes whole groups of 16 bytes: where a matrix's rows end
// inside one, it would write past them (zeros, or with an adding copy sums with
// them).  The maps of the matrices that are written therefore end at the last
// whole group, column `whole_columns`, and a lane stores (or adds) the up to 7
// elements behind it from its row of the box that is about to be sent.
template <typename T>
__host__ __device__ __forceinline__ constexpr int whole_columns(int cols) {
    return cols & ~(16 / (int)sizeof(T) - 1);
}

template <typename T>
__device__ __forceinline__ void box_tail(T* out, int64_t ld, int rows, int cols, uint32_t box, int lane, int i, int col, bool add) {
    constexpr int kGroup = 16 / sizeof(T), kBox = 128 / sizeof(T);
    const int whole = whole_columns<T>(cols);
    if (whole == cols || col + kBox <= whole || i + lane >= rows) return;
    T* p = out + (int64_t)(i + lane) * ld;
#pragma unroll 1  // seldom run: short code matters more
    for (int c = whole; c < cols; ++c) {
        const uint32_t at = piece(box, lane, (c - col) / kGroup) + (c - col) % kGroup * (int)sizeof(T);
        if constexpr (sizeof(T) == 4) {
            const float x = lds1(at);
            p[c] = add ? p[c] + x : x;
        } else {
            uint16_t x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
            reinterpret_cast<uint16_t*>(p)[c] = x;
        }
    }
}

template <int KIND>
__device__ __forceinline__ void box_activate(const LinearEpi& e, float (&v)[32]) {
    if constexpr (KIND == KIND_ACT) {
        if (e.act == ACT_GELU) {
            DPRED_EACH32(v[x] = activate<ACT_GELU>(v[x]);)
        } else if (e.act == ACT_SILU) {
            DPRED_EACH32(v[x] = activate<ACT_SILU>(v[x]);)
        } else if (e.act == ACT_RELU) {
            DPRED_EACH32(v[x] = activate<ACT_RELU>(v[x]);)
        }
    }
}

// Residual (added) or stored pre-activation (its gradient multiplies).
template <int KIND>
__device__ __forceinline__ void box_combine(const LinearEpi& e, uint32_t box, int lane, int h, float (&v)[32]) {
    uint4 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = box_get(box, lane, 4 * h + k);
    if constexpr (KIND == KIND_GRAD) {
        if (e.act == ACT_GELU) {
            DPRED_EACH32(v[x] *= activate_grad<ACT_GELU>(bf16_of(q[x / 8], x % 8));)
        } else if (e.act == ACT_SILU) {
            DPRED_EACH32(v[x] *= activate_grad<ACT_SILU>(bf16_of(q[x / 8], x % 8));)
        } else {
            DPRED_EACH32(v[x] *= activate_grad<ACT_RELU>(bf16_of(q[x / 8], x % 8));)
        }
    } else {
        DPRED_EACH32(v[x] += bf16_of(q[x / 8], x % 8);)
    }
}

template <int KIND, int BN, bool PROMOTE>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ Args g, const __grid_constant__ TileParams tp) {
    using namespace mma;
    const LinearEpi& e = tp.e;
    constexpr int S = tile_stages<BN>();
    constexpr uint32_t kA = 128 * 128, kB = BN / 2 * 128, kStage = kA + kB;
    constexpr uint32_t kCols = 2 * BN;
    constexpr int kHalf = BN / 2;  // columns per epilogue warp
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[S], empty[S], consumed[S], acc_full[2], acc_empty[2], in_full[8];
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const bool row_sums = sums_rows(KIND) && tp.row_sum != nullptr;
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int total = g.tiles_per_batch * g.batch;
    const int chunk = PROMOTE ? kPromoteBlocks : g.kblocks;

    if (threadIdx.x == 0) {
        prefetch_map(&ma);
        prefetch_map(&mb);
        for (int s = 0; s < S; ++s) {
            tma::mbar_init(&full[s], 1);   // the even CTA's expected bytes (both CTAs' copies)
            tma::mbar_init(&empty[s], row_sums ? 3 : 1);  // the issuing thread's commit, this CTA's summing warps
            tma::mbar_init(&consumed[s], 1);  // another commit of the same products, for the odd CTA's summing warps
        }
        for (int a = 0; a < 2; ++a) {
            tma::mbar_init(&acc_full[a], 1);
            tma::mbar_init(&acc_empty[a], 16);  // eight epilogue warps of each CTA
        }
        for (int w = 0; w < 8; ++w) tma::mbar_init(&in_full[w], 1);
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<2>(tma::smem_addr(&tmem_slot), kCols);
    fence_before();
    cluster_sync();
    fence_after();
    const uint32_t tmem = tmem_slot;
    if (g.release) grid_launch_dependents();
    grid_wait();

    if (warp == 0) {
        if (elect_one()) {
            int s = 0, round = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += pairs) {
                const int batch = tile / g.tiles_per_batch;
                int tm, tn;
                tile_at(g, tile - batch * g.tiles_per_batch, 256, BN, tm, tn);
                const int i0 = tm * 256 + (int)rank * 128, j0 = tn * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < g.kblocks; ++kb) {
                    if (round && !tma::mbar_wait(&empty[s], (round - 1) & 1)) {
                        record_device_error(g.err, DPRED_E_TIMEOUT);
                        ok = false;
                        break;
                    }
                    const uint32_t a = base + s * kStage, b = a + kA, bar = tma::smem_addr(&full[s]);
                    if (rank == 0) tma::mbar_arrive_expect_tx(&full[s], 2 * kStage);
                    const int k0 = kb * kBlockK;
                    if (g.a_mn) {
                        load_box_pair(a, &ma, bar, i0, k0, batch);
                        load_box_pair(a + 8192, &ma, bar, i0 + 64, k0, batch);
                    } else {
                        load_box_pair(a, &ma, bar, k0, i0, batch);
                    }
                    if (g.b_mn) {
#pragma unroll
                        for (int c = 0; c < BN / 128; ++c) load_box_pair(b + c * 8192, &mb, bar, j0 + c * 64, k0, batch);
                    } else {
                        load_box_pair(b, &mb, bar, k0, j0, batch);
                    }
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                }
            }
            if (!ok) {  // copies in flight land within microseconds, or never: leave after a bounded pause
                const long long t0 = clock64();
                while (clock64() - t0 < 20000000LL) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const uint64_t da0 = operand_desc(base, g.a_mn), db0 = operand_desc(base + kA, g.b_mn);
            const uint32_t sa = g.a_mn ? 128 : 2, sb = g.b_mn ? 128 : 2;  // 16 reduction elements, in 16-byte units
            const uint32_t idesc = instr_desc(256, BN, g.bf16, g.a_mn, g.b_mn);
            int s = 0, round = 0, fill = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += pairs) {
                for (int kb = 0; kb < g.kblocks && ok; ++fill) {
                    const int a = fill & 1;
                    if (fill >= 2 && !tma::mbar_wait(&acc_empty[a], (fill / 2 - 1) & 1)) {
                        record_device_error(g.err, DPRED_E_TIMEOUT);
                        ok = false;
                        break;
                    }
                    fence_after();
                    const int stop = min(kb + chunk, g.kblocks);
                    for (int first = kb; kb < stop; ++kb) {
                        if (!tma::mbar_wait(&full[s], round & 1)) {
                            record_device_error(g.err, DPRED_E_TIMEOUT);
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint64_t da = da0 + s * (kStage >> 4), db = db0 + s * (kStage >> 4);
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            issue<2>(tmem + a * BN, da + k * sa, db + k * sb, idesc, kb != first || k != 0);
                        commit<2>(tma::smem_addr(&empty[s]));
                        if (row_sums) commit<2>(tma::smem_addr(&consumed[s]));
                        if (++s == S) {
                            s = 0;
                            ++round;
                        }
                    }
                    if (ok) commit<2>(tma::smem_addr(&acc_full[a]));
                }
            }
        }
        __syncwarp();
    } else if (warp < kEpilogueWarp0) {
        if (row_sums) {
            const int red_group = lane / 8, piece_of = lane % 8;
            int s = 0, round = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += pairs) {
                int tm, tn;
                tile_at(g, tile, 256, BN, tm, tn);
                const int i = tm * 256 + (int)rank * 128 + (warp - 2) * 64;
                const bool mine = tn == 0 && i < g.m;
                float sum[8] = {};
                for (int kb = 0; kb < g.kblocks; ++kb) {
                    ok = __all_sync(0xFFFFFFFFu, rank == 0 ? tma::mbar_wait(&full[s], round & 1)
                                                           : mbar_wait_cluster(&consumed[s], round & 1));
                    if (!ok) break;
                    if (rank != 0) {
                        fence_after();
                        tma::fence_proxy_async_shared();  // copies wrote what is read next
                    }
                    if (mine) {
                        const uint32_t box = base + s * kStage + (warp - 2) * 8192;
                        uint4 v[16];
#pragma unroll
                        for (int r = 0; r < 16; ++r) v[r] = box_get(box, r * 4 + red_group, piece_of);
                        float part[8] = {};
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            add_bf16x2(part[0], part[1], v[r].x);
                            add_bf16x2(part[2], part[3], v[r].y);
                            add_bf16x2(part[4], part[5], v[r].z);
                            add_bf16x2(part[6], part[7], v[r].w);
                        }
#pragma unroll
                        for (int c = 0; c < 8; ++c) {  // formed here: no read is under way when the stage is given back
                            sum[c] += part[c];
                            asm volatile("" : "+f"(sum[c])::"memory");
                        }
                    }
                    __syncwarp();
                    if (lane == 0) tma::mbar_arrive(&empty[s]);
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                }
                if (ok && mine) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        sum[c] += __shfl_xor_sync(0xFFFFFFFFu, sum[c], 8);
                        sum[c] += __shfl_xor_sync(0xFFFFFFFFu, sum[c], 16);
                        const int row = i + piece_of * 8 + c;
                        if (red_group == 0 && row < g.m) {
                            float* o = tp.row_sum + row;
                            *o = tp.row_sum_add ? *o + sum[c] : sum[c];
                        }
                    }
                }
            }
            if (!ok && lane == 0) record_device_error(g.err, DPRED_E_TIMEOUT);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - kEpilogueWarp0) / 4;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * kHalf;
        const uint32_t box = base + S * kStage + (warp - kEpilogueWarp0) * kBoxBytes;
        uint64_t* in_bar = &in_full[warp - kEpilogueWarp0];
        uint32_t in_parity = 0;
        const uint32_t drained0 = map_rank(tma::smem_addr(&acc_empty[0]), 0), drained1 = map_rank(tma::smem_addr(&acc_empty[1]), 0);
        int fill = 0;
        bool ok = true;
        for (int tile = pair; tile < total && ok; tile += pairs) {
            const int batch = tile / g.tiles_per_batch;
            int tm, tn;
            tile_at(g, tile - batch * g.tiles_per_batch, 256, BN, tm, tn);
            const int i = tm * 256 + (int)rank * 128 + q * 32, j = tn * BN + half * kHalf;
            if constexpr (PROMOTE) {
                float sum[kHalf / 32][32];
#pragma unroll
                for (int c = 0; c < kHalf / 32; ++c)
#pragma unroll
                    for (int x = 0; x < 32; ++x) sum[c][x] = 0.0f;
                for (int kb = 0; kb < g.kblocks && ok; kb += chunk, ++fill) {
                    const int a = fill & 1;
                    ok = __all_sync(0xFFFFFFFFu, tma::mbar_wait(&acc_full[a], (fill / 2) & 1));
                    if (!ok) break;
                    fence_after();
#pragma unroll
                    for (int c = 0; c < kHalf / 16; ++c) {  // 16 columns: the sums take most of the registers
                        float v[16];
                        tmem_ld16(lanes + a * BN + c * 16, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; ++x) sum[c / 2][c % 2 * 16 + x] += v[x];
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(a ? drained1 : drained0);
                }
                if (ok && i < g.m) {
#pragma unroll
                    for (int c = 0; c < kHalf / 32; ++c) {
                        if (j + c * 32 >= g.n) break;
                        if (tp.stream) {
                            if (lane == 0) tma::bulk_wait_read<0>();  // the copy that last used the box
                            __syncwarp();
                            if (e.bias) {
                                float bias[32];
                                load_bias(e, g.n, j + c * 32, bias);
                                DPRED_EACH32(sum[c][x] += bias[x];)
                            }
                            block_put_row(box, lane, sum[c]);
                            box_tail(static_cast<float*>(e.out), e.o_ld, g.m, g.n, box, lane, i, j + c * 32, e.accumulate);
                            tma::fence_proxy_async_shared();
                            __syncwarp();
                            if (lane == 0 && j + c * 32 < whole_columns<float>(g.n)) {
                                if (e.accumulate)
                                    add_box(&tp.out, box, j + c * 32, i, 0);
                                else
                                    store_box(&tp.out, box, j + c * 32, i, 0);
                                tma::bulk_commit();
                            }
                        } else {
                            __syncwarp();
                            block_put_row(box, lane, sum[c]);
                            __syncwarp();
                            block_epilogue<KIND>(e, g, batch, i, j + c * 32, box, lane, false, Ahead<KIND>());
                        }
                    }
                }
            } else {
                const int a = fill & 1;
                const bool stream = KIND != KIND_LINEAR && tp.stream;
                const bool pre = KIND == KIND_ACT && e.pre_out;
                const bool in = KIND == KIND_GRAD || (KIND != KIND_LINEAR && e.res);
                auto request = [&](int col) {  // lane 0: what the epilogue of 64 columns from here reads, into the box
                    tma::mbar_arrive_expect_tx(in_bar, kBoxBytes);
                    load_box(box, &tp.in, tma::smem_addr(in_bar), col, i, 0);
                };
                auto arrived = [&]() {
                    ok = __all_sync(0xFFFFFFFFu, tma::mbar_wait(in_bar, in_parity)) && ok;
                    in_parity ^= 1;
                };
                auto send = [&](const CUtensorMap* map, void* to, int64_t ld, int col) {  // the box, complete, to its matrix
                    box_tail(static_cast<__nv_bfloat16*>(to), ld, g.m, g.n, box, lane, i, col, false);
                    tma::fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0 && col < whole_columns<__nv_bfloat16>(g.n)) {
                        store_box(map, box, col, i, 0);
                        tma::bulk_commit();
                    }
                };
                auto box_free = [&]() {  // the copies sent have read the box
                    if (lane == 0) tma::bulk_wait_read<0>();
                    __syncwarp();
                };
                const bool early = stream && in && !pre && i < g.m && j < g.n;
                if (early) {
                    box_free();
                    if (lane == 0) request(j);
                }
                ok = __all_sync(0xFFFFFFFFu, tma::mbar_wait(&acc_full[a], (fill / 2) & 1));
                if (!ok) {
                    if (early) tma::mbar_wait(in_bar, in_parity);  // no copy may land after this CTA has left
                    break;
                }
                ++fill;
                fence_after();
                if (stream) {
#pragma unroll 1
                    for (int c = 0; c < kHalf; c += 64) {
                        const int col = j + c;
                        const bool live = i < g.m && col < g.n;  // the same in the whole warp
                        float v[2][32], bias[32];
                        __syncwarp();
                        if (live) load_bias(e, g.n, col, bias);
                        tmem_ld32(lanes + a * BN + c, v[0]);
                        tmem_ld32(lanes + a * BN + c + 32, v[1]);
                        tmem_wait_ld();
                        if (c + 64 == kHalf) {  // the accumulator is in registers: the next tile may overwrite it
                            fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(a ? drained1 : drained0);
                        }
                        if (!live) continue;
                        DPRED_EACH32(v[0][x] += bias[x];)
                        load_bias(e, g.n, min(col + 32, g.n - 1), bias);
                        DPRED_EACH32(v[1][x] += bias[x];)
                        if (pre) {
                            box_free();
                            box_put(box, lane, 0, v[0]);
                            box_put(box, lane, 1, v[1]);
                            send(&tp.pre, e.pre_out, e.p_ld, col);
                        }
                        box_activate<KIND>(e, v[0]);
                        box_activate<KIND>(e, v[1]);
                        if (!in || pre || c) box_free();  // (a box requested before the accumulator is not in use)
                        if (in) {
                            if ((pre || c) && lane == 0) request(col);
                            arrived();
                            if (!ok) break;
                            box_combine<KIND>(e, box, lane, 0, v[0]);
                            box_combine<KIND>(e, box, lane, 1, v[1]);
                        }
                        if (KIND == KIND_PLAIN && tp.direct && col + 64 <= g.n) {
                            if (i + lane < g.m) {
                                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + (i + lane) * e.o_ld + col;
                                store16_bf16(o, &v[0][0]);
                                store16_bf16(o + 16, &v[0][16]);
                                store16_bf16(o + 32, &v[1][0]);
                                store16_bf16(o + 48, &v[1][16]);
                            }
                            continue;
                        }
                        box_put(box, lane, 0, v[0]);
                        box_put(box, lane, 1, v[1]);
                        send(&tp.out, e.out, e.o_ld, col);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < kHalf; c += 32) {
                        float v[32];
                        __syncwarp();
                        tmem_ld32(lanes + a * BN + c, v);
                        tmem_wait_ld();
                        if (c + 32 == kHalf) {
                            fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(a ? drained1 : drained0);
                        }
                        if (i < g.m && j + c < g.n) {
                            block_put_row(box, lane, v);
                            __syncwarp();
                            block_epilogue<KIND>(e, g, batch, i, j + c, box, lane, false, Ahead<KIND>());
                        }
                    }
                }
            }
        }
        if (lane == 0) tma::bulk_wait<0>();  // shared memory stays valid until its last copy is done
        if (!ok && lane == 0) record_device_error(g.err, DPRED_E_TIMEOUT);
        __syncwarp();
    }
    fence_before();
    cluster_sync();  // no CTA leaves while the other may still signal it or read its shared memory
    if (warp == 1) {
        fence_after();
        tmem_free<2>(tmem, kCols);
    }
}

// ------------------------------------------------------------ host interface --

// One operand: `rows` rows of `cols` 16-bit elements, `ld` elements apart,
// `batch` of them `bstride` elements apart; 16-byte aligned (base and strides).
struct Operand {
    const void* p;
    int64_t rows, cols, ld, bstride;
    bool reduce_rows;  // the reduction runs over the rows (MN-major); else over the columns (K-major)
};

struct Plan {
    Args args;
    Operand a, b;
    float* row_sum;   // args.row_sums: where to (a.reduce_rows)
    int row_sum_add;
    int fp32_result;  // the result is stored in fp32: keep the accumulators' truncation below its precision
};

}  // namespace gemm
}  // namespace dpred
