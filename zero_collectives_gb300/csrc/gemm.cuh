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
    KIND_APPLY = 3,   // Newton-Schulz: the next X, as two fp16 terms
    KIND_FINAL = 4,   // Newton-Schulz: the last X, stored or applied to a weight
};

// A linear layer's epilogue.  In order: t += bias; pre_out = t; t = act(t);
// t += residual; t *= act'(z); t += what the output holds; out = t.
struct LinearEpi {
    void* out;
    const void* bias;
    const __nv_bfloat16* res;
    __nv_bfloat16* pre_out;
    const __nv_bfloat16* z;
    int64_t o_rs, o_cs, r_rs, r_cs, p_rs, p_cs, z_rs, z_cs;  // element strides along i and j
    int out_f32, bias_f32, bias_on_row, act, accumulate;
    int vec;  // every matrix present is contiguous along j with 16-byte aligned rows
};

// One matrix of a Newton-Schulz batch as its last product writes it.
struct FinalOut {
    void* p;
    int64_t rs, cs;   // element strides along i and j
    float step;       // multiplies the orthogonalised value (negative: subtracted from the weight)
    int vec;
};
constexpr int kMaxBatch = 64;  // matrices per Newton-Schulz launch (their output table travels in the launch)

struct NsEpi {
    __half* gram;      // [batch, r, ldr] off-diagonal of X X^T, scaled (in for POLY, out for GRAM)
    __half* poly;      // [batch, r, ldr] off-diagonal of the polynomial, scaled
    float* gram_diag;  // [batch, ldr]
    float* coef;       // [batch, ldr] a + diagonal of the polynomial
    const __half* hi_in;  // [batch, r, ldc]
    const __half* lo_in;
    __half* hi;
    __half* lo;
    int64_t ldr, ldc;
    float alpha;       // multiplies the accumulator
    float off_scale, off_inv;  // GRAM, POLY: scale of the stored off-diagonals (a power of two), its reciprocal
    float a, b, c;     // the polynomial's coefficients
    float keep;        // FINAL: factor of the old weight (0: store)
    int out_f32;       // FINAL
    FinalOut out[kMaxBatch];
};

struct Args {
    int m, n;            // rows of A, rows of B
    int kblocks;         // reduction blocks of kBlockK
    int batch;
    int tiles_m, tiles_n, tiles_per_batch;
    int symmetric;       // only elements i <= j are needed (the epilogue mirrors them)
    int a_mn, b_mn;      // operand majors
    int split;           // CTAs of a cluster that share the reduction
    int regions;         // split kernel: accumulators that share a CTA's part of the reduction
    int bf16;
    int* err;
};

template <int KIND>
struct EpiOf {
    using T = NsEpi;
};
template <>
struct EpiOf<KIND_LINEAR> {
    using T = LinearEpi;
};

// ------------------------------------------------------------- activations --

// The logistic function; its two approximations (exponential and reciprocal,
// both within 2 ulp or so in fp32) are far below the bf16 rounding of what is stored.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// gelu is the tanh form: 0.5 z (1 + tanh(u)) = z * logistic(2 u), u = sqrt(2/pi) (z + 0.044715 z^3).
constexpr float kGeluQ = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

__device__ __forceinline__ float activate(float z, int act) {
    if (act == ACT_RELU) return z > 0.0f ? z : 0.0f;
    if (act == ACT_GELU) return z * logistic(kGeluQ * z * fmaf(kGeluC, z * z, 1.0f));
    if (act == ACT_SILU) return z * logistic(z);
    return z;
}

__device__ __forceinline__ float activate_grad(float z, int act) {
    if (act == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == ACT_GELU) {
        // beyond |z| = 1000 the logistic is 0 or 1 exactly; the clamp keeps z^2 finite there
        const float z2 = fminf(z * z, 1e6f);
        const float p = logistic(kGeluQ * z * fmaf(kGeluC, z2, 1.0f));
        return fmaf(z * p * (1.0f - p), kGeluQ * fmaf(3.0f * kGeluC, z2, 1.0f), p);
    }
    if (act == ACT_SILU) {
        const float p = logistic(z);
        return fmaf(z * p, 1.0f - p, p);
    }
    return 1.0f;
}

// ---------------------------------------------------------------- epilogue --

__device__ __forceinline__ float load_bf16(const __nv_bfloat16* p) { return bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p)); }

__device__ __forceinline__ void load8_bf16(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    f[0] = bf16_lo(q.x); f[1] = bf16_hi(q.x); f[2] = bf16_lo(q.y); f[3] = bf16_hi(q.y);
    f[4] = bf16_lo(q.z); f[5] = bf16_hi(q.z); f[6] = bf16_lo(q.w); f[7] = bf16_hi(q.w);
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

__device__ __forceinline__ void load8_half(const __half* p, float (&f)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        f[2 * k] = t.x;
        f[2 * k + 1] = t.y;
    }
}

__device__ __forceinline__ void store8_half(__half* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

// V consecutive columns of one row (V = 8, or 4 where eight CTAs share 32
// columns).  i < m is guaranteed by the caller; columns past n are skipped.
template <int V>
__device__ __forceinline__ void epilogue(const LinearEpi& e, const Args& g, int batch, int i, int j0, float (&t)[V]) {
    (void)batch;
    const bool whole = V == 8 && e.vec && j0 + 8 <= g.n;
    if (e.bias) {
        if (e.bias_on_row) {
            const float b = e.bias_f32 ? static_cast<const float*>(e.bias)[i]
                                       : load_bf16(static_cast<const __nv_bfloat16*>(e.bias) + i);
#pragma unroll
            for (int c = 0; c < V; ++c) t[c] += b;
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c)
                if (j0 + c < g.n)
                    t[c] += e.bias_f32 ? static_cast<const float*>(e.bias)[j0 + c]
                                       : load_bf16(static_cast<const __nv_bfloat16*>(e.bias) + j0 + c);
        }
    }
    if constexpr (V == 8) {
        if (whole) {
            float f[8];
            if (e.pre_out) store8_bf16(e.pre_out + (int64_t)i * e.p_rs + j0, t);
            if (!e.z && e.act) {
#pragma unroll
                for (int c = 0; c < 8; ++c) t[c] = activate(t[c], e.act);
            }
            if (e.res) {
                load8_bf16(e.res + (int64_t)i * e.r_rs + j0, f);
#pragma unroll
                for (int c = 0; c < 8; ++c) t[c] += f[c];
            }
            if (e.z) {
                load8_bf16(e.z + (int64_t)i * e.z_rs + j0, f);
#pragma unroll
                for (int c = 0; c < 8; ++c) t[c] *= activate_grad(f[c], e.act);
            }
            if (e.out_f32) {
                float* o = static_cast<float*>(e.out) + (int64_t)i * e.o_rs + j0;
                if (e.accumulate) {
                    load8_f32(o, f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) t[c] += f[c];
                }
                store8_f32(o, t);
            } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + (int64_t)i * e.o_rs + j0;
                if (e.accumulate) {
                    load8_bf16(o, f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) t[c] += f[c];
                }
                store8_bf16(o, t);
            }
            return;
        }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int j = j0 + c;
        if (j >= g.n) break;
        float x = t[c];
        if (e.pre_out) e.pre_out[(int64_t)i * e.p_rs + (int64_t)j * e.p_cs] = __float2bfloat16_rn(x);
        if (!e.z) x = activate(x, e.act);
        if (e.res) x += load_bf16(e.res + (int64_t)i * e.r_rs + (int64_t)j * e.r_cs);
        if (e.z) x *= activate_grad(load_bf16(e.z + (int64_t)i * e.z_rs + (int64_t)j * e.z_cs), e.act);
        const int64_t at = (int64_t)i * e.o_rs + (int64_t)j * e.o_cs;
        if (e.out_f32) {
            float* o = static_cast<float*>(e.out) + at;
            *o = e.accumulate ? *o + x : x;
        } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + at;
            *o = __float2bfloat16_rn(e.accumulate ? load_bf16(o) + x : x);
        }
    }
}

// Stores V off-diagonal values of row i and their mirror image (a symmetric
// product computes only i <= j; each pair is written by the one element that
// holds it).  The diagonal itself goes to fp32 elsewhere and is stored as 0.
template <int V>
__device__ __forceinline__ void store_symmetric(__half* d, int64_t ld, const Args& g, int i, int j0,
                                                const float (&t)[V]) {
    if (j0 > i && j0 + V <= g.n && V == 8) {
        float f[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = t[c % V];
        store8_half(d + (int64_t)i * ld + j0, f);
    } else {
#pragma unroll
        for (int c = 0; c < V; ++c)
            if (j0 + c >= i && j0 + c < g.n) d[(int64_t)i * ld + j0 + c] = __float2half_rn(j0 + c == i ? 0.0f : t[c]);
    }
#pragma unroll
    for (int c = 0; c < V; ++c)  // lanes hold consecutive i: one run of the mirrored row
        if (j0 + c > i && j0 + c < g.n) d[(int64_t)(j0 + c) * ld + i] = __float2half_rn(t[c]);
}

template <int KIND, int V>
__device__ __forceinline__ void epilogue_ns(const NsEpi& e, const Args& g, int batch, int i, int j0, float (&t)[V]) {
    if constexpr (KIND == KIND_GRAM) {
        if (j0 + V <= i) return;  // below the diagonal
        __half* d = e.gram + (int64_t)batch * g.m * e.ldr;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const float x = t[c] * e.alpha;
            if (j0 + c == i) e.gram_diag[(int64_t)batch * e.ldr + i] = x;
            t[c] = x * e.off_scale;
        }
        store_symmetric<V>(d, e.ldr, g, i, j0, t);
    } else if constexpr (KIND == KIND_POLY) {
        // With A = D + E (D diagonal, E the stored off-diagonal):
        //   A^2 = D^2 + D E + E D + E^2, so off the diagonal
        //   (b A + c A^2)_ij = (b + c (d_i + d_j)) E_ij + c (E^2)_ij
        // and on it b d_i + c d_i^2 + c (E^2)_ii.
        if (j0 + V <= i) return;
        const float* diag = e.gram_diag + (int64_t)batch * e.ldr;
        const __half* a = e.gram + ((int64_t)batch * g.m + i) * e.ldr + j0;
        const float di = diag[i];
        float x[8], dj[8];
        if (V == 8) {  // rows and diagonals are padded to a multiple of 8
            if (j0 >= g.n) return;
            load8_half(a, x);
            load8_f32(diag + j0, dj);
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                x[c] = j0 + c < g.n ? __half2float(a[c]) : 0.0f;
                dj[c] = j0 + c < g.n ? diag[j0 + c] : 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const float sq = t[c] * e.alpha;
            if (j0 + c == i) e.coef[(int64_t)batch * e.ldr + i] = e.a + fmaf(e.c, fmaf(di, di, sq), e.b * di);
            t[c] = fmaf(fmaf(e.c, di + dj[c], e.b), x[c] * e.off_inv, e.c * sq) * e.off_scale;
        }
        store_symmetric<V>(e.poly + (int64_t)batch * g.m * e.ldr, e.ldr, g, i, j0, t);
    } else {
        // X' = (a + diagonal) X + E X: the large part of the polynomial is its
        // diagonal, which multiplies X in full precision (both fp16 terms).
        const float k = e.coef[(int64_t)batch * e.ldr + i];
        const int64_t at = ((int64_t)batch * g.m + i) * e.ldc + j0;
        static_assert(V == 8 || V == 4, "column groups");
        float hi[8], lo[8];
        if constexpr (V == 8) {
            if (j0 >= g.n) return;
            load8_half(e.hi_in + at, hi);  // rows are padded to a multiple of 8 columns
            load8_half(e.lo_in + at, lo);
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const bool in = j0 + c < g.n;
                hi[c] = in ? __half2float(e.hi_in[at + c]) : 0.0f;
                lo[c] = in ? __half2float(e.lo_in[at + c]) : 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < V; ++c) t[c] = fmaf(k, hi[c] + lo[c], t[c] * e.alpha);
        if constexpr (KIND == KIND_APPLY) {
            float h[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) h[c] = c < V ? __half2float(__float2half_rn(t[c % V])) : 0.0f;
            if constexpr (V == 8) {
                store8_half(e.hi + at, h);
#pragma unroll
                for (int c = 0; c < 8; ++c) h[c] = t[c] - h[c];
                store8_half(e.lo + at, h);
            } else {
#pragma unroll
                for (int c = 0; c < V; ++c)
                    if (j0 + c < g.n) {
                        e.hi[at + c] = __float2half_rn(t[c]);
                        e.lo[at + c] = __float2half_rn(t[c] - h[c]);
                    }
            }
        } else {
            const FinalOut& f = e.out[batch];
            if (V == 8 && f.vec && j0 + 8 <= g.n) {
                const int64_t o = (int64_t)i * f.rs + j0;
                float w[8], x[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) x[c] = t[c % V] * f.step;
                if (e.out_f32) {
                    float* p = static_cast<float*>(f.p) + o;
                    if (e.keep != 0.0f) {
                        load8_f32(p, w);
#pragma unroll
                        for (int c = 0; c < 8; ++c) x[c] = fmaf(e.keep, w[c], x[c]);
                    }
                    store8_f32(p, x);
                } else {
                    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(f.p) + o;
                    if (e.keep != 0.0f) {
                        load8_bf16(p, w);
#pragma unroll
                        for (int c = 0; c < 8; ++c) x[c] = fmaf(e.keep, w[c], x[c]);
                    }
                    store8_bf16(p, x);
                }
                return;
            }
#pragma unroll
            for (int c = 0; c < V; ++c) {
                if (j0 + c >= g.n) break;
                const int64_t o = (int64_t)i * f.rs + (int64_t)(j0 + c) * f.cs;
                float x = t[c] * f.step;
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
}

template <int KIND, int V>
__device__ __forceinline__ void apply_epilogue(const typename EpiOf<KIND>::T& e, const Args& g, int batch, int i, int j0,
                                               float (&t)[V]) {
    if constexpr (KIND == KIND_LINEAR)
        epilogue<V>(e, g, batch, i, j0, t);
    else
        epilogue_ns<KIND, V>(e, g, batch, i, j0, t);
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
// accumulator in tensor memory, added in fp32 registers at the end: the tensor
// cores' accumulators truncate, about 1.9e-8 of the sum per 16-element step.

constexpr int kSplitThreads = 192;  // producer warp, issuing warp, four epilogue warps

template <int BN>
__host__ __device__ constexpr int split_stages() {
    return BN == 32 ? 5 : BN == 64 ? 4 : 3;
}
template <int BN>
__host__ __device__ constexpr int split_smem() {  // stages + alignment; barriers are static
    return split_stages<BN>() * (128 * 128 + BN * 128) + 1024;
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

// Adds V columns of one row over the cluster's partial tiles, in rank order.
template <int KIND, int V>
__device__ __forceinline__ void reduce_columns(const typename EpiOf<KIND>::T& e, const Args& g, int batch, int i, int j0,
                                               uint32_t at) {
    float t[V];
#pragma unroll
    for (int x = 0; x < V; ++x) t[x] = 0.0f;
    for (int p = 0; p < g.split; ++p) {
        const uint32_t from = mma::map_rank(at, p);
#pragma unroll
        for (int x = 0; x < V; ++x) t[x] += mma::ld_cluster(from + x * 512);
    }
    apply_epilogue<KIND, V>(e, g, batch, i, j0, t);
}

template <int KIND, int BN>
__global__ void __launch_bounds__(kSplitThreads)
    split_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const __grid_constant__ Args g, const __grid_constant__ typename EpiOf<KIND>::T e) {
    using namespace mma;
    constexpr int S = split_stages<BN>();
    constexpr uint32_t kA = 128 * 128, kStage = kA + BN * 128;
    constexpr uint32_t kCols = 256;  // two CTAs per SM together allocate all 512
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[S], empty[S], done;
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
    const int regions = min(g.regions, nkb);

    if (threadIdx.x == 0) {
        if (g.kblocks) {
            prefetch_map(&ma);
            prefetch_map(&mb);
        }
        for (int s = 0; s < S; ++s) {
            tma::mbar_init(&full[s], 1);
            tma::mbar_init(&empty[s], 1);
        }
        tma::mbar_init(&done, 1);
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<1>(tma::smem_addr(&tmem_slot), kCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    grid_launch_dependents();
    grid_wait();

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int it = 0; it < nkb; ++it) {
                const int s = it % S;
                if (it >= S && !tma::mbar_wait(&empty[s], (it / S - 1) & 1)) {
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
            }
            if (!ok)  // let the copies in flight land before the CTA can leave
                for (int it = issued > S ? issued - S : 0; it < issued; ++it) tma::mbar_wait(&full[it % S], (it / S) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = instr_desc(128, BN, g.bf16, g.a_mn, g.b_mn);
            int region = 0;
            for (int it = 0; it < nkb; ++it) {
                const int s = it % S;
                bool first = it == 0;
                if (region + 1 < regions && it >= nkb * (region + 1) / regions) {
                    ++region;
                    first = true;
                }
                if (!tma::mbar_wait(&full[s], (it / S) & 1)) {
                    record_device_error(g.err, DPRED_E_TIMEOUT);
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t a = base + s * kStage, b = a + kA;
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k) {
                    const uint64_t da = operand_desc(a + (g.a_mn ? k * 2048 : k * 32), g.a_mn);
                    const uint64_t db = operand_desc(b + (g.b_mn ? k * 2048 : k * 32), g.b_mn);
                    issue<1>(tmem + region * BN, da, db, idesc, !first || k != 0);
                }
                commit<1>(tma::smem_addr(&empty[s]));
            }
            if (ok && nkb) commit<1>(tma::smem_addr(&done));
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // tensor-memory lanes 32 q .. 32 q + 31 belong to this warp
        if (nkb && !tma::mbar_wait(&done, 0)) {
            record_device_error(g.err, DPRED_E_TIMEOUT);
            ok = false;
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        fence_after();
        const int r = q * 32 + lane, i = tm * 128 + r;
        if (g.split == 1) {
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 32) {
                float v[32];
                __syncwarp();
                read_regions<BN>(tmem + ((uint32_t)(q * 32) << 16) + c0, ok ? regions : 0, v);
                if (i < g.m && ok) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        float t[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) t[x] = v[c + x];
                        apply_epilogue<KIND, 8>(e, g, batch, i, tn * BN + c0 + c, t);
                    }
                }
            }
        } else {
            // partial tile to this CTA's shared memory, column by column (the
            // pipeline's stages are free: every load was consumed)
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 32) {
                float v[32];
                __syncwarp();
                read_regions<BN>(tmem + ((uint32_t)(q * 32) << 16) + c0, ok ? regions : 0, v);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((c0 + c) * 128 + r) * 4), "f"(v[c]) : "memory");
            }
        }
        fence_before();
    }
    if (g.split > 1) {
        cluster_sync();
        if (warp >= 2) {
            const int r = (warp & 3) * 32 + lane, i = tm * 128 + r;
            const int per = BN / g.split, c_lo = rank * per;
            if (i < g.m && ok) {
                if (per % 8 == 0) {
                    for (int c = 0; c < per; c += 8) reduce_columns<KIND, 8>(e, g, batch, i, tn * BN + c_lo + c, base + ((c_lo + c) * 128 + r) * 4);
                } else {
                    for (int c = 0; c < per; c += 4) reduce_columns<KIND, 4>(e, g, batch, i, tn * BN + c_lo + c, base + ((c_lo + c) * 128 + r) * 4);
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

constexpr int kTileThreads = 320;  // producer warp, issuing warp, eight epilogue warps
constexpr int kPromoteBlocks = 8;

template <int BN>
__host__ __device__ constexpr int tile_stages() {
    return BN == 256 ? 6 : 8;
}
template <int BN>
__host__ __device__ constexpr int tile_smem() {
    return tile_stages<BN>() * (128 * 128 + BN / 2 * 128) + 1024;
}

template <int KIND, int BN, bool PROMOTE>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ Args g, const __grid_constant__ typename EpiOf<KIND>::T e) {
    using namespace mma;
    constexpr int S = tile_stages<BN>();
    constexpr uint32_t kA = 128 * 128, kB = BN / 2 * 128, kStage = kA + kB;
    constexpr uint32_t kCols = 2 * BN;
    constexpr int kHalf = BN / 2;  // columns per epilogue warp
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int total = g.tiles_per_batch * g.batch;
    const int chunk = PROMOTE ? kPromoteBlocks : g.kblocks;

    if (threadIdx.x == 0) {
        prefetch_map(&ma);
        prefetch_map(&mb);
        for (int s = 0; s < S; ++s) {
            tma::mbar_init(&full[s], 1);   // the even CTA's expected bytes (both CTAs' copies)
            tma::mbar_init(&empty[s], 1);  // the issuing thread's commit
        }
        for (int a = 0; a < 2; ++a) {
            tma::mbar_init(&acc_full[a], 1);
            tma::mbar_init(&acc_empty[a], 16);  // eight epilogue warps of each CTA
        }
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<2>(tma::smem_addr(&tmem_slot), kCols);
    fence_before();
    cluster_sync();
    fence_after();
    const uint32_t tmem = tmem_slot;
    grid_launch_dependents();
    grid_wait();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += pairs) {
                const int batch = tile / g.tiles_per_batch;
                int tm, tn;
                tile_at(g, tile - batch * g.tiles_per_batch, 256, BN, tm, tn);
                const int i0 = tm * 256 + (int)rank * 128, j0 = tn * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < g.kblocks; ++kb, ++it) {
                    const int s = it % S;
                    if (it >= S && !tma::mbar_wait(&empty[s], (it / S - 1) & 1)) {
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
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = instr_desc(256, BN, g.bf16, g.a_mn, g.b_mn);
            int it = 0, fill = 0;
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
                    for (int first = kb; kb < stop; ++kb, ++it) {
                        const int s = it % S;
                        if (!tma::mbar_wait(&full[s], (it / S) & 1)) {
                            record_device_error(g.err, DPRED_E_TIMEOUT);
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint32_t pa = base + s * kStage, pb = pa + kA;
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k) {
                            const uint64_t da = operand_desc(pa + (g.a_mn ? k * 2048 : k * 32), g.a_mn);
                            const uint64_t db = operand_desc(pb + (g.b_mn ? k * 2048 : k * 32), g.b_mn);
                            issue<2>(tmem + a * BN, da, db, idesc, kb != first || k != 0);
                        }
                        commit<2>(tma::smem_addr(&empty[s]));
                    }
                    if (ok) commit<2>(tma::smem_addr(&acc_full[a]));
                }
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) / 4;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * kHalf;
        const uint32_t drained0 = map_rank(tma::smem_addr(&acc_empty[0]), 0), drained1 = map_rank(tma::smem_addr(&acc_empty[1]), 0);
        int fill = 0;
        bool ok = true;
        for (int tile = pair; tile < total && ok; tile += pairs) {
            const int batch = tile / g.tiles_per_batch;
            int tm, tn;
            tile_at(g, tile - batch * g.tiles_per_batch, 256, BN, tm, tn);
            const int i = tm * 256 + (int)rank * 128 + q * 32 + lane, j = tn * BN + half * kHalf;
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
                    for (int c = 0; c < kHalf / 32; ++c) {
                        float v[32];
                        tmem_ld32(lanes + a * BN + c * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) sum[c][x] += v[x];
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(a ? drained1 : drained0);
                }
                if (ok && i < g.m) {
#pragma unroll
                    for (int c = 0; c < kHalf / 8; ++c) {
                        float t[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) t[x] = sum[c / 4][(c % 4) * 8 + x];
                        if (j + c * 8 < g.n) apply_epilogue<KIND, 8>(e, g, batch, i, j + c * 8, t);
                    }
                }
            } else {
                const int a = fill & 1;
                ok = __all_sync(0xFFFFFFFFu, tma::mbar_wait(&acc_full[a], (fill / 2) & 1));
                if (!ok) break;
                ++fill;
                fence_after();
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 32) {
                    float v[32];
                    __syncwarp();
                    tmem_ld32(lanes + a * BN + c, v);
                    tmem_wait_ld();
                    if (c + 32 == kHalf) {  // the accumulator is in registers: the next tile may overwrite it
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(a ? drained1 : drained0);
                    }
                    if (i < g.m && j + c < g.n) {
#pragma unroll
                        for (int x = 0; x < 32; x += 8) {
                            float t[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) t[y] = v[x + y];
                            apply_epilogue<KIND, 8>(e, g, batch, i, j + c + x, t);
                        }
                    }
                }
            }
        }
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
    int fp32_result;  // the result is stored in fp32: keep the accumulators' truncation below its precision
};

}  // namespace gemm
}  // namespace dpred
