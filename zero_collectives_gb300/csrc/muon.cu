// muon.cu -- orthogonalised updates: dpred_newton_schulz and dpred_muon_step.
//
// Reduce-to-owner (DeepSpeed issue #8700) leaves every whole reduced gradient
// matrix on one rank, which is what this update needs: it mixes all rows and
// columns of a matrix.  For a matrix G with r = min(rows, cols):
//
//     X = U / (|U|_F + eps)                     U = G, or the momentum's
//     repeat:  A = X X^T  (r x r)
//              X = a X + (b A + c A^2) X
//
// (X on its wide side; the polynomial is odd, so the transpose commutes with it.)
//
// Precision.  What limits a step's result is the rounding of X and of the
// polynomial to the 16 bits that the matrix instructions take.  Three choices
// keep the products at the 16-bit rate with an error of 2e-4 to 1e-3 of the
// result (against 1e-2 to 3e-2 with bf16 everywhere, 1e-3 to 4e-3 with plain fp16):
//  - operands are fp16 (11 significant bits, bf16 has 8); X is scaled by a
//    power of two near sqrt(cols), which brings its entries near 1;
//  - the diagonals of A and of the polynomial stay in fp32: the polynomial is
//    near a multiple of the identity, so its diagonal is the only large part;
//  - X carries a second, 8-bit term (about 15 bits together), and that diagonal
//    multiplies both: only the products with the small off-diagonal part and the
//    Gram product see the leading term alone.
// Sums, norms, diagonals and accumulators are fp32.
//
// A and the polynomial are symmetric: only tiles that hold an element i <= j
// are computed, and the epilogue writes each value twice.
#include <algorithm>
#include <cmath>
#include <vector>

#include "gemm_host.cuh"
#include "muon_chain.cuh"
#include "muon_small.cuh"

namespace dpred {
namespace gemm {
namespace {

constexpr int kMaxSteps = 32;
constexpr int kNormBlocks = 256;  // partial sums of squares per matrix (at most)
constexpr int kTile = 64;         // the element-wise passes transpose tiles of 64 x 64

// How a block of the element-wise passes covers a tile of 4096 elements: a
// thread has 4 columns of every `step`-th row, four times.
struct Pass {
    int r, c, step, width;
    __device__ __forceinline__ explicit Pass(bool square) {
        const int shift = square ? 4 : 6;  // 64 x 64, or 16 x 256: whole kilobytes of a row
        r = threadIdx.x >> shift;
        c = (threadIdx.x & ((1 << shift) - 1)) * 4;
        step = 256 >> shift;
        width = 4 << shift;
    }
};

// One matrix of a launch as the element-wise passes see it.
struct MatIn {
    const void* g;
    float* mom;        // null: U = G
    int64_t ldg, ldm;
    int transposed;    // X is the transpose (more rows than columns)
    int g_vec, m_vec;  // 4-element groups of G / the momentum are aligned
};

struct NormArgs {
    MatIn in[kMaxBatch];
    int64_t r, c;             // X is r x c, r <= c; the caller's matrix is that or its transpose
    float mu;
    int nesterov;
    float* partial;           // [batch, kNormBlocks]
    unsigned* counter;        // [batch] finished tiles of the chained products, cleared here
    int blocks;               // partials written per matrix
    float eps, scale;
    __half* hi;               // [batch, r, ldc]
    uint8_t* lo;
    int64_t ldc;
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, int valid, bool vec, float (&f)[4]) {
    if (vec && valid >= 4) {
        if constexpr (sizeof(T) == 2) {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            f[0] = bf16_lo(q.x); f[1] = bf16_hi(q.x); f[2] = bf16_lo(q.y); f[3] = bf16_hi(q.y);
        } else {
            const float4 q = *reinterpret_cast<const float4*>(p);
            f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        f[c] = 0.0f;
        if (c < valid) {
            if constexpr (sizeof(T) == 2)
                f[c] = load_bf16(reinterpret_cast<const __nv_bfloat16*>(p) + c);
            else
                f[c] = reinterpret_cast<const float*>(p)[c];
        }
    }
}

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float warps[8];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < 8; ++w) v += warps[w];
    return v;
}

// m = mu m + g (written back), u = g + mu m or m; the block's share of |U|^2.
// Bandwidth bound: reads g and m and writes m once.
template <typename Tg>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ NormArgs a) {
    mma::grid_launch_dependents();
    mma::grid_wait();
    const MatIn& in = a.in[blockIdx.y];
    const Tg* g = static_cast<const Tg*>(in.g);
    const int64_t rows = in.transposed ? a.c : a.r, cols = in.transposed ? a.r : a.c;
    const Pass p(false);
    const int64_t tr = (rows + 4 * p.step - 1) / (4 * p.step), tc = (cols + p.width - 1) / p.width;
    float sum = 0.0f;
    for (int64_t t = blockIdx.x; t < tr * tc; t += gridDim.x) {
        const int64_t i0 = t / tc * 4 * p.step + p.r, j = t % tc * p.width + p.c;
        const int valid = (int)(cols - j);
        if (valid <= 0) continue;
        float gv[4][4], mv[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + p.step * u;
            if (i < rows) {
                load4(g + i * in.ldg + j, valid, in.g_vec, gv[u]);
                if (in.mom) load4(in.mom + i * in.ldm + j, valid, in.m_vec, mv[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + p.step * u;
            if (i >= rows) continue;
            if (in.mom) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mv[u][k] = fmaf(a.mu, mv[u][k], gv[u][k]);
                    gv[u][k] = a.nesterov ? fmaf(a.mu, mv[u][k], gv[u][k]) : mv[u][k];
                }
                float* m = in.mom + i * in.ldm + j;
                if (in.m_vec && valid >= 4) {
                    *reinterpret_cast<float4*>(m) = make_float4(mv[u][0], mv[u][1], mv[u][2], mv[u][3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < valid) m[k] = mv[u][k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < valid) sum = fmaf(gv[u][k], gv[u][k], sum);
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        a.partial[blockIdx.y * kNormBlocks + blockIdx.x] = sum;
        if (blockIdx.x == 0) a.counter[blockIdx.y] = 0;
    }
}

// X = scale * U / (|U| + eps) on its wide side, as two terms (see split8).  The
// partial sums are added in one fixed order by every block.
template <typename Tg>
__global__ void __launch_bounds__(256, 8) scale_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float tile[kTile][kTile + 1];
    mma::grid_launch_dependents();
    mma::grid_wait();
    const MatIn& in = a.in[blockIdx.y];
    const Tg* g = static_cast<const Tg*>(in.g);
    const float total = block_sum(threadIdx.x < a.blocks ? a.partial[blockIdx.y * kNormBlocks + threadIdx.x] : 0.0f);
    const float f = norm_factor(a.scale, total, a.eps);
    const int64_t rows = in.transposed ? a.c : a.r, cols = in.transposed ? a.r : a.c;
    const Pass p(in.transposed);
    const int64_t tr = (rows + 4 * p.step - 1) / (4 * p.step), tc = (cols + p.width - 1) / p.width;
    const int64_t xr = a.r, xc = a.c;
    __half* hi = a.hi + (int64_t)blockIdx.y * xr * a.ldc;
    uint8_t* lo = a.lo + (int64_t)blockIdx.y * xr * a.ldc;
    const int r = p.r, c = p.c;
    for (int64_t t = blockIdx.x; t < tr * tc; t += gridDim.x) {
        const int64_t i0 = t / tc * 4 * p.step, j0 = t % tc * p.width;
        float x[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + r + p.step * u;
            const int valid = (int)(cols - j0 - c);
            if (i < rows && valid > 0) {
                float m[4];
                load4(g + i * in.ldg + j0 + c, valid, in.g_vec, x[u]);
                if (in.mom) load4(in.mom + i * in.ldm + j0 + c, valid, in.m_vec, m);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (in.mom) x[u][k] = a.nesterov ? fmaf(a.mu, m[k], x[u][k]) : m[k];
                    x[u][k] *= f;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[u][k] = 0.0f;
            }
        }
        if (in.transposed) {
            __syncthreads();
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) tile[r + 16 * u][c + k] = x[u][k];
            __syncthreads();
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) x[u][k] = tile[c + k][r + 16 * u];
        }
        const int64_t xi0 = in.transposed ? j0 : i0, xj = (in.transposed ? i0 : j0) + c;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = xi0 + r + p.step * u;
            if (i >= xr || xj >= xc) continue;  // rows are padded to 8 columns, so a group of 4 always fits
            const float t[8] = {x[u][0], x[u][1], x[u][2], x[u][3]};
            uint4 h;
            uint2 l;
            split8(t, h, l);
            *reinterpret_cast<uint2*>(hi + i * a.ldc + xj) = make_uint2(h.x, h.y);
            *reinterpret_cast<uint32_t*>(lo + i * a.ldc + xj) = l.x;
        }
    }
}

// -------------------------------------------------------------------- host --

int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }
int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// One matrix of a call, in the caller's order and orientation.
struct Item {
    MatIn in;
    void* out;
    int64_t rows, cols, ldo;
    float step;  // factor of the orthogonalised value in the output
};

struct Layout {
    int64_t r, c, ldr, ldc;
    int64_t x, gram, diag, per;  // bytes of one leading term of X, of one r x r matrix, of one diagonal, of everything per matrix
};

Layout layout_of(int64_t rows, int64_t cols) {
    Layout l;
    l.r = std::min(rows, cols);
    l.c = std::max(rows, cols);
    l.ldr = round8(l.r);
    l.ldc = round8(l.c);
    l.x = l.r * l.ldc * 2;
    l.gram = l.r * l.ldr * 2;
    l.diag = l.ldr * 4;
    // X: leading term twice (read and written by the same product), trailing term; four r x r matrices and their
    // diagonals; partial sums; counter
    l.per = 2 * l.x + l.x / 2 + kSquares * (l.gram + l.diag) + kNormBlocks * 4 + 4;
    return l;
}
constexpr int kRegions = 5 + 2 * kSquares;  // regions of a group's workspace, each rounded up to 256 bytes

int64_t group_bytes(const Layout& l, int count) { return l.per * count + 256 * kRegions; }

struct Params {
    int g_dtype, out_dtype, nesterov, steps;
    float mu, keep, eps, a, b, c;
};

// The matrices of one shape (or of its transpose) in one launch.
struct Group {
    const Item* const* items;
    int count;
    Layout l;
    // workspace
    __half *hi[2], *square[kSquares];
    uint8_t* lo;
    float *diag[kSquares], *partial;
    unsigned* counter;
    float scale;
};

void place(Group& g, char*& ws) {
    auto take = [&](int64_t bytes) {
        char* p = ws;
        ws += align256(bytes);
        return p;
    };
    const Layout& l = g.l;
    g.hi[0] = reinterpret_cast<__half*>(take(l.x * g.count));
    g.hi[1] = reinterpret_cast<__half*>(take(l.x * g.count));
    g.lo = reinterpret_cast<uint8_t*>(take(l.x / 2 * g.count));
    for (int k = 0; k < kSquares; ++k) {
        g.square[k] = reinterpret_cast<__half*>(take(l.gram * g.count));
        g.diag[k] = reinterpret_cast<float*>(take(l.diag * g.count));
    }
    g.partial = reinterpret_cast<float*>(take((int64_t)kNormBlocks * 4 * g.count));
    // entries of X: near 1 after scaling by about sqrt(c); an orthogonal row of length c has entries near 1/sqrt(c)
    g.scale = std::exp2(std::round(0.5f * std::log2((float)std::min<int64_t>(l.c, 65536))));
}

// The element-wise passes: momentum, norm, X as two fp16 terms.
int start_group(const Group& g, const Params& q, cudaStream_t s) {
    const Layout& l = g.l;
    NormArgs n = {};
    n.r = l.r;
    n.c = l.c;
    n.mu = q.mu;
    n.nesterov = q.nesterov;
    n.partial = g.partial;
    n.counter = g.counter;
    n.eps = q.eps;
    n.scale = g.scale;
    n.hi = g.hi[0];
    n.lo = g.lo;
    n.ldc = l.ldc;
    const int gs = q.g_dtype == DPRED_F32 ? 4 : 2;
    for (int k = 0; k < g.count; ++k) {
        MatIn& in = n.in[k];
        in = g.items[k]->in;
        in.transposed = g.items[k]->rows > g.items[k]->cols;
        in.g_vec = reinterpret_cast<uintptr_t>(in.g) % (4 * gs) == 0 && (g.items[k]->rows <= 1 || in.ldg % 4 == 0);
        in.m_vec = reinterpret_cast<uintptr_t>(in.mom) % 16 == 0 && (g.items[k]->rows <= 1 || in.ldm % 4 == 0);
    }
    const int64_t tiles = ((l.r + kTile - 1) / kTile) * ((l.c + kTile - 1) / kTile);
    // the norm's blocks are resident at once (four to an SM); the scaling's, of a tile each, follow one another
    const int64_t resident = std::max<int64_t>(1, 4 * sm_count() / g.count);
    n.blocks = (int)std::min<int64_t>(std::min<int64_t>(tiles, kNormBlocks), resident);
    const dim3 grid1((unsigned)n.blocks, (unsigned)g.count);
    const dim3 grid2((unsigned)std::min<int64_t>(tiles, 65536), (unsigned)g.count);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid1;
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const bool f32 = q.g_dtype == DPRED_F32;
    cudaError_t err = cudaLaunchKernelEx(&cfg, f32 ? norm_kernel<float> : norm_kernel<__nv_bfloat16>, n);
    cfg.gridDim = grid2;
    if (err == cudaSuccess) err = cudaLaunchKernelEx(&cfg, f32 ? scale_kernel<float> : scale_kernel<__nv_bfloat16>, n);
    return err == cudaSuccess ? DPRED_OK : cuda_error(err, "orthogonalised update launch");
}

NsEpi epilogue_of_group(const Group& g, const Params& q) {
    NsEpi e = {};
    e.gram = g.square[0];
    e.poly = g.square[1];
    e.gram_diag = g.diag[0];
    e.coef = g.diag[1];
    e.lo = g.lo;
    e.ldr = g.l.ldr;
    e.ldc = g.l.ldc;
    e.a = q.a;
    e.b = q.b;
    e.c = q.c;
    e.keep = q.keep;
    e.out_f32 = q.out_dtype == DPRED_F32;
    e.alpha = 1.0f / (g.scale * g.scale);
    return e;
}

FinalOut output_of(const Group& g, int k, const Params& q) {
    const Item& it = *g.items[k];
    FinalOut o;
    o.p = it.out;
    o.ld = it.ldo;
    o.step = it.step / g.scale;
    o.vec = reinterpret_cast<uintptr_t>(o.p) % 16 == 0 && (it.rows <= 1 || o.ld * (q.out_dtype == DPRED_F32 ? 4 : 2) % 16 == 0);
    o.transposed = it.rows > it.cols;
    return o;
}

int blocks_of(int64_t n) { return (int)((n + mma::kBlockK - 1) / mma::kBlockK); }

// A group's products of one step: 0 Gram, 1 polynomial, 2 apply.
Plan product_plan(const Group& g, int product, int buffer) {
    const Layout& l = g.l;
    Plan p = {};
    p.args.batch = g.count;
    p.args.err = device_error_word();
    p.args.m = (int)l.r;
    p.args.n = (int)(product == 2 ? l.c : l.r);
    p.args.symmetric = product < 2;
    p.args.b_mn = product == 2;
    p.args.kblocks = blocks_of(product == 0 ? l.c : l.r);
    p.args.split_only = 1;
    const Operand x = {g.hi[buffer], l.r, l.c, l.ldc, l.r * l.ldc, product == 2};
    const Operand a = {g.square[product == 1 ? 0 : 1], l.r, l.r, l.ldr, l.r * l.ldr, false};
    p.a = product == 0 ? x : a;
    p.b = product == 1 ? a : x;
    return p;
}

// One launch per product: the matrices of a group that are too small, or too few, for the chained kernel.
// last: nothing of the call follows this group.
int run_products(const Group& g, const Params& q, bool last, cudaStream_t s) {
    NsParams n = {};
    NsEpi& e = n.e;
    e = epilogue_of_group(g, q);
    for (int k = 0; k < g.count; ++k) n.table[k] = output_of(g, k, q);
    for (int step = 0; step < q.steps; ++step) {
        Plan p = product_plan(g, 0, step & 1);
        p.args.release = 1;
        int rc = run<KIND_GRAM>(p, n, s);
        if (rc != DPRED_OK) return rc;
        p = product_plan(g, 1, step & 1);
        p.args.release = 1;
        rc = run<KIND_POLY>(p, n, s);
        if (rc != DPRED_OK) return rc;
        e.hi_in = g.hi[step & 1];
        e.hi = g.hi[(step + 1) & 1];
        p = product_plan(g, 2, step & 1);
        p.args.release = !last || step + 1 < q.steps;
        rc = step + 1 < q.steps ? run<KIND_APPLY>(p, n, s) : run<KIND_FINAL>(p, n, s);
        if (rc != DPRED_OK) return rc;
    }
    return DPRED_OK;
}

// A matrix's products.  A plain step is Gram, polynomial, apply.  A double
// step works out two steps from one Gram product: with P = p(A), the next Gram
// matrix is A' = P A P (everything is a polynomial of A and commutes), so
//     A, P = p(A), T = P A, A' = P T, P' = p(A'), Q = P' P, X = Q X
// reads and writes X once and trades a Gram and an apply product (3 r^2 c flops,
// the symmetric halves counted) for three r x r ones (3 r^3).  A' inherits A's
// rounding, amplified for the small singular values as one more plain step
// would amplify X's; three steps in a row measured 1.2e-3 to 1.9e-3, two 2e-4 to 1e-3.
// Matrices: 0 = A, A'; 1 = P; 2 = T, Q; 3 = P'.
int chain_program(ChainOp* op, int steps, bool pairs) {
    int n = 0;
    uint8_t x = 0, squares = 0, applies = 0;
    auto add = [&](uint8_t kind, uint8_t a, uint8_t b, uint8_t out) {
        op[n++] = {kind, a, b, out, x, squares, applies, 0};
        if (kind < CHAIN_APPLY)
            ++squares;
        else
            ++applies;
    };
    while (steps > 0) {
        const bool two = pairs && steps >= 2;
        steps -= two ? 2 : 1;
        add(CHAIN_GRAM, 0, 0, 0);
        add(CHAIN_POLY, 0, 0, 1);
        if (two) {
            add(CHAIN_MUL, 1, 0, 2);
            add(CHAIN_MUL, 1, 2, 0);
            add(CHAIN_POLY, 0, 0, 3);
            add(CHAIN_MUL, 3, 1, 2);
        }
        add(steps ? CHAIN_APPLY : CHAIN_FINAL, two ? 2 : 1, 0, 0);
        x ^= 1;
    }
    return n;
}

// Double steps pay where the products with X are much the longer ones (plain
// -> double): 6 of 1024 x 4096 437 -> 393 us, 6 of 300 x 3000 241 -> 221, 12 of
// 512 x 2048 233 -> 237; 4 of 1024 x 2048 234 -> 251, 8 of 1024 x 1024 223 -> 252.
bool double_steps(const Layout& l) { return l.c >= 3 * l.r; }

int run_chained(const std::vector<Group>& groups, const Params& q, cudaStream_t s) {
    ChainArgs a = {};
    a.groups = (int)groups.size();
    a.counter = groups[0].counter;  // the groups' counters are neighbours
    a.err = device_error_word();
    const int ops[2] = {chain_program(a.program[0], q.steps, false), chain_program(a.program[1], q.steps, true)};
    int first = 0, squares = 0, applies = 0;
    for (size_t i = 0; i < groups.size(); ++i) {
        const Group& g = groups[i];
        ChainGroup& d = a.g[i];
        for (int k = 0; k < 2; ++k) {
            Operand x = {g.hi[k], g.l.r, g.l.c, g.l.ldc, g.l.r * g.l.ldc, false};
            int rc = make_map(x, g.count, 128, false, &d.x[k]);
            if (rc != DPRED_OK) return rc;
            x.reduce_rows = true;
            if ((rc = make_map(x, g.count, 128, false, &d.xt[k])) != DPRED_OK) return rc;
            d.hi[k] = g.hi[k];
        }
        for (int k = 0; k < kSquares; ++k) {
            for (int t = 0; t < 2; ++t) {
                const Operand m = {g.square[k], g.l.r, g.l.r, g.l.ldr, g.l.r * g.l.ldr, t == 1};
                const int rc = make_map(m, g.count, 128, false, &d.square[k][t]);
                if (rc != DPRED_OK) return rc;
            }
            d.sq[k] = g.square[k];
            d.diag[k] = g.diag[k];
        }
        d.e = epilogue_of_group(g, q);
        d.r = (int)g.l.r;
        d.c = (int)g.l.c;
        d.count = g.count;
        d.first = first;
        d.tiles_r = (d.r + 255) / 256;
        d.tiles_c = (d.c + 255) / 256;
        d.square_tiles = d.tiles_r * (d.tiles_r + 1) / 2;
        d.program = double_steps(g.l);
        d.ops = ops[d.program];
        a.ops = std::max(a.ops, d.ops);
        squares += d.square_tiles * d.count;
        applies += d.tiles_r * d.tiles_c * d.count;
        for (int k = 0; k < g.count; ++k) a.out[first + k] = output_of(g, k, q);
        first += g.count;
    }
    a.most = std::max(squares, applies);
    return run_chain(a, s);
}

// Estimated times (us) of the two ways, fitted to batches of 1 to 12 matrices
// from 160 x 2500 to 2048 x 4096 (most within 12%).  The chained kernel is bound
// by one matrix's chain of products (a tile costs 0.3 a reduction block and 5.5 to
// start, drain and hand over) and by its tiles' total over the CTA pairs.
// Either side, chained against one by one: 1 of 1024 x 1024 171 and 126 us, 3 of
// them 175 and 189, 12 of them 263 and 550.
double chained_time(const std::vector<Group>& groups, int steps) {
    double work = 0, chain = 0;
    for (const Group& g : groups) {
        const double tr = (double)((g.l.r + 255) / 256), tc = (double)((g.l.c + 255) / 256), sym = tr * (tr + 1) / 2;
        const double kc = 0.3 * blocks_of(g.l.c), kr = 0.3 * blocks_of(g.l.r);
        const int twos = double_steps(g.l) ? steps / 2 : 0, passes = steps - twos, squares = steps + 3 * twos;
        work += g.count * (passes * (sym * std::max(kc, 7.6) + tr * tc * std::max(kr, 7.6)) + squares * sym * std::max(kr, 7.6));
        chain = std::max(chain, passes * (kc + kr + 2 * 5.5) + squares * (kr + 5.5));
    }
    return 2.5 + std::hypot(1.1 * chain, 1.1 * work / (sm_count() / 2));
}

double products_time(const Group& g, int steps) {
    double t = 0;
    for (int p = 0; p < 3; ++p) t += estimate(product_plan(g, p, 0).args, false);
    return steps * t;
}

// Matrices of one shape, or of its transpose, share launches.
bool same_shape(const Item* x, const Item* y) {
    return std::min(x->rows, x->cols) == std::min(y->rows, y->cols) && std::max(x->rows, x->cols) == std::max(y->rows, y->cols);
}

// Takes out the matrices that fit the single-launch kernel (muon_small.cu).
std::vector<const Item*> take_small(std::vector<const Item*>& v) {
    std::vector<const Item*> small;
    size_t kept = 0;
    for (const Item* it : v) (small_split(it->rows, it->cols) ? small.push_back(it) : void(v[kept++] = it));
    v.resize(kept);
    return small;
}

int run_small_items(std::vector<const Item*>& v, const Params& q, bool last, cudaStream_t s) {
    std::stable_sort(v.begin(), v.end(),
                     [](const Item* x, const Item* y) { return small_split(x->rows, x->cols) < small_split(y->rows, y->cols); });
    SmallArgs a = {};
    a.steps = q.steps;
    a.nesterov = q.nesterov;
    a.g_f32 = q.g_dtype == DPRED_F32;
    a.out_f32 = q.out_dtype == DPRED_F32;
    a.mu = q.mu;
    a.eps = q.eps;
    a.a = q.a;
    a.b = q.b;
    a.c = q.c;
    a.keep = q.keep;
    a.err = device_error_word();
    for (size_t i = 0; i < v.size();) {
        a.split = small_split(v[i]->rows, v[i]->cols);
        for (a.count = 0; i < v.size() && a.count < kSmallBatch && small_split(v[i]->rows, v[i]->cols) == a.split; ++i) {
            const Item& it = *v[i];
            a.m[a.count++] = {it.in.g, it.in.mom, it.out, it.in.ldg, it.in.ldm, it.ldo, (int)it.rows, (int)it.cols, it.step};
        }
        a.release = !last || i < v.size();
        const int rc = run_small(a, s);
        if (rc != DPRED_OK) return rc;
    }
    return DPRED_OK;
}

// The launches of a call: matrices of one shape are neighbours, and a launch
// takes up to kMaxBatch matrices of up to kChainGroups shapes.
std::vector<std::vector<Group>> launches_of(std::vector<const Item*>& v) {
    std::stable_sort(v.begin(), v.end(), [](const Item* x, const Item* y) {
        const int64_t a = std::min(x->rows, x->cols), b = std::min(y->rows, y->cols);
        return a != b ? a < b : std::max(x->rows, x->cols) < std::max(y->rows, y->cols);
    });
    std::vector<std::vector<Group>> launches;
    int room = 0;
    for (size_t i = 0; i < v.size();) {
        size_t j = i;
        while (j < v.size() && same_shape(v[i], v[j])) ++j;
        while (i < j) {
            if (room == 0 || launches.back().size() == (size_t)kChainGroups) {
                launches.emplace_back();
                room = kMaxBatch;
            }
            Group g = {};
            g.items = &v[i];
            g.count = (int)std::min<size_t>(j - i, room);
            g.l = layout_of(v[i]->rows, v[i]->cols);
            launches.back().push_back(g);
            room -= g.count;
            i += g.count;
        }
    }
    return launches;
}

int64_t workspace_of(const std::vector<std::vector<Group>>& launches) {
    int64_t need = 0;
    for (const auto& groups : launches) {
        int64_t bytes = 0;
        for (const Group& g : groups) bytes += group_bytes(g.l, g.count);
        need = std::max(need, bytes);
    }
    return need;
}

int run_items(std::vector<Item>& items, const Params& q, void* workspace, size_t workspace_bytes, cudaStream_t s) {
    std::vector<const Item*> v;
    for (const Item& it : items)
        if (it.rows > 0 && it.cols > 0) v.push_back(&it);
    std::vector<const Item*> small = take_small(v);
    std::vector<std::vector<Group>> launches = launches_of(v);
    const int64_t need = workspace_of(launches);
    if (need && (!workspace || (int64_t)workspace_bytes < need))
        return set_error(DPRED_E_SIZE, "workspace of %zu bytes, %lld needed", workspace ? workspace_bytes : (size_t)0, (long long)need);
    if (need && reinterpret_cast<uintptr_t>(workspace) % 256)
        return set_error(DPRED_E_ALIGN, "workspace is not 256-byte aligned");
    int rc = run_small_items(small, q, launches.empty(), s);
    for (size_t i = 0; i < launches.size() && rc == DPRED_OK; ++i) {
        std::vector<Group>& groups = launches[i];
        char* ws = static_cast<char*>(workspace);
        unsigned* counter = reinterpret_cast<unsigned*>(ws);
        ws += 256;  // counters of up to kMaxBatch matrices
        double separate = 0;
        for (Group& g : groups) {
            place(g, ws);
            g.counter = counter;
            counter += g.count;
            separate += products_time(g, q.steps);
            if ((rc = start_group(g, q, s)) != DPRED_OK) return rc;
        }
        if (chained_time(groups, q.steps) < separate) {
            rc = run_chained(groups, q, s);
        } else {
            for (size_t k = 0; k < groups.size() && rc == DPRED_OK; ++k)
                rc = run_products(groups[k], q, i + 1 == launches.size() && k + 1 == groups.size(), s);
        }
    }
    return rc;
}

int check_dtype(int dt, const char* what) {
    return dt == DPRED_BF16 || dt == DPRED_F32 ? DPRED_OK : set_error(DPRED_E_INVAL, "unknown %s type %d", what, dt);
}

int check_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return set_error(DPRED_E_INVAL, "a negative size (%lld x %lld)", (long long)rows, (long long)cols);
    if (rows > (1 << 20) || cols > (1 << 20) || std::min(rows, cols) > 65536)
        return set_error(DPRED_E_SIZE, "a matrix of %lld x %lld: at most 2^20 on the long and 65536 on the short side",
                         (long long)rows, (long long)cols);
    return DPRED_OK;
}

int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int esize, const char* name) {
    if (rows == 0 || cols == 0) return DPRED_OK;
    if (!p) return set_error(DPRED_E_INVAL, "%s is null", name);
    if (reinterpret_cast<uintptr_t>(p) % esize) return set_error(DPRED_E_ALIGN, "%s is not aligned to its element size", name);
    if (rows > 1 && ld < cols)
        return set_error(DPRED_E_SIZE, "%s: row stride %lld is less than its %lld columns", name, (long long)ld, (long long)cols);
    return DPRED_OK;
}

// Whether two of `batch` matrices that start `stride` elements apart share an
// element: any layout without one is accepted, side by side in wider rows as
// well as one after another.
bool matrices_overlap(int batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    if (batch > 1 && stride < cols) return true;
    if (rows == 1) ld = cols;  // it has no row stride
    const int64_t last = (rows - 1) * ld;
    for (int64_t k = 1, d = stride; k < batch && d < last + cols; ++k, d += stride) {
        const int64_t shift = d / ld, column = d % ld;  // the later matrix against the rows of the earlier one
        if ((shift < rows && column < cols) || (shift + 1 < rows && ld - column < cols)) return true;
    }
    return false;
}

int check_params(int steps, const float* coeffs, float eps) {
    if (steps < 1 || steps > kMaxSteps) return set_error(DPRED_E_INVAL, "steps %d outside 1..%d", steps, kMaxSteps);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return set_error(DPRED_E_INVAL, "eps must be finite and not negative");
    if (coeffs)
        for (int k = 0; k < 3; ++k)
            if (!std::isfinite(coeffs[k])) return set_error(DPRED_E_INVAL, "a coefficient is not finite");
    return DPRED_OK;
}

void set_coeffs(Params& q, const float* coeffs) {
    // the quintic whose slope at 0 is as steep as keeps [0, 1] within about 0.7 .. 1.2
    q.a = coeffs ? coeffs[0] : 3.4445f;
    q.b = coeffs ? coeffs[1] : -4.7750f;
    q.c = coeffs ? coeffs[2] : 2.0315f;
}

template <typename F>
int guarded(F f) {  // no C++ exception leaves a C entry point
    try {
        return f();
    } catch (const std::exception& e) {
        return set_error(DPRED_E_INVAL, "host failure: %s", e.what());
    }
}

}  // namespace
}  // namespace gemm
}  // namespace dpred

using namespace dpred;
using namespace dpred::gemm;

extern "C" size_t dpred_newton_schulz_workspace_bytes(int32_t batch, int64_t rows, int64_t cols) {
    if (batch <= 0 || rows <= 0 || cols <= 0 || check_shape(rows, cols) != DPRED_OK) return 0;
    if (small_split(rows, cols)) return 0;
    return (size_t)group_bytes(layout_of(rows, cols), std::min(batch, kMaxBatch));
}

extern "C" int dpred_newton_schulz(int32_t batch, int64_t rows, int64_t cols, int32_t in_dtype, const void* in, int64_t ld,
                                   int64_t batch_stride, int32_t out_dtype, void* out, int64_t ldo,
                                   int64_t out_batch_stride, int32_t steps, const float* coeffs, float eps,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc;
        if (batch < 0) return set_error(DPRED_E_INVAL, "batch < 0");
        if ((rc = check_shape(rows, cols)) != DPRED_OK || (rc = check_params(steps, coeffs, eps)) != DPRED_OK ||
            (rc = check_dtype(in_dtype, "input")) != DPRED_OK || (rc = check_dtype(out_dtype, "output")) != DPRED_OK)
            return rc;
        if (batch == 0 || rows == 0 || cols == 0) return DPRED_OK;
        const int is = in_dtype == DPRED_F32 ? 4 : 2, os = out_dtype == DPRED_F32 ? 4 : 2;
        if ((rc = check_matrix(in, rows, cols, ld, is, "in")) != DPRED_OK || (rc = check_matrix(out, rows, cols, ldo, os, "out")) != DPRED_OK)
            return rc;
        if (batch > 1 && batch_stride < 0) return set_error(DPRED_E_SIZE, "a negative batch stride");
        if (matrices_overlap(batch, rows, cols, ldo, out_batch_stride))
            return set_error(DPRED_E_SIZE, "output matrices overlap (batch stride %lld)", (long long)out_batch_stride);
        Params q = {};
        q.g_dtype = in_dtype;
        q.out_dtype = out_dtype;
        q.steps = steps;
        q.eps = eps;
        set_coeffs(q, coeffs);
        std::vector<Item> items(batch);
        for (int k = 0; k < batch; ++k) {
            Item& it = items[k];
            it.in = {static_cast<const char*>(in) + (int64_t)k * batch_stride * is, nullptr, ld, 0, 0, 0, 0};
            it.out = static_cast<char*>(out) + (int64_t)k * out_batch_stride * os;
            it.rows = rows;
            it.cols = cols;
            it.ldo = ldo;
            it.step = 1.0f;
        }
        return run_items(items, q, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    });
}

extern "C" size_t dpred_muon_workspace_bytes(const dpred_muon_matrix* mats, int32_t n) {
    if (!mats || n <= 0) return 0;
    size_t need = 0;
    guarded([&]() -> int {
        std::vector<Item> items(n);
        std::vector<const Item*> v;
        for (int k = 0; k < n; ++k) {
            if (check_shape(mats[k].rows, mats[k].cols) != DPRED_OK) return DPRED_E_SIZE;
            items[k].rows = mats[k].rows;
            items[k].cols = mats[k].cols;
            if (mats[k].rows > 0 && mats[k].cols > 0) v.push_back(&items[k]);
        }
        take_small(v);
        need = (size_t)workspace_of(launches_of(v));
        return DPRED_OK;
    });
    return need;
}

extern "C" int dpred_muon_step(const dpred_muon_matrix* mats, int32_t n, int32_t w_dtype, int32_t g_dtype, float lr,
                               float momentum, int32_t nesterov, float weight_decay, int32_t steps, const float* coeffs,
                               float eps, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc;
        if (n < 0 || (n > 0 && !mats)) return set_error(DPRED_E_INVAL, "mats is null or n < 0");
        if ((rc = check_params(steps, coeffs, eps)) != DPRED_OK || (rc = check_dtype(w_dtype, "weight")) != DPRED_OK ||
            (rc = check_dtype(g_dtype, "gradient")) != DPRED_OK)
            return rc;
        if (!std::isfinite(lr) || !std::isfinite(momentum) || !std::isfinite(weight_decay))
            return set_error(DPRED_E_INVAL, "lr, momentum and weight_decay must be finite");
        Params q = {};
        q.g_dtype = g_dtype;
        q.out_dtype = w_dtype;
        q.nesterov = nesterov != 0;
        q.steps = steps;
        q.mu = momentum;
        q.keep = 1.0f - lr * weight_decay;
        q.eps = eps;
        set_coeffs(q, coeffs);
        const int gs = g_dtype == DPRED_F32 ? 4 : 2, wsz = w_dtype == DPRED_F32 ? 4 : 2;
        std::vector<Item> items(n);
        for (int k = 0; k < n; ++k) {
            const dpred_muon_matrix& m = mats[k];
            if ((rc = check_shape(m.rows, m.cols)) != DPRED_OK ||
                (rc = check_matrix(m.weight, m.rows, m.cols, m.ldw, wsz, "weight")) != DPRED_OK ||
                (rc = check_matrix(m.momentum, m.rows, m.cols, m.ldm, 4, "momentum")) != DPRED_OK ||
                (rc = check_matrix(m.grad, m.rows, m.cols, m.ldg, gs, "grad")) != DPRED_OK)
                return rc;
            if (m.reserved != 0) return set_error(DPRED_E_INVAL, "a matrix's reserved field is not 0");
            if (!std::isfinite(m.scale)) return set_error(DPRED_E_INVAL, "a matrix's scale is not finite");
            Item& it = items[k];
            it.in = {m.grad, m.momentum, m.ldg, m.ldm, 0, 0, 0};
            it.out = m.weight;
            it.rows = m.rows;
            it.cols = m.cols;
            it.ldo = m.ldw;
            it.step = -lr * m.scale;
        }
        return run_items(items, q, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    });
}
