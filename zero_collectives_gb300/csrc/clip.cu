// clip.cu -- the global gradient norm and clipping: dpred_grad_norm and
// dpred_clip_grads.
//
// After the reduction (DeepSpeed issue #8700) every gradient lies on its owner;
// before the update they are scaled together:
//
//     n = sqrt(sum of g^2 over all gradients),  c = min(1, max_norm / (n + eps)),
//     g = c g.
//
// One launch sums squares, a second forms n and c from its partial sums and
// scales; where c is 1 it reads and writes nothing more.  Both walk the same
// table of units of 16 KB; it travels inside the launch.
//
// Bandwidth bound: each gradient is read, then read and written.  The second
// launch takes the units in the opposite order, so that what the first read last
// is still in L2.
#include <algorithm>
#include <vector>

#include "layers.cuh"

namespace dpred {
namespace layers {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16384;         // bytes of a unit: four 16-byte vectors a thread
constexpr int kNarrow = 512;         // rows below this many bytes are taken element by element
constexpr int kMaxBlocks = 2048;     // partial sums a launch can leave
constexpr int kSmallTable = 32, kMidTable = 256, kTable = 768;  // pieces that travel in a launch (1, 10 and 31 KB)
constexpr int kMaxUnits = 0x3FFFFFFF;  // of a launch

// One gradient as the kernels see it.
struct Piece {
    char* p;
    int64_t cols, ld;
    int32_t rows, unit0;  // its first unit in the launch
    int32_t per;          // rows of a unit, or minus the units of a row
    int32_t f32;
};
static_assert(sizeof(Piece) == 40, "Piece layout");

template <int CAP>
struct Table {
    int32_t n, units;
    Piece piece[CAP];
};
static_assert(sizeof(Table<kTable>) < 32000, "a launch's arguments");

// A sum of squares over the whole range of the type.  A chunk of up to 32
// squares is added in fp32; chunks between 2^-90 and 2^80 go to a compensated
// pair of fp32 (its error stays near 2^-24 of the sum however many there are;
// an fp64 addition per chunk would cost as much as the loads), the few others
// are formed again from scaled values and added in fp64.
struct Squares {
    float hi = 0.0f, lo = 0.0f;
    double far = 0.0;

    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N]) {
        float q[4] = {};
#pragma unroll
        for (int k = 0; k < N; ++k) q[k & 3] = fmaf(x[k], x[k], q[k & 3]);
        const float c = (q[0] + q[1]) + (q[2] + q[3]);
        if (c >= 0x1p-90f && c <= 0x1p80f) {
            const float s = hi + c, t = s - hi;
            lo += (hi - (s - t)) + (c - t);
            hi = s;
            return;
        }
        const bool small = c < 0x1p-90f;  // zeros most of the time
        const float f = small ? 0x1p100f : 0x1p-70f;
        float d = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float y = x[k] * f;
            d = fmaf(y, y, d);
        }
        if (d != 0.0f) far += (double)d * (small ? 0x1p-200 : 0x1p140);
    }
    __device__ __forceinline__ double total() const { return far + ((double)hi + (double)lo); }
};

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double warps[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) v += warps[w];
    return v;
}

// The 16-byte vectors of a type.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(const uint4& q, float* f) {
        f[0] = bf16_lo(q.x); f[1] = bf16_hi(q.x); f[2] = bf16_lo(q.y); f[3] = bf16_hi(q.y);
        f[4] = bf16_lo(q.z); f[5] = bf16_hi(q.z); f[6] = bf16_lo(q.w); f[7] = bf16_hi(q.w);
    }
    static __device__ __forceinline__ uint4 scaled(const uint4& q, float c) {
        return make_uint4(pack_bf16x2(bf16_lo(q.x) * c, bf16_hi(q.x) * c), pack_bf16x2(bf16_lo(q.y) * c, bf16_hi(q.y) * c),
                          pack_bf16x2(bf16_lo(q.z) * c, bf16_hi(q.z) * c), pack_bf16x2(bf16_lo(q.w) * c, bf16_hi(q.w) * c));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(const uint4& q, float* f) {
        f[0] = __uint_as_float(q.x); f[1] = __uint_as_float(q.y); f[2] = __uint_as_float(q.z); f[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 scaled(const uint4& q, float c) {
        return make_uint4(__float_as_uint(__uint_as_float(q.x) * c), __float_as_uint(__uint_as_float(q.y) * c),
                          __float_as_uint(__uint_as_float(q.z) * c), __float_as_uint(__uint_as_float(q.w) * c));
    }
};

template <bool SCALE, typename T>
__device__ __forceinline__ void one(T* p, Squares& s, float c) {
    const float x[1] = {load1(p)};
    if constexpr (SCALE)
        store1(p, x[0] * c);
    else
        s.add(x);
}

// Vectors [v0, v1) of the n elements at p, counted from the first 16-byte
// boundary, with the elements before it and after the last whole vector; by
// threads id, id + step, ...
template <bool SCALE, typename T>
__device__ __forceinline__ void span(T* p, int64_t n, int64_t v0, int64_t v1, bool first, bool last, int id, int step, Squares& s, float c) {
    constexpr int N = Vec<T>::N;
    const int64_t head = min(n, (int64_t)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
    const int64_t whole = (n - head) / N, tail = head + whole * N;
    uint4* v = reinterpret_cast<uint4*>(p + head);
    if (v1 > whole) v1 = whole;
    for (int64_t i = v0 + id; i < v1; i += 4 * step) {
        uint4 q[4];
        if (i + 3 * step < v1) {
#pragma unroll
            for (int u = 0; u < 4; ++u) q[u] = v[i + u * step];
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) q[u] = i + u * step < v1 ? v[i + u * step] : make_uint4(0, 0, 0, 0);
        }
        if constexpr (SCALE) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < v1) v[i + u * step] = Vec<T>::scaled(q[u], c);
        } else {
            float x[4 * N];
#pragma unroll
            for (int u = 0; u < 4; ++u) Vec<T>::widen(q[u], x + u * N);
            s.add(x);
        }
    }
    if (first)
        for (int64_t i = id; i < head; i += step) one<SCALE>(p + i, s, c);
    if (last)
        for (int64_t i = tail + id; i < n; i += step) one<SCALE>(p + i, s, c);
}

template <bool SCALE, typename T>
__device__ __forceinline__ void unit_of(const Piece& pc, int k, Squares& s, float c) {
    T* p = reinterpret_cast<T*>(pc.p);
    if (pc.per < 0) {  // part of one row
        const int row = k / -pc.per, part = k % -pc.per;
        constexpr int64_t kVecs = kUnit / 16;
        span<SCALE>(p + row * pc.ld, pc.cols, part * kVecs, (part + 1) * kVecs, part == 0, part == -pc.per - 1, threadIdx.x, kThreads, s, c);
        return;
    }
    const int64_t r0 = (int64_t)k * pc.per, r1 = min(r0 + pc.per, (int64_t)pc.rows);
    if (pc.cols * (int)sizeof(T) >= kNarrow) {  // a warp per row
        for (int64_t r = r0 + threadIdx.x / 32; r < r1; r += kThreads / 32)
            span<SCALE>(p + r * pc.ld, pc.cols, 0, pc.cols, true, true, threadIdx.x % 32, 32, s, c);
        return;
    }
    const uint32_t cols = (uint32_t)pc.cols, total = (uint32_t)(r1 - r0) * cols;
    for (uint32_t i = threadIdx.x; i < total; i += kThreads) one<SCALE>(p + (r0 + i / cols) * pc.ld + i % cols, s, c);
}

template <bool SCALE, typename A>
__device__ __forceinline__ void do_unit(const A& t, int unit, int& at, Squares& s, float c) {
    // units come in order: the piece of one lies near that of the one before
    if constexpr (SCALE)
        while (t.piece[at].unit0 > unit) --at;
    else
        while (at + 1 < t.n && t.piece[at + 1].unit0 <= unit) ++at;
    const Piece& pc = t.piece[at];
    if (pc.f32)
        unit_of<SCALE, float>(pc, unit - pc.unit0, s, c);
    else
        unit_of<SCALE, __nv_bfloat16>(pc, unit - pc.unit0, s, c);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<CAP> t, double* __restrict__ partial) {
    mma::grid_launch_dependents();
    mma::grid_wait();
    Squares s;
    int at = 0;
    for (int u = blockIdx.x; u < t.units; u += gridDim.x) do_unit<false>(t, u, at, s, 0.0f);
    const double v = block_sum(s.total());
    if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The sum of the partial sums, in one fixed order, in every thread.
__device__ __forceinline__ double total_of(const double* partial, int n) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v += partial[i];
    return block_sum(v);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* __restrict__ partial, int n, float* __restrict__ out) {
    mma::grid_wait();
    const double v = total_of(partial, n);
    if (threadIdx.x == 0) out[0] = (float)sqrt(v);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<CAP> t, const double* __restrict__ partial, int n,
                                                         float max_norm, float eps, float* __restrict__ out) {
    __shared__ float coefficient;
    mma::grid_wait();
    const double sum = total_of(partial, n);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum), down = norm + (double)eps;
        const double q = down == 0.0 ? 1.0 : (double)max_norm / down;
        const float c = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
        coefficient = c;
        if (blockIdx.x == 0 && out) {
            out[0] = (float)norm;
            out[1] = c;
        }
    }
    __syncthreads();
    const float c = coefficient;
    if (c == 1.0f) return;
    Squares s;
    int at = t.n - 1;
    for (int u = t.units - 1 - (int)blockIdx.x; u >= 0; u -= gridDim.x) do_unit<true>(t, u, at, s, c);
}

// -------------------------------------------------------------------- host --

struct Chunk {  // the pieces of one launch
    std::vector<Piece> pieces;
    int units = 0;
};

int check_grads(const dpred_grad_tensor* g, int n) {
    if (n < 0 || (n > 0 && !g)) return set_error(DPRED_E_INVAL, "grads is null or n < 0");
    for (int k = 0; k < n; ++k) {
        const dpred_grad_tensor& t = g[k];
        if (t.rows < 0 || t.cols < 0) return set_error(DPRED_E_INVAL, "gradient %d: a negative size (%lld x %lld)", k, (long long)t.rows, (long long)t.cols);
        if (!dtype_ok(t.dtype)) return set_error(DPRED_E_INVAL, "gradient %d: unknown type %d", k, t.dtype);
        if (t.counted != 0 && t.counted != 1) return set_error(DPRED_E_INVAL, "gradient %d: counted must be 0 or 1", k);
        if (t.rows > 0x7FFFFFFF || t.cols > ((int64_t)1 << 40))
            return set_error(DPRED_E_SIZE, "gradient %d: %lld x %lld is too large", k, (long long)t.rows, (long long)t.cols);
        const int rc = check_matrix(t.data, t.rows, t.cols, t.ld, esize(t.dtype), "a gradient");
        if (rc != DPRED_OK) return rc;
    }
    return DPRED_OK;
}

// Whether two gradients share a byte.  Rows of one stride may lie between one
// another's; where that cannot be told from the strides, ranges that meet overlap.
struct Range {
    uintptr_t lo, hi;  // first byte, one past the last
    int64_t row, step, rows;
};

bool overlap(const Range& a, const Range& b) {  // a.lo <= b.lo < a.hi
    const int64_t step = a.rows > 1 ? a.step : b.step;
    if ((a.rows > 1 && b.rows > 1 && a.step != b.step) || (a.rows <= 1 && b.rows <= 1)) return true;
    const int64_t column = (int64_t)((b.lo - a.lo) % (uintptr_t)step);
    return column < a.row || step - column < b.row;
}

bool any_overlap(const dpred_grad_tensor* g, int n) {
    std::vector<Range> v;
    v.reserve(n);
    for (int k = 0; k < n; ++k) {
        if (g[k].rows == 0 || g[k].cols == 0) continue;
        const int64_t es = esize(g[k].dtype), row = g[k].cols * es, step = g[k].rows > 1 ? g[k].ld * es : row;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(g[k].data);
        v.push_back({lo, lo + (uintptr_t)((g[k].rows - 1) * step + row), row, step, g[k].rows});
    }
    if (!std::is_sorted(v.begin(), v.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; }))
        std::sort(v.begin(), v.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    std::vector<Range> open;  // ranges that reach past the present start
    for (const Range& r : v) {
        size_t kept = 0;
        for (size_t k = 0; k < open.size(); ++k) {
            if (open[k].hi <= r.lo) continue;
            if (overlap(open[k], r)) return true;
            open[kept++] = open[k];
        }
        open.resize(kept);
        open.push_back(r);
    }
    return false;
}

// The launches over the gradients (the counted ones, or all).
int plan(const dpred_grad_tensor* g, int n, bool counted_only, std::vector<Chunk>& out) {
    for (int k = 0; k < n; ++k) {
        const dpred_grad_tensor& t = g[k];
        if (t.rows == 0 || t.cols == 0 || (counted_only && !t.counted)) continue;
        const int es = esize(t.dtype);
        const bool flat = t.rows == 1 || t.ld == t.cols;
        Piece p = {};
        p.p = static_cast<char*>(t.data);
        p.rows = flat ? 1 : (int32_t)t.rows;
        p.cols = flat ? t.rows * t.cols : t.cols;
        p.ld = t.ld;
        p.f32 = t.dtype == DPRED_F32;
        const int64_t bytes = p.cols * es;
        int64_t units;
        if (p.rows == 1 || bytes > kUnit) {
            const int64_t row_units = (bytes + kUnit - 1) / kUnit;
            units = row_units * p.rows;
            p.per = (int32_t)-std::min<int64_t>(row_units, 0x7FFFFFFF);
        } else {
            p.per = (int32_t)std::max<int64_t>(1, kUnit / bytes);
            units = (p.rows + p.per - 1) / p.per;
        }
        if (out.empty() || (int)out.back().pieces.size() == kTable) out.emplace_back();
        if (units > kMaxUnits - (int64_t)out.back().units) return set_error(DPRED_E_SIZE, "gradient %d is too large", k);
        p.unit0 = out.back().units;
        out.back().units += (int)units;
        out.back().pieces.push_back(p);
    }
    return DPRED_OK;
}

// Eight blocks of an SM hold 128 KB of loads in flight.
int blocks_of(const Chunk& c) { return std::max(1, std::min({c.units, 8 * sm_count(), kMaxBlocks})); }

template <int CAP>
Table<CAP> table_of(const Chunk& c) {
    Table<CAP> t;
    t.n = (int)c.pieces.size();
    t.units = c.units;
    std::copy(c.pieces.begin(), c.pieces.end(), t.piece);
    return t;
}

cudaError_t launch_squares(const Chunk& c, double* partial, cudaStream_t s) {
    if (c.pieces.size() <= kSmallTable)
        return launch(squares_kernel<kSmallTable>, dim3(blocks_of(c)), kThreads, 0, s, table_of<kSmallTable>(c), partial);
    if (c.pieces.size() <= kMidTable)
        return launch(squares_kernel<kMidTable>, dim3(blocks_of(c)), kThreads, 0, s, table_of<kMidTable>(c), partial);
    return launch(squares_kernel<kTable>, dim3(blocks_of(c)), kThreads, 0, s, table_of<kTable>(c), partial);
}

cudaError_t launch_scale(const Chunk& c, const double* partial, int n, float max_norm, float eps, float* out, cudaStream_t s) {
    if (c.pieces.size() <= kSmallTable)
        return launch(scale_kernel<kSmallTable>, dim3(blocks_of(c)), kThreads, 0, s, table_of<kSmallTable>(c), partial, n, max_norm, eps, out);
    if (c.pieces.size() <= kMidTable)
        return launch(scale_kernel<kMidTable>, dim3(blocks_of(c)), kThreads, 0, s, table_of<kMidTable>(c), partial, n, max_norm, eps, out);
    return launch(scale_kernel<kTable>, dim3(blocks_of(c)), kThreads, 0, s, table_of<kTable>(c), partial, n, max_norm, eps, out);
}

// A partial sum per block and launch; calls that count nothing launch one block.
size_t workspace_of(int64_t n) {
    const int64_t launches = std::max<int64_t>(1, (n + kTable - 1) / kTable);
    return (size_t)launches * kMaxBlocks * sizeof(double);
}

int run_squares(const std::vector<Chunk>& chunks, double* partial, int& n, cudaStream_t s) {
    n = 0;
    for (const Chunk& c : chunks) {
        const cudaError_t e = launch_squares(c, partial + n, s);
        if (e != cudaSuccess) return cuda_error(e, "gradient norm launch");
        n += blocks_of(c);
    }
    return DPRED_OK;
}

}  // namespace
}  // namespace layers
}  // namespace dpred

using namespace dpred;
using namespace dpred::layers;

extern "C" size_t dpred_clip_workspace_bytes(int32_t n) { return n < 0 ? 0 : workspace_of(n); }

extern "C" int dpred_grad_norm(const dpred_grad_tensor* grads, int32_t n, float* norm, void* workspace, size_t workspace_bytes,
                               void* stream) {
    return guarded([&]() -> int {
        int rc = check_grads(grads, n);
        if (rc != DPRED_OK) return rc;
        if (!norm) return set_error(DPRED_E_INVAL, "norm is null");
        if (reinterpret_cast<uintptr_t>(norm) % 4) return set_error(DPRED_E_ALIGN, "norm is not aligned to 4 bytes");
        if ((rc = check_workspace(workspace, workspace_bytes, workspace_of(n))) != DPRED_OK) return rc;
        std::vector<Chunk> chunks;
        if ((rc = plan(grads, n, true, chunks)) != DPRED_OK) return rc;
        double* partial = static_cast<double*>(workspace);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        int sums = 0;
        if ((rc = run_squares(chunks, partial, sums, s)) != DPRED_OK) return rc;
        const cudaError_t e = launch(norm_kernel, dim3(1), kThreads, 0, s, partial, sums, norm);
        return e == cudaSuccess ? DPRED_OK : cuda_error(e, "gradient norm launch");
    });
}

extern "C" int dpred_clip_grads(const dpred_grad_tensor* grads, int32_t n, float max_norm, float eps, float* result, void* workspace,
                                size_t workspace_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_grads(grads, n);
        if (rc != DPRED_OK) return rc;
        if (!(max_norm >= 0.0f) || !std::isfinite(max_norm)) return set_error(DPRED_E_INVAL, "max_norm must be finite and not negative");
        if (!(eps >= 0.0f) || !std::isfinite(eps)) return set_error(DPRED_E_INVAL, "eps must be finite and not negative");
        if (!result) return set_error(DPRED_E_INVAL, "result is null");
        if (reinterpret_cast<uintptr_t>(result) % 4) return set_error(DPRED_E_ALIGN, "result is not aligned to 4 bytes");
        if ((rc = check_workspace(workspace, workspace_bytes, workspace_of(n))) != DPRED_OK) return rc;
        if (any_overlap(grads, n)) return set_error(DPRED_E_SIZE, "two gradients share memory: each would be scaled more than once");
        std::vector<Chunk> counted, all;
        if ((rc = plan(grads, n, true, counted)) != DPRED_OK || (rc = plan(grads, n, false, all)) != DPRED_OK) return rc;
        if (all.empty()) all.emplace_back();  // no gradient: norm 0
        double* partial = static_cast<double*>(workspace);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        int sums = 0;
        if ((rc = run_squares(counted, partial, sums, s)) != DPRED_OK) return rc;
        for (size_t k = 0; k < all.size(); ++k) {
            const cudaError_t e = launch_scale(all[k], partial, sums, max_norm, eps, k == 0 ? result : nullptr, s);
            if (e != cudaSuccess) return cuda_error(e, "clipping launch");
        }
        return DPRED_OK;
    });
}
