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
// table of units of 16 KB; it travels inside the launch.  Few units are done by
// one cluster in one launch.
//
// Bandwidth bound: each gradient is read, then read and written.  Every block has
// the same stretch in both launches and takes it in the opposite order in the
// second, so that what the first read last is still in L2.
#include <algorithm>
#include <vector>

#include "layers.cuh"

namespace dpred {
namespace layers {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16384;         // bytes of a unit: four 16-byte vectors a thread
// Strided rows below this many bytes are taken element by element, others by a warp
// each.  Clipping 64 MB, by elements / by warps: fp32 rows of 384 bytes 50 / 70 us, of 512
// 43 / 41, of 1024 43 / 29; bf16 of 128 bytes 168 / 289, of 256 166 / 157, of 512 165 / 81.
constexpr int kNarrow = 512;
constexpr int kBlocksPerSm = 3;      // each with up to 32 KB of loads in flight, in 80 registers a thread
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

// Four 16-byte vectors of a type, widened piece by piece.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float2 pair(const uint4& q, int i) {
        const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
        return make_float2(bf16_lo(w), bf16_hi(w));
    }
    static __device__ __forceinline__ uint4 scaled(const uint4& q, float c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = mul2(pair(q, i), make_float2(c, c));
            w[i] = pack_bf16x2(f.x, f.y);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float2 pair(const uint4& q, int i) {
        return i == 0 ? make_float2(__uint_as_float(q.x), __uint_as_float(q.y)) : make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
    }
    static __device__ __forceinline__ uint4 scaled(const uint4& q, float c) {
        const float2 a = mul2(pair(q, 0), make_float2(c, c)), b = mul2(pair(q, 1), make_float2(c, c));
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
};

// A sum of squares over the whole range of the type.  A chunk of up to 32
// squares is added in fp32; chunks between 2^-90 and 2^80 go to a compensated
// pair of fp32 (its error stays near 2^-24 of the sum however many there are;
// an fp64 addition per chunk would cost as much as the loads), the few others
// are formed again from scaled values and added in fp64.
struct Squares {
    float hi = 0.0f, lo = 0.0f;
    double far = 0.0;

    template <typename T>
    __device__ __forceinline__ void add(const uint4 (&q)[4]) {
        float2 t[2] = {};
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int i = 0; i < Vec<T>::N / 2; ++i) {
                const float2 f = Vec<T>::pair(q[v], i);
                t[v & 1] = fma2(f, f, t[v & 1]);
            }
        const float c = (t[0].x + t[0].y) + (t[1].x + t[1].y);
        if (!near(c)) {
            const bool small = c < 0x1p-90f;  // zeros most of the time
            const float f = small ? 0x1p100f : 0x1p-70f;
            float d = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int i = 0; i < Vec<T>::N / 2; ++i) {
                    const float2 x = Vec<T>::pair(q[v], i);
                    d = fmaf(x.x * f, x.x * f, d);
                    d = fmaf(x.y * f, x.y * f, d);
                }
            apart(d, small);
        }
    }
    __device__ __forceinline__ void add(float x) {
        if (near(x * x)) return;
        const bool small = x * x < 0x1p-90f;
        const float y = x * (small ? 0x1p100f : 0x1p-70f);
        apart(y * y, small);
    }
    __device__ __forceinline__ bool near(float c) {
        if (!(c >= 0x1p-90f && c <= 0x1p80f)) return false;
        const float s = hi + c, t = s - hi;
        lo += (hi - (s - t)) + (c - t);
        hi = s;
        return true;
    }
    __device__ __forceinline__ void apart(float d, bool small) {
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

template <bool SCALE, typename T>
__device__ __forceinline__ void one(T* p, Squares& s, float c) {
    const float x = load1(p);
    if constexpr (SCALE)
        store1(p, x * c);
    else
        s.add(x);
}

// A row's elements before the first 16-byte boundary, its whole vectors, and what
// is left behind them.
template <typename T>
struct Row {
    T* p;
    int64_t n, head, whole;
    __device__ __forceinline__ Row(T* p, int64_t n) : p(p), n(n) {
        head = min(n, (int64_t)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
        whole = (n - head) / Vec<T>::N;
    }
    __device__ __forceinline__ uint4* vectors() const { return reinterpret_cast<uint4*>(p + head); }
    template <bool SCALE>
    __device__ __forceinline__ void edges(bool first, bool last, int id, int step, Squares& s, float c) const {
        if (first)
            for (int64_t i = id; i < head; i += step) one<SCALE>(p + i, s, c);
        if (last)
            for (int64_t i = head + whole * Vec<T>::N + id; i < n; i += step) one<SCALE>(p + i, s, c);
    }
};

// Past L1: nothing is read twice by one SM (the norm of 402.8M: 133 -> 121 us).
__device__ __forceinline__ void load_four(uint4 (&q)[4], const uint4* v, int i, int n, int step) {
    if (n >= 4 * step) {
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = __ldcg(v + i + u * step);
        return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = i + u * step < n ? v[i + u * step] : make_uint4(0, 0, 0, 0);
}

template <bool SCALE, typename T>
__device__ __forceinline__ void take_four(const uint4 (&q)[4], uint4* v, int i, int n, int step, Squares& s, float c) {
    if constexpr (SCALE) {
        if (n >= 4 * step) {
#pragma unroll
            for (int u = 0; u < 4; ++u) v[i + u * step] = Vec<T>::scaled(q[u], c);
            return;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * step < n) v[i + u * step] = Vec<T>::scaled(q[u], c);
    } else {
        s.add<T>(q);
    }
}

// What a block has in flight of a unit: the vectors of a stretch of one row.
struct Stretch {
    uint4* v;
    int n;  // vectors, at most 4 for each thread
    int f32;
};

constexpr int kVecs = kUnit / 16;
static_assert(kVecs == 4 * kThreads, "four vectors a thread");

// The units of a row between its first and last that are full: nothing has to be
// worked out for them.
struct Inside {
    int lo = 0, hi = 0;  // units
    uint4* v = nullptr;  // of lo
    int f32 = 0;
};

// A unit of whole rows, or the edges of a stretch; the stretch itself is returned.
template <bool SCALE, typename T>
__device__ __forceinline__ Stretch begin_unit(const Piece& pc, int unit, Squares& s, float c, Inside& in) {
    T* p = reinterpret_cast<T*>(pc.p);
    const int k = unit - pc.unit0;
    if (pc.per < 0) {  // part of one row
        const int row = pc.per == -1 ? k : k / -pc.per, part = pc.per == -1 ? 0 : k % -pc.per, last = -pc.per - 1;
        const Row<T> r(p + row * pc.ld, pc.cols);
        r.template edges<SCALE>(part == 0, part == last, threadIdx.x, kThreads, s, c);
        in = {unit - part + 1, unit - part + (int)min(r.whole / kVecs, (int64_t)last), r.vectors() + kVecs, sizeof(T) == 4};
        const int64_t left = r.whole - (int64_t)part * kVecs;
        return {r.vectors() + (int64_t)part * kVecs, (int)max((int64_t)0, min(left, (int64_t)kVecs)), sizeof(T) == 4};
    }
    const int64_t r0 = (int64_t)k * pc.per, r1 = min(r0 + pc.per, (int64_t)pc.rows);
    if (pc.cols * (int)sizeof(T) >= kNarrow) {  // a warp per row
        const int lane = threadIdx.x % 32;
        for (int64_t i = r0 + threadIdx.x / 32; i < r1; i += kThreads / 32) {
            const Row<T> r(p + i * pc.ld, pc.cols);
            uint4* v = r.vectors();
            const int n = (int)r.whole;  // the row is within a unit
            for (int j = 0; j < n; j += 128) {
                uint4 q[4];
                load_four(q, v + j, lane, n - j, 32);
                take_four<SCALE, T>(q, v + j, lane, n - j, 32, s, c);
            }
            r.template edges<SCALE>(true, true, lane, 32, s, c);
        }
    } else {
        const uint32_t cols = (uint32_t)pc.cols, total = (uint32_t)(r1 - r0) * cols;
        for (uint32_t i = threadIdx.x; i < total; i += kThreads) one<SCALE>(p + (r0 + i / cols) * pc.ld + i % cols, s, c);
    }
    return {nullptr, 0, 0};
}

// The piece that unit lies in.
template <typename A>
__device__ __forceinline__ int piece_of(const A& t, int unit) {
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.piece[mid].unit0 <= unit)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Block `block` of `blocks` has a stretch of the units and loads the next one while
// it works on the one before.  Squares go up, scaling goes down.  (Units dealt out
// in turn cost a search of the table each: the norm of 402.8M took 146 us.)
template <bool SCALE, typename A>
__device__ __forceinline__ void walk(const A& t, int block, int blocks, Squares& s, float c) {
    const int u0 = (int)((int64_t)t.units * block / blocks), u1 = (int)((int64_t)t.units * (block + 1) / blocks);
    const int first = SCALE ? u1 - 1 : u0, step = SCALE ? -1 : 1;
    int at = piece_of(t, first);
    Inside in;
    auto begin = [&](int unit) -> Stretch {
        if (SCALE ? unit < u0 : unit >= u1) return {nullptr, 0, 0};
        if (unit >= in.lo && unit < in.hi) return {in.v + (int64_t)(unit - in.lo) * kVecs, kVecs, in.f32};
        if constexpr (SCALE)
            while (t.piece[at].unit0 > unit) --at;
        else
            while (at + 1 < t.n && t.piece[at + 1].unit0 <= unit) ++at;
        const Piece& pc = t.piece[at];
        return pc.f32 ? begin_unit<SCALE, float>(pc, unit, s, c, in) : begin_unit<SCALE, __nv_bfloat16>(pc, unit, s, c, in);
    };
    auto take = [&](const uint4 (&q)[4], const Stretch& u) {
        if (u.n <= 0) return;
        if (u.f32)
            take_four<SCALE, float>(q, u.v, threadIdx.x, u.n, kThreads, s, c);
        else
            take_four<SCALE, __nv_bfloat16>(q, u.v, threadIdx.x, u.n, kThreads, s, c);
    };
    uint4 qa[4], qb[4];
    Stretch a = begin(first);
    load_four(qa, a.v, threadIdx.x, a.n, kThreads);
    for (int unit = first; SCALE ? unit >= u0 : unit < u1; unit += 2 * step) {
        const Stretch b = begin(unit + step);
        load_four(qb, b.v, threadIdx.x, b.n, kThreads);
        take(qa, a);
        a = begin(unit + 2 * step);
        load_four(qa, a.v, threadIdx.x, a.n, kThreads);
        take(qb, b);
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) squares_kernel(const __grid_constant__ Table<CAP> t, double* __restrict__ partial) {
    mma::grid_launch_dependents();
    mma::grid_wait();
    Squares s;
    walk<false>(t, blockIdx.x, gridDim.x, s, 0.0f);
    const double v = block_sum(s.total());
    if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The sum of the partial sums, in one fixed order, in every thread.
__device__ __forceinline__ double total_of(const double* partial, int n) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v += partial[i];
    return block_sum(v);
}

// The factor of the gradients; a NaN stays one.  Where none was counted it is 1.
__device__ __forceinline__ float factor(bool counted, double norm, float max_norm, float eps) {
    if (!counted) return 1.0f;
    const double down = norm + (double)eps;
    const double q = down == 0.0 ? 1.0 : (double)max_norm / down;
    return q >= 1.0 ? 1.0f : (float)q;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* __restrict__ partial, int n, float* __restrict__ out) {
    mma::grid_wait();
    const double v = total_of(partial, n);
    if (threadIdx.x == 0) out[0] = (float)sqrt(v);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) scale_kernel(const __grid_constant__ Table<CAP> t, const double* __restrict__ partial, int n,
                                                                       float max_norm, float eps, float* __restrict__ out) {
    __shared__ float coefficient;
    mma::grid_wait();
    const double sum = total_of(partial, n);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        coefficient = factor(n > 0, norm, max_norm, eps);
        if (blockIdx.x == 0 && out) {
            out[0] = (float)norm;
            out[1] = coefficient;
        }
    }
    __syncthreads();
    const float c = coefficient;
    if (c == 1.0f) return;
    Squares s;
    walk<true>(t, blockIdx.x, gridDim.x, s, c);
}

// Few units in one launch: the blocks of a cluster exchange their sums through
// distributed shared memory, and the host launches once.  A call into a given result,
// one launch / two: 1 unit 6.3 / 10.7 us, 32 units 9.4 / 10.5, 48 units 10.7 / 10.4,
// 64 units 12.0 / 10.4; in a captured graph 8 units 6.6 / 6.8, 64 units 12.2 / 7.0.
constexpr int kCluster = 8;
constexpr int kFewUnits = 8 * kCluster;

template <bool SCALE>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    cluster_kernel(const __grid_constant__ Table<kSmallTable> t, int counted, float max_norm, float eps, float* __restrict__ out) {
    __shared__ double mine;
    mma::grid_wait();
    const int rank = (int)mma::cluster_rank();
    Squares s;
    struct {  // the counted pieces come first
        int32_t n, units;
        const Piece* piece;
    } const part = {counted, counted < t.n ? t.piece[counted].unit0 : t.units, t.piece};
    walk<false>(part, rank, kCluster, s, 0.0f);
    const double v = block_sum(s.total());
    if (threadIdx.x == 0) mine = v;
    mma::cluster_sync();
    double sum = 0.0;
    for (int k = 0; k < kCluster; ++k) {
        const uint32_t at = mma::map_rank(tma::smem_addr(&mine), k);
        const float lo = mma::ld_cluster(at), hi = mma::ld_cluster(at + 4);
        sum += __hiloint2double(__float_as_int(hi), __float_as_int(lo));
    }
    mma::cluster_sync();  // no block leaves while its sum is read
    const double norm = sqrt(sum);
    const float c = SCALE ? factor(counted > 0, norm, max_norm, eps) : 1.0f;
    if (rank == 0 && threadIdx.x == 0) {
        out[0] = (float)norm;
        if (SCALE) out[1] = c;
    }
    if (SCALE && c != 1.0f) walk<true>(t, rank, kCluster, s, c);
}

// -------------------------------------------------------------------- host --

// The pieces of one launch, the counted ones first.
struct Chunk {
    Table<kTable> t;
    int counted, counted_units;
};

int check_grads(const dpred_grad_tensor* g, int n) {
    if (n < 0 || (n > 0 && !g)) return set_error(DPRED_E_INVAL, "grads is null or n < 0");
    for (int k = 0; k < n; ++k) {
        const dpred_grad_tensor& t = g[k];
        if (t.rows < 0 || t.cols < 0) return set_error(DPRED_E_INVAL, "gradient %d: a negative size (%lld x %lld)", k, (long long)t.rows, (long long)t.cols);
        if (!dtype_ok(t.dtype)) return set_error(DPRED_E_INVAL, "gradient %d: unknown type %d", k, t.dtype);
        if (t.counted != 0 && t.counted != 1) return set_error(DPRED_E_INVAL, "gradient %d: counted must be 0 or 1", k);
        // sizes in bytes, and differences of addresses, fit 64 bits
        const int64_t most = (int64_t)1 << 60;
        if (t.rows > 0x7FFFFFFF || t.cols > ((int64_t)1 << 40) || (t.rows > 1 && t.ld > most / t.rows))
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

Range range_of(const dpred_grad_tensor& g) {
    const int64_t es = esize(g.dtype), row = g.cols * es, step = g.rows > 1 ? g.ld * es : row;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(g.data);
    return {lo, lo + (uintptr_t)((g.rows - 1) * step + row), row, step, g.rows};
}

bool any_overlap(const dpred_grad_tensor* g, int n) {
    // one after another in memory, as views of a buffer are: nothing to sort
    bool apart = true;
    uintptr_t end = 0;
    for (int k = 0; k < n && apart; ++k) {
        if (g[k].rows == 0 || g[k].cols == 0) continue;
        const Range r = range_of(g[k]);
        apart = r.lo >= end;
        end = r.hi;
    }
    if (apart) return false;
    std::vector<Range> v;
    v.reserve(n);
    for (int k = 0; k < n; ++k)
        if (g[k].rows > 0 && g[k].cols > 0) v.push_back(range_of(g[k]));
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

// The launches over the counted gradients and, behind them, over the others.
int plan(const dpred_grad_tensor* g, int n, bool counted_only, std::vector<Chunk>& out) {
    for (int i = 0; i < (counted_only ? n : 2 * n); ++i) {
        const int k = i < n ? i : i - n;
        const dpred_grad_tensor& t = g[k];
        if (t.rows == 0 || t.cols == 0 || t.counted != (i < n)) continue;
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
            units = ((int64_t)p.rows + p.per - 1) / p.per;
        }
        if (out.empty() || out.back().t.n == kTable) {
            out.emplace_back();
            out.back().t.n = out.back().t.units = out.back().counted = out.back().counted_units = 0;
        }
        Chunk& c = out.back();
        if (units > kMaxUnits - (int64_t)c.t.units) return set_error(DPRED_E_SIZE, "gradient %d is too large", k);
        p.unit0 = c.t.units;
        c.t.units += (int)units;
        c.t.piece[c.t.n++] = p;
        if (i < n) {
            c.counted = c.t.n;
            c.counted_units = c.t.units;
        }
    }
    return DPRED_OK;
}

int blocks_of(int units) { return std::max(1, std::min({units, kBlocksPerSm * sm_count(), kMaxBlocks})); }

// The first n pieces, in a table of no more than needed.
template <int CAP>
Table<CAP> table_of(const Chunk& c, int n, int units) {
    Table<CAP> t;
    t.n = n;
    t.units = units;
    std::copy(c.t.piece, c.t.piece + n, t.piece);
    return t;
}

cudaError_t launch_squares(const Chunk& c, double* partial, cudaStream_t s) {
    const int n = c.counted, u = c.counted_units;
    const dim3 grid(blocks_of(u));
    if (n <= kSmallTable) return launch(squares_kernel<kSmallTable>, grid, kThreads, 0, s, table_of<kSmallTable>(c, n, u), partial);
    if (n <= kMidTable) return launch(squares_kernel<kMidTable>, grid, kThreads, 0, s, table_of<kMidTable>(c, n, u), partial);
    return launch(squares_kernel<kTable>, grid, kThreads, 0, s, table_of<kTable>(c, n, u), partial);
}

cudaError_t launch_scale(const Chunk& c, const double* partial, int sums, float max_norm, float eps, float* out, cudaStream_t s) {
    const int n = c.t.n, u = c.t.units;
    const dim3 grid(blocks_of(u));
    if (n <= kSmallTable) return launch(scale_kernel<kSmallTable>, grid, kThreads, 0, s, table_of<kSmallTable>(c, n, u), partial, sums, max_norm, eps, out);
    if (n <= kMidTable) return launch(scale_kernel<kMidTable>, grid, kThreads, 0, s, table_of<kMidTable>(c, n, u), partial, sums, max_norm, eps, out);
    return launch(scale_kernel<kTable>, grid, kThreads, 0, s, c.t, partial, sums, max_norm, eps, out);
}

// A partial sum per block and launch; calls that count nothing launch one block.
size_t workspace_of(int64_t n) {
    const int64_t launches = std::max<int64_t>(1, (n + kTable - 1) / kTable);
    return (size_t)launches * kMaxBlocks * sizeof(double);
}

int run_squares(const std::vector<Chunk>& chunks, double* partial, int& sums, cudaStream_t s) {
    sums = 0;
    for (const Chunk& c : chunks) {
        if (c.counted == 0) continue;
        const cudaError_t e = launch_squares(c, partial + sums, s);
        if (e != cudaSuccess) return cuda_error(e, "gradient norm launch");
        sums += blocks_of(c.counted_units);
    }
    return DPRED_OK;
}

bool few(const std::vector<Chunk>& c) { return c.empty() || (c.size() == 1 && c[0].t.units <= kFewUnits && c[0].t.n <= kSmallTable); }

template <bool SCALE>
int run_cluster(const std::vector<Chunk>& chunks, float max_norm, float eps, float* out, cudaStream_t s) {
    Table<kSmallTable> t;
    t.n = t.units = 0;
    if (!chunks.empty()) t = table_of<kSmallTable>(chunks[0], chunks[0].t.n, chunks[0].t.units);
    const int counted = chunks.empty() ? 0 : chunks[0].counted;
    const cudaError_t e = launch(cluster_kernel<SCALE>, dim3(kCluster), kThreads, 0, s, t, counted, max_norm, eps, out);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "gradient norm launch");
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
        if (few(chunks)) return run_cluster<false>(chunks, 0.0f, 0.0f, norm, s);
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
        std::vector<Chunk> all;
        if ((rc = plan(grads, n, false, all)) != DPRED_OK) return rc;
        double* partial = static_cast<double*>(workspace);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        if (few(all)) return run_cluster<true>(all, max_norm, eps, result, s);
        int sums = 0;
        if ((rc = run_squares(all, partial, sums, s)) != DPRED_OK) return rc;
        for (size_t k = 0; k < all.size(); ++k) {
            const cudaError_t e = launch_scale(all[k], partial, sums, max_norm, eps, k == 0 ? result : nullptr, s);
            if (e != cudaSuccess) return cuda_error(e, "clipping launch");
        }
        return DPRED_OK;
    });
}
