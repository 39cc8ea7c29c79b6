// block_norm.cuh -- what the block norm and its gradient share: how threads
// cover rows, sums over a row, weights, argument checks.
#pragma once

#include <algorithm>

#include "layers.cuh"

namespace dpred {
namespace layers {

constexpr int kMaxWidth = 16384;

// `lanes` threads (a power of two, whole warps) hold a row, 8 * vecs columns each.
// More columns a thread mean fewer instructions a row (what a row takes besides
// its elements, some 150 for each of its warps, is most of it at 8 columns), fewer
// columns a shorter way through a single one.
struct RowShape {
    int lanes, vecs, threads;
};
inline RowShape shape_of(int64_t d, int most_vecs) {
    RowShape q = {32, 1, 256};
    while (q.vecs < most_vecs && q.lanes * 8 * q.vecs < d) q.vecs *= 2;
    while (q.lanes < 512 && q.lanes * 8 * q.vecs < d) q.lanes *= 2;
    while (q.lanes * 8 * q.vecs < d) q.vecs *= 2;
    q.threads = std::max(q.lanes, 256);  // of a block without a ring
    return q;
}

#ifdef __CUDACC__

// A thread's first column of its v-th group of 8.
template <bool VEC>
__device__ __forceinline__ int first(int v, int id, int lanes) {
    return v * 8 * lanes + (VEC ? 8 * id : id);
}

// All threads of a row group.
__device__ __forceinline__ void group_sync(int group, int lanes) {
    if (lanes == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
}

// Sums over the threads of a row are formed of their sums times 1 / lanes, and times
// lanes / d they are means.  Powers of two round nothing, and no row overflows whose
// threads' own sums, of at most 32 products, do not.
__device__ __forceinline__ float share_of(int lanes) { return __uint_as_float(0x7F000000u - __float_as_uint((float)lanes)); }
__device__ __forceinline__ float mean_of(int lanes, int d) { return (float)lanes * (1.0f / (float)d); }

// Sums over the threads of a row, the same in all of them.  A row of several
// warps has a barrier of its own; one per sum is enough, since sums in turn use
// two places: whoever writes to one again has passed the barrier in between,
// and so has everyone who read it.
struct RowSum {
    int lanes, group, turn = 0;
    __device__ __forceinline__ RowSum(int lanes, int group) : lanes(lanes), group(group) {}

    template <int N>
    __device__ __forceinline__ void operator()(float (&s)[N]) {
        __shared__ float4 warps[2][16];
        static_assert(N <= 4, "sums at once");
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) s[n] += __shfl_xor_sync(0xFFFFFFFFu, s[n], o);
        if (lanes == 32) return;
        const int warp = threadIdx.x / 32, first_warp = group * (lanes / 32);
        if (threadIdx.x % 32 == 0) warps[turn][warp] = make_float4(s[0], N > 1 ? s[1 % N] : 0.0f, N > 2 ? s[2 % N] : 0.0f, N > 3 ? s[3 % N] : 0.0f);
        group_sync(group, lanes);
        float4 t = warps[turn][first_warp];
        for (int w = 1; w < lanes / 32; ++w) {
            const float4 x = warps[turn][first_warp + w];
            t.x += x.x;
            if (N > 1) t.y += x.y;
            if (N > 2) t.z += x.z;
            if (N > 3) t.w += x.w;
        }
        s[0] = t.x;
        if (N > 1) s[1 % N] = t.y;
        if (N > 2) s[2 % N] = t.z;
        if (N > 3) s[3 % N] = t.w;
        turn ^= 1;
    }
};

#endif  // __CUDACC__

constexpr int kMaxStages = 8, kMaxGroups = 16, kSegments = 5;
// Shared memory of a block that has an SM to itself; what is left of it lets the
// next launch's small blocks start beside it.
constexpr int kRoom = 220 * 1024;
constexpr int kBarrierBytes = kMaxGroups * kMaxStages * 8;

// One matrix of a ring, and all of them.
struct Segment {
    const char* p;       // null: not there
    int64_t pitch;       // bytes between rows
    uint32_t bytes, at;  // of a row; where it lies in a slot
    uint32_t div, last;  // rows of the stream that share one of it; its last row
};
struct Rows {
    Segment seg[kSegments];
    uint32_t used;
    int32_t stages, slot_bytes;
    int* err;
    // vec: rows of whole 16-byte pieces; other rows take a piece more than they fill.
    void add(int k, bool vec, const void* p, int64_t m, int64_t ld, int64_t d, int es, int64_t div = 1) {
        const uint32_t bytes = (uint32_t)(d * es);
        seg[k] = {static_cast<const char*>(p), ld * es, bytes, used, (uint32_t)div, (uint32_t)(m / div - 1)};
        used += vec ? bytes : (bytes + 15) / 16 * 16 + 16;
    }
    void drop(int k) {  // the one added last
        used = seg[k].at;
        seg[k] = {};
    }
    int slot() const { return (int)((used + 127) / 128 * 128); }
};

// The ring of a block that has an SM to itself, in `room` bytes: as many row groups
// as may have two slots each (up to `most` threads), then as many slots.  0: not
// even one group may.
inline int ring_groups(const RowShape& q, int slot_bytes, int room, int most) {
    return std::min({kMaxGroups, most / q.lanes, (room - kBarrierBytes) / (2 * slot_bytes)});
}
inline int ring_stages(int groups, int slot_bytes, int room) { return std::min(kMaxStages, (room - kBarrierBytes) / (groups * slot_bytes)); }

#ifdef __CUDACC__

// Rows on their way from global to shared memory by bulk copies: each row group
// of a block has a ring of `stages` slots, and its first thread asks for rows
// ahead of the one that the group works on.  A slot holds one row of up to five
// matrices.
//
// Bulk copies move whole 16-byte pieces.  A row that does not fill its first and
// last piece (VEC false) comes with its neighbours' share of them, which nobody
// looks at, and lies in the slot as far behind a 16-byte boundary as in memory.
// Nothing is read before the matrix or behind it: elements that lie in such a piece
// are copied one by one.
template <bool VEC>
struct Ring {
    uint64_t* full;
    char* slots;
    int stages, slot_bytes;
    int to = 0, from = 0;  // the slot that the next request fills, that the next row comes from
    uint32_t phase = 0;
    int* err;
    long long budget = tma::kWaitBudgetCycles;

    __device__ __forceinline__ Ring(const Rows& in, char* smem, int group)
        : full(reinterpret_cast<uint64_t*>(smem) + group * kMaxStages),
          slots(smem + kBarrierBytes + group * in.stages * in.slot_bytes),
          stages(in.stages), slot_bytes(in.slot_bytes), err(in.err) {}

    // All threads of the block.
    __device__ __forceinline__ void start(int id) {
        if (id == 0) {
            for (int k = 0; k < stages; ++k) tma::mbar_init(full + k, 1);
            tma::fence_barrier_init();
        }
        __syncthreads();
    }

    static __device__ __forceinline__ uintptr_t down(uintptr_t x) { return x & ~(uintptr_t)15; }
    static __device__ __forceinline__ uintptr_t up(uintptr_t x) { return (x + 15) & ~(uintptr_t)15; }

    // Called by the group's first thread, for rows in the order in which take() is called.
    __device__ __forceinline__ void request(const Segment (&seg)[kSegments], int64_t row) {
        char* slot = slots + to * slot_bytes;
        uint32_t all = 0;
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < kSegments; ++k)
                if (seg[k].p) all += seg[k].bytes;
            tma::mbar_arrive_expect_tx(full + to, all);
#pragma unroll
            for (int k = 0; k < kSegments; ++k)
                if (seg[k].p) tma::bulk_load(slot + seg[k].at, row_of(seg[k], row), seg[k].bytes, full + to);
        } else {
            for (int k = 0; k < kSegments; ++k)
                if (seg[k].p) {
                    const Pieces x(seg[k], row_of(seg[k], row));
                    all += x.bytes();
                    if (!x.whole()) {
                        x.copy_rest(slot + seg[k].at);
                        tma::fence_proxy_async_shared();  // bulk copies write these bytes when the slot takes another row
                    }
                }
            tma::mbar_arrive_expect_tx(full + to, all);
            for (int k = 0; k < kSegments; ++k)
                if (seg[k].p) {
                    const Pieces x(seg[k], row_of(seg[k], row));
                    if (x.bytes()) tma::bulk_load(slot + seg[k].at + (x.lo - down(x.s)), reinterpret_cast<const void*>(x.lo), x.bytes(), full + to);
                }
        }
        to = to + 1 == stages ? 0 : to + 1;
    }

    static __device__ __forceinline__ const char* row_of(const Segment& seg, int64_t row) { return seg.p + (seg.div == 1 ? row : row / seg.div) * seg.pitch; }

    // A row [s, e) and the pieces [lo, hi) that may be copied for it.
    struct Pieces {
        uintptr_t s, e, lo, hi;
        __device__ __forceinline__ Pieces(const Segment& seg, const char* row) {
            const uintptr_t start = reinterpret_cast<uintptr_t>(seg.p), end = start + seg.last * seg.pitch + seg.bytes;
            s = reinterpret_cast<uintptr_t>(row);
            e = s + seg.bytes;
            lo = max(down(s), up(start));
            hi = min(up(e), down(end));
        }
        __device__ __forceinline__ uint32_t bytes() const { return lo < hi ? (uint32_t)(hi - lo) : 0; }
        __device__ __forceinline__ bool whole() const { return lo <= s && hi >= e; }
        // What lies before and behind them, element by element.
        __device__ __forceinline__ void copy_rest(char* place) const {
            char* there = place - down(s);  // an address plus this is its place
            const uintptr_t head = lo < hi ? lo : e;
            for (uintptr_t x = s; x < head; x += 2) *reinterpret_cast<uint16_t*>(there + x) = *reinterpret_cast<const uint16_t*>(x);
            for (uintptr_t x = max(head, hi); x < e; x += 2) *reinterpret_cast<uint16_t*>(there + x) = *reinterpret_cast<const uint16_t*>(x);
        }
    };

    // Where a row of a matrix (at `row` in memory) lies in its slot.
    template <typename T>
    static __device__ __forceinline__ const T* in(const char* slot, const Segment& seg, const T* row) {
        return reinterpret_cast<const T*>(slot + seg.at + (VEC ? 0 : reinterpret_cast<uintptr_t>(row) % 16));
    }

    // The slot of the next row, once it is there.  A wait that gives up is
    // reported, and the ones after it give up at once: the block still ends.
    __device__ __forceinline__ const char* take() {
        if (!tma::mbar_wait(full + from, phase, budget)) {
            record_device_error(err, DPRED_E_TIMEOUT);
            budget = 1000;
        }
        const char* slot = slots + from * slot_bytes;
        if (++from == stages) {
            from = 0;
            phase ^= 1;
        }
        return slot;
    }
};

#endif  // __CUDACC__

// A weight vector, or gate rows, of either type; p is null where there is none.
struct Weight {
    const void* p;
    int32_t f32;
    int64_t ld;
#ifdef __CUDACC__
    // One element; 1 where there is no weight.
    __device__ __forceinline__ float at(int64_t row, int c) const {
        if (!p) return 1.0f;
        return f32 ? static_cast<const float*>(p)[row * ld + c] : load1(static_cast<const __nv_bfloat16*>(p) + row * ld + c);
    }
    template <bool VEC>
    __device__ __forceinline__ F8 load(int64_t row, int c0, int step, int d) const {
        if (f32) {
            Cols<float, VEC> q;
            q.load(static_cast<const float*>(p) + row * ld, c0, step, d);
            return widen(q);
        }
        Cols<__nv_bfloat16, VEC> q;
        q.load(static_cast<const __nv_bfloat16*>(p) + row * ld, c0, step, d);
        return widen(q);
    }
#endif
};

#ifdef __CUDACC__

// Weights of a row in shared memory, in fp32 and in the order in which threads
// take them, so that the loop over rows has no flags, types or bank conflicts: a
// thread's columns lie together, their 16-byte pieces exchanged among themselves
// so that eight threads in a row read eight different bank groups (VEC), or
// column by column.  Columns from d on are 0.
template <bool VEC, int VPT>
struct Staged {
    float* at;
    int lanes;
    // Where thread id has column k of its v-th eight.
    __device__ __forceinline__ int place(int v, int id, int k) const {
        if (!VEC) return (v * 8 + k) * lanes + id;
        constexpr int kPieces = 2 * VPT;  // of 4 columns
        const int turn = id / (8 / kPieces) & (kPieces - 1);
        return (id * kPieces + ((v * 2 + k / 4) ^ turn)) * 4 + k % 4;
    }
    __device__ __forceinline__ F8 get(int v, int id) const {
        F8 f;
        if constexpr (VEC) {
            const float4 a = *reinterpret_cast<const float4*>(at + place(v, id, 0)), b = *reinterpret_cast<const float4*>(at + place(v, id, 4));
            f.p[0] = make_float2(a.x, a.y); f.p[1] = make_float2(a.z, a.w); f.p[2] = make_float2(b.x, b.y); f.p[3] = make_float2(b.z, b.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f.p[i] = make_float2(at[place(v, id, 2 * i)], at[place(v, id, 2 * i + 1)]);
        }
        return f;
    }
};

// All threads of a block: f(column, it is one, place) for every column that their
// vectors cover; f is to load its weights before it writes any, and 0 behind the row.
template <bool VEC, int VPT, typename F>
__device__ __forceinline__ void fill(int lanes, int d, F f) {
    const Staged<VEC, VPT> s = {nullptr, lanes};
    for (int i = threadIdx.x; i < VPT * 8 * lanes; i += blockDim.x) {
        const int k = VEC ? i % 8 : i / lanes % 8, id = VEC ? i / 8 % lanes : i % lanes, v = i / (8 * lanes);
        const int c = column<VEC>(first<VEC>(v, id, lanes), lanes, k);
        f(c, c < d, s.place(v, id, k));
    }
}
inline __host__ __device__ int staged_floats(int lanes, int vecs) { return 8 * lanes * vecs; }

#endif  // __CUDACC__

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
    const struct { const void* p; int32_t dt; const char* name; } w[] = {
        {n.post, n.post_dtype, "post"}, {n.gate, n.gate_dtype, "gate"}, {n.pre, n.pre_dtype, "pre"}};
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
