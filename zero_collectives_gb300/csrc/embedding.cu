// embedding.cu -- the token embedding and its gradient: dpred_embedding and
// dpred_embedding_grad.
//
//     y[t]  = scale W[id(t)]
//     dW[v] = (dW[v] +) scale * sum of dy[t] over the tokens t with id(t) = v
//
// The embedding is the largest task of a bucket flush (98304 x 1024 of the
// 402.8M parameters).  Its gradient is summed in fp32 in one fixed order: the
// tokens of a row in ascending t, in runs of 4 to 32 positions of the sorted order
// whose sums are then added in ascending order.  Three launches:
//
//  sort   Tokens are ordered by the low bits of their id, then by the rest, then
//         by t.  Every block owns the ids with its low bits (frequent ids lie next
//         to each other, so this spreads them) and reads all ids: it counts those
//         with lower low bits (where its tokens start in the order) and those of
//         each of its rows, per warp, then places its tokens.  No block waits for
//         another.  Reading T ids per SM from L2 costs T / 30000 us, a ninth at
//         most of what T rows of 2 KB take from HBM.
//  sum    A warp takes a run of positions and 256 columns, eight rows in flight.
//         Rows whose tokens lie inside the run are written; what continues from or
//         into other runs is left as a partial sum.  Work is the same whatever the
//         ids are: one row with all tokens is cut like any other.  Where the whole
//         table is stored, other blocks write the rows without a token.
//  join   Adds the partial sums of the rows that were cut.
//
// Bandwidth bound: dy is read once and each row of dW written once (read and
// written once where it is added to, and only where a token is).
#include <algorithm>

#include "layers.cuh"

namespace dpred {
namespace layers {
namespace {

// ------------------------------------------------------------------- lookup --

constexpr int kLookThreads = 256;

struct LookArgs {
    const void* ids;
    const void* w;
    void* y;
    int64_t t, v, ldw, ldy;
    int32_t d, id64;
    float scale;
    int* err;
};

// The id of token t, -1 where it is outside the table or t behind the last token.
__device__ __forceinline__ int64_t checked_id(const LookArgs& a, int64_t t, bool report) {
    if (t >= a.t) return -1;
    const int64_t id = a.id64 ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t];
    if (id >= 0 && id < a.v) return id;
    if (report) record_device_error(a.err, DPRED_E_BOUNDS);
    return -1;
}

// `lanes` threads of a warp cover a row, CH vectors of 8 columns each at a time; a
// thread has 8 vectors in flight, of 8 / CH rows.  (More rows for each warp in turn,
// with the next ids asked for meanwhile: 11.0 us a call with warm caches instead of 9.9
// for 16384 tokens of 1024 columns.  From cold caches the kernel takes 11.2-12.9 us.)
template <typename TW, typename TY, int CH>
__global__ void __launch_bounds__(kLookThreads) lookup_kernel(const __grid_constant__ LookArgs a, int lanes) {
    constexpr int R = 8 / CH;
    mma::grid_wait();
    const int lane = threadIdx.x & (lanes - 1), sub = 32 / lanes, part = threadIdx.x % 32 / lanes;
    const int64_t step = (int64_t)gridDim.x * (kLookThreads / 32) * sub * R;
    for (int64_t t0 = ((int64_t)blockIdx.x * (kLookThreads / 32) + threadIdx.x / 32) * sub * R + part; t0 < a.t; t0 += step) {
        int64_t id[R];
#pragma unroll
        for (int u = 0; u < R; ++u) id[u] = checked_id(a, t0 + u * sub, lane == 0);
        for (int c0 = 0; c0 < a.d; c0 += CH * lanes * 8) {
            Eight<TW> q[R][CH];
#pragma unroll
            for (int u = 0; u < R; ++u)
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const int c = c0 + (k * lanes + lane) * 8;
                    if (id[u] >= 0 && c < a.d)
                        q[u][k].load(static_cast<const TW*>(a.w) + id[u] * a.ldw + c);
                    else
                        q[u][k] = {};
                }
#pragma unroll
            for (int u = 0; u < R; ++u) {
                const int64_t t = t0 + u * sub;
                if (t >= a.t) continue;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const int c = c0 + (k * lanes + lane) * 8;
                    if (c < a.d) store_cols<true>(static_cast<TY*>(a.y) + t * a.ldy, c, 0, a.d, widen(q[u][k]) * splat(a.scale));
                }
            }
        }
    }
}

// Rows without 16-byte alignment: a warp per row, element by element (16384 tokens of
// 777 columns 12.1 us, floor 5.4; of 1024 in rows of 1027 15.4, floor 7.0).
template <typename TW, typename TY>
__global__ void __launch_bounds__(kLookThreads) lookup_any_kernel(const __grid_constant__ LookArgs a) {
    mma::grid_wait();
    const int lane = threadIdx.x % 32;
    for (int64_t t = (int64_t)blockIdx.x * (kLookThreads / 32) + threadIdx.x / 32; t < a.t; t += (int64_t)gridDim.x * (kLookThreads / 32)) {
        const int64_t id = checked_id(a, t, lane == 0);
        const TW* w = static_cast<const TW*>(a.w) + (id < 0 ? 0 : id * a.ldw);
        TY* y = static_cast<TY*>(a.y) + t * a.ldy;
        for (int c0 = lane; c0 < a.d; c0 += 256) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = id >= 0 && c0 + 32 * k < a.d ? load1(w + c0 + 32 * k) * a.scale : 0.0f;
            store_cols<false>(y, c0, 32, a.d, f);
        }
    }
}

// --------------------------------------------------------------------- sort --

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxRows = 4096;            // of a block
constexpr int kCounters = 160 * 1024;     // bytes: one for each of its rows and warps
constexpr int kHeld = 16;                 // ids that a thread has in flight
constexpr int kList = 96;                 // tokens of the block that a warp lists

struct SortArgs {
    const void* ids;
    int64_t t;
    uint32_t v, padding;  // this id's tokens give no gradient; kNoId: none
    int32_t shift;        // the low bits of an id say which block has it
    int32_t rows;         // rows of a block, a multiple of 32
    int32_t warps;        // warps that share the tokens
    int32_t* key;         // [t] id of a sorted position
    int32_t* order;       // [t] its token
    uint32_t* met;        // [blocks][rows / 32] bits: rows with a token (null: not wanted)
    int32_t* count;       // sorted positions in all
    int* err;
};
constexpr uint32_t kNoId = 0xFFFFFFFFu;

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// An id, or kNoId where it gives no gradient.
template <typename I>
__device__ __forceinline__ uint32_t usable_id(const SortArgs& a, int64_t t, bool& outside) {
    const I id = static_cast<const I*>(a.ids)[t];
    if constexpr (sizeof(I) == 8) {
        if (static_cast<uint64_t>(id) >= a.v) {
            outside = true;
            return kNoId;
        }
    } else if (static_cast<uint32_t>(id) >= a.v) {
        outside = true;
        return kNoId;
    }
    return static_cast<uint32_t>(id) == a.padding ? kNoId : static_cast<uint32_t>(id);
}

// How many tokens of a row a warp has met, then how many of the row come before
// its next one; two rows in a word where no count passes 16 bits (HALF).
template <bool HALF>
struct Counters {
    uint32_t* w;
    __device__ __forceinline__ uint32_t* word(int row) const { return w + (HALF ? row / 2 : row); }
    __device__ __forceinline__ uint32_t one(int row) const { return HALF && (row & 1) ? 0x10000u : 1u; }
    __device__ __forceinline__ int get(int row) const { return HALF ? (*word(row) >> (row & 1) * 16) & 0xFFFF : *word(row); }
};

template <typename I, bool HALF>
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint32_t counters[];  // [warps][words]
    __shared__ int below[kSortWarps], sums[kSortWarps], starts[kMaxRows];
    __shared__ uint32_t bits[kMaxRows / 32];
    __shared__ int2 lists[kSortWarps][kList];  // row and token, in order
    mma::grid_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, words = HALF ? a.rows / 2 : a.rows;
    const uint32_t mask = (1u << a.shift) - 1, me = blockIdx.x, rows = a.rows, before_me = (1u << lane) - 1;
    for (int i = threadIdx.x * 4; i < a.warps * words; i += kSortThreads * 4) *reinterpret_cast<int4*>(counters + i) = make_int4(0, 0, 0, 0);
    if (threadIdx.x < kMaxRows / 32) bits[threadIdx.x] = 0;
    __syncthreads();
    mma::grid_wait();
    // each warp has one stretch of the tokens, a multiple of 32
    const int64_t per = (a.t + a.warps * 32 - 1) / (a.warps * 32) * 32;
    const int64_t t0 = warp * per, t1 = warp < a.warps ? min(a.t, t0 + per) : 0;
    const Counters<HALF> mine = {counters + warp * words};
    int2* list = lists[warp];
    int less = 0, listed = 0;
    bool outside = false;
    for (int64_t base = t0; base < t1; base += 32 * kHeld) {
        uint32_t id[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int64_t t = base + 32 * u + lane;
            id[u] = t < t1 ? usable_id<I>(a, t, outside) : kNoId;
        }
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            // kNoId has the highest low bits and no row
            less += (id[u] & mask) < me;
            const uint32_t row = id[u] >> a.shift;
            const bool here = (id[u] & mask) == me && row < rows;
            const unsigned met = __ballot_sync(0xFFFFFFFFu, here);
            if (here) {
                const int at = listed + __popc(met & before_me);
                if (at < kList) list[at] = make_int2((int)row, (int)(base + 32 * u + lane));
                atomicAdd(mine.word(row), mine.one(row));
            }
            listed += __popc(met);
        }
    }
    if (outside && blockIdx.x == 0) record_device_error(a.err, DPRED_E_BOUNDS);
    less = warp_sum(less);
    if (lane == 0) below[warp] = less;
    __syncthreads();
    // over the warps, what comes before each one's tokens of a row; a thread has up
    // to 4 rows next to each other
    constexpr int kPer = HALF ? 2 : 1;  // rows of a word
    const int each = (words + kSortThreads - 1) / kSortThreads, w0 = min((int)threadIdx.x * each, words), w1 = min(w0 + each, words);
    int total = 0;
    uint32_t sum[kMaxRows / kSortThreads];
#pragma unroll
    for (int i = 0; i < kMaxRows / kSortThreads; ++i) {
        sum[i] = 0;
        if (w0 + i >= w1) continue;
#pragma unroll 8
        for (int w = 0; w < a.warps; ++w) {
            uint32_t& c = counters[w * words + w0 + i];
            const uint32_t n = c;
            c = sum[i];
            sum[i] += n;
        }
        const int r = (w0 + i) * kPer;
        const uint32_t some = HALF ? ((sum[i] & 0xFFFF) != 0) | ((sum[i] >> 16 != 0) << 1) : sum[i] != 0;
        if (some && a.met) atomicOr(bits + r / 32, some << r % 32);
        total += HALF ? (sum[i] & 0xFFFF) + (sum[i] >> 16) : sum[i];
    }
    // where each row starts in the order
    int before = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) sums[warp] = before;
    before -= total;
    __syncthreads();
    before += warp_sum(lane < warp ? sums[lane] : 0) + warp_sum(below[lane]);
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == kSortThreads - 1) *a.count = before + total;
    if (a.met && threadIdx.x < a.rows / 32) a.met[(int64_t)blockIdx.x * (a.rows / 32) + threadIdx.x] = bits[threadIdx.x];
#pragma unroll
    for (int i = 0; i < kMaxRows / kSortThreads; ++i) {
        if (w0 + i >= w1) continue;
        starts[(w0 + i) * kPer] = before;
        if (HALF) {
            before += sum[i] & 0xFFFF;
            starts[(w0 + i) * 2 + 1] = before;
            before += sum[i] >> 16;
        } else {
            before += sum[i];
        }
    }
    __syncthreads();
    // up to 32 tokens in ascending order, row by row
    auto place = [&](bool here, uint32_t row, int token) {
        unsigned left = __ballot_sync(0xFFFFFFFFu, here);
        while (left) {
            const uint32_t r = __shfl_sync(0xFFFFFFFFu, row, __ffs(left) - 1);
            const unsigned same = __ballot_sync(0xFFFFFFFFu, here && row == r);
            left &= ~same;
            const int at = starts[r] + mine.get(r) + __popc(same & before_me);
            __syncwarp();
            if (same >> lane & 1) {
                a.key[at] = (int32_t)(r << a.shift | me);
                a.order[at] = token;
                if ((same >> lane) == 1u) *mine.word(r) += mine.one(r) * __popc(same);  // the last of them
            }
            __syncwarp();
        }
    };
    if (listed <= kList) {
        for (int i = 0; i < listed; i += 32) {
            const int2 e = list[min(i + lane, kList - 1)];
            place(i + lane < listed, e.x, e.y);
        }
        return;
    }
    for (int64_t base = t0; base < t1; base += 32 * kHeld) {
        uint32_t id[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int64_t t = base + 32 * u + lane;
            id[u] = t < t1 ? usable_id<I>(a, t, outside) : kNoId;
        }
#pragma unroll
        for (int u = 0; u < kHeld; ++u) place((id[u] & mask) == me && (id[u] >> a.shift) < rows, id[u] >> a.shift, (int)(base + 32 * u + lane));
    }
}

// ---------------------------------------------------------------------- sum --

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kSlab = 256;      // columns of a warp
constexpr int kFillRows = 8;    // rows of a warp that writes zeros
constexpr int kMostRun = 32;    // positions of a run

struct SumArgs {
    const void* dy;
    void* dw;
    const int32_t *key, *order, *count;
    const uint32_t* met;   // null: rows without a token stay as they are
    float *head, *tail;    // [runs][d] partial sums: of the row that began before the run, of the one that goes on behind it
    int64_t ldy, ldw, v;
    int32_t d, slabs, run;  // run: positions, a power of two
    int32_t shift, rows;    // as in SortArgs
    int64_t runs, sum_blocks;
    float scale;
};

// A lane's first column of a slab.
template <bool VEC>
__device__ __forceinline__ int first_column(int base, int lane) {
    return VEC ? base + lane * 8 : base + lane;
}

__device__ __forceinline__ F8 plus(const F8& a, const F8& b) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = make_float2(a.p[i].x + b.p[i].x, a.p[i].y + b.p[i].y);
    return f;
}

// ADD: the sums are added to rows of dw, which are asked for with the last of
// their tokens' rows.
template <typename TG, typename TW, bool VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumArgs a) {
    if (a.runs > 1) mma::grid_launch_dependents();  // another launch of the call follows
    mma::grid_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    TW* dw = static_cast<TW*>(a.dw);
    if (blockIdx.x >= a.sum_blocks) {  // zeros for the rows without a token
        const int64_t v0 = ((blockIdx.x - a.sum_blocks) * kSumWarps + warp) * kFillRows, id = v0 + lane;
        bool met = true;
        if (lane < kFillRows && id < a.v) {
            const int64_t block = id & ((1 << a.shift) - 1), r = id >> a.shift;
            met = a.met[block * (a.rows / 32) + r / 32] >> (r % 32) & 1;
        }
        const unsigned without = __ballot_sync(0xFFFFFFFFu, !met);
        const F8 zero = splat(0.0f);
#pragma unroll
        for (int r = 0; r < kFillRows; ++r)
            if (without >> r & 1)
                for (int base = 0; base < a.d; base += kSlab) store_cols<VEC>(dw + (v0 + r) * a.ldw, first_column<VEC>(base, lane), 32, a.d, zero);
        return;
    }
    const int64_t item = (int64_t)blockIdx.x * kSumWarps + warp, run = item / a.slabs;
    const int c0 = first_column<VEC>((int)(item % a.slabs) * kSlab, lane);
    const int64_t n = *a.count, p0 = run * a.run;
    if (p0 >= n) return;
    const int len = (int)min((int64_t)a.run, n - p0);
    const int32_t key = lane < len ? a.key[p0 + lane] : -1, token = lane < len ? a.order[p0 + lane] : 0;
    const int32_t after = p0 + len < n ? a.key[p0 + len] : -1, ahead = p0 > 0 ? a.key[p0 - 1] : -1;
    const int32_t next = __shfl_down_sync(0xFFFFFFFFu, key, 1);
    // positions that end a row's share of this run; the row that began before, and the one that goes on behind it
    const unsigned ends = __ballot_sync(0xFFFFFFFFu, lane < len && (lane == len - 1 || key != next));
    const unsigned head = __shfl_sync(0xFFFFFFFFu, key, 0) == ahead ? ends & (0u - ends) : 0u;
    const unsigned tail = __shfl_sync(0xFFFFFFFFu, key, len - 1) == after ? (1u << (len - 1)) & ~head : 0u;
    const unsigned whole = ends & ~head & ~tail;
    const TG* dy = static_cast<const TG*>(a.dy);
    const F8 scale = splat(a.scale);
    F8 sum = splat(0.0f);
    constexpr int U = ADD ? 4 : 8;
    for (int i = 0; i < len; i += U) {
        Cols<TG, VEC> q[U];
        Cols<TW, VEC> old[ADD ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = __shfl_sync(0xFFFFFFFFu, token, (i + u) % 32), row = __shfl_sync(0xFFFFFFFFu, key, (i + u) % 32);
            if (i + u < len) q[u].load(dy + t * a.ldy, c0, 32, a.d);
            if (ADD && (whole >> (i + u) & 1)) old[ADD ? u : 0].load(dw + row * a.ldw, c0, 32, a.d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = __shfl_sync(0xFFFFFFFFu, key, (i + u) % 32);
            if (i + u >= len) continue;
            sum = plus(sum, widen(q[u]));
            if (!(ends >> (i + u) & 1)) continue;
            if (head >> (i + u) & 1)
                store_cols<VEC>(a.head + run * a.d, c0, 32, a.d, sum);
            else if (tail >> (i + u) & 1)
                store_cols<VEC>(a.tail + run * a.d, c0, 32, a.d, sum);
            else
                store_cols<VEC>(dw + row * a.ldw, c0, 32, a.d, ADD ? fma8(sum, scale, widen(old[ADD ? u : 0])) : sum * scale);
            sum = splat(0.0f);
        }
    }
}

// The rows that begin in a run and go on behind it: the tail there and the heads of
// the runs that follow.  A warp looks at one run; it adds a few heads itself, and
// leaves a longer row to all warps of the block, whose shares are added in order.
// 16384 tokens stored, 8192 added: 48.5 and 21.2 us; with 2 heads 49.2 and 22.0, with
// 32 heads 52.2 and 23.2.
constexpr int kFewHeads = 8;

template <bool VEC>
__device__ __forceinline__ F8 sum_heads(const SumArgs& a, int64_t q0, int64_t q1, int c0) {
    F8 sum = splat(0.0f);
    constexpr int U = 4;
    for (int64_t q = q0; q < q1; q += U) {
        Cols<float, VEC> f[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + u < q1) f[u].load(a.head + (q + u) * a.d, c0, 32, a.d);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + u < q1) sum = plus(sum, widen(f[u]));
    }
    return sum;
}

template <bool VEC, bool ADD, typename TW>
__device__ __forceinline__ void leave(TW* p, int c0, int d, const F8& sum, float scale) {
    if (ADD) {
        Cols<TW, VEC> old;
        old.load(p, c0, 32, d);
        store_cols<VEC>(p, c0, 32, d, fma8(sum, splat(scale), widen(old)));
    } else {
        store_cols<VEC>(p, c0, 32, d, sum * splat(scale));
    }
}

template <typename TW, bool VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const __grid_constant__ SumArgs a) {
    __shared__ float part[kSumWarps][kSlab];
    __shared__ int64_t heads[kSumWarps];
    mma::grid_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int c0 = first_column<VEC>((int)(blockIdx.x % a.slabs) * kSlab, lane);
    const int64_t run0 = (int64_t)(blockIdx.x / a.slabs) * kSumWarps, run = run0 + warp, n = *a.count, p0 = run * a.run;
    TW* dw = static_cast<TW*>(a.dw);
    int64_t more = 0;  // runs behind this one that begin with the row that begins here
    if (p0 + a.run < n) {
        const int32_t row = a.key[p0 + a.run - 1], after = a.key[p0 + a.run], first = a.key[p0], ahead = p0 > 0 ? a.key[p0 - 1] : -1;
        if (after == row && !(first == row && ahead == row)) {
            const int64_t runs = (n + a.run - 1) / a.run;
            for (;;) {
                const int64_t r = run + 1 + more + lane;
                const unsigned same = __ballot_sync(0xFFFFFFFFu, r < runs && a.key[min(r, runs - 1) * a.run] == row);
                const int k = same == 0xFFFFFFFFu ? 32 : __ffs(~same) - 1;
                more += k;
                if (k < 32) break;
            }
            if (more <= kFewHeads) {
                Cols<float, VEC> first_part;
                first_part.load(a.tail + run * a.d, c0, 32, a.d);
                leave<VEC, ADD>(dw + (int64_t)row * a.ldw, c0, a.d, plus(widen(first_part), sum_heads<VEC>(a, run + 1, run + 1 + more, c0)), a.scale);
            }
        }
    }
    if (lane == 0) heads[warp] = more;
    __syncthreads();
    for (int w = 0; w < kSumWarps; ++w) {
        const int64_t k = heads[w], q0 = run0 + w + 1;
        if (k <= kFewHeads) continue;
        const F8 mine = sum_heads<VEC>(a, q0 + k * warp / kSumWarps, q0 + k * (warp + 1) / kSumWarps, c0);
        __syncthreads();  // the row before is done with part
#pragma unroll
        for (int i = 0; i < 8; ++i) part[warp][i * 32 + lane] = mine.get(i);
        __syncthreads();
        if (warp) continue;
        Cols<float, VEC> first_part;
        first_part.load(a.tail + (q0 - 1) * a.d, c0, 32, a.d);
        F8 sum = widen(first_part);
        for (int x = 0; x < kSumWarps; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum.p[i].x += part[x][2 * i * 32 + lane];
                sum.p[i].y += part[x][(2 * i + 1) * 32 + lane];
            }
        leave<VEC, ADD>(dw + (int64_t)a.key[q0 * a.run] * a.ldw, c0, a.d, sum, a.scale);
    }
}

// --------------------------------------------------------------------- host --

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
int64_t slabs_of(int64_t d) { return (d + kSlab - 1) / kSlab; }

// Positions of a run: 32 where that leaves 2048 warps (13 to an SM) or more, fewer
// where there are fewer tokens, so that they keep the SMs busy too.  (1024 warps:
// the gradient of 8192 tokens takes 27 us instead of 21; 8192: of 16384 51 instead of 48.)
int run_of(int64_t t, int64_t d) {
    int run = kMostRun;
    while (run > 4 && t * slabs_of(d) < (int64_t)2048 * run) run /= 2;
    return run;
}
int64_t runs_of(int64_t t, int64_t d) { return (t + run_of(t, d) - 1) / run_of(t, d); }

// How the ids are dealt out: to 128 blocks, or to more where a block would have
// more than kMaxRows rows.
struct Deal {
    int shift, rows;
};
Deal deal_of(int64_t v) {
    Deal q = {7, 0};
    while (((v - 1) >> q.shift) + 1 > kMaxRows) ++q.shift;
    q.rows = (int)((((v - 1) >> q.shift) + 1 + 31) / 32 * 32);
    return q;
}

struct Space {
    int64_t key, order, met, count, head, tail, bytes;
};
Space space_of(int64_t t, int64_t v, int64_t d) {
    Space s;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t p = at;
        at += align256(n);
        return p;
    };
    const Deal q = deal_of(v);
    s.key = take(t * 4);
    s.order = take(t * 4);
    s.met = take(((int64_t)q.rows << q.shift) / 8);
    s.count = take(4);
    s.head = take(runs_of(t, d) * d * 4);
    s.tail = take(runs_of(t, d) * d * 4);
    s.bytes = at;
    return s;
}

int check_sizes(int64_t t, int64_t v, int64_t d, int32_t id_bytes) {
    if (t < 0 || v < 0 || d < 0) return set_error(DPRED_E_INVAL, "a negative size (%lld, %lld, %lld)", (long long)t, (long long)v, (long long)d);
    if (t > 0x3FFFFFFF || v > 0x3FFFFFFF || d > (1 << 20))
        return set_error(DPRED_E_SIZE, "%lld tokens, %lld rows of %lld: at most 2^30 - 1, 2^30 - 1 and 2^20", (long long)t, (long long)v, (long long)d);
    if (id_bytes != 4 && id_bytes != 8) return set_error(DPRED_E_INVAL, "ids of %d bytes: 4 or 8", id_bytes);
    return DPRED_OK;
}

int check_ids(const void* ids, int64_t t, int32_t id_bytes) {
    if (t > 0 && !ids) return set_error(DPRED_E_INVAL, "ids is null");
    if (reinterpret_cast<uintptr_t>(ids) % id_bytes) return set_error(DPRED_E_ALIGN, "ids is not aligned to its element size");
    return DPRED_OK;
}

template <typename TW, typename TY, int CH>
cudaError_t launch_rows(const LookArgs& a, int lanes, cudaStream_t s) {
    const int64_t per = (int64_t)(kLookThreads / 32) * (32 / lanes) * (8 / CH), blocks = (a.t + per - 1) / per;
    return launch(lookup_kernel<TW, TY, CH>, dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)), kLookThreads, 0, s, a, lanes);
}

template <typename TW, typename TY>
cudaError_t launch_lookup(const LookArgs& a, bool vec, cudaStream_t s) {
    if (!vec) return launch(lookup_any_kernel<TW, TY>, dim3((unsigned)std::min<int64_t>((a.t + 7) / 8, 1 << 20)), kLookThreads, 0, s, a);
    int lanes = 1;
    while (lanes < 32 && lanes * 8 < a.d) lanes *= 2;
    if (a.d <= 256) return launch_rows<TW, TY, 1>(a, lanes, s);
    if (a.d <= 512) return launch_rows<TW, TY, 2>(a, lanes, s);
    if (a.d <= 1024) return launch_rows<TW, TY, 4>(a, lanes, s);
    return launch_rows<TW, TY, 8>(a, lanes, s);
}

template <typename I, bool HALF>
cudaError_t launch_sort(const SortArgs& q, unsigned blocks, int per_warp, cudaStream_t s) {
    static bool done[64];
    const cudaError_t e = ensure_smem_attr(sort_kernel<I, HALF>, kCounters, done);
    return e == cudaSuccess ? launch(sort_kernel<I, HALF>, dim3(blocks), kSortThreads, (size_t)q.warps * per_warp, s, q) : e;
}

template <typename TG, typename TW, bool VEC, bool ADD>
cudaError_t launch_sums(const SumArgs& a, unsigned blocks, cudaStream_t s) {
    const cudaError_t e = launch(sum_kernel<TG, TW, VEC, ADD>, dim3(blocks), kSumThreads, 0, s, a);
    if (e != cudaSuccess || a.runs <= 1) return e;
    return launch(join_kernel<TW, VEC, ADD>, dim3((unsigned)((a.runs - 1 + kSumWarps - 1) / kSumWarps * a.slabs)), kSumThreads, 0, s, a);
}

template <typename TG, typename TW>
cudaError_t launch_sums(const SumArgs& a, bool vec, bool add, unsigned blocks, cudaStream_t s) {
    if (vec) return add ? launch_sums<TG, TW, true, true>(a, blocks, s) : launch_sums<TG, TW, true, false>(a, blocks, s);
    return add ? launch_sums<TG, TW, false, true>(a, blocks, s) : launch_sums<TG, TW, false, false>(a, blocks, s);
}

}  // namespace
}  // namespace layers
}  // namespace dpred

using namespace dpred;
using namespace dpred::layers;

extern "C" int dpred_embedding(int64_t t, int64_t v, int64_t d, int32_t id_bytes, const void* ids, int32_t w_dtype, const void* w, int64_t ldw,
                               float scale, int32_t out_dtype, void* y, int64_t ldy, void* stream) {
    int rc = check_sizes(t, v, d, id_bytes);
    if (rc != DPRED_OK || (rc = check_dtype(w_dtype, "w")) != DPRED_OK || (rc = check_dtype(out_dtype, "y")) != DPRED_OK) return rc;
    if (!std::isfinite(scale)) return set_error(DPRED_E_INVAL, "scale is not finite");
    if (t == 0 || d == 0) return DPRED_OK;
    const int ws = esize(w_dtype), ys = esize(out_dtype);
    if ((rc = check_ids(ids, t, id_bytes)) != DPRED_OK || (rc = check_matrix(w, v, d, ldw, ws, "w")) != DPRED_OK ||
        (rc = check_matrix(y, t, d, ldy, ys, "y")) != DPRED_OK)
        return rc;
    const LookArgs a = {ids, w, y, t, v, ldw, ldy, (int32_t)d, id_bytes == 8, scale, device_error_word()};
    const bool vec = d % 8 == 0 && aligned_rows(w, v, ldw, ws) && aligned_rows(y, t, ldy, ys);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool out_f32 = out_dtype == DPRED_F32;
    cudaError_t e;
    if (w_dtype == DPRED_F32)
        e = out_f32 ? launch_lookup<float, float>(a, vec, s) : launch_lookup<float, __nv_bfloat16>(a, vec, s);
    else
        e = out_f32 ? launch_lookup<__nv_bfloat16, float>(a, vec, s) : launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "embedding launch");
}

extern "C" size_t dpred_embedding_grad_workspace_bytes(int64_t t, int64_t v, int64_t d) {
    if (t < 0 || v <= 0 || d <= 0 || check_sizes(t, v, d, 4) != DPRED_OK) return 0;
    return (size_t)space_of(t, v, d).bytes;
}

extern "C" int dpred_embedding_grad(int64_t t, int64_t v, int64_t d, int32_t id_bytes, const void* ids, int64_t padding, int32_t g_dtype,
                                    const void* dy, int64_t lddy, float scale, int32_t accumulate, int32_t out_dtype, void* dw, int64_t lddw,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_sizes(t, v, d, id_bytes);
    if (rc != DPRED_OK || (rc = check_dtype(g_dtype, "dy")) != DPRED_OK || (rc = check_dtype(out_dtype, "dw")) != DPRED_OK) return rc;
    if (!std::isfinite(scale)) return set_error(DPRED_E_INVAL, "scale is not finite");
    if (padding < -1 || padding >= std::max<int64_t>(v, 1))
        return set_error(DPRED_E_INVAL, "padding %lld outside -1..%lld", (long long)padding, (long long)v - 1);
    const int gs = esize(g_dtype), ws = esize(out_dtype);
    if (v == 0 || d == 0) return DPRED_OK;
    if ((rc = check_ids(ids, t, id_bytes)) != DPRED_OK || (rc = check_matrix(dy, t, d, lddy, gs, "dy")) != DPRED_OK ||
        (rc = check_matrix(dw, v, d, lddw, ws, "dw")) != DPRED_OK)
        return rc;
    if (t == 0 && accumulate) return DPRED_OK;
    const int64_t slabs = slabs_of(d), runs = runs_of(t, d), sum_blocks = (runs * slabs + kSumWarps - 1) / kSumWarps;
    const int64_t blocks = sum_blocks + (accumulate ? 0 : (v + kSumWarps * kFillRows - 1) / (kSumWarps * kFillRows));
    if (blocks > 0x7FFFFFFF || runs * slabs > 0x7FFFFFFF)
        return set_error(DPRED_E_SIZE, "%lld tokens of %lld columns are too many", (long long)t, (long long)d);
    const Space sp = space_of(t, v, d);
    if ((rc = check_workspace(workspace, workspace_bytes, (size_t)sp.bytes)) != DPRED_OK) return rc;
    char* base = static_cast<char*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Deal deal = deal_of(v);

    SortArgs q = {};
    q.ids = ids;
    q.t = t;
    q.v = (uint32_t)v;
    q.padding = padding < 0 ? kNoId : (uint32_t)padding;
    q.shift = deal.shift;
    q.rows = deal.rows;
    // a set of counters for each 128 tokens, so that few tokens clear few, as far as there is room
    const bool half = t <= 0xFFFF;
    const int per_warp = deal.rows * (half ? 2 : 4);
    q.warps = (int32_t)std::max<int64_t>(1, std::min<int64_t>({kSortWarps, t / 128, kCounters / per_warp}));
    q.key = reinterpret_cast<int32_t*>(base + sp.key);
    q.order = reinterpret_cast<int32_t*>(base + sp.order);
    q.met = accumulate ? nullptr : reinterpret_cast<uint32_t*>(base + sp.met);
    q.count = reinterpret_cast<int32_t*>(base + sp.count);
    q.err = device_error_word();
    const unsigned grid = 1u << deal.shift;
    cudaError_t e = id_bytes == 8 ? (half ? launch_sort<int64_t, true>(q, grid, per_warp, s) : launch_sort<int64_t, false>(q, grid, per_warp, s))
                                  : (half ? launch_sort<int32_t, true>(q, grid, per_warp, s) : launch_sort<int32_t, false>(q, grid, per_warp, s));
    if (e != cudaSuccess) return cuda_error(e, "embedding gradient launch");

    SumArgs a = {};
    a.dy = dy;
    a.dw = dw;
    a.key = q.key;
    a.order = q.order;
    a.count = q.count;
    a.met = q.met;
    a.head = reinterpret_cast<float*>(base + sp.head);
    a.tail = reinterpret_cast<float*>(base + sp.tail);
    a.ldy = lddy;
    a.ldw = lddw;
    a.v = v;
    a.d = (int32_t)d;
    a.slabs = (int32_t)slabs;
    a.run = run_of(t, d);
    a.shift = deal.shift;
    a.rows = deal.rows;
    a.runs = runs;
    a.sum_blocks = sum_blocks;
    a.scale = scale;
    const bool vec = d % 8 == 0 && aligned_rows(dy, t, lddy, gs) && aligned_rows(dw, v, lddw, ws), add = accumulate != 0;
    const bool out_f32 = out_dtype == DPRED_F32;
    const unsigned n = (unsigned)blocks;
    if (g_dtype == DPRED_F32)
        e = out_f32 ? launch_sums<float, float>(a, vec, add, n, s) : launch_sums<float, __nv_bfloat16>(a, vec, add, n, s);
    else
        e = out_f32 ? launch_sums<__nv_bfloat16, float>(a, vec, add, n, s) : launch_sums<__nv_bfloat16, __nv_bfloat16>(a, vec, add, n, s);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "embedding gradient launch");
}
