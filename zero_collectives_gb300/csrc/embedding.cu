// embedding.cu -- the token embedding and its gradient: dpred_embedding and
// dpred_embedding_grad.
//
//     y[t]  = scale W[id(t)]
//     dW[v] = (dW[v] +) scale * sum of dy[t] over the tokens t with id(t) = v
//
// The embedding is the largest task of a bucket flush (98304 x 1024 of the
// 402.8M parameters).  Its gradient is summed in fp32 in one fixed order: the
// tokens of a row in ascending t, in runs of kRun positions of the sorted order
// whose sums are then added in ascending order.  Three launches:
//
//  sort   Every CTA owns a range of ids and reads all ids: it counts those below
//         its range (where its tokens start in the sorted order) and those of
//         each of its rows, per warp, then places its tokens.  The order is
//         stable and no CTA waits for another.  Reading T ids per SM from L2
//         costs T / 30000 us, a ninth at most of what T rows of 2 KB take from
//         HBM.
//  sum    A warp takes kRun sorted positions and 256 columns, eight rows in
//         flight.  Rows whose tokens lie inside its positions are written;
//         what continues from or into other positions is left as a partial sum.
//         Work is the same whatever the ids are: one row with all tokens is cut
//         like any other.  Where the whole table is stored, other blocks write
//         the rows without a token.
//  join   Adds the partial sums of the rows that were cut.
//
// Bandwidth bound: dy is read once and each row of dW written once (read and
// written once where it is added to, and only where a token is).
#include <algorithm>

#include "layers.cuh"

namespace dpred {
namespace layers {
namespace {

template <typename I>
__device__ __forceinline__ int64_t id_at(const I* ids, int64_t t) {
    return (int64_t)ids[t];
}

// ------------------------------------------------------------------- lookup --

constexpr int kLookThreads = 256, kLookRows = 4;

struct LookArgs {
    const void* ids;
    const void* w;
    void* y;
    int64_t t, v, ldw, ldy;
    int32_t d, id64;
    float scale;
    int* err;
};

// `lanes` threads cover a row in steps, kLookRows rows at a time.
template <typename TW, typename TY, bool VEC>
__global__ void __launch_bounds__(kLookThreads) lookup_kernel(const __grid_constant__ LookArgs a, int lanes) {
    mma::grid_wait();
    const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = kLookThreads / lanes;
    const TW* w = static_cast<const TW*>(a.w);
    TY* y = static_cast<TY*>(a.y);
    const int64_t step = (int64_t)gridDim.x * groups;
    for (int64_t t0 = (int64_t)blockIdx.x * groups + group; t0 < a.t; t0 += step * kLookRows) {
        int64_t id[kLookRows];
#pragma unroll
        for (int u = 0; u < kLookRows; ++u) {
            const int64_t t = t0 + u * step;
            id[u] = -1;
            if (t < a.t) {
                id[u] = a.id64 ? id_at(static_cast<const int64_t*>(a.ids), t) : id_at(static_cast<const int32_t*>(a.ids), t);
                if (id[u] < 0 || id[u] >= a.v) {
                    id[u] = -1;
                    if (lane == 0) record_device_error(a.err, DPRED_E_BOUNDS);
                }
            }
        }
        if constexpr (VEC) {
            for (int c = lane * 8; c < a.d; c += lanes * 8) {
                Eight<TW> q[kLookRows];
#pragma unroll
                for (int u = 0; u < kLookRows; ++u)
                    if (id[u] >= 0) q[u].load(w + id[u] * a.ldw + c);
#pragma unroll
                for (int u = 0; u < kLookRows; ++u) {
                    if (t0 + u * step >= a.t) continue;
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = id[u] >= 0 ? q[u][k] * a.scale : 0.0f;
                    store8(y + (t0 + u * step) * a.ldy + c, f);
                }
            }
        } else {
            for (int c = lane; c < a.d; c += lanes) {
                float f[kLookRows];
#pragma unroll
                for (int u = 0; u < kLookRows; ++u) f[u] = id[u] >= 0 ? load1(w + id[u] * a.ldw + c) * a.scale : 0.0f;
#pragma unroll
                for (int u = 0; u < kLookRows; ++u)
                    if (t0 + u * step < a.t) store1(y + (t0 + u * step) * a.ldy + c, f[u]);
            }
        }
    }
}

// --------------------------------------------------------------------- sort --

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxRange = 1024;  // ids of a CTA: a counter for each and every warp, 128 KB
constexpr int kRun = 32;         // sorted positions of a warp in the sums

struct SortArgs {
    const void* ids;
    int64_t padding;  // this id's tokens give no gradient; INT64_MIN: none
    int64_t t, v;
    int32_t range;    // ids of a CTA, a multiple of 32
    int32_t warps;    // warps that share the tokens
    int32_t* key;     // [t] id of a sorted position
    int32_t* order;   // [t] its token
    uint32_t* met;    // a bit per id: it has a token (null: not wanted)
    int32_t* count;   // sorted positions in all
    int* err;
};

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ int counts[];  // [warps][range]: tokens of a row that a warp has met, then where its next one goes
    __shared__ int below[kSortWarps], sums[kSortWarps];
    mma::grid_launch_dependents();
    mma::grid_wait();
    const I* ids = static_cast<const I*>(a.ids);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t lo = (int64_t)blockIdx.x * a.range;
    const int rows = (int)min((int64_t)a.range, a.v - lo);
    for (int i = threadIdx.x; i < a.warps * a.range; i += kSortThreads) counts[i] = 0;
    __syncthreads();
    // each warp has one stretch of the tokens, a multiple of 32
    const int64_t per = (a.t + a.warps * 32 - 1) / (a.warps * 32) * 32;
    const int64_t t0 = warp * per, t1 = warp < a.warps ? min(a.t, t0 + per) : 0;
    int* mine = counts + warp * a.range;
    int less = 0;
    bool outside = false;
    constexpr int U = 8;
    for (int64_t t = t0 + lane; t < t1; t += 32 * U) {
        int64_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = t + 32 * u < t1 ? id_at(ids, t + 32 * u) : a.v;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + 32 * u >= t1) continue;
            const bool good = id[u] >= 0 && id[u] < a.v;
            outside |= !good && id[u] != a.padding;
            if (!good || id[u] == a.padding) continue;
            less += id[u] < lo;
            const int64_t r = id[u] - lo;
            if (r >= 0 && r < rows) atomicAdd(mine + r, 1);
        }
    }
    if (outside && blockIdx.x == 0) record_device_error(a.err, DPRED_E_BOUNDS);
    less = warp_sum(less);
    if (lane == 0) below[warp] = less;
    __syncthreads();
    // the rows' tokens in all; an exclusive sum over rows, then over the warps of a row
    int total = 0;
    if ((int)threadIdx.x < rows)
        for (int w = 0; w < a.warps; ++w) total += counts[w * a.range + threadIdx.x];
    if (a.met) {
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, total != 0);
        if (lane == 0 && warp * 32 < rows) a.met[lo / 32 + warp] = bits;
    }
    int before = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) sums[warp] = before;
    before -= total;
    __syncthreads();
    int start = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        start += below[w];
        if (w < warp) before += sums[w];
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == kSortThreads - 1) *a.count = start + before + total;
    if ((int)threadIdx.x < rows) {
        int at = start + before;
        for (int w = 0; w < a.warps; ++w) {
            int& c = counts[w * a.range + threadIdx.x];
            const int n = c;
            c = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t t = t0 + lane; t - lane < t1; t += 32 * U) {
        int64_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = t + 32 * u < t1 ? id_at(ids, t + 32 * u) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = id[u] - lo;
            const bool here = id[u] >= 0 && r >= 0 && r < rows && id[u] != a.padding;
            if (!__any_sync(0xFFFFFFFFu, here)) continue;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, here ? (int)r : -1 - lane);
            if (here) {
                const int rank = __popc(same & ((1u << lane) - 1));
                const int at = mine[r] + rank;
                a.key[at] = (int32_t)id[u];
                a.order[at] = (int32_t)(t + 32 * u);
            }
            __syncwarp();
            if (here && lane == __ffs(same) - 1) mine[r] += __popc(same);
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------- sum --

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kSlab = 256;      // columns of a warp
constexpr int kFillRows = 8;    // rows of a warp that writes zeros

struct SumArgs {
    const void* dy;
    void* dw;
    const int32_t *key, *order, *count;
    const uint32_t* met;   // null: rows without a token stay as they are
    float *head, *tail;    // [runs][d] partial sums: of the row that began before the run, of the one that goes on behind it
    int64_t ldy, ldw, v;
    int32_t d, slabs;
    int64_t runs, sum_blocks;
    float scale;
    int32_t accumulate;
};

// A lane's first column of a slab.
template <bool VEC>
__device__ __forceinline__ int first_column(int base, int lane) {
    return VEC ? base + lane * 8 : base + lane;
}

// A finished row into the gradient.
template <bool VEC, typename T>
__device__ __forceinline__ void leave(T* p, int c0, int d, const float (&sum)[8], float scale, bool add) {
    float f[8];
    if (add) {
        Cols<T, VEC> old;
        old.load(p, c0, 32, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = fmaf(sum[k], scale, old[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = sum[k] * scale;
    }
    store_cols<VEC>(p, c0, 32, d, f);
}

template <typename TG, typename TW, bool VEC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumArgs a) {
    if (a.runs > 1) mma::grid_launch_dependents();  // another launch of the call follows
    mma::grid_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    TW* dw = static_cast<TW*>(a.dw);
    if (blockIdx.x >= a.sum_blocks) {  // zeros for the rows without a token
        const int64_t r0 = ((blockIdx.x - a.sum_blocks) * kSumWarps + warp) * kFillRows;
        const float zero[8] = {};
        if (r0 >= a.v) return;
        const uint32_t bits = a.met[r0 / 32] >> (r0 % 32);
        for (int r = 0; r < kFillRows && r0 + r < a.v; ++r) {
            if (bits >> r & 1) continue;
            for (int base = 0; base < a.d; base += kSlab) store_cols<VEC>(dw + (r0 + r) * a.ldw, first_column<VEC>(base, lane), 32, a.d, zero);
        }
        return;
    }
    const int64_t item = (int64_t)blockIdx.x * kSumWarps + warp, run = item / a.slabs;
    const int c0 = first_column<VEC>((int)(item % a.slabs) * kSlab, lane);
    const int64_t n = *a.count, p0 = run * kRun;
    if (p0 >= n) return;
    const int len = (int)min((int64_t)kRun, n - p0);
    const int32_t key = lane < len ? a.key[p0 + lane] : -1, token = lane < len ? a.order[p0 + lane] : 0;
    const bool goes_on = p0 + len < n && a.key[p0 + len] == __shfl_sync(0xFFFFFFFFu, key, len - 1);
    bool began_before = p0 > 0 && a.key[p0 - 1] == __shfl_sync(0xFFFFFFFFu, key, 0);
    const TG* dy = static_cast<const TG*>(a.dy);
    float sum[8] = {};
    constexpr int U = 8;
    for (int i = 0; i < len; i += U) {
        Cols<TG, VEC> q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = __shfl_sync(0xFFFFFFFFu, token, i + u);
            if (i + u < len) q[u].load(dy + t * a.ldy, c0, 32, a.d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t now = __shfl_sync(0xFFFFFFFFu, key, i + u), next = __shfl_sync(0xFFFFFFFFu, key, (i + u + 1) % 32);
            if (i + u >= len) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += q[u][k];
            const bool last = i + u + 1 == len;
            if (!last && now == next) continue;
            if (began_before)
                store_cols<VEC>(a.head + run * a.d, c0, 32, a.d, sum);
            else if (last && goes_on)
                store_cols<VEC>(a.tail + run * a.d, c0, 32, a.d, sum);
            else
                leave<VEC>(dw + now * a.ldw, c0, a.d, sum, a.scale, a.accumulate);
            began_before = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
        }
    }
}

// The row that begins in this run and goes on behind it: its tail here and the
// heads of the runs that follow.  The block's warps share them, and the shares
// are added in order.
template <typename TW, bool VEC>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const __grid_constant__ SumArgs a) {
    __shared__ float part[kSumWarps][kSlab];
    mma::grid_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t run = blockIdx.x / a.slabs, n = *a.count, p0 = run * kRun;
    const int c0 = first_column<VEC>((int)(blockIdx.x % a.slabs) * kSlab, lane);
    if (p0 + kRun >= n) return;
    const int32_t row = a.key[p0 + kRun - 1];
    if (a.key[p0 + kRun] != row) return;
    if (a.key[p0] == row && p0 > 0 && a.key[p0 - 1] == row) return;  // it began before
    // runs behind this one that begin with the row
    const int64_t runs = (n + kRun - 1) / kRun;
    int64_t more = 1;
    for (;;) {
        const int64_t r = run + 1 + more + lane;
        const unsigned same = __ballot_sync(0xFFFFFFFFu, r < runs && a.key[r * kRun] == row);
        const int k = same == 0xFFFFFFFFu ? 32 : __ffs(~same) - 1;
        more += k;
        if (k < 32) break;
    }
    const int64_t q0 = run + 1 + more * warp / kSumWarps, q1 = run + 1 + more * (warp + 1) / kSumWarps;
    float sum[8] = {};
    constexpr int U = 4;
    for (int64_t q = q0; q < q1; q += U) {
        Cols<float, VEC> f[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + u < q1) f[u].load(a.head + (q + u) * a.d, c0, 32, a.d);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + u < q1)
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += f[u][k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) part[warp][k * 32 + lane] = sum[k];
    __syncthreads();
    if (warp) return;
    Cols<float, VEC> first;
    first.load(a.tail + run * a.d, c0, 32, a.d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        sum[k] = first[k];
        for (int w = 0; w < kSumWarps; ++w) sum[k] += part[w][k * 32 + lane];
    }
    leave<VEC>(static_cast<TW*>(a.dw) + row * a.ldw, c0, a.d, sum, a.scale, a.accumulate);
}

// --------------------------------------------------------------------- host --

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
int64_t runs_of(int64_t t) { return (t + kRun - 1) / kRun; }

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
    s.key = take(t * 4);
    s.order = take(t * 4);
    s.met = take((v + 31) / 32 * 4);
    s.count = take(4);
    s.head = take(runs_of(t) * d * 4);
    s.tail = take(runs_of(t) * d * 4);
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

template <typename TW, typename TY>
cudaError_t launch_lookup(const LookArgs& a, bool vec, cudaStream_t s) {
    const int items = vec ? (a.d + 7) / 8 : a.d;
    int lanes = 1;
    while (lanes < items && lanes < kLookThreads) lanes *= 2;
    const int64_t groups = kLookThreads / lanes;
    // a row at a time while that gives every SM its blocks, then kLookRows at once
    const int64_t blocks = std::min<int64_t>((a.t + groups - 1) / groups, std::max<int64_t>((a.t + groups * kLookRows - 1) / (groups * kLookRows), 8 * sm_count()));
    const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 20));
    return vec ? launch(lookup_kernel<TW, TY, true>, grid, kLookThreads, 0, s, a, lanes) : launch(lookup_kernel<TW, TY, false>, grid, kLookThreads, 0, s, a, lanes);
}

template <typename TG, typename TW>
cudaError_t launch_sums(const SumArgs& a, bool vec, unsigned blocks, cudaStream_t s) {
    cudaError_t e = vec ? launch(sum_kernel<TG, TW, true>, dim3(blocks), kSumThreads, 0, s, a) : launch(sum_kernel<TG, TW, false>, dim3(blocks), kSumThreads, 0, s, a);
    if (e != cudaSuccess || a.runs <= 1) return e;
    const dim3 grid((unsigned)((a.runs - 1) * a.slabs));
    return vec ? launch(join_kernel<TW, true>, grid, kSumThreads, 0, s, a) : launch(join_kernel<TW, false>, grid, kSumThreads, 0, s, a);
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
    const cudaError_t e = w_dtype == DPRED_F32 ? (out_dtype == DPRED_F32 ? launch_lookup<float, float>(a, vec, s) : launch_lookup<float, __nv_bfloat16>(a, vec, s))
                                               : (out_dtype == DPRED_F32 ? launch_lookup<__nv_bfloat16, float>(a, vec, s) : launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, vec, s));
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
    if (padding < -1 || padding >= std::max<int64_t>(v, 1)) return set_error(DPRED_E_INVAL, "padding %lld outside -1..%lld", (long long)padding, (long long)v - 1);
    const int gs = esize(g_dtype), ws = esize(out_dtype);
    if (v == 0 || d == 0) return DPRED_OK;
    if ((rc = check_ids(ids, t, id_bytes)) != DPRED_OK || (rc = check_matrix(dy, t, d, lddy, gs, "dy")) != DPRED_OK ||
        (rc = check_matrix(dw, v, d, lddw, ws, "dw")) != DPRED_OK)
        return rc;
    if (t == 0 && accumulate) return DPRED_OK;
    const int64_t slabs = (d + kSlab - 1) / kSlab, sum_blocks = (runs_of(t) * slabs + kSumWarps - 1) / kSumWarps;
    const int64_t blocks = sum_blocks + (accumulate ? 0 : (v + kSumWarps * kFillRows - 1) / (kSumWarps * kFillRows));
    if (blocks > 0x7FFFFFFF || runs_of(t) * slabs > 0x7FFFFFFF)
        return set_error(DPRED_E_SIZE, "%lld tokens of %lld columns are too many", (long long)t, (long long)d);
    const Space sp = space_of(t, v, d);
    if ((rc = check_workspace(workspace, workspace_bytes, (size_t)sp.bytes)) != DPRED_OK) return rc;
    char* base = static_cast<char*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);

    SortArgs q = {};
    q.ids = ids;
    q.padding = padding < 0 ? INT64_MIN : padding;
    q.t = t;
    q.v = v;
    // one CTA per SM where its counters fit; a counter row for each 128 tokens, so that few tokens clear few counters
    q.range = (int32_t)std::min<int64_t>(kMaxRange, ((v + sm_count() - 1) / sm_count() + 31) / 32 * 32);
    q.warps = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kSortWarps, t / 128));
    q.key = reinterpret_cast<int32_t*>(base + sp.key);
    q.order = reinterpret_cast<int32_t*>(base + sp.order);
    q.met = accumulate ? nullptr : reinterpret_cast<uint32_t*>(base + sp.met);
    q.count = reinterpret_cast<int32_t*>(base + sp.count);
    q.err = device_error_word();
    const int smem = q.warps * q.range * 4;
    static bool done32[64], done64[64];
    cudaError_t e = id_bytes == 8 ? ensure_smem_attr(sort_kernel<int64_t>, kSortWarps * kMaxRange * 4, done64) : ensure_smem_attr(sort_kernel<int32_t>, kSortWarps * kMaxRange * 4, done32);
    if (e != cudaSuccess) return cuda_error(e, "embedding gradient set-up");
    const dim3 grid((unsigned)((v + q.range - 1) / q.range));
    e = id_bytes == 8 ? launch(sort_kernel<int64_t>, grid, kSortThreads, smem, s, q) : launch(sort_kernel<int32_t>, grid, kSortThreads, smem, s, q);
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
    a.runs = runs_of(t);
    a.sum_blocks = sum_blocks;
    a.scale = scale;
    a.accumulate = accumulate != 0;
        const bool vec = d % 8 == 0 && aligned_rows(dy, t, lddy, gs) && aligned_rows(dw, v, lddw, ws);
    e = g_dtype == DPRED_F32 ? (out_dtype == DPRED_F32 ? launch_sums<float, float>(a, vec, (unsigned)blocks, s) : launch_sums<float, __nv_bfloat16>(a, vec, (unsigned)blocks, s))
                             : (out_dtype == DPRED_F32 ? launch_sums<__nv_bfloat16, float>(a, vec, (unsigned)blocks, s) : launch_sums<__nv_bfloat16, __nv_bfloat16>(a, vec, (unsigned)blocks, s));
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "embedding gradient launch");
}
