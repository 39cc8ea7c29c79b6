// muon_chain.cu -- every product of the orthogonalised updates of a batch, as
// one launch of the tile kernel's pipeline.
//
// Launched one by one, the three products of a step leave most SMs idle at
// every boundary: 8 matrices of 1024 x 1024 are 80 symmetric tiles for 76 CTA
// pairs, twice as long as 76.  Here the pairs walk one list of tiles in the order
// (product, matrix): the first matrices' next product starts while the
// last ones' current product is still running.  What a tile needs is its own
// matrix's previous product, complete: a counter per matrix says so (it counts
// the epilogue warps whose part of a tile is in memory), and since the
// list is in dependency order and all pairs are resident (a cooperative
// launch), every wait ends.  Waits are bounded all the same.
//
// The symmetric products store only their tiles on and above the diagonal.
// Where a later product needs the part below, it loads the mirror image as an
// operand of the other major (rows and columns exchanged), which the matrix
// instruction takes as it is: writing the mirror image cost the epilogue a
// transposition through shared memory and the same stores again.
//
// Measured: 12 of 1024 x 1024 (5 steps) 264 us, 6 of 1024 x 4096 392 us.  With
// tiles to spare (48 of 1024 x 1024) a tile takes 8.5 us and its reduction alone
// 5: X's two terms, 192 KB in and out, share the SM's way to L2 with 512 KB of
// operands.  With few (one matrix) the chain of products bounds it.
#include "muon_chain.cuh"

namespace dpred {
namespace gemm {
namespace {

constexpr int kBN = 256;
constexpr int kStages = 6;
// The producer is at most this many tiles ahead of the epilogue: two accumulators, a tile in every stage.
constexpr int kReady = 16;
static_assert(kReady > 2 + kStages + 1, "a tile's barrier is reused before it was waited for");
constexpr uint32_t kStageBytes = 2 * 128 * 128;
constexpr int kSmem = kStages * (int)kStageBytes + 8 * (int)kBlockBytes + 1024;

// A pair's position in the list of tiles.
struct Cursor {
    int at = 0, offset;  // product (of every matrix's program), tile within it
    // of the tile at this position
    int group, batch, tm, tn;
    ChainOp op;

    __device__ __forceinline__ Cursor(int first) : offset(first) {}

    __device__ __forceinline__ bool settle(const ChainArgs& a) {
        for (; at < a.ops; ++at) {
            int t = offset;
            for (group = 0; group < a.groups; ++group) {
                const ChainGroup& g = a.g[group];
                if (at >= g.ops) continue;
                op = a.program[g.program][at];
                const bool square = op.kind < CHAIN_APPLY;
                const int per = square ? g.square_tiles : g.tiles_r * g.tiles_c, n = per * g.count;
                if (t < n) {
                    batch = t / per;
                    t -= batch * per;
                    if (square) {  // row tm starts at the diagonal
                        for (tm = 0; t >= g.tiles_r - tm; ++tm) t -= g.tiles_r - tm;
                        tn = tm + t;
                    } else {
                        tm = t % g.tiles_r;
                        tn = t / g.tiles_r;
                    }
                    return true;
                }
                t -= n;
            }
            offset = t;
        }
        return false;
    }

    // What the matrix's counter must have reached before this product may start.
    __device__ __forceinline__ unsigned needed(const ChainGroup& g) const {
        return 16u * (unsigned)(op.squares * g.square_tiles + op.applies * g.tiles_r * g.tiles_c);
    }
    __device__ __forceinline__ int reduction(const ChainGroup& g) const { return op.kind == CHAIN_GRAM ? g.c : g.r; }
    // A row block of a stored r x r matrix exists from its diagonal tile on:
    // reduction indexes below these are loaded from the mirror image.  X as the
    // second factor is MN-major throughout.
    __device__ __forceinline__ int a_from() const { return op.kind == CHAIN_GRAM ? 0 : tm * 256; }
    __device__ __forceinline__ int b_from() const { return op.kind == CHAIN_GRAM ? 0 : op.kind >= CHAIN_APPLY ? 0x7FFFFFFF : tn * 256; }
};

__device__ __forceinline__ bool wait_counter(const unsigned* p, unsigned need) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= need) return true;
    const long long t0 = clock64();
    do {
        __nanosleep(64);
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        if (v >= need) return true;
    } while (clock64() - t0 <= tma::kWaitBudgetCycles);
    return false;
}

// One tile's epilogue by one warp: 32 rows of 128 columns.
template <int KIND>
__device__ __forceinline__ bool tile_epilogue(const NsEpi& e, const Args& g, int batch, int i, int j, uint32_t acc,
                                              uint32_t block, int lane, uint64_t* full, uint32_t parity, uint32_t drained) {
    // the next block's operands are loaded while this one is worked on; two factors (MUL) would not fit the
    // registers twice, and theirs are loaded at the block
    constexpr bool kNext = KIND != KIND_MUL;
    Ahead<KIND> ahead;
    load_ahead<KIND>(e, g, batch, i, j, lane, ahead);
    if (!__all_sync(0xFFFFFFFFu, tma::mbar_wait(full, parity))) return false;
    mma::fence_after();
#pragma unroll 1
    for (int c = 0; c < kBN / 2; c += 32) {
        float v[32];
        __syncwarp();
        mma::tmem_ld32(acc + c, v);
        mma::tmem_wait_ld();
        if (c + 32 == kBN / 2) {  // the accumulator is in registers: the next tile may overwrite it
            mma::fence_before();
            __syncwarp();
            if (lane == 0) mma::mbar_arrive_cluster(drained);
        }
        if (i < g.m && j + c < g.n) {
            block_put_row(block, lane, v);
            if constexpr (kNext) {
                const Ahead<KIND> now = ahead;
                if (c + 32 < kBN / 2) load_ahead<KIND>(e, g, batch, i, j + c + 32, lane, ahead);
                __syncwarp();
                block_epilogue<KIND>(e, g, batch, i, j + c, block, lane, false, now);
            } else {
                __syncwarp();
                block_epilogue<KIND>(e, g, batch, i, j + c, block, lane, false, ahead);
                if (c + 32 < kBN / 2) load_ahead<KIND>(e, g, batch, i, j + c + 32, lane, ahead);
            }
        }
    }
    return true;
}

// 32 bytes, past the first-level cache (other SMs wrote them earlier in this launch).
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// tile_epilogue<KIND_APPLY> where X's rows are whole 32-column chunks: a lane
// keeps the row that it has in tensor memory, and both terms of X come and go
// in 32-byte pieces (whole sectors) without a pass through shared memory.  All
// of X that the tile reads is requested before its accumulators are waited for.
// 12 of 1024 x 1024: 291 us against 304 through shared memory (what remains for
// rows that end inside a chunk).
struct XChunk {
    uint32_t h[2][8], l[8];
};

__device__ __forceinline__ bool apply_rows(const NsEpi& e, const Args& g, int batch, int i, int j, uint32_t acc, int lane,
                                           uint64_t* full, uint32_t parity, uint32_t drained) {
    const int row = i + lane;
    const bool live = row < g.m;
    const int64_t at = ((int64_t)batch * g.m + row) * e.ldc + j;
    XChunk ahead[kBN / 64] = {};
    auto load = [&](int c, XChunk& x) {
        if (live && j + c < g.n) {
            load32(e.hi_in + at + c, x.h[0]);
            load32(e.hi_in + at + c + 16, x.h[1]);
            load32(e.lo + at + c, x.l);
        }
    };
#pragma unroll
    for (int c = 0; c < kBN / 2; c += 32) load(c, ahead[c / 32]);
    const float k = live ? __ldcg(e.coef + (int64_t)batch * e.ldr + row) : 0.0f;
    if (!__all_sync(0xFFFFFFFFu, tma::mbar_wait(full, parity))) return false;
    mma::fence_after();
#pragma unroll
    for (int c = 0; c < kBN / 2; c += 32) {
        float v[32];
        __syncwarp();
        mma::tmem_ld32(acc + c, v);
        mma::tmem_wait_ld();
        if (c + 32 == kBN / 2) {  // the accumulator is in registers: the next tile may overwrite it
            mma::fence_before();
            __syncwarp();
            if (lane == 0) mma::mbar_arrive_cluster(drained);
        }
        XChunk& now = ahead[c / 32];
        if (live && j + c < g.n) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t(&hw)[8] = now.h[p / 2];
                const int o = p % 2 * 4;
                float x[8];
                join8(make_uint4(hw[o], hw[o + 1], hw[o + 2], hw[o + 3]), make_uint2(now.l[2 * p], now.l[2 * p + 1]), x);
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] = fmaf(k, x[q], v[8 * p + q]);
                uint4 h;
                uint2 l;
                split8(x, h, l);
                hw[o] = h.x;
                hw[o + 1] = h.y;
                hw[o + 2] = h.z;
                hw[o + 3] = h.w;
                now.l[2 * p] = l.x;
                now.l[2 * p + 1] = l.y;
            }
            store32(e.hi + at + c, now.h[0]);
            store32(e.hi + at + c + 16, now.h[1]);
            store32(e.lo + at + c, now.l);
        }
    }
    return true;
}

__global__ void __launch_bounds__(kTileThreads, 1) chain_kernel(const __grid_constant__ ChainArgs a) {
    using namespace mma;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], stored[2], taken[2], ready[kReady];
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tma::mbar_init(&full[s], 1);
            tma::mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tma::mbar_init(&acc_full[i], 1);
            tma::mbar_init(&acc_empty[i], 16);
            tma::mbar_init(&stored[i], 8);  // the CTA's epilogue warps
            tma::mbar_init(&taken[i], 1);   // the releasing thread
        }
        for (int i = 0; i < kReady; ++i) tma::mbar_init(&ready[i], 1);
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<2>(tma::smem_addr(&tmem_slot), 512);
    fence_before();
    cluster_sync();
    fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        if (elect_one()) {
            int s = 0, round = 0, fill = 0;
            bool ok = true;
            for (Cursor at(pair); ok && at.settle(a); at.offset += pairs, ++fill) {
                const ChainGroup& g = a.g[at.group];
                if (!wait_counter(a.counter + g.first + at.batch, at.needed(g))) {
                    record_device_error(a.err, DPRED_E_TIMEOUT);
                    ok = false;
                    break;
                }
                tma::mbar_arrive(&ready[fill % kReady]);
                fence_proxy_async();  // what other SMs stored is about to be read by copies
                const ChainOp op = at.op;
                const CUtensorMap* ma = op.kind == CHAIN_GRAM ? &g.x[op.x] : g.square[op.a];
                const CUtensorMap* mb = op.kind >= CHAIN_APPLY ? &g.xt[op.x] : op.kind == CHAIN_GRAM ? ma : g.square[op.b];
                const int n = at.reduction(g), a_from = at.a_from(), b_from = at.b_from();
                const int i0 = at.tm * 256 + (int)rank * 128, j0 = at.tn * 256 + (int)rank * 128;
                for (int k0 = 0; k0 < n; k0 += kBlockK) {
                    if (round && !tma::mbar_wait(&empty[s], (round - 1) & 1)) {
                        record_device_error(a.err, DPRED_E_TIMEOUT);
                        ok = false;
                        break;
                    }
                    const uint32_t pa = base + s * kStageBytes, pb = pa + 128 * 128, bar = tma::smem_addr(&full[s]);
                    if (rank == 0) tma::mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                    if (k0 < a_from) {
                        load_box_pair(pa, ma + 1, bar, i0, k0, at.batch);
                        load_box_pair(pa + 8192, ma + 1, bar, i0 + 64, k0, at.batch);
                    } else {
                        load_box_pair(pa, ma, bar, k0, i0, at.batch);
                    }
                    if (k0 < b_from) {
                        const CUtensorMap* mt = op.kind >= CHAIN_APPLY ? mb : mb + 1;
                        load_box_pair(pb, mt, bar, j0, k0, at.batch);
                        load_box_pair(pb + 8192, mt, bar, j0 + 64, k0, at.batch);
                    } else {
                        load_box_pair(pb, mb, bar, k0, j0, at.batch);
                    }
                    if (++s == kStages) {
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
            const uint64_t dk = operand_desc(base, false), dm = operand_desc(base, true);
            int s = 0, round = 0, fill = 0;
            bool ok = true;
            for (Cursor at(pair); ok && at.settle(a); at.offset += pairs, ++fill) {
                const ChainGroup& g = a.g[at.group];
                const int n = at.reduction(g), acc = fill & 1, a_from = at.a_from(), b_from = at.b_from();
                if (fill >= 2 && !tma::mbar_wait(&acc_empty[acc], (fill / 2 - 1) & 1)) {
                    record_device_error(a.err, DPRED_E_TIMEOUT);
                    break;
                }
                fence_after();
                for (int k0 = 0; k0 < n; k0 += kBlockK) {
                    // the copies may wait for other SMs' tiles first, hence twice the budget
                    if (!tma::mbar_wait(&full[s], round & 1, 2 * tma::kWaitBudgetCycles)) {
                        record_device_error(a.err, DPRED_E_TIMEOUT);
                        ok = false;
                        break;
                    }
                    fence_after();
                    const bool am = k0 < a_from, bm = k0 < b_from;
                    const uint64_t da = (am ? dm : dk) + s * (kStageBytes >> 4), db = (bm ? dm : dk) + s * (kStageBytes >> 4) + (128 * 128 >> 4);
                    const uint32_t idesc = instr_desc(256, kBN, false, am, bm), sa = am ? 128 : 2, sb = bm ? 128 : 2;
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k)
                        issue<2>(tmem + acc * kBN, da + k * sa, db + k * sb, idesc, k0 != 0 || k != 0);
                    commit<2>(tma::smem_addr(&empty[s]));
                    if (++s == kStages) {
                        s = 0;
                        ++round;
                    }
                }
                if (ok) commit<2>(tma::smem_addr(&acc_full[acc]));
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // Makes finished tiles known to the other SMs.  The release waits until the CTA's stores have
        // reached L2, about 4000 cycles, which the epilogue's warps spend on their next tile (12 of
        // 1024 x 1024: 266 us, 290 with every epilogue warp releasing its own part).
        if (elect_one()) {
            int fill = 0;
            for (Cursor at(pair); at.settle(a); at.offset += pairs, ++fill) {
                const int acc = fill & 1;
                // a tile's epilogue may wait for its operands and for its accumulators first
                if (!tma::mbar_wait(&stored[acc], (fill / 2) & 1, 3 * tma::kWaitBudgetCycles)) {
                    record_device_error(a.err, DPRED_E_TIMEOUT);
                    break;
                }
                tma::mbar_arrive(&taken[acc]);
                fence_proxy_async();  // these stores will be read by other SMs' copies
                asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(a.counter + a.g[at.group].first + at.batch), "r"(8u)
                             : "memory");
            }
        }
        __syncwarp();
    } else if (warp >= kEpilogueWarp0) {
        const int q = warp & 3, half = (warp - kEpilogueWarp0) / 4;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * (kBN / 2);
        const uint32_t block = base + kStages * kStageBytes + (warp - kEpilogueWarp0) * kBlockBytes;
        const uint32_t drained0 = map_rank(tma::smem_addr(&acc_empty[0]), 0), drained1 = map_rank(tma::smem_addr(&acc_empty[1]), 0);
        int fill = 0;
        bool ok = true;
        for (Cursor at(pair); ok && at.settle(a); at.offset += pairs, ++fill) {
            const ChainGroup& g = a.g[at.group];
            const int acc = fill & 1;
            const ChainOp op = at.op;
            if (op.kind != CHAIN_GRAM) {  // the epilogue reads what earlier products stored, as the producer has seen
                ok = __all_sync(0xFFFFFFFFu, tma::mbar_wait(&ready[fill % kReady], (fill / kReady) & 1, 2 * tma::kWaitBudgetCycles));
                if (!ok) break;
            }
            NsEpi e = g.e;
            e.out = a.out + g.first;
            Args d;
            d.m = g.r;
            d.n = op.kind >= CHAIN_APPLY ? g.c : g.r;
            const int i = at.tm * 256 + (int)rank * 128 + q * 32, j = at.tn * 256 + half * (kBN / 2);
            const uint32_t from = lanes + acc * kBN, parity = (fill / 2) & 1, drained = acc ? drained1 : drained0;
            e.gram = g.sq[op.kind == CHAIN_POLY ? op.a : op.out];
            e.gram_diag = g.diag[op.kind == CHAIN_POLY ? op.a : op.out];
            e.poly = g.sq[op.out];
            e.coef = g.diag[op.kind == CHAIN_POLY ? op.out : op.a];
            e.m1 = g.sq[op.a];
            e.d1 = g.diag[op.a];
            e.m2 = g.sq[op.b];
            e.d2 = g.diag[op.b];
            e.hi_in = g.hi[op.x];
            e.hi = g.hi[op.x ^ 1];
            switch (op.kind) {
                case CHAIN_GRAM: ok = tile_epilogue<KIND_GRAM>(e, d, at.batch, i, j, from, block, lane, &acc_full[acc], parity, drained); break;
                case CHAIN_POLY: ok = tile_epilogue<KIND_POLY>(e, d, at.batch, i, j, from, block, lane, &acc_full[acc], parity, drained); break;
                case CHAIN_MUL: ok = tile_epilogue<KIND_MUL>(e, d, at.batch, i, j, from, block, lane, &acc_full[acc], parity, drained); break;
                case CHAIN_APPLY:
                    if (g.c % 32 == 0) {
                        ok = apply_rows(e, d, at.batch, i, j, from, lane, &acc_full[acc], parity, drained);
                        break;
                    }
                    ok = tile_epilogue<KIND_APPLY>(e, d, at.batch, i, j, from, block, lane, &acc_full[acc], parity, drained); break;
                default: ok = tile_epilogue<KIND_FINAL>(e, d, at.batch, i, j, from, block, lane, &acc_full[acc], parity, drained); break;
            }
            __syncwarp();
            if (lane == 0 && ok) {
                if (fill >= 2) ok = tma::mbar_wait(&taken[acc], (fill / 2 - 1) & 1);
                if (ok) tma::mbar_arrive(&stored[acc]);
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        if (!ok && lane == 0) record_device_error(a.err, DPRED_E_TIMEOUT);
        __syncwarp();
    }
    fence_before();
    cluster_sync();  // no CTA leaves while the other may still signal it or read its shared memory
    if (warp == 1) {
        fence_after();
        tmem_free<2>(tmem, 512);
    }
}

}  // namespace

int run_chain(const ChainArgs& a, cudaStream_t s) {
    static bool attr[64] = {};
    cudaError_t err = ensure_smem_attr(chain_kernel, kSmem, attr);
    if (err != cudaSuccess) return cuda_error(err, "shared-memory limit of the chained products");
    const int pairs = resident_pairs(reinterpret_cast<const void*>(chain_kernel), kTileThreads, kSmem);
    if (pairs < 1) return set_error(DPRED_E_CUDA, "no CTA pair fits on this device");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (a.most < pairs ? a.most : pairs)));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, chain_kernel, a);
    return err == cudaSuccess ? DPRED_OK : cuda_error(err, "chained products launch");
}

}  // namespace gemm
}  // namespace dpred
