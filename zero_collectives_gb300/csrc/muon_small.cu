// muon_small.cu -- one launch for a whole orthogonalised update of matrices of
// up to 128 x 2048.
//
// The general path takes 17 launches, each a few microseconds whatever the
// size.  Here a cluster keeps a matrix on chip for the whole update: each of
// its 1 to 8 CTAs holds up to 256 columns of X, and a step is
//   Gram    every CTA multiplies its own columns, 128 x 128 partial sums; they
//           are added through distributed shared memory, each CTA summing a
//           band of rows in rank order and sending the result to all;
//   poly    every CTA computes the whole 128 x 128 polynomial;
//   apply   every CTA updates its own columns in place.
// The arithmetic is that of the general path (muon.cu), except that X's second
// term is the rest of it in fp32: a thread owns the same row and columns in every step, so X stays in
// its registers and only the fp16 operand goes through shared memory.
// Operand tiles lie in the 128-byte swizzle, 64 columns wide: the same bytes
// serve the Gram product as K-major rows and the apply product as an MN-major
// operand.  What bounds it is latency: three dependent products a step, with
// two cluster barriers (about 1100 cycles each) where there is a cluster.
#include "muon_small.cuh"

#include <algorithm>

namespace dpred {
namespace gemm {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t kChunk = 128 * 128;           // 128 rows x 64 columns of fp16
constexpr float kOffScale = 256.0f;
// shared memory: X operand (4 chunks), E (2), partial sums (128 x 128 fp32; P
// lies over them).  X passes through as fp32 once, over X and the partial sums.
constexpr uint32_t kX = 0, kPart = 4 * kChunk, kP = kPart, kE = 8 * kChunk;
constexpr uint32_t kSmem = 10 * kChunk + 1024;

// Byte of element (row, col) of a matrix stored in 64-column chunks.
__device__ __forceinline__ uint32_t at(int row, int col) {
    return (col >> 6) * kChunk + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}
// 16-byte piece c4 of a row of `pieces` pieces of fp32.
template <int PIECES>
__device__ __forceinline__ uint32_t f32_at(int row, int c4) { return row * (PIECES * 16) + ((c4 ^ (row & 7)) << 4); }

__device__ __forceinline__ uint4 ldsq(uint32_t a) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(a) : "memory");
    return q;
}
__device__ __forceinline__ void stsq(uint32_t a, uint4 q) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
__device__ __forceinline__ void sts1(uint32_t a, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
    if constexpr (sizeof(T) == 2)
        return load_bf16(reinterpret_cast<const __nv_bfloat16*>(p));
    else
        return *p;
}

// Takes v[lane] out of v (0 stays in its place), without a branch per element.
__device__ __forceinline__ float take_lane(float (&v)[32], int lane) {
    float d = 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) {
        d = q == lane ? v[q] : d;
        v[q] = q == lane ? 0.0f : v[q];
    }
    return d;
}

// The passes between global memory and the fp32 stage work on 32 values a
// thread: 8 stored rows (major0 + 16 k) by 4 columns (minor0 + 32 q) of the
// CTA's part of the matrix (rows x cols as stored; T: X is its transpose).
// Addresses are clamped to valid elements rather than branched around, so that
// all loads are in flight together.
template <bool T>
__device__ __forceinline__ uint32_t stage_at(int major, int minor) {
    const int i = T ? minor : major, j = T ? major : minor;
    return f32_at<64>(i, j >> 2) + (j & 3) * 4;
}

// U (the gradient, or the updated momentum's) to the stage, zeros past the
// matrix; returns the sum of its squares.
template <typename Tg, bool T>
__device__ __forceinline__ float load_update(const SmallArgs& a, const SmallMat& m, uint32_t stage, int j0, int rows, int cols,
                                             int major0, int minor0) {
    const Tg* g = static_cast<const Tg*>(m.g) + (T ? (int64_t)j0 * m.ldg : j0);
    float* mom = m.mom ? m.mom + (T ? (int64_t)j0 * m.ldm : j0) : nullptr;
    int col[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) col[q] = min(minor0 + 32 * q, cols - 1);
    float u[8][4], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const Tg* p = g + (int64_t)min(major0 + 16 * k, rows - 1) * m.ldg;
#pragma unroll
        for (int q = 0; q < 4; ++q) u[k][q] = load1(p + col[q]);
    }
    if (mom) {
        float v[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float* p = mom + (int64_t)min(major0 + 16 * k, rows - 1) * m.ldm;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[k][q] = p[col[q]];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float* p = mom + (int64_t)(major0 + 16 * k) * m.ldm;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[k][q] = fmaf(a.mu, v[k][q], u[k][q]);
                if (major0 + 16 * k < rows && minor0 + 32 * q < cols) p[minor0 + 32 * q] = v[k][q];
                u[k][q] = a.nesterov ? fmaf(a.mu, v[k][q], u[k][q]) : v[k][q];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (!(major0 + 16 * k < rows && minor0 + 32 * q < cols)) u[k][q] = 0.0f;
            sum = fmaf(u[k][q], u[k][q], sum);
            sts1(stage + stage_at<T>(major0 + 16 * k, minor0 + 32 * q), u[k][q]);  // inside the 128 x 256 of the stage
        }
    return sum;
}

// The result, from the stage to the output (or the weight).
template <typename To, bool T>
__device__ __forceinline__ void store_update(const SmallArgs& a, const SmallMat& m, uint32_t stage, int j0, int rows, int cols,
                                             int major0, int minor0) {
    To* out = static_cast<To*>(m.out) + (T ? (int64_t)j0 * m.ldo : j0);
    int col[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) col[q] = min(minor0 + 32 * q, cols - 1);
    float v[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const To* p = out + (int64_t)min(major0 + 16 * k, rows - 1) * m.ldo;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k][q] = a.keep != 0.0f ? load1(p + col[q]) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        To* p = out + (int64_t)(major0 + 16 * k) * m.ldo + minor0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float y = fmaf(a.keep, v[k][q], lds1(stage + stage_at<T>(major0 + 16 * k, minor0 + 32 * q)));
            if (major0 + 16 * k < rows && minor0 + 32 * q < cols) {
                if constexpr (sizeof(To) == 2)
                    p[32 * q] = __float2bfloat16_rn(y);
                else
                    p[32 * q] = y;
            }
        }
    }
}

// S: CTAs of the cluster.
template <typename Tg, int S>
__global__ void __launch_bounds__(kThreads, 1) small_kernel(const __grid_constant__ SmallArgs a) {
    using namespace mma;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float diag[kSmallRows];
    __shared__ float coef[kSmallRows], warp_sum[16], rank_sum[8];
    const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const SmallMat& m = a.m[blockIdx.x / S];
    const bool transposed = m.rows > m.cols;
    const int r = transposed ? m.cols : m.rows, c = transposed ? m.rows : m.cols;
    const int chunks = (c + 63) / 64, ch0 = chunks * rank / S, nch = chunks * (rank + 1) / S - ch0;
    const int j0 = ch0 * 64, w = min(nch * 64, c - j0);  // this CTA's columns (none where nch = 0)
    auto barrier = [&]() {
        fence_before();
        if constexpr (S > 1)
            cluster_sync();
        else
            __syncthreads();
        fence_after();
    };

    if (threadIdx.x == 0) {
        tma::mbar_init(&done, 1);
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<1>(tma::smem_addr(&tmem_slot), 512);
    if (a.release) grid_launch_dependents();
    grid_wait();

    // U to shared memory as fp32 (rows and columns past the matrix as zeros), and its sum of squares
    float sum = 0.0f;
    const int rows = transposed ? w : r, cols = transposed ? r : w;  // of this CTA's part, as stored
    if (nch) {
        const int rows_all = transposed ? nch * 64 : 128, cols_all = transposed ? 128 : nch * 64;
        for (int i0 = 0; i0 < rows_all; i0 += 128)
            for (int c0 = 0; c0 < cols_all; c0 += 128)
                sum += transposed ? load_update<Tg, true>(a, m, base, j0, rows, cols, i0 + warp, c0 + lane)
                                  : load_update<Tg, false>(a, m, base, j0, rows, cols, i0 + warp, c0 + lane);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    barrier();  // with a cluster: the other CTAs have started, so their shared memory may be written
    const uint32_t tmem = tmem_slot;
    float norm = 0.0f;
    for (int k = 0; k < 16; ++k) norm += warp_sum[k];
    if constexpr (S > 1) {
        if (threadIdx.x < S) st_cluster(map_rank(tma::smem_addr(&rank_sum[rank]), threadIdx.x), norm);
        cluster_sync();
        norm = 0.0f;
#pragma unroll
        for (int p = 0; p < S; ++p) norm += rank_sum[p];
    }
    // entries of X near 1 (see muon.cu); a power of two
    const float scale = exp2f(rintf(0.5f * log2f((float)c)));
    const float f = norm_factor(scale, norm, a.eps);

    // Every thread owns a row (its tensor-memory lane) and columns quarter * 32 + 128 h + 0..31, h = 0, 1.
    const int row = (warp & 3) * 32 + lane, quarter = warp >> 2;
    float x[2][32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = quarter * 32 + 128 * h;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float v[4] = {};
            if (j < nch * 64) lds4(base + f32_at<64>(row, j / 4 + q), v);
#pragma unroll
            for (int y = 0; y < 4; ++y) x[h][4 * q + y] = v[y] * f;
        }
    }
    __syncthreads();
    auto store_operand = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = quarter * 32 + 128 * h;
            if (j < nch * 64) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    stsq(base + kX + at(row, j + 8 * q),
                         make_uint4(pack_half2(x[h][8 * q], x[h][8 * q + 1]), pack_half2(x[h][8 * q + 2], x[h][8 * q + 3]),
                                    pack_half2(x[h][8 * q + 4], x[h][8 * q + 5]), pack_half2(x[h][8 * q + 6], x[h][8 * q + 7])));
            }
        }
    };
    store_operand();

    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), acc = lanes + 256;
    const uint32_t idesc = instr_desc(128, 128, false, false, false);
    const bool diagonal = quarter == (warp & 3);  // this thread's 32 columns of a 128 x 128 matrix hold its diagonal element
    uint32_t phase = 0;
    bool ok = true;
    // Every product is issued by one thread and waited for by all.
    auto wait_product = [&]() {
        if (ok && !tma::mbar_wait(&done, phase)) {
            record_device_error(a.err, DPRED_E_TIMEOUT);
            ok = false;
        }
        phase ^= 1;
        __syncwarp();
        fence_after();
    };

    for (int step = 0; step < a.steps; ++step) {
        // ------------------------------------------------------------- Gram
        tma::fence_proxy_async_shared();
        fence_before();
        __syncthreads();
        if (warp == 0) {
            if (elect_one()) {
                fence_after();
                const uint64_t d = operand_desc(base + kX, false);
                for (int k = 0; k < nch * 4; ++k) {
                    const uint64_t dk = d + (k >> 2) * (kChunk >> 4) + (k & 3) * 2;
                    issue<1>(tmem + 256, dk, dk, idesc, k != 0);
                }
                commit<1>(tma::smem_addr(&done));
            }
            __syncwarp();
        }
        wait_product();
        const float alpha = 1.0f / (scale * scale);
        {
            float v[32];
            if (nch) {
                tmem_ld32(acc + quarter * 32, v);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = 0.0f;
            }
            if constexpr (S == 1) {  // straight to the operand: off-diagonal in fp16, diagonal in fp32
                if (diagonal) diag[row] = take_lane(v, lane) * alpha;
                const float to = alpha * kOffScale;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    stsq(base + kE + at(row, quarter * 32 + 8 * q),
                         make_uint4(pack_half2(v[8 * q] * to, v[8 * q + 1] * to), pack_half2(v[8 * q + 2] * to, v[8 * q + 3] * to),
                                    pack_half2(v[8 * q + 4] * to, v[8 * q + 5] * to), pack_half2(v[8 * q + 6] * to, v[8 * q + 7] * to)));
                tma::fence_proxy_async_shared();
                barrier();
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    sts4(base + kPart + f32_at<32>(row, quarter * 8 + q), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                cluster_sync();
                // 128 / S rows of 32 pieces; every load of this thread in flight at once
                constexpr int kEach = 8 / S;
                float t[kEach][S][4];
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const int i = 128 / S * rank + warp + 16 * k;
#pragma unroll
                    for (int p = 0; p < S; ++p) ld_cluster4(map_rank(base + kPart + f32_at<32>(i, lane), p), t[k][p]);
                }
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const int i = 128 / S * rank + warp + 16 * k;
                    float z[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        z[y] = t[k][0][y];
#pragma unroll
                        for (int p = 1; p < S; ++p) z[y] += t[k][p][y];
                        z[y] *= alpha;
                    }
                    if (lane == i / 4) {
                        const float d = i % 4 == 0 ? z[0] : i % 4 == 1 ? z[1] : i % 4 == 2 ? z[2] : z[3];
#pragma unroll
                        for (int p = 0; p < S; ++p) st_cluster(map_rank(tma::smem_addr(&diag[i]), p), d);
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) z[y] = lane * 4 + y == i ? 0.0f : z[y] * kOffScale;
                    const uint32_t lo = pack_half2(z[0], z[1]), hi = pack_half2(z[2], z[3]), to = base + kE + at(i, lane * 4);
#pragma unroll
                    for (int p = 0; p < S; ++p) st_cluster2(map_rank(to, p), lo, hi);
                }
                fence_proxy_async();
                barrier();
            }
        }
        // ------------------------------------------------------------- polynomial
        if (warp == 0) {
            if (elect_one()) {
                fence_proxy_async();
                const uint64_t d = operand_desc(base + kE, false);
                for (int k = 0; k < 8; ++k) {
                    const uint64_t dk = d + (k >> 2) * (kChunk >> 4) + (k & 3) * 2;
                    issue<1>(tmem + 256, dk, dk, idesc, k != 0);
                }
                commit<1>(tma::smem_addr(&done));
            }
            __syncwarp();
        }
        // while it runs: this thread's factors of E
        const float di = diag[row], lin = fmaf(a.c, di, a.b), sq = a.c / kOffScale;  // E^2 is scaled by 256^2, the result by 256
        uint4 e8[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) e8[q] = ldsq(base + kE + at(row, quarter * 32 + 8 * q));
        wait_product();
        {
            float v[32];
            tmem_ld32(acc + quarter * 32, v);
            tmem_wait_ld();
            if (diagonal)  // E's stored diagonal is 0, so P's becomes 0 too
                coef[row] = a.a + fmaf(a.c, fmaf(di, di, take_lane(v, lane) * (1.0f / (kOffScale * kOffScale))), a.b * di);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float e[8], dj[8], t[8];
                half8(e8[q], e);
                lds4(tma::smem_addr(&diag[quarter * 32 + 8 * q]), dj);
                lds4(tma::smem_addr(&diag[quarter * 32 + 8 * q + 4]), dj + 4);
#pragma unroll
                for (int y = 0; y < 8; ++y) t[y] = fmaf(fmaf(a.c, dj[y], lin), e[y], sq * v[8 * q + y]);
                stsq(base + kP + at(row, quarter * 32 + 8 * q),
                     make_uint4(pack_half2(t[0], t[1]), pack_half2(t[2], t[3]), pack_half2(t[4], t[5]), pack_half2(t[6], t[7])));
            }
        }
        // ------------------------------------------------------------- apply
        tma::fence_proxy_async_shared();
        fence_before();
        __syncthreads();
        if (warp == 0) {
            if (elect_one()) {
                fence_after();
                if (nch) {
                    const uint32_t id = instr_desc(128, nch * 64, false, false, true);
                    const uint64_t da = operand_desc(base + kP, false);
                    // MN-major: 64-column chunks kChunk apart, 8 reduction rows 1024 bytes apart
                    const uint64_t db = operand_desc(base + kX, true, kChunk);
                    for (int k = 0; k < 8; ++k)
                        issue<1>(tmem, da + (k >> 2) * (kChunk >> 4) + (k & 3) * 2, db + k * 128, id, k != 0);
                }
                commit<1>(tma::smem_addr(&done));
            }
            __syncwarp();
        }
        wait_product();
        const float k1 = coef[row], inv = 1.0f / kOffScale;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = quarter * 32 + 128 * h;
            if (j < nch * 64) {  // the same in the whole warp
                float v[32];
                tmem_ld32(lanes + j, v);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 32; ++q) x[h][q] = fmaf(k1, x[h][q], v[q] * inv);
            }
        }
        if (step + 1 < a.steps) store_operand();
    }

    // the result, through shared memory so that global rows are written by whole warps
    __syncthreads();
    const float scl = m.step / scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = quarter * 32 + 128 * h;
        if (j < nch * 64) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                sts4(base + f32_at<64>(row, j / 4 + q), x[h][4 * q] * scl, x[h][4 * q + 1] * scl, x[h][4 * q + 2] * scl,
                     x[h][4 * q + 3] * scl);
        }
    }
    __syncthreads();
    if (nch && ok) {
        for (int i0 = 0; i0 < rows; i0 += 128)
            for (int c0 = 0; c0 < cols; c0 += 128) {
                if (a.out_f32)
                    transposed ? store_update<float, true>(a, m, base, j0, rows, cols, i0 + warp, c0 + lane)
                               : store_update<float, false>(a, m, base, j0, rows, cols, i0 + warp, c0 + lane);
                else
                    transposed ? store_update<__nv_bfloat16, true>(a, m, base, j0, rows, cols, i0 + warp, c0 + lane)
                               : store_update<__nv_bfloat16, false>(a, m, base, j0, rows, cols, i0 + warp, c0 + lane);
            }
    }
    barrier();  // no CTA leaves while another may still read its shared memory
    if (warp == 1) tmem_free<1>(tmem, 512);
}

template <typename Tg, int S>
int launch(const SmallArgs& a, cudaStream_t s) {
    static bool attr[64] = {};
    auto kernel = small_kernel<Tg, S>;
    cudaError_t e = ensure_smem_attr(kernel, (int)kSmem, attr);
    if (e != cudaSuccess) return cuda_error(e, "shared-memory limit of a small orthogonalised update");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.count * a.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.split;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? DPRED_OK : cuda_error(e, "small orthogonalised update launch");
}

template <typename Tg>
int launch_split(const SmallArgs& a, cudaStream_t s) {
    switch (a.split) {
        case 1: return launch<Tg, 1>(a, s);
        case 2: return launch<Tg, 2>(a, s);
        case 4: return launch<Tg, 4>(a, s);
        default: return launch<Tg, 8>(a, s);
    }
}

}  // namespace

int small_split(int64_t rows, int64_t cols) {
    const int64_t r = std::min(rows, cols), c = std::max(rows, cols);
    if (r > kSmallRows || c > kSmallCols) return 0;
    int s = 1;
    while (c > (int64_t)s * 256) s *= 2;
    return s;
}

int run_small(const SmallArgs& a, cudaStream_t s) { return a.g_f32 ? launch_split<float>(a, s) : launch_split<__nv_bfloat16>(a, s); }

}  // namespace gemm
}  // namespace dpred
