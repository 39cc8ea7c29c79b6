// muon_small.cu -- one launch for a whole orthogonalised update of matrices of
// up to 128 x 2048.
//
// The general path takes 17 launches, each a few microseconds whatever the
// size.  Here a cluster keeps a matrix in shared memory for the whole update:
// each of its 1 to 8 CTAs holds up to 256 columns of X (both fp16 terms), and
// a step is
//   Gram    every CTA multiplies its own columns, 128 x 128 partial sums; they
//           are added through distributed shared memory, each CTA summing a
//           band of rows in rank order and sending the result to all;
//   poly    every CTA computes the whole 128 x 128 polynomial;
//   apply   every CTA updates its own columns in place.
// The arithmetic and its precision are those of the general path (muon.cu).
// Tiles lie in the 128-byte swizzle, 64 columns wide: the same bytes serve the
// Gram product as K-major rows and the apply product as an MN-major operand.
// What bounds it is latency: 2 cluster barriers and 3 dependent products a step.
#include "muon_small.cuh"

#include <algorithm>

namespace dpred {
namespace gemm {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t kChunk = 128 * 128;           // 128 rows x 64 columns of fp16
constexpr float kOffScale = 256.0f;
// shared memory: X leading terms, X trailing terms (4 chunks each), E (2), partial sums (128 x 128 fp32; P lies over them)
constexpr uint32_t kHi = 0, kLo = 4 * kChunk, kE = 8 * kChunk, kPart = 10 * kChunk, kP = kPart;
constexpr uint32_t kSmem = 14 * kChunk + 1024;

// Byte of element (row, col) of a matrix stored in 64-column chunks.
__device__ __forceinline__ uint32_t at(int row, int col) {
    return (col >> 6) * kChunk + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}
// 16-byte piece c4 of a row of the fp32 partial sums.
__device__ __forceinline__ uint32_t part_at(int row, int c4) { return row * 512 + ((c4 ^ (row & 7)) << 4); }

__device__ __forceinline__ void sts2(uint32_t a, float x) {
    const __half h = __float2half_rn(x);
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(*reinterpret_cast<const uint16_t*>(&h)) : "memory");
}
__device__ __forceinline__ uint4 ldsq(uint32_t a) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(a) : "memory");
    return q;
}
__device__ __forceinline__ void stsq(uint32_t a, uint4 q) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
    if constexpr (sizeof(T) == 2)
        return load_bf16(reinterpret_cast<const __nv_bfloat16*>(p));
    else
        return *p;
}

template <typename Tg>
__global__ void __launch_bounds__(kThreads, 1) small_kernel(const __grid_constant__ SmallArgs a) {
    using namespace mma;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ float diag[kSmallRows], coef[kSmallRows], warp_sum[16], rank_sum[8];
    const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_rank(), S = a.split;
    const SmallMat& m = a.m[blockIdx.x / S];
    const bool transposed = m.rows > m.cols;
    const int r = transposed ? m.cols : m.rows, c = transposed ? m.rows : m.cols;
    const int chunks = (c + 63) / 64, ch0 = chunks * rank / S, nch = chunks * (rank + 1) / S - ch0;
    const int j0 = ch0 * 64, w = min(nch * 64, c - j0);  // this CTA's columns (none where w <= 0)

    if (threadIdx.x == 0) {
        tma::mbar_init(&done, 1);
        tma::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<1>(tma::smem_addr(&tmem_slot), 512);
    for (uint32_t b = threadIdx.x * 16; b < (uint32_t)nch * kChunk; b += kThreads * 16) {
        stsq(base + kHi + b, make_uint4(0, 0, 0, 0));
        stsq(base + kLo + b, make_uint4(0, 0, 0, 0));
    }
    grid_launch_dependents();
    grid_wait();

    // U in registers, 64 values a thread: along the stored rows (rows warp + 16 k,
    // columns lane + 32 q of X; or of its transpose, columns warp + 16 k, rows lane + 32 q)
    const Tg* g = static_cast<const Tg*>(m.g);
    float u[64], sum = 0.0f;
    const int n_major = transposed ? 16 : 8, n_minor = transposed ? 4 : 8;
#pragma unroll
    for (int x = 0; x < 64; ++x) {
        const int major = warp + 16 * (transposed ? x >> 2 : x >> 3), minor = lane + 32 * (transposed ? x & 3 : x & 7);
        const int i = transposed ? minor : major, j = transposed ? major : minor;
        u[x] = 0.0f;
        if (i < r && j < w) u[x] = load1(g + (transposed ? (int64_t)(j0 + j) * m.ldg + i : (int64_t)i * m.ldg + j0 + j));
    }
    (void)n_major;
    (void)n_minor;
    if (m.mom) {
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
            float v[32];
#pragma unroll
            for (int y = 0; y < 32; ++y) {
                const int x = h + y;
                const int major = warp + 16 * (transposed ? x >> 2 : x >> 3), minor = lane + 32 * (transposed ? x & 3 : x & 7);
                const int i = transposed ? minor : major, j = transposed ? major : minor;
                v[y] = 0.0f;
                if (i < r && j < w) v[y] = m.mom[transposed ? (int64_t)(j0 + j) * m.ldm + i : (int64_t)i * m.ldm + j0 + j];
            }
#pragma unroll
            for (int y = 0; y < 32; ++y) {
                const int x = h + y;
                const int major = warp + 16 * (transposed ? x >> 2 : x >> 3), minor = lane + 32 * (transposed ? x & 3 : x & 7);
                const int i = transposed ? minor : major, j = transposed ? major : minor;
                if (i < r && j < w) {
                    v[y] = fmaf(a.mu, v[y], u[x]);
                    m.mom[transposed ? (int64_t)(j0 + j) * m.ldm + i : (int64_t)i * m.ldm + j0 + j] = v[y];
                    u[x] = a.nesterov ? fmaf(a.mu, v[y], u[x]) : v[y];
                }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 64; ++x) sum = fmaf(u[x], u[x], sum);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    fence_before();
    cluster_sync();  // the other CTAs have started: their shared memory may be written
    fence_after();
    const uint32_t tmem = tmem_slot;
    if (threadIdx.x < S) {
        float t = 0.0f;
        for (int k = 0; k < 16; ++k) t += warp_sum[k];
        st_cluster(map_rank(tma::smem_addr(&rank_sum[rank]), threadIdx.x), t);
    }
    cluster_sync();
    float norm = 0.0f;
    for (int p = 0; p < S; ++p) norm += rank_sum[p];
    // entries of X near 1 (see muon.cu); a power of two
    const float scale = exp2f(rintf(0.5f * log2f((float)c)));
    const float f = scale / (sqrtf(norm) + a.eps);
#pragma unroll
    for (int x = 0; x < 64; ++x) {
        const int major = warp + 16 * (transposed ? x >> 2 : x >> 3), minor = lane + 32 * (transposed ? x & 3 : x & 7);
        const int i = transposed ? minor : major, j = transposed ? major : minor;
        if (i < r && j < w) {
            const float v = u[x] * f, h = __half2float(__float2half_rn(v));
            sts2(base + kHi + at(i, j), h);
            sts2(base + kLo + at(i, j), v - h);
        }
    }

    // Every thread owns a tensor-memory row and a quarter of its columns.
    const int row = (warp & 3) * 32 + lane, quarter = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), acc = lanes + 256;
    const uint32_t idesc = instr_desc(128, 128, false, false, false);
    uint32_t phase = 0;
    bool ok = true;
    // one product: issued by one thread, waited for by all; the operands were
    // written by this CTA (or its peers, before a cluster barrier)
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
                const uint64_t d = operand_desc(base + kHi, false);
                for (int k = 0; k < nch * 4; ++k) {
                    const uint64_t dk = d + (k >> 2) * (kChunk >> 4) + (k & 3) * 2;
                    issue<1>(tmem + 256, dk, dk, idesc, k != 0);
                }
                commit<1>(tma::smem_addr(&done));
            }
            __syncwarp();
        }
        wait_product();
        {
            float v[32];
            if (nch) {
                tmem_ld32(acc + quarter * 32, v);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = 0.0f;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) sts4(base + kPart + part_at(row, quarter * 8 + x), v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
        }
        cluster_sync();
        const float alpha = 1.0f / (scale * scale);
        for (int t = threadIdx.x; t < 128 / S * 32; t += kThreads) {
            const int i = 128 / S * rank + t / 32, c4 = t % 32;
            float v[4];
            cluster_get(base + kPart + part_at(i, c4), S, v);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                v[x] *= alpha;
                if (c4 * 4 + x == i) {
                    for (int p = 0; p < S; ++p) st_cluster(map_rank(tma::smem_addr(&diag[i]), p), v[x]);
                    v[x] = 0.0f;
                }
                v[x] *= kOffScale;
            }
            const uint32_t lo = pack_half2(v[0], v[1]), hi = pack_half2(v[2], v[3]), to = base + kE + at(i, c4 * 4);
            for (int p = 0; p < S; ++p) st_cluster2(map_rank(to, p), lo, hi);
        }
        fence_proxy_async();
        fence_before();
        cluster_sync();
        // ------------------------------------------------------------- polynomial
        if (warp == 0) {
            if (elect_one()) {
                fence_after();
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
        wait_product();
        {
            float v[32];
            tmem_ld32(acc + quarter * 32, v);
            tmem_wait_ld();
            const float di = diag[row], lin = fmaf(a.c, di, a.b), sq = a.c / kOffScale;  // E^2 is scaled by 256^2, the result by 256
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = quarter * 32 + x * 8;
                float e8[8], t[8];
                half8(ldsq(base + kE + at(row, j)), e8);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    t[y] = fmaf(fmaf(a.c, diag[j + y], lin), e8[y], sq * v[8 * x + y]);
                    if (j + y == row) {
                        coef[row] = a.a + fmaf(a.c, fmaf(di, di, v[8 * x + y] / (kOffScale * kOffScale)), a.b * di);
                        t[y] = 0.0f;
                    }
                }
                stsq(base + kP + at(row, j), pack8(t));
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
                    const uint64_t db = operand_desc(base + kHi, true, kChunk);
                    for (int k = 0; k < 8; ++k)
                        issue<1>(tmem, da + (k >> 2) * (kChunk >> 4) + (k & 3) * 2, db + k * 128, id, k != 0);
                }
                commit<1>(tma::smem_addr(&done));
            }
            __syncwarp();
        }
        wait_product();
        const bool last = step + 1 == a.steps;
        const float k1 = coef[row], inv = 1.0f / kOffScale;
        for (int j = quarter * 32; j < nch * 64; j += 128) {
            float v[32];
            tmem_ld32(lanes + j, v);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t p = at(row, j + 8 * x);
                float h[8], l[8];
                half8(ldsq(base + kHi + p), h);
                half8(ldsq(base + kLo + p), l);
#pragma unroll
                for (int y = 0; y < 8; ++y) v[8 * x + y] = fmaf(k1, h[y] + l[y], v[8 * x + y] * inv);
                if (!last) {
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        h[y] = __half2float(__float2half_rn(v[8 * x + y]));
                        l[y] = v[8 * x + y] - h[y];
                    }
                    stsq(base + kHi + p, pack8(h));
                    stsq(base + kLo + p, pack8(l));
                }
            }
            if (last && ok && row < r) {
                const float scl = m.step / scale;
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    if (j + x >= w) break;
                    const int64_t o = transposed ? (int64_t)(j0 + j + x) * m.ldo + row : (int64_t)row * m.ldo + j0 + j + x;
                    const float y = v[x] * scl;
                    if (a.out_f32) {
                        float* q = static_cast<float*>(m.out) + o;
                        *q = a.keep != 0.0f ? fmaf(a.keep, *q, y) : y;
                    } else {
                        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(m.out) + o;
                        *q = __float2bfloat16_rn(a.keep != 0.0f ? fmaf(a.keep, load_bf16(q), y) : y);
                    }
                }
            }
            __syncwarp();
        }
    }
    fence_before();
    cluster_sync();  // no CTA leaves while another may still read its shared memory
    if (warp == 1) {
        fence_after();
        tmem_free<1>(tmem, 512);
    }
}

template <typename Tg>
int launch(const SmallArgs& a, cudaStream_t s) {
    static bool attr[64] = {};
    auto kernel = small_kernel<Tg>;
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

}  // namespace

int small_split(int64_t rows, int64_t cols) {
    const int64_t r = std::min(rows, cols), c = std::max(rows, cols);
    if (r > kSmallRows || c > kSmallCols) return 0;
    int s = 1;
    while (c > (int64_t)s * 256) s *= 2;
    return s;
}

int run_small(const SmallArgs& a, cudaStream_t s) { return a.g_f32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s); }

}  // namespace gemm
}  // namespace dpred
