// muon_small.cuh -- orthogonalised updates of small matrices, whole in one launch.
#pragma once

#include "gemm.cuh"

namespace dpred {
namespace gemm {

constexpr int kSmallRows = 128;                  // shorter side, at most
constexpr int kSmallCols = 2048;                 // longer side, at most (8 CTAs x 256 columns)
constexpr int kSmallBatch = 64;                  // matrices per launch

struct SmallMat {
    const void* g;
    float* mom;          // null: U = G
    void* out;
    int64_t ldg, ldm, ldo;
    int rows, cols;      // as stored; X is the matrix or its transpose, shorter side first
    float step;          // factor of the orthogonalised value in the output
};

struct SmallArgs {
    SmallMat m[kSmallBatch];
    int count;
    int split;           // CTAs of a cluster, each holding a run of X's columns
    int steps, nesterov, g_f32, out_f32;
    int release;         // a later launch of the same call follows
    float mu, eps, a, b, c, keep;
    int* err;
};

// CTAs that a matrix of this shape takes (0: it is too large).
int small_split(int64_t rows, int64_t cols);
int run_small(const SmallArgs& a, cudaStream_t s);

}  // namespace gemm
}  // namespace dpred
