// muon_chain.cuh -- the products of whole orthogonalised updates in one launch.
#pragma once

#include "gemm_host.cuh"

namespace dpred {
namespace gemm {

constexpr int kChainGroups = 8;  // shapes per launch

// The matrices of one shape: X is r x c (r <= c), `count` of them.
struct ChainGroup {
    CUtensorMap x[2];     // X's leading term, K-major (boxes of 128 rows), two buffers
    CUtensorMap xt[2];    // the same as an MN-major operand
    CUtensorMap gram[2];  // K-major, MN-major
    CUtensorMap poly[2];
    NsEpi e;
    __half* hi[2];
    int r, c, count, first; // first: index of the group's first matrix (counter, output entry)
    int tiles_r, tiles_c;   // 256 x 256 tiles of the r x r products' rows, of X's columns
    int gram_tiles;         // tiles of a symmetric product
    float gram_alpha;       // factor of the Gram accumulators
};

struct ChainArgs {
    ChainGroup g[kChainGroups];
    FinalOut out[kMaxBatch];
    int groups, steps;
    int gram_total, apply_total;  // tiles of all matrices, per phase
    unsigned* counter;            // [matrices], 0 at launch: epilogue warps that have finished a tile
    int* err;
};

int run_chain(const ChainArgs& a, cudaStream_t s);

}  // namespace gemm
}  // namespace dpred
