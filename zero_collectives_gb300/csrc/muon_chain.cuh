// muon_chain.cuh -- the products of whole orthogonalised updates in one launch.
#pragma once

#include "gemm_host.cuh"

namespace dpred {
namespace gemm {

constexpr int kChainGroups = 8;   // shapes per launch
constexpr int kChainOps = 112;    // products of one matrix, at most (32 steps)
constexpr int kSquares = 4;       // r x r matrices in memory: see chain_program()

enum ChainKind : uint8_t { CHAIN_GRAM, CHAIN_POLY, CHAIN_MUL, CHAIN_APPLY, CHAIN_FINAL };

// One product of a matrix's program.
struct ChainOp {
    uint8_t kind;
    uint8_t a, b, out;        // r x r matrices: factors (POLY: a; APPLY, FINAL: a times X), result
    uint8_t x;                // which of the two buffers holds X's leading term
    uint8_t squares, applies; // r x r products and products with X before this one
    uint8_t reserved;
};

// The matrices of one shape: X is r x c (r <= c), `count` of them.
struct ChainGroup {
    CUtensorMap x[2];             // X's leading term, K-major (boxes of 128 rows), two buffers
    CUtensorMap xt[2];            // the same as an MN-major operand
    CUtensorMap square[kSquares][2];  // the r x r matrices, K-major and MN-major
    NsEpi e;
    __half* hi[2];
    __half* sq[kSquares];
    float* diag[kSquares];
    int r, c, count, first;       // first: index of the group's first matrix (counter, output entry)
    int tiles_r, tiles_c;         // 256 x 256 tiles of the r x r products' rows, of X's columns
    int square_tiles;             // tiles of a symmetric product
    int program, ops;             // which program, and its length
};

struct ChainArgs {
    ChainGroup g[kChainGroups];
    FinalOut out[kMaxBatch];
    ChainOp program[2][kChainOps];
    int groups, ops;              // the longest program
    int most;                     // tiles of the largest product
    unsigned* counter;            // [matrices], 0 at launch: epilogue warps that have finished a tile
    int* err;
};

int run_chain(const ChainArgs& a, cudaStream_t s);

}  // namespace gemm
}  // namespace dpred
