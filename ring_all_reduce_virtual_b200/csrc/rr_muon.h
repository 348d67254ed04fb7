// rr_muon.h -- layouts, parameter blocks and launchers of the orthogonalisation
// and the Muon step (rr_muon.cu, rr_muon_gemm.cu, host side rr_muon_api.cu).
// Not part of the C ABI.
//
// A value of the iteration is kept as two fp16 halves, v = (hi + lo) / scale
// with hi = fp16(v * scale) and lo = fp16(v * scale - hi): 22 bits for values
// within 2^-12 of the largest, which the scale (a power of two) puts just
// below fp16's largest.  One fp16 (or bf16) misses the exact polynomial by
// 2e-3 to 2e-2 (1e-2 to 2e-1): the steps multiply what they round by up to
// 3.4445 each wherever a singular value is small.
//
// A matrix of halves lies in blocks of 64 x 64 (8 KB), rows and columns padded
// to multiples of 128 with zeros.  Block (i, j) is number ((i / 2) * columns of
// blocks + j) * 2 + i % 2: the two blocks of 128 rows follow one another.
// Within a block, row r has 128 bytes whose 16-byte pieces are permuted, piece
// c lying at c ^ (r % 8): the 128-byte swizzle of the tensor core's operands.
// So a block is copied to shared memory as it is, and serves as an operand
// with its rows along K or with its columns along K.
#pragma once

#include "rr_internal.h"

namespace rr {

constexpr uint32_t kBlk = 64;                   // rows and columns of a block
constexpr uint32_t kBlkElems = kBlk * kBlk;
constexpr uint32_t kPad = 128;                  // rows and columns are padded to multiples of this

__host__ __device__ constexpr uint32_t pad_up(uint32_t x) { return (x + kPad - 1) / kPad * kPad; }

// Offset (halves) of block (i, j) in a matrix of `nbj` columns of blocks.
__host__ __device__ constexpr uint64_t block_at(uint32_t i, uint32_t j, uint32_t nbj)
{
    return (((uint64_t)(i >> 1) * nbj + j) * 2 + (i & 1)) * kBlkElems;
}

// Offset (halves) of the 16-byte piece that begins at element (r, c).
__host__ __device__ constexpr uint64_t piece_at(uint32_t r, uint32_t c, uint32_t nbj)
{
    return block_at(r / kBlk, c / kBlk, nbj) + (r % kBlk) * kBlk + ((((c % kBlk) >> 3) ^ (r & 7u)) << 3);
}

// A blocked matrix: the two halves.
struct Halves {
    uint16_t* hi;
    uint16_t* lo;
};

// One product of a launch: out = alpha * op(a) op(b)^T + beta * c + diag * 1,
// on tiles of 256 rows and `tile_n` columns.  A symmetric matrix is formed and
// kept on and below the diagonal of its 256 x 256 tiles; an operand's block
// above it is read as the transpose of the one below.
struct MuonProduct {
    Halves a, b, c, out;   // c.hi NULL: none
    uint32_t a_nbj, b_nbj, o_nbj;  // columns of blocks: operands, out (and c)
    uint32_t mt, nu, kb;   // units of 128 rows, of 128 columns, blocks along K
    uint32_t tile0;        // the launch's first tile of this product
    uint8_t a_mn, b_mn;    // the operand's rows run along K (not its columns)
    uint8_t a_low, b_low;  // the operand is symmetric, kept on and below the diagonal
    uint32_t side;         // diag goes to the first `side` elements of the diagonal
    uint8_t sym, pad_[3];  // the result is symmetric
    float alpha, beta, diag;
};

constexpr int kMuonMats = 24;     // matrices per launch: parameter blocks below 4 KB,
constexpr int kMuonProducts = 30; // which larger ones cost the host 3-5 us more
constexpr uint32_t kNormParts = 256;  // partial sums of squares per matrix, at most
constexpr uint32_t kPrepTile = 8192;  // elements of a tile of the first pass

struct MuonGemmParams {
    MuonProduct q[kMuonProducts];
    int n;
    uint32_t tile_n;       // 128 or 256
    uint32_t tiles;
    unsigned int* waits;   // bulk_wait_counters()
    uint32_t hold, spin;   // as in BulkParams
};

// What the elementwise passes need of a matrix.
struct MuonMat {
    const void* g;         // gradient, or the matrix itself
    float* m;              // momentum; NULL: orthogonalize
    uint32_t rows, cols;
    uint32_t part0, parts; // its partial sums
    Halves x;
    uint32_t tile0;        // first tile of the launch, 128 rows x 64 columns
    uint8_t dtype, out_dtype, vec, pad_;
    uint32_t out;          // muon: index of its first pointer in MuonFinishParams::out
    float factor;          // muon: lr * the shape's factor
};

struct MuonPrepParams {
    MuonMat mat[kMuonMats];
    int n;
    double* partial;
    float momentum;
    int nesterov;
    float eps;
    float scale;           // of the first X
};

constexpr int kMuonPtrs = 128;
struct MuonFinishParams {
    MuonMat mat[kMuonMats];
    int n;
    int nranks;            // outputs per matrix
    float inv;             // 1 / the scale of X
    float keep;            // muon: 1 - lr * weight decay
    void* out[kMuonPtrs];  // matrix-major
};

cudaError_t launch_muon_squares(const MuonPrepParams& p, uint32_t parts, cudaStream_t s);
cudaError_t launch_muon_pack(const MuonPrepParams& p, uint32_t tiles, cudaStream_t s);
cudaError_t launch_muon_finish(const MuonFinishParams& p, uint32_t tiles, cudaStream_t s);
// Fills in the tiles and the waits and launches.
cudaError_t launch_muon_gemm(MuonGemmParams& p, cudaStream_t s);

}  // namespace rr
