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

// The products of all matrices of a call's group run in one launch, as a list
// of tiles of 256 rows and `tile_n` columns that pairs of CTAs take in order.
//
// A product: out = alpha * a b^T + beta * c + diag * 1.  Of a matrix with
// m <= n sides, X is rows x cols and the others m x m:
//   kGram    X X^T, or X^T X of a tall matrix (symmetric)
//   kSquare  two symmetric m x m matrices that commute (symmetric)
//   kApply   Q X, or X Q of a tall matrix
// A symmetric matrix is formed and kept on and below the diagonal of its
// 256 x 256 tiles; an operand's block above it is read as the transpose of the
// one below.
enum MuonKind : int { kGram = 0, kSquare = 1, kApply = 2 };

// Buffers of a matrix: 0 and 1 are X's, kSquares and up the m x m ones.
constexpr uint8_t kSquares = 2, kNoBuffer = 255;

struct MuonOp {
    float alpha, beta, diag;
    uint8_t kind, a, b, c, out;  // buffers; c kNoBuffer: none.  kApply: a is Q, b is X
    uint8_t level;               // reads what its matrix's earlier levels wrote
    uint8_t chunk;               // stages of 64 of K that an accumulator collects
    uint8_t pad_;
};

struct MuonWork {
    uint16_t* x[2];
    uint16_t* squares;
    uint32_t rows, cols;
    uint16_t op0, ops;           // its products in MuonGemmParams::op, in the order of their levels
};

// Matrices per group, and per launch that takes them whole.  While one waits for a
// level of its own, others have tiles: 24 layers of width 256, bf16, in groups of 24
// / 128: 960 / 450 us, 12 of 1024: 5620 / 5570.
constexpr int kMuonMats = 128;
constexpr int kMuonOps = 200;         // different products of a launch, at most
constexpr int kMuonSeq = 768;         // products of a launch, those of like matrices counted once
// Of parameter blocks below 4 KB: larger ones cost the host 3-5 us.
constexpr int kMuonMatsSmall = 24, kMuonOpsSmall = 60, kMuonSeqSmall = 400;
constexpr uint32_t kMuonCounters = 160;  // words of the workspace: the next tile, each matrix's finished parts
constexpr uint32_t kNormParts = 256;  // partial sums of squares per matrix, at most
constexpr uint32_t kPrepTile = 8192;  // elements of a tile of the first pass

struct MuonGemmHead {
    uint32_t n, nseq;
    uint32_t tile_n[3];    // of each kind of product: 128 or 256
    uint32_t* counters;
    unsigned int* waits;   // bulk_wait_counters()
    uint32_t hold, spin;   // as in BulkParams
};
template <int MATS, int OPS, int SEQ>
struct MuonGemmParamsT : MuonGemmHead {
    MuonWork work[MATS];
    MuonOp op[OPS];
    uint32_t seq[SEQ];     // the products in order, of neighbouring matrices of one shape: first | how many << 8 | number << 16
};
using MuonGemmParams = MuonGemmParamsT<kMuonMats, kMuonOps, kMuonSeq>;

// Sides of a matrix's product, in units of 128 rows and columns, and its tiles.
struct MuonSides {
    uint32_t mt, nu;
};

__host__ __device__ inline MuonSides muon_sides(uint32_t rows, uint32_t cols, int kind)
{
    const uint32_t mu = pad_up(rows < cols ? rows : cols) / 128;
    if (kind == kApply) return {pad_up(rows) / 128, pad_up(cols) / 128};
    return {mu, mu};
}

// Column tiles of row tile i of a symmetric result.
__host__ __device__ inline uint32_t muon_sym_tiles(uint32_t i, uint32_t nu, uint32_t per)
{
    const uint32_t units = 2 * i + 2 < nu ? 2 * i + 2 : nu;
    return (units + per - 1) / per;
}

__host__ __device__ inline uint32_t muon_tiles(uint32_t rows, uint32_t cols, int kind, uint32_t tile_n)
{
    const MuonSides s = muon_sides(rows, cols, kind);
    const uint32_t per = tile_n / 128, r = (s.mt + 1) / 2;
    if (kind == kApply) return r * ((s.nu + per - 1) / per);
    // the sum of muon_sym_tiles over the row tiles
    return per == 2 ? r * (r + 1) / 2 : r * (r + 1) - (s.mt & 1);
}

// What the elementwise passes need of a matrix.
struct MuonMat {
    const void* g;         // gradient, or the matrix itself
    float* m;              // momentum; NULL: orthogonalize
    uint32_t rows, cols;
    uint32_t part0, parts; // its partial sums
    Halves x;
    uint32_t tile0;        // first tile of the launch, 128 rows x 64 columns
    uint8_t dtype, out_dtype;
    // Neighbours in a row that lie on their common size everywhere, 8 (on 16 bytes), 2
    // or 1: of gradient and momentum, of the outputs.
    uint8_t vec, out_vec;
    uint32_t out;          // muon: index of its first pointer in MuonFinishParams::out
    float factor;          // muon: lr * the shape's factor
};

struct MuonPrepHead {
    int n;
    double* partial;
    uint32_t* counters;    // zeroed by the first pass
    float momentum;
    int nesterov;
    float eps;
    float scale;           // of the first X
};
template <int MATS>
struct MuonPrepParamsT : MuonPrepHead {
    MuonMat mat[MATS];
};
using MuonPrepParams = MuonPrepParamsT<kMuonMats>;

constexpr int kMuonPtrs = 1024, kMuonPtrsSmall = 128;  // outputs of a launch
struct MuonFinishHead {
    int n;
    int nranks;            // outputs per matrix
    float inv;             // 1 / the scale of X
    float keep;            // muon: 1 - lr * weight decay
};
template <int MATS, int PTRS>
struct MuonFinishParamsT : MuonFinishHead {
    MuonMat mat[MATS];
    void* out[PTRS];       // matrix-major
};
using MuonFinishParams = MuonFinishParamsT<kMuonMats, kMuonPtrs>;

// Matrices that one launch takes whole (rr_muon_small.cu): a cluster each.
constexpr uint32_t kMuonSmallSide = 128, kMuonSmallCtas = 8;
constexpr int kMuonMaxSteps = 50;

// A step's factors: A = gram P, B = poly_a A + poly A A, X = apply_x X + apply B X.
struct MuonSmallStep {
    float gram, poly, poly_a, apply, apply_x;
};

struct MuonSmallHead {
    int n;
    uint32_t ctas;           // per cluster: of the longest matrix
    int nranks;
    int steps, nesterov;
    float momentum, eps, keep;
    float scale, inv;        // of the first X; 1 / that of the last
    unsigned int* waits;     // bulk_wait_counters()
    uint32_t hold, spin;     // as in BulkParams
    MuonSmallStep step[kMuonMaxSteps];
};
template <int MATS, int PTRS>
struct MuonSmallParamsT : MuonSmallHead {
    MuonMat mat[MATS];       // x, part0, parts and tile0 unused
    void* out[PTRS];         // matrix-major
};
using MuonSmallParams = MuonSmallParamsT<kMuonMats, kMuonPtrs>;

cudaError_t launch_muon_squares(const MuonPrepParams& p, uint32_t parts, cudaStream_t s);
cudaError_t launch_muon_pack(const MuonPrepParams& p, uint32_t tiles, cudaStream_t s);
cudaError_t launch_muon_finish(const MuonFinishParams& p, uint32_t tiles, cudaStream_t s);
// The products of a group: tile_n, waits, hold and spin are filled in here.
cudaError_t launch_muon_gemm(MuonGemmParams& p, int nops, cudaStream_t s);

// waits, hold and spin are filled in here.
cudaError_t launch_muon_small(MuonSmallParams& p, cudaStream_t s);

}  // namespace rr
