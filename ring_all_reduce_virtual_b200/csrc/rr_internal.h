// rr_internal.h -- kernel parameter blocks and launchers shared between the
// host dispatcher (rr_api.cu) and the kernels (rr_kernels.cu, rr_bucket.cu).
// Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace rr {

constexpr int kMaxRanksH = 64;

// Rule-driven collectives over N rank buffers (one-shot all-reduce in ring
// or tree order, reduce-scatter, all-gather, all-to-all).
struct RankParams {
    const void* in[kMaxRanksH];
    void* out[kMaxRanksH];
    int n;          // ranks
    int vec_ok;     // all in[] agree modulo 16 bytes, and all out[] do
    float divisor;  // AVG's divisor (the rank count)
    int pad_;
    uint64_t C;     // chunk / part length in elements
    uint64_t count; // elements per rank buffer (all-reduce)
    uint64_t nseg;  // segments
    uint64_t tps;   // tiles per segment
    uint64_t lo;    // one-shot all-reduce: element range [lo, hi) of every
    uint64_t hi;    //   rank processed by this launch
    int owner_only; // one-shot all-reduce: write chunk c only to rank c (two-shot's first shot)
    int pad2_;
    unsigned int* waits;  // the bulk-copy kernels' wait counters on the launching device
                          // (bulk_wait_counters(); NULL keeps a call off those kernels)
};

// One segment of a table-driven step (a ring step, a tree level): fold
// in0 op in1 (in0 on the left) into out, or copy in0 into out when the step
// has one input.
struct StepSeg {
    const void* in0;
    const void* in1;
    void* out;
    uint64_t len;
};

struct StepParams {
    StepSeg seg[2 * kMaxRanksH];  // one per rank, or two (the double ring's two directions)
    int nseg;
    int nin;        // 2: fold, 1: copy
    int vec_ok;     // every segment's pointers agree modulo 16 bytes
    float divisor;  // AVG's divisor when this step finishes the fold
    uint64_t tps;
};

// The ring, double-ring and tree schedules in one launch.  The schedules'
// data dependencies run along (chunk, tile) chains: tile t of chunk k at
// ring step s reads only what step s-1 wrote to tile t of chunk k (on the
// previous rank), and a tree level reads only what the level below wrote to
// the same elements.  So one CTA carries its tile through every step, each
// thread on the same elements at every step (it reads what it wrote itself),
// and no CTA waits for another.
struct ChainParams {
    void* buf[kMaxRanksH];
    int n;
    int vec_ok;      // every buffer at the same 16-byte phase (required: the chains run the vector path)
    float divisor;   // AVG's divisor
    int nhalf;       // ring: 1 (the whole buffer, clockwise); double ring: 2 (half 1 counter-clockwise)
    uint64_t count;  // elements per rank
    uint64_t H;      // the double ring's first element of half 1 (count for the ring)
    uint64_t C[2];   // chunk size of each half
    uint64_t tps;    // tiles per chunk (ring) or per buffer (tree)
};

// Bucket launches: one launch covers up to kMaxBucketTensors tensors of one
// bucket and up to kMaxBucketPtrs gradient pointers (tensor-major: entry
// t * n + r is rank r's copy of the launch's t-th tensor).
constexpr int kMaxBucketPtrs = 2048;
constexpr int kMaxBucketTensors = 384;
constexpr int kMaxBucketSegs = kMaxBucketTensors + kMaxRanksH;

// Work items of the bucket kernels are numbered through per-segment prefix
// sums of their tile counts, so segments of very different lengths launch no
// empty CTAs: work item w belongs to the segment s with
// tile0[s] <= w < tile0[s + 1].
struct BucketCopyParams {
    const void* grad[kMaxBucketPtrs];      // pack: sources; unpack: destinations
    void* bucket[kMaxRanksH];              // fp32 bucket of each rank
    uint64_t toff[kMaxBucketTensors];      // element offset of tensor t in the bucket
    uint64_t tlen[kMaxBucketTensors];      // elements of tensor t
    uint64_t tile0[kMaxBucketTensors + 1]; // first work item of tensor t (n ranks x its tiles)
    int n;
    int nt;
    float divisor;
    int pad_;
};

// A fused bucket segment: elements [off, off + len) of launch tensor t, all
// in the bucket's chunk c (their fold starts on rank c).
struct BucketSeg {
    uint32_t t;
    uint32_t c;
    uint64_t off;
    uint64_t len;
};

struct BucketFoldParams {
    void* grad[kMaxBucketPtrs];
    BucketSeg seg[kMaxBucketSegs];
    uint64_t tile0[kMaxBucketSegs + 1];  // first work item (tile) of segment s
    int n;
    int nseg;
    int vec_ok;
    float divisor;
};

// Global norm and clipping (rr_clip.cu).  A launch of the norm covers up to
// CAP tensors of one type and writes one fp64 partial sum of squares per CTA;
// a small table keeps the parameter block of a short list small.
constexpr int kNormCtas = 592;        // CTAs of a norm launch: 4 on each of 148 SMs
constexpr int kNormTensors = 1024;    // tensors per launch
constexpr int kNormTensorsSmall = 160;  // a parameter block below 4 KB: larger ones cost the host 3-5 us per launch
template <int CAP>
struct NormParamsT {
    const void* ptr[CAP];
    uint64_t len[CAP];
    uint64_t tile0[CAP + 1];  // first work item (tile) of tensor t
    double* partial;          // this launch's slots, one per CTA
    float* clear;             // the launch zeroes this word (NULL: it does not); see ClipArgs::lost
    int nt;
    int pad_;
};
using NormParams = NormParamsT<kNormTensors>;

// What a launch that needs the norm reads: the partial sums of squares, and
// the clipping's arguments.
struct ClipArgs {
    const double* partial;
    int npartial;
    int in_l2;    // the set is small enough for L2 to hold much of it between the passes
    float max_norm;
    float eps;
    float* norm;  // where the launch writes the norm (NULL: it does not)
    // The norm's word in a call whose scaling waits for copies (NULL: none does).
    // A tile that a wait gave up on makes it NaN, before or after the norm is
    // written: a launch of the pass before zeroes it, and both go through
    // atomicMax, by whose order a NaN's bits are above every norm's.
    float* lost;
};

// The clipping's second pass: rank 0's copy of each tensor, scaled, into
// every rank's (entry t * n + r of ptr is rank r's copy of tensor t).
constexpr int kScaleTensors = 512;
constexpr int kScaleTensorsSmall = 64;
template <int CAP, int PTRS>
struct ScaleParamsT {
    void* ptr[PTRS];
    uint64_t len[CAP];
    uint64_t tile0[CAP + 1];
    uint8_t vec[CAP];  // every rank's copy of the tensor at one 16-byte phase
    ClipArgs clip;
    int n;
    int nt;
};
constexpr int kScalePtrs = 2048;
constexpr int kScalePtrsSmall = 256;
using ScaleParams = ScaleParamsT<kScaleTensors, kScalePtrs>;

// Embedding lookup and gradient (rr_embed.cu).  ids: int32 or int64 (ids64).
struct EmbedLookupParams {
    const void* ids[kMaxRanksH];
    const void* table[kMaxRanksH];
    void* out[kMaxRanksH];
    uint32_t T;     // tokens per rank
    uint32_t M;     // tokens of all ranks
    uint64_t V;     // table rows
    uint32_t D;     // row width
    int ids64;
    float scale;
};

struct EmbedGradParams {
    const void* ids[kMaxRanksH];
    const void* dout[kMaxRanksH];
    void* grad[kMaxRanksH];  // nout of them
    int64_t padding;         // this id adds nothing
    uint64_t V;
    uint32_t T, M, D;
    int ids64;
    int nout;
    int accumulate;
    float factor;            // scale, over the rank count for AVG
    // workspace
    uint32_t* key[2];        // sort buffers: token ids ...
    uint32_t* pos[2];        // ... and positions (rank * T + token)
    uint32_t* counts;        // per pass, tile and digit
    float* part;             // partial sums of runs that cross a block: [2][nblk][Dp]
    uint32_t* arrived;       // per slice: warps that have summed (few tokens)
    int passes, bits;        // of the sort: digits, and bits per digit
    uint32_t ntiles;
    uint32_t K, nblk, Dp;    // sorted positions per block, blocks, padded row width
};

// The clipped sync's first pass over a short range: BucketFoldParams with a
// parameter block below 4 KB.
constexpr int kParkPtrsSmall = 256;
constexpr int kParkSegsSmall = 48;
struct ParkSmallParams {
    void* grad[kParkPtrsSmall];
    BucketSeg seg[kParkSegsSmall];
    uint64_t tile0[kParkSegsSmall + 1];
    int n;
    int nseg;
    int vec_ok;
    float divisor;
};

enum DType : int { kF32 = 0, kBF16 = 1, kI32 = 2, kF16 = 3 };
enum Kind : int {
    kOneshotRing = 0,
    kOneshotTree = 1,
    kReduceScatter = 2,
    kAllGather = 3,
    kAllToAll = 4,
    kChunkBroadcast = 5  // chunk c of rank c copied to chunk c of every other rank
};

// Vectors per thread per tile: kernels that fold N inputs keep N loads per
// vector in flight and use few vectors; kernels with one or two inputs use
// more vectors to keep as many loads in flight.
constexpr int kVptReduce = 2;
constexpr int kVptMove = 4;

// Vectors per thread of the N-input folds (one-shot all-reduce, reduce-scatter,
// fused bucket sync, tree-order one-shot).  These kernels are also compiled for
// fixed rank counts (2, 3, 4, 8, 16; the bucket kernel 2, 4, 8): with the
// count known the compiler unrolls every rank loop, needs few registers and
// keeps N * 2 loads per thread in flight at high occupancy.  Other counts run
// a variant with a runtime rank count.
inline int reduce_vpt(int) { return kVptReduce; }

// Elements one fold tile covers (for sizing tiles per segment on the host),
// and one bucket pack/unpack tile.
uint64_t tile_elems(int dtype, int vpt);
uint64_t bucket_tile_elems(int grad_dtype);

// Launch configuration: one CTA per work item (a tile of a segment), up to
// the grid limit; kernels loop over the rest.
constexpr uint64_t kMaxGrid = 0x7fffffffull;

// Launchers: return the launch's cudaError_t.  `op` is an rr_op_t value.
cudaError_t launch_rank_kernel(int kind, int dtype, int op, const RankParams& p, cudaStream_t s);
cudaError_t launch_step(int dtype, int op, const StepParams& p, cudaStream_t s);
// The whole ring schedule (p.nhalf 1) or double ring (2) in one launch, and
// the whole tree schedule (reduce levels, then broadcast levels) in one launch;
// wire: the ring's bf16 wire format (fp32 buffers, SUM or AVG).
cudaError_t launch_ring_chain(int dtype, int op, bool wire, const ChainParams& p, cudaStream_t s);
uint64_t chain_tile_elems(int dtype);  // elements of one chain tile (ChainParams::tps counts these)
cudaError_t launch_tree_chain(int dtype, int op, const ChainParams& p, cudaStream_t s);
// bf16 wire (fp32 buffers, SUM or AVG): the fused one-shot, and a reduce-scatter
// step (wire 1: the step completes its chunks; 2: it does not).
cudaError_t launch_oneshot_wire(int op, const RankParams& p, uint64_t work, cudaStream_t s);
cudaError_t launch_step_wire(int op, int wire, const StepParams& p, cudaStream_t s);
// The bulk-copy kernels' two wait counters on the current device (tiles whose
// bounded wait ran out; of those, tiles whose copies were not seen to land),
// looked up once per device; NULL if the lookup fails.
unsigned int* bulk_wait_counters();
// Takes (reads and clears, atomically on the device) both counters of the
// current device.  Synchronous.
cudaError_t take_bulk_timeouts(unsigned int* ran_out, unsigned int* in_flight);
// cudaFuncGetAttributes(...).binaryVersion of one of the library's kernels.
cudaError_t kernel_binary_version(int* version);
cudaError_t launch_bucket_pack(int grad_dtype, const BucketCopyParams& p, cudaStream_t s);
cudaError_t launch_bucket_unpack(int grad_dtype, int op, const BucketCopyParams& p, cudaStream_t s);
// pdl: launch the bulk-copy sync as a programmatic dependent of the stream's
// previous kernel (its CTAs scheduled while a previous sync drains): for
// back-to-back syncs, not for syncs that run beside other work (the reducer),
// whose waiting CTAs would hold SMs that work could use.
cudaError_t launch_bucket_fold(int grad_dtype, int op, const BucketFoldParams& p, cudaStream_t s,
                               uint64_t max_grid = kMaxGrid, bool pdl = false);

// Global norm and clipping.  parked (16-bit types): the values are fp32 sums
// whose upper halves lie in rank 0's buffers and lower halves in rank 1's.
uint64_t norm_tile_elems(int dtype);
uint64_t scale_tile_elems(int dtype, bool parked, bool bulk);
cudaError_t launch_norm(int dtype, const NormParams& p, int* slots, cudaStream_t s);
cudaError_t launch_norm_join(const double* in, int64_t count, double* out, int* slots, cudaStream_t s);
cudaError_t launch_norm_finish(const ClipArgs& a, cudaStream_t s);
cudaError_t launch_clip_scale(int dtype, bool parked, bool bulk, const ScaleParams& p, cudaStream_t s);
// Bytes written from which the scaling runs by bulk copies, against by the
// threads: 4 x 64 MB 60.4 and 68.9 us, 4 x 32 MB 31.2 and 33.7, 4 x 16 MB 20.0 and
// 20.4, 1 x 32 MB 18.1 and 18.3, 1 x 16 MB 13.6 and 12.5 (its CTAs are short, and
// each sums the partials).
constexpr uint64_t kBulkClipBytes = 64ull << 20;
// One rank's bytes up to which the scaling stores with an evict-first hint, so
// that the values the norm left in L2 are read there: 4 x 104 MB 104.6 -> 99.9
// us; above L2's 126 MB the hint costs (8 x 666 MB: 1773 -> 1794).
constexpr uint64_t kKeepBytes = 126ull << 20;
constexpr int kJoinCtas = 128;        // partials that launch_norm_join leaves
constexpr int kMaxPartials = 1280;    // partials that a launch sums itself
// The clipped sync's first pass: fold, park the sums, one partial per tile;
// clear (or NULL): a word that the launch zeroes (ClipArgs::lost).
uint64_t park_tile_elems(int grad_dtype, int n);
cudaError_t launch_bucket_park(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, double* partial,
                               float* clear, cudaStream_t s);
// Norm (scale false) or clipping of a small set in one launch: whether it is
// one (the tensors' prefix sums are filled in), and the launch.
bool clip_small_plan(int dtype, ParkSmallParams& p, int ntensors);
cudaError_t launch_clip_small(int dtype, bool scale, const ParkSmallParams& f, const ClipArgs& clip, cudaStream_t s);
// The other way: a first pass that only sums the squares, and a second that
// folds again and writes the scaled values to every rank; which one a call
// takes.
bool clip_folds_twice(int n, int grad_dtype);
cudaError_t launch_bucket_squares(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, double* partial,
                                  float* clear, cudaStream_t s);
cudaError_t launch_bucket_scaled(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, const ClipArgs& clip,
                                 cudaStream_t s);

// Embedding.  vec: elements per access, which divides the row width and
// suits every address; out_dtype: the gradient's type, dtype or fp32.
cudaError_t launch_embed_lookup(int dtype, int vec, const EmbedLookupParams& p, cudaStream_t s);
cudaError_t launch_embed_sort(const EmbedGradParams& p, int* launches, cudaStream_t s);
cudaError_t launch_embed_reduce(int dtype, int out_dtype, int vec, const EmbedGradParams& p, int* launches,
                                cudaStream_t s);
// Keys per CTA of a sort pass: 65536 tokens' gradient 109.7 / 104.6 / 105.4 us with
// 2048 / 1024 / 512, 16384 tokens' 196.9 / 191.5 / 188.5 (more tiles spread a pass
// over more SMs; each CTA reads every tile's counts, so many tokens want few).
constexpr uint32_t kSortTile = 1024;
constexpr int kSortMaxBits = 9;        // bits per digit, at most
// Tokens that are sorted by counting smaller ids, in one launch: against the
// radix sort's three, 1024 tokens' gradient 16.4 and 21.1 us, 2048 tokens' 21.1
// and 22.9, 3000 tokens' 27.4 and 25.9.
constexpr uint32_t kRankMax = 2048;
// Tiles from which a sort pass scans its counts in a launch of its own instead
// of every CTA summing all of them, which grows with the square of the tiles:
// at 512 tiles 152 us for the call against 266.
constexpr uint32_t kScanTiles = 1024;
// Blocks up to which an adding call's sums join their cut runs themselves: 300
// tokens of width 515, call after call, 16.8 us in three launches and 14.8 in two (a
// run over all 64 is then one warp's 16 rounds of loads per slice).
constexpr uint32_t kJoinHere = 64;
constexpr uint32_t kEmbedCols = 256;   // columns of a warp's slice of a row

}  // namespace rr

namespace rr {
// Kernel parameter blocks must fit the 32,764-byte kernel parameter limit.
static_assert(sizeof(RankParams) <= 32764, "RankParams too large");
static_assert(sizeof(StepParams) <= 32764, "StepParams too large");
static_assert(sizeof(ChainParams) <= 32764, "ChainParams too large");
static_assert(sizeof(BucketCopyParams) <= 32764, "BucketCopyParams too large");
static_assert(sizeof(BucketFoldParams) <= 32764, "BucketFoldParams too large");
static_assert(sizeof(NormParams) <= 32764, "NormParams too large");
static_assert(sizeof(ScaleParams) <= 32764, "ScaleParams too large");
}  // namespace rr
