// rr_muon_gemm.cu -- the products of the Newton-Schulz iteration on the fifth
// generation tensor cores: all steps of a group of matrices in one launch
// (rr_muon.h), for operands and results held as two fp16 halves.  A product of
// two such values is three products of halves, lo hi + hi lo + hi hi (lo lo is
// below 2^-22), in one fp32 accumulator.
//
// Two CTAs on neighbouring SMs share a tile of 256 x 256 (or 256 x 128): each
// copies its 128 rows of A and its half of B's (cp.async.bulk, both halves of 64
// of K a stage, 64 KB, three stages), and the first one's instructions multiply
// out of both: 196 operations a byte from L2, against 85 of one CTA's tile of
// 128 x 256 with K gone through three times.  Of a CTA's warps two copy, one
// issues the products (in the second CTA: tells the first that a stage has
// landed), eight take accumulators out of tensor memory.
//
// The tensor cores' sums are cut off, not rounded: a long one comes out low by
// 2^-25 and more a term (a sum of 8192 positive products by 1.5e-5).  So an
// accumulator collects a few stages only (MuonOp::chunk); the eight warps add it to sums in
// their registers, rounded to nearest, while the other accumulator fills.
//
// A pair takes the next tile of the list from a counter, and begins it once its
// matrix's earlier levels are finished, which another counter says.  A tile
// waits only for tiles before it in the list, which are then in the hands of
// pairs that run, so the waits end whatever the number of pairs that run at a
// time.  Against a launch per level, SMs do not idle at the end of each level
// while another matrix has work, and a level of a small matrix does not cost a
// launch.
//
// Results leave through shared memory, 4 KB a warp: a thread has a row of the
// tile, whose 16-byte pieces lie 128 bytes from the next row's; written to L2
// from there they took the warps longer than the products took.
//
// Every wait is bounded (rr_bulk.cuh): one that runs out is counted, the CTA's
// warps stop, wait (bounded) for copies and products in flight, give their
// tensor memory back and leave; what the call writes is then undefined.
#include <algorithm>
#include <cstddef>

#include <cuda_fp16.h>

#include "rr_bulk.cuh"
#include "rr_launch.cuh"
#include "rr_muon.h"
#include "rr_muon_device.cuh"

namespace rr {

namespace {

constexpr int kMaxStages = 4;
constexpr uint32_t kPairs = 74;                // pairs of SMs
constexpr uint32_t kTileN = 256;
constexpr uint32_t kPlane = 128 * kBlk * 2;    // one half of 128 rows (or columns) of an operand's stage
// A's hi and lo, B's hi and lo: three stages where tiles may have 256 columns, four
// where all have 128 -- a stage's way round (copies from L2, the other CTA's word,
// products, the word back) takes 2.3 us, which the products of 128 columns do not
// fill otherwise.
template <bool WIDE>
struct Ring {
    static constexpr int kStages = WIDE ? 3 : 4;
    static constexpr uint32_t kPlaneB = WIDE ? kPlane : kPlane / 2;
    static constexpr uint32_t kBytes = 2 * kPlane + 2 * kPlaneB;
};
constexpr uint32_t kRingBytes = 3 * 4 * kPlane;
static_assert(Ring<true>::kStages * Ring<true>::kBytes == kRingBytes && Ring<false>::kStages * Ring<false>::kBytes == kRingBytes);
constexpr int kTakers = 8;                     // warps that take accumulators out
constexpr int kGemmThreads = 128 + 32 * kTakers;
// Registers a thread: 168 at the launch (65536 over 384 threads), of which the
// first four warps give 112 back and the takers have 56 more: their sums are
// 128.  128 x 56 + 256 x 224 = 384 x 168.
constexpr int kFewRegs = 56, kManyRegs = 224;
static_assert(128 * kFewRegs + 32 * kTakers * kManyRegs <= 168 * kGemmThreads, "more than the launch has");
constexpr uint32_t kOutBytes = 32 * kBlk * 2;  // a warp's 32 rows of a block
constexpr int kSlots = 4;                      // tiles handed on to the CTA's other warps
constexpr uint32_t kSmem = kRingBytes + kTakers * kOutBytes + 1024 + 512;  // from a 1024-byte boundary; the rest
constexpr uint32_t kEnd = 0xffffffffu;
constexpr uint32_t kFull = 0xffffffffu;

struct Slot {
    uint32_t seq;   // in the list of products; kEnd: no more tiles
    uint32_t i, j;  // the tile: 256 rows, tile_n columns
    uint32_t mat;
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];  // of a stage: its copies have landed; its products are done
    uint64_t other[kMaxStages];                // first CTA: the second's copies have landed
    uint64_t ready[2], taken[2];             // of an accumulator: finished; read out by both CTAs (in the first)
    uint64_t told[kSlots], heard[kSlots];    // of a slot: filled; read by all of both CTAs (in the first)
    uint64_t drained;
    alignas(16) Slot slot[kSlots];
    uint32_t tmem;
    uint32_t stop;
    uint32_t begun_b;                        // stages that copies of B were begun for
};
static_assert(sizeof(Bars) <= 512 && offsetof(Bars, slot) % 16 == 0, "kSmem counts 512 bytes; slots are written whole");
// Who reads a slot: the first CTA's copies of B, products and takers, the second's copies, messages and takers.
constexpr uint32_t kHearers = 2 + kTakers + 3 + kTakers;

// ---------------------------------------------------------------- barriers

__device__ __forceinline__ void give_up(Bars* b, unsigned int* waits)
{
    if (atomicExch(&b->stop, 1u) == 0) atomicAdd(&waits[0], 1u);
}

// Bounded; false as well once another warp of the CTA has given up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Bars* b, unsigned int* waits, uint32_t spin)
{
    const uint32_t at = muon_smem(bar);
    for (uint32_t i = 0; i < spin; ++i) {
        if (muon_try_wait(at, parity)) return true;
        if (*(volatile uint32_t*)&b->stop) return false;
    }
    give_up(b, waits);
    return false;
}

// The same for a whole warp, one lane of which looks.  (A shuffle orders no memory:
// what the others read or copy next is ordered by a warp's barrier or an instruction
// of the whole warp behind this.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars* b, unsigned int* waits, uint32_t spin)
{
    uint32_t ok = 0;
    if ((threadIdx.x & 31) == 0) ok = wait_for(bar, parity, b, waits, spin);
    return __shfl_sync(kFull, ok, 0) != 0;
}

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(muon_smem(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(muon_smem(bar)) : "memory");
}

// An arrival on the first CTA's barrier, from either CTA.
__device__ __forceinline__ void first_arrive(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .b32 at;\n\tmapa.shared::cluster.u32 at, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [at];\n\t}" ::"r"(muon_smem(bar))
        : "memory");
}

__device__ __forceinline__ void copy_block(uint32_t to, const uint16_t* from, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(muon_smem(bar))
                 : "memory");
}

// ------------------------------------------------------------------- tiles

// A buffer of a matrix, and its columns of blocks.
__device__ __forceinline__ Halves buffer_of(const MuonWork& w, uint32_t id, uint32_t* nbj)
{
    const uint32_t m = pad_up(min(w.rows, w.cols));
    if (id < kSquares) {
        *nbj = pad_up(w.cols) / kBlk;
        return {w.x[id], w.x[id] + (uint64_t)pad_up(w.rows) * pad_up(w.cols)};
    }
    *nbj = m / kBlk;
    const uint64_t half = (uint64_t)m * m;
    uint16_t* hi = w.squares + (id - kSquares) * 2 * half;
    return {hi, hi + half};
}

// Blocks along K.
__device__ __forceinline__ uint32_t depth_of(const MuonWork& w, int kind)
{
    const uint32_t k = kind == kGram ? max(w.rows, w.cols) : min(w.rows, w.cols);
    return (k + kBlk - 1) / kBlk;
}

// Tile t of a product.
__device__ __forceinline__ void place_of(const MuonWork& w, int kind, uint32_t tile_n, uint32_t t, uint32_t* i, uint32_t* j)
{
    const MuonSides s = muon_sides(w.rows, w.cols, kind);
    if (kind == kApply) {
        const uint32_t r = (s.mt + 1) / 2;
        *i = t % r;
        *j = t / r;
        return;
    }
    uint32_t row = 0;
    for (uint32_t n; t >= (n = muon_sym_tiles(row, s.nu, tile_n / 128)); ++row) t -= n;
    *i = row;
    *j = t;
}

// What every warp knows of its tile.
struct Tile {
    const MuonWork* w;
    const MuonOp* op;
    uint32_t i, j, per, units, mt, kb, chunk, mat;  // per: units of 128 columns of a whole tile
};

template <class P>
__device__ __forceinline__ Tile tile_at(const P& p, const Slot& s)
{
    Tile t;
    t.mat = s.mat;
    t.w = &p.work[s.mat];
    t.op = &p.op[t.w->op0 + (p.seq[s.seq] >> 16)];
    const MuonSides sides = muon_sides(t.w->rows, t.w->cols, t.op->kind);
    t.i = s.i;
    t.j = s.j;
    t.per = p.tile_n[t.op->kind] / 128;
    t.units = min(t.per, sides.nu - s.j * t.per);
    t.mt = sides.mt;
    t.kb = depth_of(*t.w, t.op->kind);
    t.chunk = t.op->chunk;
    return t;
}

// Tiles of product k of the list, of one matrix.
template <class P>
__device__ __forceinline__ uint32_t tiles_of(const P& p, uint32_t k)
{
    const uint32_t e = p.seq[k];
    const MuonWork& w = p.work[e & 255u];
    const int kind = p.op[w.op0 + (e >> 16)].kind;
    return muon_tiles(w.rows, w.cols, kind, p.tile_n[kind]);
}

// What the matrix's counter shows when the levels before op's are finished:
// every taker of both CTAs counts each tile.
template <class P>
__device__ __forceinline__ uint32_t parts_before(const P& p, const Tile& t)
{
    uint32_t tiles[3], sum = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) tiles[k] = muon_tiles(t.w->rows, t.w->cols, k, p.tile_n[k]);
    for (uint32_t o = 0; o < t.w->ops; ++o) {
        const MuonOp& op = p.op[t.w->op0 + o];
        if (op.level >= t.op->level) break;
        sum += op.kind == kGram ? tiles[kGram] : op.kind == kSquare ? tiles[kSquare] : tiles[kApply];
    }
    return sum * 2 * kTakers;
}

__device__ __forceinline__ bool parts_done(const uint32_t* counter, uint32_t need, Bars* b, unsigned int* waits, uint32_t spin)
{
    for (uint32_t i = 0; i < spin; ++i) {
        uint32_t have;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(have) : "l"(counter) : "memory");
        if (have >= need) return true;
        if (*(volatile uint32_t*)&b->stop) return false;
    }
    give_up(b, waits);
    return false;
}

// A tile into both CTAs' slot.
__device__ __forceinline__ void tell(const Slot& s, uint32_t n, Bars* b)
{
    const uint32_t k = n % kSlots, at = muon_smem(&b->slot[k]), bar = muon_smem(&b->told[k]);
    asm volatile(
        "{\n\t.reg .b32 a, r;\n\t"
        "st.shared.v4.b32 [%0], {%2, %3, %4, %5};\n\t"
        "mapa.shared::cluster.u32 r, %1, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t"
        "mapa.shared::cluster.u32 a, %0, 1;\n\t"
        "st.shared::cluster.v4.b32 [a], {%2, %3, %4, %5};\n\t"
        "mapa.shared::cluster.u32 r, %1, 1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(at),
        "r"(bar), "r"(s.seq), "r"(s.i), "r"(s.j), "r"(s.mat)
        : "memory");
}

// The next tile as it was told, for one thread; it says that it has read it.
__device__ __forceinline__ bool hear(Slot& s, uint32_t n, Bars* b, unsigned int* waits, uint32_t spin)
{
    const uint32_t k = n % kSlots;
    s.seq = kEnd;
    s.i = s.j = s.mat = 0;
    if (!wait_for(&b->told[k], (n / kSlots) & 1, b, waits, spin)) return false;
    volatile Slot* v = &b->slot[k];
    s.seq = v->seq;
    s.i = v->i;
    s.j = v->j;
    s.mat = v->mat;
    first_arrive(&b->heard[k]);
    return s.seq != kEnd;
}

__device__ __forceinline__ void share(Slot& s)
{
    s.seq = __shfl_sync(kFull, s.seq, 0);
    s.i = __shfl_sync(kFull, s.i, 0);
    s.j = __shfl_sync(kFull, s.j, 0);
    s.mat = __shfl_sync(kFull, s.mat, 0);
}

// The same for a whole warp.
__device__ __forceinline__ bool warp_hear(Slot& s, uint32_t n, Bars* b, unsigned int* waits, uint32_t spin)
{
    if ((threadIdx.x & 31) == 0) hear(s, n, b, waits, spin);
    share(s);
    return s.seq != kEnd;
}

// ---------------------------------------------------------------- products

// An arrival on the barrier of both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     muon_smem(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

// ----------------------------------------------------------------- results

// A taker's 4 KB of shared memory, 32 rows of one half of a block, in which a
// lane has its row's pieces and the warp moves whole lines.
struct OutRows {
    uint8_t* mem;

    __device__ __forceinline__ uint4* piece(int lane, int g) const
    {
        return reinterpret_cast<uint4*>(mem + lane * (kBlk * 2) + ((g ^ (lane & 7)) << 4));
    }
    __device__ __forceinline__ uint4* line(int lane, int g) const { return reinterpret_cast<uint4*>(mem) + g * 32 + lane; }
};

__device__ __forceinline__ void fetch(uint4 (&r)[8], const uint16_t* from, int lane)
{
#pragma unroll
    for (int g = 0; g < 8; ++g) r[g] = __ldcg(reinterpret_cast<const uint4*>(from) + g * 32 + lane);
}

// 64 columns of this thread's row of the sums: v[l] is column col + l.  The
// warp's part of the blocks begins at c and out.
struct Factors {
    float alpha, beta, diag;
};

__device__ __forceinline__ void put_block(float (&v)[64], const Factors& f, const Halves& c, const Halves& out, uint32_t row,
                                          uint32_t col, uint32_t side, const OutRows& o, int lane)
{
#pragma unroll
    for (int l = 0; l < 64; ++l) v[l] *= f.alpha;
    if (c.hi) {
        uint4 r[8];
        fetch(r, c.hi, lane);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int g = 0; g < 8; ++g) *o.line(lane, g) = r[g];
            __syncwarp();
            if (half == 0) fetch(r, c.lo, lane);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                float a[8];
                F16T::unpack(*o.piece(lane, g), a);
#pragma unroll
                for (int l = 0; l < 8; ++l) v[g * 8 + l] = __fmaf_rn(f.beta, a[l], v[g * 8 + l]);
            }
            __syncwarp();
        }
    }
    if (f.diag != 0.0f && row < side && row / 64 == col / 64) {
#pragma unroll
        for (int l = 0; l < 64; ++l)
            if (col + l == row) v[l] += f.diag;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            float a[8];
#pragma unroll
            for (int l = 0; l < 8; ++l) a[l] = v[g * 8 + l];
            const uint4 w = F16T::pack(a);
            *o.piece(lane, g) = w;
            if (half == 0) {  // what is left
                float r[8];
                F16T::unpack(w, r);
#pragma unroll
                for (int l = 0; l < 8; ++l) v[g * 8 + l] = a[l] - r[l];
            }
        }
        __syncwarp();
        uint4* to = reinterpret_cast<uint4*>(half ? out.lo : out.hi);
#pragma unroll
        for (int g = 0; g < 8; ++g) __stcg(to + g * 32 + lane, *o.line(lane, g));
        __syncwarp();
    }
}

// ------------------------------------------------------------- the warps

// The first CTA's lane that takes tiles off the list: the next one's number, and
// where in the list it is.
template <class P>
struct Source {
    uint32_t next, at_seq = 0, at_tile = 0, each;  // each: tiles of one matrix of at_seq's

    __device__ __forceinline__ Source() : next(0), each(0) {}
    __device__ __forceinline__ explicit Source(const P& p) : next(atomicAdd(p.counters, 1u)), each(tiles_of(p, 0)) {}

    // The n-th tile of the pair, told to all that wait for it.
    __device__ __forceinline__ void take(const P& p, Slot& s, uint32_t n, Bars* b)
    {
        for (uint32_t all; at_seq < p.nseq && next - at_tile >= (all = each * (p.seq[at_seq] >> 8 & 255u));) {
            at_tile += all;
            if (++at_seq < p.nseq) each = tiles_of(p, at_seq);
        }
        if (at_seq < p.nseq) {
            const uint32_t e = p.seq[at_seq], t = next - at_tile;
            s.seq = at_seq;
            s.mat = (e & 255u) + t / each;
            const MuonWork& w = p.work[s.mat];
            const int kind = p.op[w.op0 + (e >> 16)].kind;
            place_of(w, kind, p.tile_n[kind], t % each, &s.i, &s.j);
        }
        if (n < kSlots || wait_for(&b->heard[n % kSlots], ((n / kSlots) - 1) & 1, b, p.waits, p.spin)) {
            tell(s, n, b);
            if (s.seq != kEnd) next = atomicAdd(p.counters, 1u);  // on its way while this tile is copied
        } else {
            s.seq = kEnd;
        }
    }
};

// Copies of A's stages (IS_B 0) or B's by a warp: four blocks of 8 KB by a lane
// each, the pairs that follow one another in memory as one copy of 16 KB.  A
// copy takes its warp about 100 clocks to issue, so that one warp's four or
// eight a stage took longer than the products of a tile of 128 columns.
// Returns the stages begun.
template <bool IS_B, bool WIDE, class P>
__device__ __forceinline__ uint32_t copy_tiles(const P& p, Bars* b, uint32_t ops, uint32_t rank, int lane)
{
    const uint32_t half = lane & 1, second = lane >> 1 & 1;  // of the pair; the low halves
    const bool source = !IS_B && rank == 0;
    uint32_t it = 0;
    Source<P> from = source && lane == 0 ? Source<P>(p) : Source<P>();
    uint32_t last = kEnd, of = 0;  // the product and the matrix whose earlier levels are known to be finished
    for (uint32_t n = 0;; ++n) {
        Slot s{kEnd, 0, 0, 0};
        if (source) {
            if (lane == 0) from.take(p, s, n, b);
            share(s);
            if (s.seq == kEnd) return it;
        } else if (!warp_hear(s, n, b, p.waits, p.spin)) {
            return it;
        }
        const Tile t = tile_at(p, s);
        const bool wide = t.w->rows <= t.w->cols;
        const int kind = t.op->kind;
        const bool rows = 2 * t.i + rank < t.mt;  // else this CTA's part of the products is of no use
        // kApply: Q X, or X Q
        const uint32_t id = kind == kApply ? (IS_B == wide ? t.op->b : t.op->a) : IS_B ? t.op->b : t.op->a;
        uint32_t nbj;
        const Halves op = buffer_of(*t.w, id, &nbj);
        const bool low = id >= kSquares;
        const bool mn = !low && (kind == kGram ? !wide : wide);
        // the first of this CTA's blocks along M or N, and how many there are
        const uint32_t at = IS_B ? t.j * t.per * 2 + t.units * rank : 2 * (2 * t.i + rank);
        const uint32_t blocks = IS_B ? t.units : rows ? 2 : 0;
        const uint16_t* src = second ? op.lo : op.hi;
        const uint16_t* by_row = src + block_at(at + half, 0, nbj);  // + k * 2 blocks
        const uint16_t* by_col = src + block_at(0, at + half, nbj);  // + k / 2 * 2 nbj blocks + k % 2
        const uint32_t to = ops + (IS_B ? 2 * kPlane + second * Ring<WIDE>::kPlaneB : second * kPlane) + half * (kPlane / 2);
        const uint32_t kb = t.kb, limit = low ? (at >> 2) * 4 + 4 : mn ? 0 : kb;  // K's blocks that lie by rows
        const uint64_t pair = (uint64_t)nbj * 2 * kBlkElems;
        if (s.seq != last || s.mat != of) {  // what the operands come from is finished
            uint32_t fine = 1;
            if (lane == 0 && t.op->level > 0) fine = parts_done(p.counters + 1 + t.mat, parts_before(p, t), b, p.waits, p.spin);
            __syncwarp();  // the lanes that copy are behind the one that looked
            if (!__shfl_sync(kFull, fine, 0)) return it;
            last = s.seq;
            of = s.mat;
            asm volatile("fence.proxy.async;" ::: "memory");  // it was written by ordinary stores
        }
        for (uint32_t k = 0; k < kb; ++k, ++it) {
            constexpr int kStages = Ring<WIDE>::kStages;
            const uint32_t st = it % kStages, use = it / kStages;
            if (use > 0 && !warp_wait(&b->empty[st], (use - 1) & 1, b, p.waits, p.spin)) return it;
            uint64_t* full = &b->full[st];
            if (lane == 0)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(muon_smem(full)), "r"(blocks * kPlane) : "memory");
            __syncwarp();
            const bool whole = k < limit && blocks == 2;  // both blocks, one after the other
            if (lane < 4 && half < (whole ? 1 : blocks))
                copy_block(to + st * Ring<WIDE>::kBytes,
                           k < limit ? by_row + (uint64_t)k * 2 * kBlkElems : by_col + (k >> 1) * pair + (k & 1) * kBlkElems,
                           whole ? kPlane : kPlane / 2, full);
        }
    }
}

// The second CTA, one thread: the first one learns of its copies.
template <bool WIDE, class P>
__device__ __forceinline__ void report_copies(const P& p, Bars* b)
{
    constexpr int kStages = Ring<WIDE>::kStages;
    uint32_t stages = 0;
    Slot slot;
    for (uint32_t n = 0; hear(slot, n, b, p.waits, p.spin); ++n) {
        const uint32_t kb = tile_at(p, slot).kb;
        for (uint32_t k = 0; k < kb; ++k, ++stages) {
            const uint32_t s = stages % kStages;
            if (!wait_for(&b->full[s], (stages / kStages) & 1, b, p.waits, p.spin)) return;
            first_arrive(&b->other[s]);
        }
    }
}

// The first CTA, one thread: the products of both.
template <bool WIDE, class P>
__device__ __forceinline__ void multiply(const P& p, Bars* b, uint32_t ops, uint32_t tmem)
{
    constexpr int kStages = Ring<WIDE>::kStages;
    constexpr uint32_t kPlaneB = Ring<WIDE>::kPlaneB;
    uint32_t stages = 0, sums = 0;
    Slot slot;
    for (uint32_t n = 0; hear(slot, n, b, p.waits, p.spin); ++n) {
        const Tile t = tile_at(p, slot);
        const bool wide = t.w->rows <= t.w->cols;
        const int kind = t.op->kind;
        // K's blocks that lie by rows; both CTAs' blocks lie in one tile of 256
        const uint32_t kb = t.kb, n128 = t.units * 128;
        const uint32_t low_a = t.i * 4 + 4, low_b = (t.j * t.per / 2) * 4 + 4;
        const uint32_t a_rows = kind == kSquare || (kind == kApply && wide) ? low_a : kind == kGram && !wide ? 0 : kb;
        const uint32_t b_rows = kind == kSquare || (kind == kApply && !wide) ? low_b : kind == kGram && wide ? kb : 0;
        for (uint32_t k0 = 0; k0 < kb; k0 += t.chunk, ++sums) {
            const uint32_t acc = tmem + (sums & 1) * kTileN, k1 = min(kb, k0 + t.chunk);
            if (sums >= 2 && !wait_for(&b->taken[sums & 1], ((sums >> 1) - 1) & 1, b, p.waits, p.spin)) return;
            for (uint32_t k = k0; k < k1; ++k, ++stages) {
                const uint32_t s = stages % kStages, parity = (stages / kStages) & 1;
                if (!wait_for(&b->full[s], parity, b, p.waits, p.spin)) return;
                if (!wait_for(&b->other[s], parity, b, p.waits, p.spin)) return;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sa = ops + s * Ring<WIDE>::kBytes;
                const bool a_mn = k >= a_rows, b_mn = k >= b_rows;
                const uint32_t inst = muon_instruction(256, n128, a_mn, b_mn);
                const uint32_t astep = (a_mn ? 2048u : 32u) >> 4, bstep = (b_mn ? 2048u : 32u) >> 4;  // 16 of K
                const uint64_t ah = muon_operand(sa, a_mn, 8192), al = muon_operand(sa + kPlane, a_mn, 8192);
                const uint64_t bh = muon_operand(sa + 2 * kPlane, b_mn, 8192), bl = muon_operand(sa + 2 * kPlane + kPlaneB, b_mn, 8192);
#pragma unroll
                for (uint32_t c = 0; c < kBlk / 16; ++c) muon_mma<2>(acc, al + c * astep, bh + c * bstep, inst, k > k0 || c > 0);
#pragma unroll
                for (uint32_t c = 0; c < kBlk / 16; ++c) muon_mma<2>(acc, ah + c * astep, bl + c * bstep, inst, true);
#pragma unroll
                for (uint32_t c = 0; c < kBlk / 16; ++c) muon_mma<2>(acc, ah + c * astep, bh + c * bstep, inst, true);
                commit(&b->empty[s]);
            }
            commit(&b->ready[sums & 1]);
        }
    }
}

// One tile's results: a warp reads the quarter of the accumulator's rows that is
// its own, and COLS columns, half of them.  False: a wait ran out.
template <int COLS, class P>
__device__ __forceinline__ bool take_tile(const P& p, Bars* b, uint32_t tmem, const OutRows& o, uint32_t rank, int warp, int lane,
                                          const Tile& t, uint32_t& sums)
{
    const uint32_t quarter = warp & 3, col0 = ((warp - 4) >> 2) * COLS;
    const uint32_t unit = 2 * t.i + rank;  // of 128 rows
    const uint32_t row0 = unit * 128 + quarter * 32, col = t.j * t.per * 128 + col0;
    const bool mine = unit < t.mt;
    // where the results go and what of, looked up while the products run
    uint32_t nbj;
    Halves out = buffer_of(*t.w, t.op->out, &nbj), c{nullptr, nullptr};
    const uint64_t at = block_at(row0 / kBlk, col / kBlk, nbj) + row0 % kBlk * kBlk;
    out = {out.hi + at, out.lo + at};
    if (t.op->c != kNoBuffer) {
        c = buffer_of(*t.w, t.op->c, &nbj);  // of out's shape
        c = {c.hi + at, c.lo + at};
    }
    const uint32_t side = min(t.w->rows, t.w->cols);
    const Factors f{t.op->alpha, t.op->beta, t.op->diag};
    float sum[COLS];
#pragma unroll
    for (int l = 0; l < COLS; ++l) sum[l] = 0.0f;
    for (uint32_t k0 = 0; k0 < t.kb; k0 += t.chunk, ++sums) {
        if (!warp_wait(&b->ready[sums & 1], (sums >> 1) & 1, b, p.waits, p.spin)) return false;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t acc = tmem + (quarter * 32 << 16) + (sums & 1) * kTileN + col0;
        constexpr int kAtOnce = COLS == 64 ? 2 : 1;  // as the registers allow
#pragma unroll
        for (int h = 0; h < COLS / 32; h += kAtOnce) {
            uint32_t bits[kAtOnce][32];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) muon_load_acc(acc + (h + u) * 32, bits[u]);
            muon_acc_landed();
#pragma unroll
            for (int l = 0; l < 32 * kAtOnce; ++l) sum[h * 32 + l] += __uint_as_float(bits[l / 32][l % 32]);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) first_arrive(&b->taken[sums & 1]);
    }
    if (mine) {
#pragma unroll
        for (int h = 0; h < COLS / 64; ++h) {
            float v[64];
#pragma unroll
            for (int l = 0; l < 64; ++l) v[l] = sum[h * 64 + l];
            constexpr uint64_t next = 2 * kBlkElems;  // the block beside it
            put_block(v, f, {c.hi ? c.hi + h * next : nullptr, c.lo + h * next}, {out.hi + h * next, out.lo + h * next}, row0 + lane,
                      col + h * 64, side, o, lane);
        }
    }
    return true;
}

template <bool WIDE, class P>
__device__ __forceinline__ void take_tiles(const P& p, Bars* b, uint32_t tmem, const OutRows& o, uint32_t rank, int warp, int lane)
{
    uint32_t sums = 0;
    Slot slot;
    for (uint32_t n = 0; warp_hear(slot, n, b, p.waits, p.spin); ++n) {
        const Tile t = tile_at(p, slot);
        if (!(WIDE && t.units == 2 ? take_tile<WIDE ? 128 : 64>(p, b, tmem, o, rank, warp, lane, t, sums)
                                   : take_tile<64>(p, b, tmem, o, rank, warp, lane, t, sums)))
            return;
        __syncwarp();
        if (lane == 0)  // this part is there, of every lane's stores
            asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.counters + 1 + t.mat) : "memory");
    }
}

template <bool WIDE, class P>
__global__ void __launch_bounds__(kGemmThreads, 1) muon_gemm_kernel(const __grid_constant__ P p)
{
    extern __shared__ uint8_t raw_smem[];
    uint8_t* base = raw_smem + ((1024u - (muon_smem(raw_smem) & 1023u)) & 1023u);
    uint8_t* out_rows = base + kRingBytes;
    Bars* b = reinterpret_cast<Bars*>(out_rows + kTakers * kOutBytes);
    const uint32_t ops = muon_smem(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;  // in its pair
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            bar_init(&b->full[s], 2 + p.hold);
            bar_init(&b->empty[s], 1);
            bar_init(&b->other[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(&b->ready[s], 1);
            bar_init(&b->taken[s], 2 * kTakers);
        }
        for (int s = 0; s < kSlots; ++s) {
            bar_init(&b->told[s], 1);
            bar_init(&b->heard[s], kHearers);
        }
        bar_init(&b->drained, 1);
        b->stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(muon_smem(&b->tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    cluster_arrive();
    cluster_wait();  // both CTAs' barriers are set up
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = b->tmem;
    pdl_begin();

    uint32_t begun = 0;  // stages, of a copying warp
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0) {
            begun = copy_tiles<false, WIDE>(p, b, ops, rank, lane);
            __syncwarp();
        } else if (warp == 2) {
            begun = copy_tiles<true, WIDE>(p, b, ops, rank, lane);
            if (lane == 0) b->begun_b = begun;
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0) {
                if (rank != 0) report_copies<WIDE>(p, b);
                else multiply<WIDE>(p, b, ops, tmem);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        take_tiles<WIDE>(p, b, tmem, OutRows{out_rows + (warp - 4) * kOutBytes}, rank, warp, lane);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (b->stop) {  // a wait ran out: what is in flight ends before the CTA's memory goes
        if (threadIdx.x == 0) {
            constexpr int kStages = Ring<WIDE>::kStages;
            const uint32_t least = min(begun, b->begun_b);
            begun = max(begun, b->begun_b);
            for (uint32_t k = least; k < begun; ++k) bar_arrive(&b->full[k % kStages]);  // for the warp that got less far
            if (p.hold)
                for (uint32_t k = 0; k < kStages && k < begun; ++k) bar_arrive(&b->full[k]);
            for (uint32_t back = 1; back <= kStages && back <= begun; ++back) {
                const uint32_t last = begun - back;
                bool landed = false;
                for (uint32_t i = 0; i < p.spin && !landed; ++i)
                    landed = muon_try_wait(muon_smem(&b->full[last % kStages]), (last / kStages) & 1);
                if (!landed) atomicAdd(&p.waits[1], 1u);
            }
        }
        if (threadIdx.x == 32 && rank == 0) {
            commit(&b->drained);
            for (uint32_t i = 0; i < p.spin && !muon_try_wait(muon_smem(&b->drained), 0); ++i) {
            }
        }
        __syncwarp();
    }
    // neither CTA leaves while the other may read its operands or arrive on its barriers
    cluster_arrive();
    cluster_wait();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <bool WIDE, class P>
cudaError_t launch_as(const P& p, uint32_t pairs, cudaStream_t s)
{
    const cudaError_t e = allow_smem<muon_gemm_kernel<WIDE, P>>(kSmem);
    return e != cudaSuccess ? e : launch_pdl_clusters(muon_gemm_kernel<WIDE, P>, 2 * pairs, kGemmThreads, kSmem, 2, s, p);
}

// Tiles of one product of each matrix.
uint32_t tiles_of_all(const MuonGemmParams& p, int kind, uint32_t tile_n)
{
    uint32_t sum = 0;
    for (uint32_t k = 0; k < p.n; ++k) sum += muon_tiles(p.work[k].rows, p.work[k].cols, kind, tile_n);
    return sum;
}

}  // namespace

cudaError_t launch_muon_gemm(MuonGemmParams& p, int nops, cudaStream_t s)
{
    if (p.nseq == 0) return cudaSuccess;
    RankParams rp{};
    rp.waits = bulk_wait_counters();
    if (!rp.waits) return cudaErrorSymbolNotFound;
    const BulkParams bp = bulk_params(rp);
    p.waits = rp.waits;
    p.hold = bp.hold;
    // A tile may wait for a whole level of its matrix, which of the largest that fit
    // the memory takes a second or two.
    p.spin = bp.hold ? bp.spin : 1u << 26;
    // Tiles of 256 columns where those of a square product, which most levels are,
    // keep half of the pairs of SMs busy, and for Q X where every pair has one;
    // narrower ones, twice as many, are done sooner.  One / four layers of width 512,
    // bf16, in tiles of 256: 351 / 444 us, of 128: 297 / 467; two of 1000, fp16: 975
    // and 1218.
    const bool wide = tiles_of_all(p, kSquare, 256) >= kPairs / 2;
    uint32_t widest = 0;
    for (int kind = 0; kind < 3; ++kind) {
        p.tile_n[kind] = wide && (kind != kApply || tiles_of_all(p, kind, 256) >= kPairs) ? 256 : 128;
        widest = std::max(widest, tiles_of_all(p, kind, p.tile_n[kind]));
    }
    const uint32_t pairs = std::min(kPairs, 2 * widest);  // two products of a matrix may run side by side
    if (p.n > kMuonMatsSmall || nops > kMuonOpsSmall || p.nseq > kMuonSeqSmall)
        return wide ? launch_as<true>(p, pairs, s) : launch_as<false>(p, pairs, s);
    MuonGemmParamsT<kMuonMatsSmall, kMuonOpsSmall, kMuonSeqSmall> q;
    static_cast<MuonGemmHead&>(q) = p;
    std::copy_n(p.work, p.n, q.work);
    std::copy_n(p.op, nops, q.op);
    std::copy_n(p.seq, p.nseq, q.seq);
    return wide ? launch_as<true>(q, pairs, s) : launch_as<false>(q, pairs, s);
}

}  // namespace rr
