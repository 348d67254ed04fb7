// rr_muon_gemm.cu -- the products of the Newton-Schulz iteration on the fifth
// generation tensor cores: a group of matrices in one launch,
//     out = alpha * op(A) op(B)^T + beta * C
// for operands and results held as two fp16 halves (rr_muon.h).  A product of
// two such values is three products of halves, lo hi + hi lo + hi hi (lo lo is
// below 2^-22), in one fp32 accumulator.
//
// Two CTAs on neighbouring SMs share a tile of 256 x 256 (or 256 x 128): each
// copies its 128 rows of A and its half of B's (cp.async.bulk, both halves of 64
// of K a stage, 64 KB, three stages), and the first one's instructions multiply
// out of both.  That is what the L2 cache can feed: 196 operations a byte,
// against 85 of one CTA's tile of 128 x 256 with K gone through three times
// (796 TFLOP/s at 16 matrices of width 2048, all of it waiting for L2).
// Of a CTA's warps one copies, one issues the products (in the second CTA: tells
// the first that a stage has landed), eight take accumulators out of tensor
// memory.
//
// The tensor cores' sums are cut off, not rounded: a long one comes out low by
// 2^-25 and more a term (a sum of 8192 positive products by 1.5e-5).  So an
// accumulator collects kChunk stages only; the eight warps add it to sums in
// their registers, rounded to nearest, while the other accumulator fills.
//
// Results leave through shared memory, 4 KB a warp: a thread has a row of the
// tile, whose 16-byte pieces lie 128 bytes from the next row's; written to L2
// from there they took the warps longer than the products (8 x 2048 x 2048, one
// step: 803 us against 633 without them).  Laid into 32 rows of a block they go
// out as one copy.
//
// Every wait is bounded (rr_bulk.cuh): one that runs out is counted, the CTA's
// warps stop, wait (bounded) for copies and products in flight, give their
// tensor memory back and leave; what the call writes is then undefined.
#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "rr_bulk.cuh"
#include "rr_launch.cuh"
#include "rr_muon.h"

namespace rr {

namespace {

constexpr int kStages = 3;
constexpr uint32_t kPairs = 74;                // pairs of SMs
constexpr uint32_t kChunk = 4;                 // stages an accumulator collects
constexpr uint32_t kTileN = 256;
constexpr uint32_t kPlane = 128 * kBlk * 2;    // one half of 128 rows (or columns) of an operand's stage
constexpr uint32_t kStageBytes = 4 * kPlane;   // A's hi and lo, B's hi and lo
constexpr int kTakers = 8;                     // warps that take accumulators out
constexpr int kGemmThreads = 128 + 32 * kTakers;
// Registers a thread: 168 at the launch (65536 over 384 threads), of which the
// first four warps give 112 back and the takers have 56 more: their sums are
// 128.  128 x 56 + 256 x 224 = 384 x 168.
constexpr int kFewRegs = 56, kManyRegs = 224;
static_assert(128 * kFewRegs + 32 * kTakers * kManyRegs <= 168 * kGemmThreads, "more than the launch has");
constexpr uint32_t kOutBytes = 32 * kBlk * 2;  // a warp's 32 rows of a block
constexpr uint32_t kSmem = kStages * kStageBytes + kTakers * kOutBytes + 1024 + 256;  // from a 1024-byte boundary; barriers

struct Bars {
    uint64_t full[kStages], empty[kStages];  // of a stage: its copies have landed; its products are done
    uint64_t other[kStages];                 // first CTA: the second's copies have landed
    uint64_t ready[2], taken[2];             // of an accumulator: finished; read out by both CTAs (in the first)
    uint64_t added[kTakers];                 // a taker's piece of C has landed
    uint64_t drained;
    uint32_t tmem;
    uint32_t stop;
};

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Bounded; false as well once another warp of the CTA has given up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Bars* b, unsigned int* waits, uint32_t spin)
{
    const uint32_t at = smem_of(bar);
    for (uint32_t i = 0; i < spin; ++i) {
        if (try_wait(at, parity)) return true;
        if (*(volatile uint32_t*)&b->stop) return false;
    }
    if (atomicExch(&b->stop, 1u) == 0) atomicAdd(&waits[0], 1u);
    return false;
}

// The same for a whole warp, one lane of which looks: 32 that do keep the shared
// memory busy for the warps that copy and multiply.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars* b, unsigned int* waits, uint32_t spin)
{
    uint32_t ok = 0;
    if ((threadIdx.x & 31) == 0) ok = wait_for(bar, parity, b, waits, spin);
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(smem_of(bar)) : "memory");
}

// An arrival on the first CTA's barrier, from either CTA.
__device__ __forceinline__ void first_arrive(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .b32 at;\n\tmapa.shared::cluster.u32 at, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [at];\n\t}" ::"r"(smem_of(bar))
        : "memory");
}

__device__ __forceinline__ void copy_block(uint32_t to, const uint16_t* from, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(smem_of(bar))
                 : "memory");
}

// Where the launch's tile `w` lies: 256 rows, tile_n columns.
struct Tile {
    const MuonProduct* q;
    uint32_t i, j;
    uint32_t units;  // of 128 columns: 1 or 2
};

// Column tiles of a row tile of a symmetric result.
__host__ __device__ __forceinline__ uint32_t sym_tiles(uint32_t i, uint32_t nu, uint32_t per)
{
    const uint32_t units = 2 * i + 2 < nu ? 2 * i + 2 : nu;
    return (units + per - 1) / per;
}

__device__ __forceinline__ Tile tile_of(const MuonGemmParams& p, uint32_t w)
{
    int lo = 0, hi = p.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q[mid].tile0 <= w) lo = mid;
        else hi = mid;
    }
    Tile t;
    t.q = &p.q[lo];
    uint32_t k = w - t.q->tile0;
    const uint32_t per = p.tile_n / 128, rows = (t.q->mt + 1) / 2;
    if (t.q->sym) {
        uint32_t i = 0;
        while (k >= sym_tiles(i, t.q->nu, per)) k -= sym_tiles(i++, t.q->nu, per);
        t.i = i;
        t.j = k;
    } else {
        t.i = k % rows;
        t.j = k / rows;
    }
    t.units = min(per, t.q->nu - t.j * per);
    return t;
}

// Shared-memory descriptor of an operand in 128-byte-swizzled blocks: K along a
// block's columns (groups of 8 rows are 1024 bytes apart), or along its rows
// (groups of 8 of K 1024 bytes apart, of 64 of M or N 8192).
__device__ __forceinline__ uint64_t operand(uint32_t addr, bool mn)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(mn ? 8192u >> 4 : 1u) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp16 operands, fp32 accumulator, 256 x n over two CTAs.
__device__ __forceinline__ uint32_t instruction(uint32_t n, bool a_mn, bool b_mn)
{
    return 1u << 4 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (n >> 3) << 17 | (256u >> 4) << 24;
}

__device__ __forceinline__ void mma(uint32_t acc, uint64_t a, uint64_t b, uint32_t inst, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
        "l"(a), "l"(b), "r"(inst), "r"((uint32_t)add)
        : "memory");
}

// An arrival on the barrier of both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_of(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void load_acc(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A taker's 4 KB of shared memory, 32 rows of one half of a block.
struct OutRows {
    uint8_t* mem;
    uint64_t* bar;    // of copies into it
    uint32_t parity;  // of the next one

    __device__ __forceinline__ uint4* piece(int lane, int g) const
    {
        return reinterpret_cast<uint4*>(mem + lane * (kBlk * 2) + ((g ^ (lane & 7)) << 4));
    }
    // Free again: the copy out of it has read it.
    __device__ __forceinline__ void reuse(int lane) const
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
    }
    __device__ __forceinline__ void send(uint16_t* to, int lane) const
    {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_of(mem)), "r"(kOutBytes)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
};

// 64 columns of this thread's row: to out's block, `at` halves into it.
__device__ __forceinline__ bool put_block(const MuonProduct& q, uint64_t at, uint32_t row, uint32_t col, float (&v)[64], OutRows& o,
                                          int lane, Bars* b, const MuonGemmParams& p)
{
#pragma unroll
    for (int l = 0; l < 64; ++l) v[l] *= q.alpha;
    if (q.c.hi) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            o.reuse(lane);
            if (lane == 0) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(o.bar)), "r"(kOutBytes) : "memory");
                copy_block(smem_of(o.mem), (half ? q.c.lo : q.c.hi) + at, kOutBytes, o.bar);
            }
            const bool landed = warp_wait(o.bar, o.parity, b, p.waits, p.spin);
            o.parity ^= 1;
            if (!landed) {  // given up: the copy lands before the CTA leaves
                if (lane == 0) {
                    bool late = false;
                    for (uint32_t i = 0; i < p.spin && !late; ++i) late = try_wait(smem_of(o.bar), o.parity ^ 1);
                    if (!late) atomicAdd(&p.waits[1], 1u);
                }
                __syncwarp();
                return false;
            }
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                float a[8];
                F16T::unpack(*o.piece(lane, g), a);
#pragma unroll
                for (int l = 0; l < 8; ++l) v[g * 8 + l] = __fmaf_rn(q.beta, a[l], v[g * 8 + l]);
            }
            __syncwarp();
        }
    }
    if (q.diag != 0.0f && row < q.side) {
#pragma unroll
        for (int l = 0; l < 64; ++l)
            if (col + l == row) v[l] += q.diag;
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        o.reuse(lane);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            float a[8];
#pragma unroll
            for (int l = 0; l < 8; ++l) a[l] = v[g * 8 + l];
            const uint4 w = F16T::pack(a);
            *o.piece(lane, g) = w;
            float r[8];
            F16T::unpack(w, r);  // what is left, for the second half (unread after it)
#pragma unroll
            for (int l = 0; l < 8; ++l) v[g * 8 + l] = a[l] - r[l];
        }
        o.send((half ? q.out.lo : q.out.hi) + at, lane);
    }
    return true;
}

__global__ void __launch_bounds__(kGemmThreads, 1) muon_gemm_kernel(const __grid_constant__ MuonGemmParams p)
{
    extern __shared__ uint8_t raw_smem[];
    uint8_t* base = raw_smem + ((1024u - (smem_of(raw_smem) & 1023u)) & 1023u);
    Bars* b = reinterpret_cast<Bars*>(base + kStages * kStageBytes + kTakers * kOutBytes);
    const uint32_t ops = smem_of(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;  // in its pair
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            bar_init(&b->full[s], 1 + p.hold);
            bar_init(&b->empty[s], 1);
            bar_init(&b->other[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(&b->ready[s], 1);
            bar_init(&b->taken[s], 2 * kTakers);
        }
        for (int k = 0; k < kTakers; ++k) bar_init(&b->added[k], 1);
        bar_init(&b->drained, 1);
        b->stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&b->tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // both CTAs' barriers are set up
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = b->tmem;
    pdl_begin();

    const uint32_t first = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    uint32_t it = 0;  // the copying warp's: stages begun
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0) {
                // Copies: a stage's eight blocks of 8 KB by a lane each, the pairs that
            // follow one another in memory as one copy of 16 KB.  (One thread that
            // worked out and issued them all took 2600 clocks a stage, which the
            // products need for 1536.)
            asm volatile("fence.proxy.async;" ::: "memory");  // the operands were written by ordinary stores
            const uint32_t half = lane & 1, second = lane >> 1 & 1;  // of the pair; the low halves
            const bool is_b = lane >> 2 & 1;
            bool ok = true;
            for (uint32_t w = first; w < p.tiles && ok; w += pairs) {
                const Tile t = tile_of(p, w);
                const MuonProduct& q = *t.q;
                const bool rows = 2 * t.i + rank < q.mt;  // else this CTA's part of the products is of no use
                // the first of this CTA's blocks along M or N, and how many there are
                const uint32_t at = is_b ? t.j * (p.tile_n / kBlk) + t.units * rank : 2 * (2 * t.i + rank);
                const uint32_t blocks = is_b ? t.units : rows ? 2 : 0;
                const Halves& op = is_b ? q.b : q.a;
                const uint16_t* src = second ? op.lo : op.hi;
                const uint32_t nbj = is_b ? q.b_nbj : q.a_nbj;
                const bool mn = is_b ? q.b_mn : q.a_mn, low = is_b ? q.b_low : q.a_low;
                const uint16_t* by_row = src + block_at(at + half, 0, nbj);  // + k * 2 blocks
                const uint16_t* by_col = src + block_at(0, at + half, nbj);  // + k / 2 * 2 nbj blocks + k % 2
                const uint32_t to = ops + (is_b ? 2 * kPlane : 0) + second * kPlane + half * (kPlane / 2);
                const uint32_t bytes = (rows ? 2 * kPlane : 0) + t.units * kPlane;
                const uint32_t kb = q.kb, limit = low ? (at >> 2) * 4 + 4 : mn ? 0 : kb;  // K's blocks that lie by rows
                const uint64_t pair = (uint64_t)nbj * 2 * kBlkElems;
                for (uint32_t k = 0; k < kb; ++k, ++it) {
                    const uint32_t s = it % kStages, use = it / kStages;
                    if (use > 0) ok = warp_wait(&b->empty[s], (use - 1) & 1, b, p.waits, p.spin);
                    if (!ok) break;
                    uint64_t* full = &b->full[s];
                    if (lane == 0)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(full)), "r"(bytes) : "memory");
                    __syncwarp();
                    const bool whole = k < limit && blocks == 2;  // both blocks, one after the other
                    if (lane < 8 && half < (whole ? 1 : blocks))
                        copy_block(to + s * kStageBytes, k < limit ? by_row + (uint64_t)k * 2 * kBlkElems : by_col + (k >> 1) * pair + (k & 1) * kBlkElems,
                                   whole ? kPlane : kPlane / 2, full);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0 && rank != 0) {  // the first CTA learns of this one's copies
                uint32_t done = 0;
                bool ok = true;
                for (uint32_t w = first; w < p.tiles && ok; w += pairs) {
                    const uint32_t kb = tile_of(p, w).q->kb;
                    for (uint32_t k = 0; k < kb; ++k, ++done) {
                        const uint32_t s = done % kStages;
                        if (!(ok = wait_for(&b->full[s], (done / kStages) & 1, b, p.waits, p.spin))) break;
                        first_arrive(&b->other[s]);
                    }
                }
            } else if (lane == 0) {  // products
                uint32_t done = 0, n = 0;  // stages, accumulators
                bool ok = true;
                for (uint32_t w = first; w < p.tiles && ok; w += pairs) {
                    const Tile t = tile_of(p, w);
                    const MuonProduct& q = *t.q;
                    // K's blocks that lie by rows; both CTAs' blocks lie in one tile of 256
                    const uint32_t kb = q.kb, n128 = t.units * 128;
                    const uint32_t a_rows = q.a_low ? t.i * 4 + 4 : q.a_mn ? 0 : kb;
                    const uint32_t b_rows = q.b_low ? (t.j * p.tile_n / 256) * 4 + 4 : q.b_mn ? 0 : kb;
                    for (uint32_t k0 = 0; k0 < kb && ok; k0 += kChunk, ++n) {
                        const uint32_t acc = tmem + (n & 1) * kTileN, k1 = min(kb, k0 + kChunk);
                        if (n >= 2 && !(ok = wait_for(&b->taken[n & 1], ((n >> 1) - 1) & 1, b, p.waits, p.spin))) break;
                        for (uint32_t k = k0; k < k1; ++k, ++done) {
                            const uint32_t s = done % kStages, parity = (done / kStages) & 1;
                            if (!(ok = wait_for(&b->full[s], parity, b, p.waits, p.spin) &&
                                       wait_for(&b->other[s], parity, b, p.waits, p.spin)))
                                break;
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                            const uint32_t sa = ops + s * kStageBytes;
                            const bool a_mn = k >= a_rows, b_mn = k >= b_rows;
                            const uint32_t inst = instruction(n128, a_mn, b_mn);
                            const uint32_t astep = (a_mn ? 2048u : 32u) >> 4, bstep = (b_mn ? 2048u : 32u) >> 4;
                            const uint64_t ah = operand(sa, a_mn), al = operand(sa + kPlane, a_mn);
                            const uint64_t bh = operand(sa + 2 * kPlane, b_mn), bl = operand(sa + 3 * kPlane, b_mn);
    #pragma unroll
                            for (uint32_t c = 0; c < kBlk / 16; ++c) mma(acc, al + c * astep, bh + c * bstep, inst, k > k0 || c > 0);
#pragma unroll
                            for (uint32_t c = 0; c < kBlk / 16; ++c) mma(acc, ah + c * astep, bl + c * bstep, inst, true);
#pragma unroll
                            for (uint32_t c = 0; c < kBlk / 16; ++c) mma(acc, ah + c * astep, bh + c * bstep, inst, true);
                            commit(&b->empty[s]);
                        }
                        if (ok) commit(&b->ready[n & 1]);
                    }
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // results: a warp reads the quarter of the accumulator's rows that is its
        // own, and one of its units of 128 columns
        const uint32_t quarter = warp & 3, side = (warp - 4) >> 2;
        OutRows o{base + kStages * kStageBytes + (warp - 4) * kOutBytes, &b->added[warp - 4], 0};
        uint32_t n = 0;
        bool ok = true;
        for (uint32_t w = first; w < p.tiles && ok; w += pairs) {
            const Tile t = tile_of(p, w);
            const MuonProduct& q = *t.q;
            const bool mine = side < t.units;
            float sum[128];
#pragma unroll
            for (int l = 0; l < 128; ++l) sum[l] = 0.0f;
            for (uint32_t k0 = 0; k0 < q.kb && ok; k0 += kChunk, ++n) {
                ok = warp_wait(&b->ready[n & 1], (n >> 1) & 1, b, p.waits, p.spin);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t acc = tmem + (quarter * 32 << 16) + (n & 1) * kTileN + side * 128;
                if (mine && ok) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        load_acc(acc + c * 32, r);
#pragma unroll
                        for (int l = 0; l < 32; ++l) sum[c * 32 + l] += __uint_as_float(r[l]);
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0 && ok) first_arrive(&b->taken[n & 1]);
            }
            const uint32_t unit = 2 * t.i + rank;  // of 128 rows
            if (!ok || !mine || unit >= q.mt) continue;
            const uint32_t row0 = unit * 128 + quarter * 32, col = t.j * p.tile_n + side * 128;
            const uint64_t at = block_at(row0 / kBlk, col / kBlk, q.o_nbj) + row0 % kBlk * kBlk;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[64];
#pragma unroll
                for (int l = 0; l < 64; ++l) v[l] = sum[h * 64 + l];
                ok = ok && put_block(q, at + (uint64_t)h * 2 * kBlkElems, row0 + lane, col + h * 64, v, o, lane, b, p);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (b->stop) {  // a wait ran out: what is in flight ends before the CTA's memory goes
        if (threadIdx.x == 0) {
            if (p.hold)
                for (uint32_t k = 0; k < kStages && k < it; ++k) bar_arrive(&b->full[k]);
            for (uint32_t back = 1; back <= kStages && back <= it; ++back) {
                const uint32_t last = it - back;
                bool landed = false;
                for (uint32_t i = 0; i < p.spin && !landed; ++i)
                    landed = try_wait(smem_of(&b->full[last % kStages]), (last / kStages) & 1);
                if (!landed) atomicAdd(&p.waits[1], 1u);
            }
        }
        if (threadIdx.x == 32 && rank == 0) {
            commit(&b->drained);
            for (uint32_t i = 0; i < p.spin && !try_wait(smem_of(&b->drained), 0); ++i) {
            }
        }
        __syncwarp();
    }
    // neither CTA leaves while the other may read its operands or arrive on its barriers
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

uint32_t tiles_of(const MuonProduct& q, uint32_t tile_n)
{
    const uint32_t per = tile_n / 128, rows = (q.mt + 1) / 2;
    if (!q.sym) return rows * ((q.nu + per - 1) / per);
    uint32_t t = 0;
    for (uint32_t i = 0; i < rows; ++i) t += sym_tiles(i, q.nu, per);
    return t;
}

}  // namespace

cudaError_t launch_muon_gemm(MuonGemmParams& p, cudaStream_t s)
{
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> asked[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !asked[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(muon_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) asked[dev].store(true, std::memory_order_release);
    }
    RankParams rp{};
    rp.waits = bulk_wait_counters();
    if (!rp.waits) return cudaErrorSymbolNotFound;
    const BulkParams bp = bulk_params(rp);
    p.waits = rp.waits;
    p.hold = bp.hold;
    p.spin = bp.spin;
    // tiles of 256 columns where every pair of SMs has one; narrower ones are done sooner
    for (p.tile_n = 256;; p.tile_n = 128) {
        p.tiles = 0;
        for (int i = 0; i < p.n; ++i) {
            p.q[i].tile0 = p.tiles;
            p.tiles += tiles_of(p.q[i], p.tile_n);
        }
        if (p.tiles >= kPairs || p.tile_n == 128) break;
    }
    if (p.tiles == 0) return cudaSuccess;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * std::min(p.tiles, kPairs));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, muon_gemm_kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rr
