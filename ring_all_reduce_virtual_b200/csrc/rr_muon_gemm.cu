// rr_muon_gemm.cu -- the products of the Newton-Schulz iteration on the fifth
// generation tensor cores: a group of matrices in one launch,
//     out = alpha * op(A) op(B)^T + beta * C
// for operands and results held as two fp16 halves (rr_muon.h).  A product of
// two such values is three products of halves, lo hi + hi lo + hi hi (lo lo is
// below 2^-22), which accumulate in one fp32 accumulator: K runs three times.
//
// One CTA per SM goes through tiles of 128 x 256 (or 128 x 128) of all matrices.
// Its warps: one copies operand blocks (cp.async.bulk, 64 of K a stage, four
// stages), one issues the tensor core's instructions, four take finished
// accumulators out of tensor memory, form alpha acc + beta C, split it and store
// it; two accumulators, so that the next tile's products run meanwhile.
// A symmetric result is computed on and below the diagonal and stored twice.
//
// Every wait is bounded (rr_bulk.cuh): one that runs out is counted, the CTA's
// warps stop, wait (bounded) for copies and products in flight, give their
// tensor memory back and leave; what the call writes is then undefined.
#include <atomic>

#include <cuda_fp16.h>

#include "rr_bulk.cuh"
#include "rr_launch.cuh"
#include "rr_muon.h"

namespace rr {

namespace {

constexpr int kStages = 4;
constexpr uint32_t kTileM = 128, kTileN = 256;
constexpr uint32_t kABytes = kTileM * kBlk * 2, kBBytes = kTileN * kBlk * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr int kGemmThreads = 192;  // copies, products, four warps of results
constexpr uint32_t kSmem = kStages * kStageBytes + 1024 + 256;  // operands from a 1024-byte boundary, barriers

struct Bars {
    uint64_t full[kStages], empty[kStages];  // of a stage: its copies have landed; its products are done
    uint64_t ready[2], taken[2];             // of an accumulator: finished; read out
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
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
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

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(smem_of(bar)) : "memory");
}

__device__ __forceinline__ void copy_block(uint32_t to, const uint16_t* from, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(smem_of(bar))
                 : "memory");
}

// Where the launch's tile `w` lies.
struct Tile {
    const MuonProduct* q;
    uint32_t i, j;   // in tiles of 128 rows, of tile_n columns
    uint32_t units;  // of 128 columns: 1 or 2
};

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
    const uint32_t per = p.tile_n / 128;
    if (t.q->sym) {
        uint32_t i = 0;
        while (k >= i / per + 1) k -= i++ / per + 1;
        t.i = i;
        t.j = k;
    } else {  // tiles of one column run together: they share B, the wider operand
        t.i = k % t.q->mt;
        t.j = k / t.q->mt;
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

// Instruction descriptor: fp16 operands, fp32 accumulator, 128 x n.
__device__ __forceinline__ uint32_t instruction(uint32_t n, bool a_mn, bool b_mn)
{
    return 1u << 4 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (n >> 3) << 17 | (kTileM >> 4) << 24;
}

__device__ __forceinline__ void mma(uint32_t acc, uint64_t a, uint64_t b, uint32_t inst, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
        "l"(a), "l"(b), "r"(inst), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(bar)) : "memory");
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

__device__ __forceinline__ uint32_t pack_halves(__half a, __half b)
{
    return (uint32_t)__half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// 32 columns of the accumulator: this thread's row, columns col..col+31 of the
// result.  mirror: the same values at (column, row) as well.
__device__ __forceinline__ void put_columns(const MuonProduct& q, uint32_t row, uint32_t col, const uint32_t (&acc)[32],
                                            bool mirror)
{
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint32_t c0 = col + g * 8;
        const uint64_t at = piece_at(row, c0, q.o_nbj);
        float v[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) v[l] = q.alpha * __uint_as_float(acc[g * 8 + l]);
        if (q.c.hi) {
            const uint4 h = ld16(q.c.hi + at), l = ld16(q.c.lo + at);
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 a = pair_of(hw[k]), b = pair_of(lw[k]);
                v[2 * k] = __fmaf_rn(q.beta, a.x, __fmaf_rn(q.beta, b.x, v[2 * k]));
                v[2 * k + 1] = __fmaf_rn(q.beta, a.y, __fmaf_rn(q.beta, b.y, v[2 * k + 1]));
            }
        }
        __half hi[8], lo[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) {
            hi[l] = __float2half_rn(v[l]);
            lo[l] = __float2half_rn(v[l] - __half2float(hi[l]));
        }
        *reinterpret_cast<uint4*>(q.out.hi + at) = make_uint4(pack_halves(hi[0], hi[1]), pack_halves(hi[2], hi[3]),
                                                              pack_halves(hi[4], hi[5]), pack_halves(hi[6], hi[7]));
        *reinterpret_cast<uint4*>(q.out.lo + at) = make_uint4(pack_halves(lo[0], lo[1]), pack_halves(lo[2], lo[3]),
                                                              pack_halves(lo[4], lo[5]), pack_halves(lo[6], lo[7]));
        if (mirror) {
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                const uint64_t m = piece_at(c0 + l, row & ~7u, q.o_nbj) + (row & 7u);
                q.out.hi[m] = __half_as_ushort(hi[l]);
                q.out.lo[m] = __half_as_ushort(lo[l]);
            }
        }
    }
}

__global__ void __launch_bounds__(kGemmThreads, 1) muon_gemm_kernel(const __grid_constant__ MuonGemmParams p)
{
    extern __shared__ uint8_t raw_smem[];
    uint8_t* base = raw_smem + ((1024u - (smem_of(raw_smem) & 1023u)) & 1023u);
    Bars* b = reinterpret_cast<Bars*>(base + kStages * kStageBytes);
    const uint32_t ops = smem_of(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            bar_init(&b->full[s], 1 + p.hold);
            bar_init(&b->empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(&b->ready[s], 1);
            bar_init(&b->taken[s], 4);
        }
        bar_init(&b->drained, 1);
        b->stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&b->tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = b->tmem;
    pdl_begin();

    uint32_t it = 0;  // the copying thread's: stages begun
    if (warp == 0) {
        if (lane == 0) {  // copies
            asm volatile("fence.proxy.async;" ::: "memory");  // the operands were written by ordinary stores
            bool ok = true;
            for (uint32_t w = blockIdx.x; w < p.tiles && ok; w += gridDim.x) {
                const Tile t = tile_of(p, w);
                const MuonProduct& q = *t.q;
                const uint32_t bytes = kABytes + t.units * (kBBytes / 2);
                for (uint32_t pass = 0; pass < 3 && ok; ++pass) {  // lo hi, hi lo, hi hi: small terms first
                    const uint16_t* a = pass == 0 ? q.a.lo : q.a.hi;
                    const uint16_t* bb = pass == 1 ? q.b.lo : q.b.hi;
                    for (uint32_t k = 0; k < q.kb; ++k, ++it) {
                        const uint32_t s = it % kStages, use = it / kStages;
                        if (use > 0 && !(ok = wait_for(&b->empty[s], (use - 1) & 1, b, p.waits, p.spin))) break;
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(&b->full[s])), "r"(bytes)
                                     : "memory");
                        const uint32_t sa = ops + s * kStageBytes, sb = sa + kABytes;
                        if (!q.a_mn) {
                            copy_block(sa, a + block_at(2 * t.i, k, q.a_nbj), kABytes, &b->full[s]);
                        } else {
                            copy_block(sa, a + block_at(k, 2 * t.i, q.a_nbj), kABytes / 2, &b->full[s]);
                            copy_block(sa + kABytes / 2, a + block_at(k, 2 * t.i + 1, q.a_nbj), kABytes / 2, &b->full[s]);
                        }
                        const uint32_t n0 = t.j * (p.tile_n / kBlk);  // the tile's first block along N
                        for (uint32_t u = 0; u < t.units; ++u) {
                            const uint32_t to = sb + u * (kBBytes / 2);
                            if (!q.b_mn) {
                                copy_block(to, bb + block_at(n0 + 2 * u, k, q.b_nbj), kBBytes / 2, &b->full[s]);
                            } else {
                                copy_block(to, bb + block_at(k, n0 + 2 * u, q.b_nbj), kBBytes / 4, &b->full[s]);
                                copy_block(to + kBBytes / 4, bb + block_at(k, n0 + 2 * u + 1, q.b_nbj), kBBytes / 4, &b->full[s]);
                            }
                        }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {  // products
            uint32_t done = 0, n = 0;
            bool ok = true;
            for (uint32_t w = blockIdx.x; w < p.tiles && ok; w += gridDim.x, ++n) {
                const Tile t = tile_of(p, w);
                const MuonProduct& q = *t.q;
                const uint32_t acc = tmem + (n & 1) * kTileN;
                const uint32_t inst = instruction(t.units * 128, q.a_mn, q.b_mn);
                const uint32_t astep = (q.a_mn ? 2048u : 32u) >> 4, bstep = (q.b_mn ? 2048u : 32u) >> 4;
                if (n >= 2 && !(ok = wait_for(&b->taken[n & 1], ((n >> 1) - 1) & 1, b, p.waits, p.spin))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t steps = 3 * q.kb;
                for (uint32_t k = 0; k < steps; ++k, ++done) {
                    const uint32_t s = done % kStages;
                    if (!(ok = wait_for(&b->full[s], (done / kStages) & 1, b, p.waits, p.spin))) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t sa = ops + s * kStageBytes;
                    const uint64_t da = operand(sa, q.a_mn), db = operand(sa + kABytes, q.b_mn);
#pragma unroll
                    for (uint32_t c = 0; c < kBlk / 16; ++c) mma(acc, da + c * astep, db + c * bstep, inst, k > 0 || c > 0);
                    commit(&b->empty[s]);
                }
                if (ok) commit(&b->ready[n & 1]);
            }
        }
        __syncwarp();
    } else {
        // results: a warp reads the quarter of the accumulator's rows that is its own
        const uint32_t quarter = warp & 3;
        uint32_t n = 0;
        for (uint32_t w = blockIdx.x; w < p.tiles; w += gridDim.x, ++n) {
            const Tile t = tile_of(p, w);
            const MuonProduct& q = *t.q;
            const bool ok = wait_for(&b->ready[n & 1], (n >> 1) & 1, b, p.waits, p.spin);
            if (!__all_sync(0xffffffffu, ok)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t row = t.i * kTileM + quarter * 32 + lane;
            const uint32_t acc = tmem + (quarter * 32 << 16) + (n & 1) * kTileN;
            const uint32_t per = p.tile_n / 128;
            for (uint32_t c = 0; c < t.units * 128; c += 32) {
                uint32_t r[32];
                load_acc(acc + c, r);
                const uint32_t unit = t.j * per + c / 128;
                put_columns(q, row, t.j * p.tile_n + c, r, q.sym && unit / per < t.i / per);
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) bar_arrive(&b->taken[n & 1]);
        }
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
        if (threadIdx.x == 32) {
            commit(&b->drained);
            for (uint32_t i = 0; i < p.spin && !try_wait(smem_of(&b->drained), 0); ++i) {
            }
        }
        __syncthreads();
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

uint32_t tiles_of(const MuonProduct& q, uint32_t tile_n)
{
    const uint32_t per = tile_n / 128;
    if (!q.sym) return q.mt * ((q.nu + per - 1) / per);
    uint32_t t = 0;
    for (uint32_t i = 0; i < q.mt; ++i) t += i / per + 1;
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
    // tiles of 256 columns where every SM has one; narrower ones are done sooner
    for (p.tile_n = 256;; p.tile_n = 128) {
        p.tiles = 0;
        for (int i = 0; i < p.n; ++i) {
            p.q[i].tile0 = p.tiles;
            p.tiles += tiles_of(p.q[i], p.tile_n);
        }
        if (p.tiles >= 148 || p.tile_n == 128) break;
    }
    if (p.tiles == 0) return cudaSuccess;
    return launch_pdl(muon_gemm_kernel, dim3(p.tiles < 148 ? p.tiles : 148), kGemmThreads, kSmem, s, p);
}

}  // namespace rr
