// rr_muon_small.cu -- the whole orthogonalisation or Muon step of matrices whose
// shorter side is at most 128 and whose longer one at most 1024, in one launch:
// momentum, norm, every Newton-Schulz step, the update of every replica.
//
// A cluster has one matrix, in X's orientation of m <= n sides (a tall matrix is
// transposed as it is read and written); each of its CTAs keeps m x 128 columns
// of X in shared memory, as two fp16 halves in the blocks of rr_muon.h, and next
// to it the m x m matrices A and B, the same in all of them.  A step:
//     P = X X^T of the CTA's columns, in fp32, summed over the cluster in the
//         order of its CTAs: each sums the rows that are its own and hands their
//         halves to the others                                      -> A
//     B = b A + c A^2      (every CTA for itself)
//     X = a X + B X        (its own columns)
// Each product is one or two instructions' worth of K per 16, an accumulator for
// every 64 of K (rr_muon_gemm.cu says why), and its result goes back to shared
// memory: nothing of an iteration leaves the chip, and a step costs two cluster
// barriers.  As tiles of rr_muon_gemm.cu a level of such a matrix takes 8 us, most
// of it the way through L2: one layer of width 128 (fp32) 155 us against 70.
#include <algorithm>

#include <cuda_fp16.h>

#include "rr_bulk.cuh"
#include "rr_clip.cuh"
#include "rr_launch.cuh"
#include "rr_muon.h"
#include "rr_muon_device.cuh"

namespace rr {

namespace {

constexpr uint32_t kSide = 128;
constexpr uint32_t kPlaneBytes = kSide * kSide * 2;      // a half of an m x 128 matrix
constexpr uint32_t kMatBytes = 2 * kPlaneBytes;
constexpr uint32_t kSmallSmem = 3 * kMatBytes + 1024;    // X, A, B from a 1024-byte boundary

struct SmallShared {
    double part[kMuonSmallCtas];  // every CTA's sum of squares
    double sums[kThreads / 32];
    uint64_t done;                // the products' barrier
    uint32_t tmem;
    uint32_t stop;
};

__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

// The 16-byte piece of an m x 128 half that begins at (r, c): blocks of 64 x 64,
// the two of one column block of blocks after one another.
__device__ __forceinline__ uint4* piece(uint8_t* plane, uint32_t r, uint32_t c)
{
    return reinterpret_cast<uint4*>(plane + 2 * piece_at(r, c, 2));
}

// fp32 values of an m x 128 matrix, 4 bytes each, words permuted within a row so
// that both a row's and a column's neighbours lie in different banks.
__device__ __forceinline__ float* word(uint8_t* mem, uint32_t r, uint32_t c)
{
    return reinterpret_cast<float*>(mem) + r * kSide + (c ^ (r & 31u));
}

// 16 bytes of a row of fp32 sums, permuted by whole pieces.
__device__ __forceinline__ float4* quad(uint8_t* mem, uint32_t r, uint32_t q)
{
    return reinterpret_cast<float4*>(mem) + r * (kSide / 4) + (q ^ (r & 31u));
}

// acc = X op for K = 64 k of two 128 x 128 operands, for every k below `slabs` into
// an accumulator of its own; the CTA waits for them.  False: a wait ran out.
struct Products {
    uint32_t tmem;
    uint64_t* bar;
    uint32_t parity;
    uint32_t* stop;
    unsigned int* waits;
    uint32_t spin;

    __device__ __forceinline__ void run(uint32_t a, bool a_mn, uint32_t b, bool b_mn, uint32_t slabs)
    {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // operands were written by ordinary stores
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (*(volatile uint32_t*)stop) return;  // the same in every thread: written before a barrier
        if (threadIdx.x == 0) {
            const uint32_t inst = muon_instruction(128, 128, a_mn, b_mn);
            // rows along K: 64 rows (8 KB) a slab, 64 columns 16 KB apart; else 64 columns a slab
            const uint32_t aslab = a_mn ? 8192 : 16384, bslab = b_mn ? 8192 : 16384;
            const uint32_t astep = (a_mn ? 2048u : 32u) >> 4, bstep = (b_mn ? 2048u : 32u) >> 4;
            for (uint32_t k = 0; k < slabs; ++k) {
                const uint32_t acc = tmem + k * kSide;
                const uint64_t ah = muon_operand(a + k * aslab, a_mn, 16384), al = muon_operand(a + kPlaneBytes + k * aslab, a_mn, 16384);
                const uint64_t bh = muon_operand(b + k * bslab, b_mn, 16384), bl = muon_operand(b + kPlaneBytes + k * bslab, b_mn, 16384);
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) muon_mma<1>(acc, al + c * astep, bh + c * bstep, inst, c > 0);
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) muon_mma<1>(acc, ah + c * astep, bl + c * bstep, inst, true);
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) muon_mma<1>(acc, ah + c * astep, bh + c * bstep, inst, true);
            }
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(muon_smem(bar)) : "memory");
        }
        bool ok = false;
        for (uint32_t i = 0; i < spin && !ok; ++i) ok = muon_try_wait(muon_smem(bar), parity);
        parity ^= 1;
        if (!ok && atomicExch(stop, 1u) == 0) atomicAdd(&waits[0], 1u);
        __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    // Columns col .. col + 31 of this thread's row, summed over the accumulators.
    __device__ __forceinline__ void sums(float (&v)[32], uint32_t quarter, uint32_t col, uint32_t slabs) const
    {
        uint32_t r[2][32];
        const uint32_t at = tmem + (quarter * 32 << 16) + col;
        muon_load_acc(at, r[0]);
        if (slabs > 1) muon_load_acc(at + kSide, r[1]);
        muon_acc_landed();
#pragma unroll
        for (int l = 0; l < 32; ++l) v[l] = __uint_as_float(r[0][l]) + (slabs > 1 ? __uint_as_float(r[1][l]) : 0.0f);
    }
};

// 32 columns of a row as halves.
__device__ __forceinline__ void put_halves(uint8_t* mat, uint32_t row, uint32_t col, const float (&v)[32])
{
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float a[8], r[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) a[l] = v[g * 8 + l];
        const uint4 w = F16T::pack(a);
        F16T::unpack(w, r);
#pragma unroll
        for (int l = 0; l < 8; ++l) a[l] -= r[l];
        *piece(mat, row, col + g * 8) = w;
        *piece(mat + kPlaneBytes, row, col + g * 8) = F16T::pack(a);
    }
}

// v = beta * (the matrix's value) + alpha * v.
__device__ __forceinline__ void add_halves(uint8_t* mat, uint32_t row, uint32_t col, float alpha, float beta, float (&v)[32])
{
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float h[8], l[8];
        F16T::unpack(*piece(mat, row, col + g * 8), h);
        F16T::unpack(*piece(mat + kPlaneBytes, row, col + g * 8), l);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[g * 8 + i] = __fmaf_rn(beta, h[i], __fmaf_rn(beta, l[i], alpha * v[g * 8 + i]));
    }
}

template <class P>
__global__ void __launch_bounds__(kThreads, 1) muon_small_kernel(const __grid_constant__ P p)
{
    extern __shared__ uint8_t raw_smem[];
    __shared__ SmallShared sh;
    uint8_t* X = raw_smem + ((1024u - (muon_smem(raw_smem) & 1023u)) & 1023u);
    uint8_t *A = X + kMatBytes, *B = A + kMatBytes;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = p.ctas, rank = blockIdx.x % ctas;
    const MuonMat& t = p.mat[blockIdx.x / ctas];
    const bool wide = t.rows <= t.cols;
    const uint32_t m = wide ? t.rows : t.cols, n = wide ? t.cols : t.rows;
    const uint32_t used = (n + kSide - 1) / kSide;  // CTAs with columns
    if (rank >= used) return;  // no barrier waits for a CTA that has left
    const uint32_t n0 = rank * kSide, width = min(kSide, n - n0);
    if (tid == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(muon_smem(&sh.done)), "r"(1u + p.hold) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.stop = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(muon_smem(&sh.tmem)), "r"(256u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_begin();

    // this CTA's columns, momentum and all, as fp32 in A's place
    uint8_t* S = A;
    const uint32_t prows = wide ? m : width, pcols = wide ? width : m;  // its part of the matrix as it lies
    const uint64_t first = wide ? n0 : (uint64_t)n0 * t.cols;
    const uint32_t per = (pcols + 7) / 8;
    if (m < kSide || width < kSide) {  // what is beyond the matrix is zero
        for (uint32_t k = tid; k < kSide * kSide / 4; k += kThreads) reinterpret_cast<float4*>(S)[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncthreads();
    }
    constexpr uint32_t kAtOnce = 4;  // pieces of eight a thread has on the way
    double squares = 0.0;
    muon_with_type(t.dtype, [&]<class Ty>() {
        const auto* g = static_cast<const typename Ty::T*>(t.g);
#pragma unroll 1
        for (uint32_t k0 = tid; k0 < prows * per; k0 += kAtOnce * kThreads) {
            float v[kAtOnce][8], mo[kAtOnce][8];
            uint32_t r[kAtOnce], c[kAtOnce], left[kAtOnce];
#pragma unroll
            for (uint32_t u = 0; u < kAtOnce; ++u) {
                const uint32_t k = k0 + u * kThreads;
                r[u] = k / per;
                c[u] = (k - r[u] * per) * 8;
                left[u] = r[u] < prows ? min(8u, pcols - c[u]) : 0;
                const uint64_t e = first + (uint64_t)r[u] * t.cols + c[u];
                muon_load8<Ty>(g + e, t.vec == 8, left[u], v[u]);
                if (t.m) muon_load8<F32T>(t.m + e, t.vec == 8, left[u], mo[u]);
            }
#pragma unroll
            for (uint32_t u = 0; u < kAtOnce; ++u) {
                if (left[u] == 0) continue;
                if (t.m) {
#pragma unroll
                    for (int l = 0; l < 8; ++l) {
                        mo[u][l] = __fmaf_rn(p.momentum, mo[u][l], v[u][l]);
                        v[u][l] = p.nesterov ? __fmaf_rn(p.momentum, mo[u][l], v[u][l]) : mo[u][l];
                    }
                    muon_store8<F32T>(t.m + first + (uint64_t)r[u] * t.cols + c[u], t.vec == 8, left[u], mo[u]);
                }
#pragma unroll
                for (int l = 0; l < 8; ++l)
                    if ((uint32_t)l >= left[u]) v[u][l] = 0.0f;
                squares += sum_squares(v[u]);
#pragma unroll
                for (int l = 0; l < 8; ++l)
                    if ((uint32_t)l < left[u]) *(wide ? word(S, r[u], c[u] + l) : word(S, c[u] + l, r[u])) = v[u][l];
            }
        }
    });
    squares = cta_sum(squares, sh.sums);
    cluster_sync();  // every CTA runs, so its shared memory may be written
    if (tid < used) *cluster_at(&sh.part[rank], tid) = squares;
    cluster_sync();
    double total = 0.0;
    for (uint32_t k = 0; k < used; ++k) total += sh.part[k];
    const MuonScale f = muon_scale(sqrt(total) + (double)p.eps, p.scale);
    const uint32_t row = tid % kSide, half = tid / kSide * 64;  // a thread's part of an m x 128 matrix, elementwise
#pragma unroll 1
    for (uint32_t c = half; c < half + 64; c += 32) {
        float v[32];
#pragma unroll
        for (int l = 0; l < 32; ++l) v[l] = *word(S, row, c + l) * f.a * f.b;
        if (p.steps > 0) {
            put_halves(X, row, c, v);
        } else {
#pragma unroll
            for (int l = 0; l < 32; ++l) *word(S, row, c + l) = v[l];
        }
    }

    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    Products pr{sh.tmem, &sh.done, 0, &sh.stop, p.waits, p.spin};
    const uint32_t xs = muon_smem(X), as = muon_smem(A), bs = muon_smem(B);
    const uint32_t quarter = warp & 3, arow = quarter * 32 + lane, acol = (warp >> 2) * 64;  // of an accumulator
    const uint32_t nk = (width + 63) / 64, mk = (m + 63) / 64;
    for (int step = 0; step < p.steps; ++step) {
        const MuonSmallStep s = p.step[step];
        pr.run(xs, false, xs, false, nk);  // X X^T
#pragma unroll 1
        for (uint32_t c = acol; c < acol + 64; c += 32) {
            float v[32];
            pr.sums(v, quarter, c, nk);
#pragma unroll
            for (int g = 0; g < 8; ++g) *quad(B, arow, c / 4 + g) = make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        }
        cluster_sync();
        // 16 rows at a time, of every CTA's sums, in the order of the CTAs: two
        // groups, four CTAs' values on the way (the summing and handing out takes 5 us
        // of a step's 14 in four CTAs: 112 KB a CTA between SMs)
#pragma unroll 1
        for (uint32_t group = rank; group < kSide / 16; group += 2 * used) {
            const uint32_t c = tid % 16 * 8;
            float v[2][8] = {};
#pragma unroll 1
            for (uint32_t k0 = 0; k0 < used; k0 += 4) {
                float4 x[2][4][2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) {
                        const uint32_t r = (group + u * used) * 16 + tid / 16;
                        x[u][k][0] = x[u][k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (k0 + k < used && r < kSide) {
                            uint8_t* const of = cluster_at(B, k0 + k);
                            x[u][k][0] = *quad(of, r, c / 4);
                            x[u][k][1] = *quad(of, r, c / 4 + 1);
                        }
                    }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            v[u][4 * h] += x[u][k][h].x;
                            v[u][4 * h + 1] += x[u][k][h].y;
                            v[u][4 * h + 2] += x[u][k][h].z;
                            v[u][4 * h + 3] += x[u][k][h].w;
                        }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t r = (group + u * used) * 16 + tid / 16;
                if (r >= kSide) continue;
                float w[8];
#pragma unroll
                for (int l = 0; l < 8; ++l) v[u][l] *= s.gram;
                const uint4 hi = F16T::pack(v[u]);
                F16T::unpack(hi, w);
#pragma unroll
                for (int l = 0; l < 8; ++l) w[l] = v[u][l] - w[l];
                const uint4 lo = F16T::pack(w);
                for (uint32_t k = 0; k < used; ++k) {
                    uint8_t* const of = cluster_at(A, k);
                    *piece(of, r, c) = hi;
                    *piece(of + kPlaneBytes, r, c) = lo;
                }
            }
        }
        cluster_sync();
        pr.run(as, false, as, false, mk);  // A A
#pragma unroll 1
        for (uint32_t c = acol; c < acol + 64; c += 32) {
            float v[32];
            pr.sums(v, quarter, c, mk);
            add_halves(A, arow, c, s.poly, s.poly_a, v);
            put_halves(B, arow, c, v);
        }
        pr.run(bs, false, xs, true, mk);  // B X
#pragma unroll 1
        for (uint32_t c = acol; c < acol + 64; c += 32) {
            float v[32];
            pr.sums(v, quarter, c, mk);
            add_halves(X, arow, c, s.apply, s.apply_x, v);
            if (step + 1 < p.steps) {
                put_halves(X, arow, c, v);
            } else {
#pragma unroll
                for (int l = 0; l < 32; ++l) *word(S, arow, c + l) = v[l];
            }
        }
    }
    __syncthreads();

    muon_with_type(t.out_dtype, [&]<class Ty>() {
        using T = typename Ty::T;
        // Rows that do not begin on 16 bytes: neighbours in neighbouring lanes where many
        // replicas are written (four layers of width 90, fp32, eight replicas: 121 -> 90
        // us), else eight a lane, which starts more loads at once (17 of 105, fp16, four
        // replicas: 208 -> 194).
        if (t.out_vec < 8 && p.nranks > 4) {
#pragma unroll 1
            for (uint32_t r0 = warp; r0 < prows; r0 += 4 * (kThreads / 32)) {
                float w[16];
#pragma unroll
                for (uint32_t k = 0; k < 16; ++k) {
                    const uint32_t r = r0 + k / 4 * (kThreads / 32), c = k % 4 * 32 + lane;
                    const bool in = r < prows && c < pcols;
                    w[k] = in && t.m ? Ty::ld1(static_cast<const T*>(p.out[t.out]) + first + (uint64_t)r * t.cols + c) : 0.0f;
                }
#pragma unroll
                for (uint32_t k = 0; k < 16; ++k) {
                    const uint32_t r = r0 + k / 4 * (kThreads / 32), c = k % 4 * 32 + lane;
                    if (r >= prows || c >= pcols) continue;
                    float v = *(wide ? word(S, r, c) : word(S, c, r)) * p.inv;
                    if (t.m) v = __fmaf_rn(-t.factor, v, p.keep * w[k]);
                    const uint64_t e = first + (uint64_t)r * t.cols + c;
                    for (int o = 0; o < p.nranks; ++o) Ty::st1(static_cast<T*>(p.out[t.out + o]) + e, v);
                }
            }
            return;
        }
#pragma unroll 1
        for (uint32_t k0 = tid; k0 < prows * per; k0 += kAtOnce * kThreads) {
            float w[kAtOnce][8];
            uint32_t r[kAtOnce], c[kAtOnce], left[kAtOnce];
#pragma unroll
            for (uint32_t u = 0; u < kAtOnce; ++u) {
                const uint32_t k = k0 + u * kThreads;
                r[u] = k / per;
                c[u] = (k - r[u] * per) * 8;
                left[u] = r[u] < prows ? min(8u, pcols - c[u]) : 0;
                if (t.m)  // weights: rank 0's, updated, to every rank
                    muon_load8<Ty>(static_cast<const T*>(p.out[t.out]) + first + (uint64_t)r[u] * t.cols + c[u], t.out_vec == 8, left[u], w[u]);
            }
#pragma unroll
            for (uint32_t u = 0; u < kAtOnce; ++u) {
                if (left[u] == 0) continue;
                float v[8];
#pragma unroll
                for (int l = 0; l < 8; ++l)
                    v[l] = (uint32_t)l < left[u] ? *(wide ? word(S, r[u], c[u] + l) : word(S, c[u] + l, r[u])) * p.inv : 0.0f;
                if (t.m) {
#pragma unroll
                    for (int l = 0; l < 8; ++l) v[l] = __fmaf_rn(-t.factor, v[l], p.keep * w[u][l]);
                }
                const uint64_t e = first + (uint64_t)r[u] * t.cols + c[u];
                for (int o = 0; o < p.nranks; ++o) muon_store8<Ty>(static_cast<T*>(p.out[t.out + o]) + e, t.out_vec == 8, left[u], v);
            }
        }
    });

    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (sh.stop && tid == 0) {  // a wait ran out: the products in flight end before their memory goes
        if (p.hold) asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(muon_smem(&sh.done)) : "memory");
        bool ended = false;
        for (uint32_t i = 0; i < p.spin && !ended; ++i) ended = muon_try_wait(muon_smem(&sh.done), pr.parity ^ 1);
        if (!ended) atomicAdd(&p.waits[1], 1u);
    }
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(256u) : "memory");
}

template <class P>
cudaError_t launch_as(const P& p, cudaStream_t s)
{
    const cudaError_t e = allow_smem<muon_small_kernel<P>>(kSmallSmem);
    return e != cudaSuccess ? e : launch_pdl_clusters(muon_small_kernel<P>, p.ctas * (unsigned)p.n, kThreads, kSmallSmem, p.ctas, s, p);
}

}  // namespace

cudaError_t launch_muon_small(MuonSmallParams& p, cudaStream_t s)
{
    RankParams rp{};
    rp.waits = bulk_wait_counters();
    if (!rp.waits) return cudaErrorSymbolNotFound;
    const BulkParams bp = bulk_params(rp);
    p.waits = rp.waits;
    p.hold = bp.hold;
    p.spin = bp.spin;
    if (p.n > kMuonMatsSmall || p.n * p.nranks > kMuonPtrsSmall) return launch_as(p, s);
    MuonSmallParamsT<kMuonMatsSmall, kMuonPtrsSmall> q;
    static_cast<MuonSmallHead&>(q) = p;
    std::copy_n(p.mat, p.n, q.mat);
    std::copy_n(p.out, p.n * p.nranks, q.out);
    return launch_as(q, s);
}

}  // namespace rr
