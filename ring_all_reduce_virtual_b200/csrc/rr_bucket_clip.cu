// rr_bucket_clip.cu -- the passes of the bucket sync with clipping.  Every
// pass reads every rank's gradients and folds them in fp32 in ring order (AVG
// divided), as the fused bucket sync does; the result a cannot be written
// before the global norm is known.  Two ways:
//
//   parked      the first pass parks a: an fp32 sum whole in rank 0's buffer,
//               for 16-bit gradients its upper half in rank 0's buffer and its
//               lower half in rank 1's -- the same elements the CTA has just
//               read, so no memory beside the gradients is needed and a is
//               not rounded to 16 bits before it is scaled; the scaling (rr_clip.cu) reads
//               the halves and writes every rank.  Traffic for N ranks of S
//               elements of e bytes: 2 (N + 1) S e, 16-bit types 2 (N + 2) S e.
//   folded      the first pass only sums the squares, the second folds again
//   twice       and writes round(c a) to every rank: 3 N S e.  For 2 and 3 ranks
//               of 16-bit gradients, where that is less: 1 GB of 2 / 3 bf16 ranks
//               453 / 472 us against 595 / 500 parked (4 ranks 454 and 451).
//
// A sync, a norm and a scaling one after the other move (4 N + 1) S e.  Each
// tile of a first pass leaves one fp64 partial sum of squares.
//
// Bound by HBM: 8 ranks x 267 Mi bf16, 747 us for the first pass (7.1 TB/s of 10 S e)
// and 800 for the scaling (6.7), where the copy peak is 6.55 TB/s.
#include "rr_bulk.cuh"
#include "rr_clip.cuh"
#include "rr_launch.cuh"

namespace rr {

namespace {

// Bytes of shared memory per CTA: the tiles of all ranks.  Measured against
// 16, 24 and 40 KB: 144 MB of 3 / 5 / 8 bf16 ranks 85.6 / 78.1 / 66.1 us with 16 KB,
// 76.3 / 68.2 / 60.9 with 32 KB (fewer, longer CTAs: short sets are bound by a
// CTA's latency), 40 KB as 32; 1 GB of 8 ranks 393 and 388 us.
constexpr uint32_t kParkBytes = 32768;
// And of the passes that fold twice: 48 / 144 MB / 1 GB of 3 bf16 ranks 31.2 / 77.1 /
// 473 us with 32 KB, 29.5 / 74.0 / 469 with 24; 2 ranks alike with both.
constexpr uint32_t kTwiceBytes = 24576;

enum FoldMode : int { kPark = 0, kSquares = 1, kScaled = 2 };

template <class Fold>
struct ParkParams {
    Fold f;              // BucketFoldParams or ParkSmallParams; tile0 counts tiles of park_tile_elems
    double* partial;     // kPark, kSquares: one per tile
    ClipArgs clip;       // kScaled: what the coefficient comes from; else norm: the word to zero, or NULL
    unsigned int* waits; // as BulkParams (rr_bulk.cuh)
    uint32_t hold;
    uint32_t spin;
    uint32_t tv;         // vectors per rank per tile
    uint32_t pad_;
};
static_assert(sizeof(ParkParams<BucketFoldParams>) <= 32764, "ParkParams too large");
static_assert(sizeof(ParkParams<ParkSmallParams>) <= 4064, "a small parameter block");

template <class G>
__device__ __forceinline__ void park_one(typename G::T* p0, typename G::T* p1, uint64_t e, float a)
{
    if constexpr (sizeof(typename G::T) == 2) {
        const uint32_t b = __float_as_uint(a);
        p0[e] = (uint16_t)(b >> 16);
        p1[e] = (uint16_t)b;
    } else {
        p0[e] = a;
    }
}

// A first pass zeroes the norm's word where it is given (ClipArgs::lost).
__device__ __forceinline__ void zero_norm(const ClipArgs& a)
{
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = 0.0f;
}

// Fold of element e: the same operations as the sync's, unrounded.
template <class G, int OP, class InF>
__device__ __forceinline__ float fold_value(const InF& in, int n, uint64_t e, float divisor)
{
    float a = G::ld1(in(0) + e);
    for (int j = 1; j < n; ++j) a = apply<OP>(a, G::ld1(in(j) + e));
    return finish<OP>(a, divisor);
}

// One element's result to where the pass puts it; its square.
template <class G, int MODE, class OutF>
__device__ __forceinline__ double settle_one(const OutF& out, int n, uint64_t e, float a, const Coef& c)
{
    if constexpr (MODE == kScaled) {
        const float x = scaled(a, c);
        for (int o = 0; o < n; ++o) G::st1(out(o) + e, x);
        return 0.0;
    } else {
        if constexpr (MODE == kPark) park_one<G>(out(0), out(1), e, a);
        const float x[1] = {a};
        return sum_squares(x);
    }
}

// Ranks whose copies of a tensor share a 16-byte phase: tiles staged by bulk
// copies as in the fused bucket sync (rr_bucket.cu); results leave by bulk
// stores from slot 0, parked lower halves from slot 1.  The second pass takes
// the tiles from the last to the first: L2 still holds what was touched last.
template <class G, int OP, int NS, int MODE, class Fold>
__global__ void __launch_bounds__(kThreads) bucket_park_kernel(const __grid_constant__ ParkParams<Fold> bp)
{
    using T = typename G::T;
    constexpr int L = G::L;
    constexpr bool kSplit = sizeof(T) == 2;
    pdl_begin();
    const Fold& p = bp.f;
    const int n = NS > 0 ? NS : p.n;
    const uint32_t TV = NS > 0 ? (MODE == kPark ? kParkBytes : kTwiceBytes) / (NS > 0 ? NS : 1) / 16 : bp.tv;
    if constexpr (MODE != kScaled) zero_norm(bp.clip);
    extern __shared__ __align__(128) uint4 sm[];  // [n][TV]: slot j holds rank (c + j) mod N
    __shared__ __align__(8) uint64_t bar;
    __shared__ double sh[kThreads / 32];

    const uint64_t w = MODE == kScaled ? p.tile0[p.nseg] - 1 - blockIdx.x : blockIdx.x;
    const int s = find_segment(p.tile0, p.nseg, w);
    const uint64_t tile = w - p.tile0[s];
    const BucketSeg& sg = p.seg[s];
    const int base = (int)sg.t * n;
    const int start = (int)sg.c;
    auto in = [&](int j) {
        int r = start + j;
        if (r >= n) r -= n;
        return static_cast<const T*>(p.grad[base + r]) + sg.off;
    };
    auto out = [&](int o) { return static_cast<T*>(p.grad[base + o]) + sg.off; };
    const uint64_t len = sg.len;
    uint64_t head = (uint64_t)((L - phase_of(in(0), L)) & (L - 1));
    if (head > len) head = len;
    const uint64_t nv = (len - head) / L;
    const uint64_t tail = len - head - nv * L;
    const uint64_t v0 = tile * TV;
    const bool staged = v0 < nv;
    const uint32_t nvt = (uint32_t)(nv - v0 < TV ? nv - v0 : TV);
    const uint32_t bytes = nvt * 16u;
    const uint64_t e0 = head + v0 * L;  // 16-byte aligned in every rank's copy
    const uint32_t b = bulk_smem_addr(&bar);
    if (threadIdx.x == 0 && staged) {
        bulk_bar_init(b, bp.hold);
        asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                     ::"r"(b), "r"(bytes * (uint32_t)n) : "memory");
#pragma unroll
        for (int j = 0; j < (NS > 0 ? NS : n); ++j)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                ::"r"(bulk_smem_addr(sm + j * TV)), "l"(in(j) + e0), "r"(bytes), "r"(b)
                : "memory");
    }
    // the barrier is set up before the other threads wait on it; the second
    // pass forms the coefficient meanwhile
    Coef c{};
    if constexpr (MODE == kScaled) c = clip_coef(bp.clip, sh);
    else __syncthreads();
    double acc = 0.0;
    if (tile == 0 && (uint64_t)threadIdx.x < head + tail) {
        const uint64_t e = (uint64_t)threadIdx.x < head ? (uint64_t)threadIdx.x : head + nv * L + (threadIdx.x - head);
        acc = settle_one<G, MODE>(out, n, e, fold_value<G, OP>(in, n, e, p.divisor), c);
    }
    if (staged) {
        if (!bulk_tile_landed(b, bp.waits, bp.hold, bp.spin)) {
            // the whole CTA skips the tile: a NaN norm says that the step is lost
            if (threadIdx.x == 0) {
                if constexpr (MODE == kScaled) tile_lost(bp.clip);
                else bp.partial[w] = __longlong_as_double(0x7ff8000000000000ll);
            }
            return;
        }
        for (uint32_t v = threadIdx.x; v < nvt; v += kThreads) {
            float a[L];
            G::unpack(sm[v], a);
#pragma unroll 4
            for (int j = 1; j < (NS > 0 ? NS : n); ++j) {
                float x[L];
                G::unpack(sm[j * TV + v], x);
#pragma unroll
                for (int l = 0; l < L; ++l) a[l] = apply<OP>(a[l], x[l]);
            }
#pragma unroll
            for (int l = 0; l < L; ++l) a[l] = finish_n<OP, NS>(a[l], p.divisor);
            if constexpr (MODE == kScaled) {
#pragma unroll
                for (int l = 0; l < L; ++l) a[l] = scaled(a[l], c);
                sm[v] = G::pack(a);
                continue;
            }
            acc += sum_squares(a);
            if constexpr (MODE == kSquares) continue;
            if constexpr (kSplit) {
                uint32_t h[4], q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t b0 = __float_as_uint(a[(2 * k) % L]), b1 = __float_as_uint(a[(2 * k + 1) % L]);
                    h[k] = __byte_perm(b0, b1, 0x7632);
                    q[k] = __byte_perm(b0, b1, 0x5410);
                }
                sm[v] = make_uint4(h[0], h[1], h[2], h[3]);
                sm[TV + v] = make_uint4(q[0], q[1], q[2], q[3]);
            } else {
                sm[v] = G::pack(a);
            }
        }
        if constexpr (MODE != kSquares) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            if (threadIdx.x == 0) {
                const int nout = MODE == kScaled ? n : kSplit ? 2 : 1;
                for (int o = 0; o < nout; ++o)
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                                 ::"l"(out(o) + e0), "r"(bulk_smem_addr(sm + (MODE == kPark ? o * TV : 0))), "r"(bytes)
                                 : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        if constexpr (MODE != kScaled) acc = cta_sum(acc, sh);
        if (threadIdx.x == 0) {
            if constexpr (MODE != kScaled) bp.partial[w] = acc;
            if constexpr (MODE != kSquares) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            bulk_bar_inval(b);
        }
        return;
    }
    if constexpr (MODE != kScaled) {
        acc = cta_sum(acc, sh);
        if (threadIdx.x == 0) bp.partial[w] = acc;
    }
}

// Any ranks: element by element.
template <class G, int OP, int MODE, class Fold>
__global__ void __launch_bounds__(kThreads) bucket_park_any_kernel(const __grid_constant__ ParkParams<Fold> bp)
{
    using T = typename G::T;
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    if constexpr (MODE != kScaled) zero_norm(bp.clip);
    const Fold& p = bp.f;
    const int n = p.n;
    const Coef c = MODE == kScaled ? clip_coef(bp.clip, sh) : Coef{};
    const uint64_t w = MODE == kScaled ? p.tile0[p.nseg] - 1 - blockIdx.x : blockIdx.x;
    const int s = find_segment(p.tile0, p.nseg, w);
    const BucketSeg& sg = p.seg[s];
    const int base = (int)sg.t * n, start = (int)sg.c;
    auto in = [&](int j) {
        int r = start + j;
        if (r >= n) r -= n;
        return static_cast<const T*>(p.grad[base + r]) + sg.off;
    };
    auto out = [&](int o) { return static_cast<T*>(p.grad[base + o]) + sg.off; };
    const uint64_t te = (uint64_t)bp.tv * G::L, lo = (w - p.tile0[s]) * te;
    const uint64_t hi = sg.len < lo + te ? sg.len : lo + te;
    double acc = 0.0;
    for (uint64_t e = lo + threadIdx.x; e < hi; e += kThreads) {
        acc += settle_one<G, MODE>(out, n, e, fold_value<G, OP>(in, n, e, p.divisor), c);
    }
    if constexpr (MODE != kScaled) {
        acc = cta_sum(acc, sh);
        if (threadIdx.x == 0) bp.partial[w] = acc;
    }
}

template <class G, int OP, int MODE, class Fold>
cudaError_t park_sized(const ParkParams<Fold>& bp, cudaStream_t s)
{
    const int n = bp.f.n;
    const unsigned work = (unsigned)bp.f.tile0[bp.f.nseg];
    auto go = [&](void (*kernel)(ParkParams<Fold>), uint32_t smem) {
        return launch_pdl(kernel, dim3(work), kThreads, smem, s, bp);
    };
    if (!bp.f.vec_ok || !bp.waits) return go(bucket_park_any_kernel<G, OP, MODE, Fold>, 0);
    // compiled rank counts of the calls that get here (clip_folds_twice)
    if constexpr (MODE != kPark) {
        if (n == 2) return go(bucket_park_kernel<G, OP, 2, MODE, Fold>, kTwiceBytes);
        if (n == 3) return go(bucket_park_kernel<G, OP, 3, MODE, Fold>, kTwiceBytes);
        return cudaErrorInvalidValue;
    } else {
        switch (n) {
        case 2:
            if constexpr (sizeof(typename G::T) == 4) return go(bucket_park_kernel<G, OP, 2, MODE, Fold>, kParkBytes);
            break;
        case 4: return go(bucket_park_kernel<G, OP, 4, MODE, Fold>, kParkBytes);
        case 8: return go(bucket_park_kernel<G, OP, 8, MODE, Fold>, kParkBytes);
        case 16: return go(bucket_park_kernel<G, OP, 16, MODE, Fold>, kParkBytes);
        }
        return go(bucket_park_kernel<G, OP, 0, MODE, Fold>, bp.tv * 16u * (uint32_t)n);
    }
}

// The launch's table, as it is or as a small one.
inline void copy_table(BucketFoldParams& to, const BucketFoldParams& f, int) { to = f; }

inline void copy_table(ParkSmallParams& to, const BucketFoldParams& f, int ntensors)
{
    for (int i = 0; i < ntensors * f.n; ++i) to.grad[i] = f.grad[i];
    to.tile0[0] = 0;
    for (int i = 0; i < f.nseg; ++i) {
        to.seg[i] = f.seg[i];
        to.tile0[i + 1] = f.tile0[i + 1];
    }
    to.n = f.n;
    to.nseg = f.nseg;
    to.vec_ok = f.vec_ok;
    to.divisor = f.divisor;
}

template <int MODE, class Fold>
cudaError_t launch_table(int grad_dtype, int op, const BucketFoldParams& f, int ntensors, double* partial,
                         const ClipArgs& clip, cudaStream_t s)
{
    RankParams rp{};
    rp.waits = bulk_wait_counters();
    const BulkParams wait = bulk_params(rp, MODE == kScaled);
    ParkParams<Fold> bp;
    copy_table(bp.f, f, ntensors);
    bp.partial = partial;
    bp.clip = clip;
    bp.waits = wait.waits;
    bp.hold = wait.hold;
    bp.spin = wait.spin;
    bp.tv = (MODE == kPark ? kParkBytes : kTwiceBytes) / (uint32_t)f.n / 16u;
    bp.pad_ = 0;
    const bool avg = op == kAvg;
    switch (grad_dtype) {
    case kF32:
        if constexpr (MODE != kPark) return cudaErrorInvalidValue;  // fp32 is parked
        else return avg ? park_sized<F32T, kAvg, MODE>(bp, s) : park_sized<F32T, kSum, MODE>(bp, s);
    case kBF16: return avg ? park_sized<BF16T, kAvg, MODE>(bp, s) : park_sized<BF16T, kSum, MODE>(bp, s);
    case kF16: return avg ? park_sized<F16T, kAvg, MODE>(bp, s) : park_sized<F16T, kSum, MODE>(bp, s);
    }
    return cudaErrorInvalidValue;
}

template <int MODE>
cudaError_t launch_pass(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, double* partial,
                        const ClipArgs& clip, cudaStream_t s)
{
    if (p.tile0[p.nseg] > kMaxGrid || p.n < 2) return cudaErrorInvalidValue;
    if (p.nseg <= kParkSegsSmall && ntensors * p.n <= kParkPtrsSmall)
        return launch_table<MODE, ParkSmallParams>(grad_dtype, op, p, ntensors, partial, clip, s);
    return launch_table<MODE, BucketFoldParams>(grad_dtype, op, p, ntensors, partial, clip, s);
}

}  // namespace

uint64_t park_tile_elems(int grad_dtype, int n)
{
    const uint32_t bytes = clip_folds_twice(n, grad_dtype) ? kTwiceBytes : kParkBytes;
    return (uint64_t)(bytes / (uint32_t)n / 16u) * (grad_dtype == kF32 ? 4u : 8u);
}

bool clip_folds_twice(int n, int grad_dtype) { return n <= 3 && grad_dtype != kF32; }

cudaError_t launch_bucket_park(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, double* partial,
                               float* clear, cudaStream_t s)
{
    ClipArgs a{};
    a.norm = clear;
    return launch_pass<kPark>(grad_dtype, op, p, ntensors, partial, a, s);
}

cudaError_t launch_bucket_squares(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, double* partial,
                                  float* clear, cudaStream_t s)
{
    ClipArgs a{};
    a.norm = clear;
    return launch_pass<kSquares>(grad_dtype, op, p, ntensors, partial, a, s);
}

cudaError_t launch_bucket_scaled(int grad_dtype, int op, const BucketFoldParams& p, int ntensors, const ClipArgs& clip,
                                 cudaStream_t s)
{
    return launch_pass<kScaled>(grad_dtype, op, p, ntensors, nullptr, clip, s);
}

}  // namespace rr
