// rr_clip.cu -- the global gradient norm over many tensors, and clipping by
// it: one pass that reads every tensor and leaves a few hundred fp64 partial
// sums of squares, and one that sums those, forms the coefficient and writes
// the scaled gradients to every rank.
//
//   norm    ||g|| = sqrt(sum over tensors t and elements i of g_t[i]^2)
//   clip    c = 1 if ||g|| + eps <= max_norm else max_norm / (||g|| + eps);
//           g_r[i] = round(c * g_0[i]) on every rank r: c and the product in
//           fp32, then the rounding to the tensor's type
//
// Both are bound by HBM.  The norm of 735 MB of bf16 takes 107 us, 6.9 TB/s (a copy
// moves 6.55).  Clipping 4 replicas of 104 MB of fp16 (519 MB written and read
// once) takes 97 us, of one rank's 50 MB of fp32 25 us: the second pass finds part
// of the values in L2, but the first one shares HBM with the write-back of what
// the program wrote before.  Partial sums are joined in a fixed order (no
// atomics), so a call's bits depend only on its tensors.
#include "rr_bulk.cuh"
#include "rr_clip.cuh"
#include "rr_launch.cuh"

namespace rr {

namespace {

// 16-byte vectors per thread per tile of the norm: 32 KB a tile (4: 735 MB in 112.7
// us against 110, and with 8 CTAs per SM 114.8), and of the scaling: 16 KB of one
// rank's copy.
constexpr int kNormU = 8;
constexpr int kScaleU = 4;

__device__ __forceinline__ uint4 ld_keep(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// The squares of one tile of one tensor, as this thread's share.
template <class Ty>
__device__ __forceinline__ double tile_squares(const typename Ty::T* p, uint64_t len, uint64_t tile)
{
    constexpr int L = Ty::L;
    constexpr uint64_t TV = (uint64_t)kThreads * kNormU;
    const uint64_t tid = threadIdx.x;
    uint64_t head = (uint64_t)((L - phase_of(p, L)) & (L - 1));
    if (head > len) head = len;
    const uint64_t nv = (len - head) / L, tail = len - head - nv * L;
    double acc = 0.0;
    if (tile == 0 && tid < head + tail) {
        const float x[1] = {Ty::ld1(p + (tid < head ? tid : head + nv * L + (tid - head)))};
        acc = sum_squares(x);
    }
    const uint64_t v0 = tile * TV + tid;
    uint4 raw[kNormU];
#pragma unroll
    for (int u = 0; u < kNormU; ++u) {
        const uint64_t v = v0 + (uint64_t)u * kThreads;
        raw[u] = v < nv ? ld_keep(p + head + v * L) : make_uint4(0u, 0u, 0u, 0u);
    }
    return acc + sum_squares_of<Ty>(raw);
}

// The CTAs sweep the tiles together (each on one run of consecutive tiles: 104 MB
// 20.5 us against 19.2, 735 MB 109.3 against 107.3); a CTA's next tile is in the
// same tensor or one behind it.
template <class Ty, int CAP>
__global__ void __launch_bounds__(kThreads, 4) norm_kernel(const __grid_constant__ NormParamsT<CAP> p)
{
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.clear = 0.0f;
    const uint64_t total = p.tile0[p.nt];
    double acc = 0.0;
    int t = find_segment(p.tile0, p.nt, blockIdx.x);
    for (uint64_t w = blockIdx.x; w < total; w += gridDim.x) {
        while (w >= p.tile0[t + 1]) ++t;
        acc += tile_squares<Ty>(static_cast<const typename Ty::T*>(p.ptr[t]), p.len[t], w - p.tile0[t]);
    }
    acc = cta_sum(acc, sh);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = acc;
}

// Many partials to kJoinCtas: CTA b sums the b-th run of them.
__global__ void __launch_bounds__(kThreads) norm_join_kernel(const double* in, int64_t count, double* out)
{
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    const int64_t lo = count * blockIdx.x / gridDim.x, hi = count * (blockIdx.x + 1) / gridDim.x;
    const double v = partials_sum(in + lo, hi - lo, sh);
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const __grid_constant__ ClipArgs a)
{
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    clip_coef(a, sh);
}

// The two fp32 values whose upper halves are the word h and lower halves the
// word l.
__device__ __forceinline__ void unpark2(uint32_t h, uint32_t l, float& x, float& y)
{
    x = __uint_as_float(__byte_perm(l, h, 0x5410));
    y = __uint_as_float(__byte_perm(l, h, 0x7632));
}

// Rank 0's copy, scaled, into every rank's.  PARKED (16-bit types): the value
// is the fp32 whose upper half rank 0's copy holds and whose lower half rank
// 1's does.  A thread reads its elements of both before it writes any copy.
// The tiles run from the last to the first: what the pass before touched last
// is what L2 still holds.
template <class Ty, bool PARKED, int CAP, int PTRS>
__global__ void __launch_bounds__(kThreads, 4) clip_scale_kernel(const __grid_constant__ ScaleParamsT<CAP, PTRS> p)
{
    using T = typename Ty::T;
    constexpr int L = Ty::L;
    constexpr uint64_t TV = (uint64_t)kThreads * kScaleU;
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    Coef c{};
    const uint64_t total = p.tile0[p.nt], tid = threadIdx.x;
    const int n = p.n;
    for (uint64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const uint64_t w = total - 1 - i;
        const int t = find_segment(p.tile0, p.nt, w);
        const uint64_t tile = w - p.tile0[t], len = p.len[t];
        T* const* ptr = reinterpret_cast<T* const*>(&p.ptr[(size_t)t * n]);
        const T* src = ptr[0];
        const T* low = PARKED ? ptr[1] : ptr[0];
        uint64_t head = (uint64_t)((L - phase_of(src, L)) & (L - 1));
        if (head > len) head = len;
        const uint64_t nv = p.vec[t] ? (len - head) / L : 0, tail = len - head - nv * L;
        const uint64_t v0 = tile * TV + tid;
        uint4 raw[kScaleU], lo[PARKED ? kScaleU : 1];
#pragma unroll
        for (int u = 0; u < kScaleU; ++u) {
            const uint64_t v = v0 + (uint64_t)u * kThreads;
            if (v < nv) {
                raw[u] = ld_keep(src + head + v * L);
                if constexpr (PARKED) lo[u] = ld_keep(low + head + v * L);
            }
        }
        if (i == blockIdx.x) c = clip_coef(p.clip, sh);  // while the first tile is on the way
        auto one = [&](uint64_t e) {
            float x;
            if constexpr (PARKED) x = __uint_as_float(((uint32_t)src[e] << 16) | (uint32_t)low[e]);
            else x = Ty::ld1(src + e);
            x = scaled(x, c);
            for (int o = 0; o < n; ++o) Ty::st1(ptr[o] + e, x);
        };
        if (!p.vec[t]) {
            const uint64_t e0 = tile * TV * L;
            for (uint64_t e = e0 + tid; e < len && e < e0 + TV * L; e += kThreads) one(e);
            continue;
        }
        if (tile == 0 && tid < head + tail) one(tid < head ? tid : head + nv * L + (tid - head));
#pragma unroll
        for (int u = 0; u < kScaleU; ++u) {
            float a[L];
            if constexpr (PARKED) {
                unpark2(raw[u].x, lo[u].x, a[0], a[1]);
                unpark2(raw[u].y, lo[u].y, a[2], a[3]);
                unpark2(raw[u].z, lo[u].z, a[4], a[5]);
                unpark2(raw[u].w, lo[u].w, a[6], a[7]);
            } else {
                Ty::unpack(raw[u], a);
            }
#pragma unroll
            for (int l = 0; l < L; ++l) a[l] = scaled(a[l], c);
            raw[u] = Ty::pack(a);
        }
        for (int o = 0; o < n; ++o) {
            T* q = ptr[o] + head;
#pragma unroll
            for (int u = 0; u < kScaleU; ++u) {
                const uint64_t v = v0 + (uint64_t)u * kThreads;
                if (v < nv) stv(q + v * L, raw[u]);
            }
        }
    }
}

// The scaling of large sets: one CTA per tile, the tile (two of them where the
// values are parked in halves) brought to shared memory and sent to every
// rank by bulk copies, as the one-shot all-reduce moves its tiles.  Every CTA
// forms the coefficient while its tile is on the way.  Tensors whose copies are
// at different 16-byte phases run element by element.
struct ScaleBulkParams {
    ScaleParams s;       // tile0 counts tiles of kBulkScaleBytes in all
    unsigned int* waits; // as BulkParams (rr_bulk.cuh)
    uint32_t hold;
    uint32_t spin;
};
static_assert(sizeof(ScaleBulkParams) <= 32764, "ScaleBulkParams too large");
// Of shared memory per CTA: 4 replicas of 104 MB 104 / 105 / 115 us with 8 / 16 / 24
// KB (32 as 24), 50 MB in place 30 / 27 / 29.
constexpr uint32_t kBulkScaleBytes = 16384;

template <class Ty, bool PARKED>
__global__ void __launch_bounds__(kThreads) clip_bulk_kernel(const __grid_constant__ ScaleBulkParams bp)
{
    using T = typename Ty::T;
    constexpr int L = Ty::L;
    constexpr uint32_t TV = kBulkScaleBytes / 16 / (PARKED ? 2 : 1);
    extern __shared__ __align__(128) uint4 sm[];
    __shared__ __align__(8) uint64_t bar;
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    const ScaleParams& p = bp.s;
    const int n = p.n;
    const uint64_t w = p.tile0[p.nt] - 1 - blockIdx.x;  // last tiles first: L2 still holds what was touched last
    const int t = find_segment(p.tile0, p.nt, w);
    const uint64_t tile = w - p.tile0[t], len = p.len[t];
    T* const* ptr = reinterpret_cast<T* const*>(&p.ptr[(size_t)t * n]);
    const T* src = ptr[0];
    const T* low = PARKED ? ptr[1] : ptr[0];
    uint64_t head = (uint64_t)((L - phase_of(src, L)) & (L - 1));
    if (head > len) head = len;
    const uint64_t nv = (len - head) / L, tail = len - head - nv * L;
    const uint64_t v0 = tile * TV;
    const bool staged = p.vec[t] && v0 < nv;
    const uint32_t nvt = (uint32_t)(nv - v0 < TV ? nv - v0 : TV), bytes = nvt * 16u;
    const uint64_t e0 = head + v0 * L;
    const uint32_t b = bulk_smem_addr(&bar);
    if (threadIdx.x == 0 && staged) {
        bulk_bar_init(b, bp.hold);  // the others wait on it only after clip_coef's barrier
        asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                     ::"r"(b), "r"(bytes * (PARKED ? 2u : 1u)) : "memory");
#pragma unroll
        for (int k = 0; k < (PARKED ? 2 : 1); ++k)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         ::"r"(bulk_smem_addr(sm + k * TV)), "l"((k ? low : src) + e0), "r"(bytes), "r"(b)
                         : "memory");
    }
    const Coef c = clip_coef(p.clip, sh);
    auto one = [&](uint64_t e) {
        float x;
        if constexpr (PARKED) x = __uint_as_float(((uint32_t)src[e] << 16) | (uint32_t)low[e]);
        else x = Ty::ld1(src + e);
        x = scaled(x, c);
        for (int o = 0; o < n; ++o) Ty::st1(ptr[o] + e, x);
    };
    if (!p.vec[t]) {
        const uint64_t at = tile * TV * L;
        for (uint64_t e = at + threadIdx.x; e < len && e < at + TV * L; e += kThreads) one(e);
        return;
    }
    if (tile == 0 && threadIdx.x < head + tail)
        one(threadIdx.x < head ? threadIdx.x : head + nv * L + (threadIdx.x - head));
    if (!staged) return;
    if (!bulk_tile_landed(b, bp.waits, bp.hold, bp.spin)) {  // the whole CTA skips the tile
        if (threadIdx.x == 0) tile_lost(p.clip);
        return;
    }
    for (uint32_t v = threadIdx.x; v < nvt; v += kThreads) {
        float a[L];
        if constexpr (PARKED) {
            const uint4 h = sm[v], q = sm[TV + v];
            unpark2(h.x, q.x, a[0], a[1]);
            unpark2(h.y, q.y, a[2], a[3]);
            unpark2(h.z, q.z, a[4], a[5]);
            unpark2(h.w, q.w, a[6], a[7]);
        } else {
            Ty::unpack(sm[v], a);
        }
#pragma unroll
        for (int l = 0; l < L; ++l) a[l] = scaled(a[l], c);
        sm[v] = Ty::pack(a);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint64_t pol = evict_first_policy();
        for (int o = 0; o < n; ++o) {
            if (!PARKED && p.clip.in_l2) bulk_store_last(ptr[o] + e0, bulk_smem_addr(sm), bytes, pol);
            else
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                             ::"l"(ptr[o] + e0), "r"(bulk_smem_addr(sm)), "r"(bytes)
                             : "memory");
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        bulk_bar_inval(b);
    }
}

// The same table with fewer entries: a short list's parameter block.
template <class Small>
Small shrink(const NormParams& p)
{
    Small q{};
    for (int t = 0; t < p.nt; ++t) {
        q.ptr[t] = p.ptr[t];
        q.len[t] = p.len[t];
        q.tile0[t + 1] = p.tile0[t + 1];
    }
    q.partial = p.partial;
    q.clear = p.clear;
    q.nt = p.nt;
    return q;
}

template <class Ty>
cudaError_t norm_typed(const NormParams& p, unsigned grid, cudaStream_t s)
{
    if (p.nt <= kNormTensorsSmall)
        return launch_pdl(norm_kernel<Ty, kNormTensorsSmall>, dim3(grid), kThreads, 0, s, shrink<NormParamsT<kNormTensorsSmall>>(p));
    return launch_pdl(norm_kernel<Ty, kNormTensors>, dim3(grid), kThreads, 0, s, p);
}

template <class Ty, bool PARKED>
cudaError_t scale_typed(const ScaleParams& p, unsigned grid, cudaStream_t s)
{
    if (p.nt <= kScaleTensorsSmall && p.nt * p.n <= kScalePtrsSmall) {
        ScaleParamsT<kScaleTensorsSmall, kScalePtrsSmall> q{};
        for (int i = 0; i < p.nt * p.n; ++i) q.ptr[i] = p.ptr[i];
        for (int t = 0; t < p.nt; ++t) {
            q.len[t] = p.len[t];
            q.tile0[t + 1] = p.tile0[t + 1];
            q.vec[t] = p.vec[t];
        }
        q.clip = p.clip;
        q.n = p.n;
        q.nt = p.nt;
        return launch_pdl(clip_scale_kernel<Ty, PARKED, kScaleTensorsSmall, kScalePtrsSmall>, dim3(grid), kThreads, 0, s, q);
    }
    return launch_pdl(clip_scale_kernel<Ty, PARKED, kScaleTensors, kScalePtrs>, dim3(grid), kThreads, 0, s, p);
}

template <class Ty, bool PARKED>
cudaError_t bulk_typed(const ScaleParams& p, unsigned grid, cudaStream_t s)
{
    RankParams rp{};
    rp.waits = bulk_wait_counters();
    if (!rp.waits) return cudaErrorInvalidValue;
    const BulkParams wait = bulk_params(rp, true);
    ScaleBulkParams bp;
    bp.s = p;
    bp.waits = wait.waits;
    bp.hold = wait.hold;
    bp.spin = wait.spin;
    return launch_pdl(clip_bulk_kernel<Ty, PARKED>, dim3(grid), kThreads, kBulkScaleBytes, s, bp);
}

}  // namespace

uint64_t norm_tile_elems(int dtype) { return (uint64_t)kThreads * kNormU * (dtype == kF32 ? 4u : 8u); }
uint64_t scale_tile_elems(int dtype, bool parked, bool bulk)
{
    const uint64_t vecs = bulk ? kBulkScaleBytes / 16 / (parked && dtype != kF32 ? 2 : 1) : (uint64_t)kThreads * kScaleU;
    return vecs * (dtype == kF32 ? 4u : 8u);
}

cudaError_t launch_norm(int dtype, const NormParams& p, int* slots, cudaStream_t s)
{
    const uint64_t work = p.tile0[p.nt];
    const unsigned grid = (unsigned)(work < kNormCtas ? work : kNormCtas);
    *slots = (int)grid;
    if (grid == 0) return cudaSuccess;
    switch (dtype) {
    case kF32: return norm_typed<F32T>(p, grid, s);
    case kBF16: return norm_typed<BF16T>(p, grid, s);
    case kF16: return norm_typed<F16T>(p, grid, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_norm_join(const double* in, int64_t count, double* out, int* slots, cudaStream_t s)
{
    *slots = kJoinCtas;
    return launch_pdl(norm_join_kernel, dim3(kJoinCtas), kThreads, 0, s, in, count, out);
}

cudaError_t launch_norm_finish(const ClipArgs& a, cudaStream_t s) { return launch_pdl(norm_finish_kernel, dim3(1), kThreads, 0, s, a); }

cudaError_t launch_clip_scale(int dtype, bool parked, bool bulk, const ScaleParams& p, cudaStream_t s)
{
    const uint64_t work = p.tile0[p.nt];
    if (work == 0) return cudaSuccess;
    if (bulk) {
        if (work > kMaxGrid) return cudaErrorInvalidValue;
        switch (dtype) {
        case kF32: return bulk_typed<F32T, false>(p, (unsigned)work, s);
        case kBF16:
            return parked ? bulk_typed<BF16T, true>(p, (unsigned)work, s)
                          : bulk_typed<BF16T, false>(p, (unsigned)work, s);
        case kF16:
            return parked ? bulk_typed<F16T, true>(p, (unsigned)work, s)
                          : bulk_typed<F16T, false>(p, (unsigned)work, s);
        }
        return cudaErrorInvalidValue;
    }
    const unsigned grid = (unsigned)(work < kNormCtas ? work : kNormCtas);
    switch (dtype) {
    case kF32: return scale_typed<F32T, false>(p, grid, s);  // fp32 sums are parked whole, in rank 0's buffers
    case kBF16: return parked ? scale_typed<BF16T, true>(p, grid, s) : scale_typed<BF16T, false>(p, grid, s);
    case kF16: return parked ? scale_typed<F16T, true>(p, grid, s) : scale_typed<F16T, false>(p, grid, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace rr
