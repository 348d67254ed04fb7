// rr_clip_small.cu -- norm and clipping of a small set in one launch: a cluster
// of 8 CTAs reads the gradients once, keeps the values in registers, adds up
// the squares through distributed shared memory and writes the scaled values.
// For sets whose values fit the cluster's registers (262144 elements) and
// whose ranks' copies share a 16-byte phase per tensor.
//
// Bound by latency and by the host: the norm of 14 fp32 tensors of 50 k
// elements, call after call, 12.2 us in two launches and 10.1 in this one (its
// kernel runs 5.3 us against 2.4 + 1.8).  The clipped bucket sync keeps its two
// launches: folding on 8 SMs took 18 us for 4 ranks x 200 k fp32, the two grids 7.
#include "rr_clip.cuh"

namespace rr {

namespace {

constexpr int kSmallThreads = 1024;
constexpr int kSmallCtas = 8;

// Vectors per thread: 32 values in registers.
template <class Ty>
constexpr int kHeld = 32 / Ty::L;

struct SmallParams {
    ParkSmallParams f;  // tile0: prefix sums of the segments' whole vectors
    ClipArgs clip;
    int scale;          // 0: the norm alone
    int pad_;
};
static_assert(sizeof(SmallParams) <= 4064, "a small parameter block");

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <class Ty>
__global__ void __launch_bounds__(kSmallThreads) clip_small_kernel(const __grid_constant__ SmallParams sp)
{
    using T = typename Ty::T;
    constexpr int L = Ty::L, R = kHeld<Ty>;
    __shared__ double warps[kSmallThreads / 32];
    __shared__ double mine;  // this CTA's sum, which the others read
    pdl_begin();
    const ParkSmallParams& p = sp.f;
    const uint32_t tid = threadIdx.x, me = blockIdx.x;  // the grid is one cluster
    const int n = p.n;
    const uint32_t total = (uint32_t)p.tile0[p.nseg], per = (total + kSmallCtas - 1) / kSmallCtas;
    // vector j of this thread: its segment and first element, or false
    auto locate = [&](int j, int& s, uint64_t& e) {
        const uint32_t k = (uint32_t)j * kSmallThreads + tid, g = me * per + k;
        if (k >= per || g >= total) return false;
        s = find_segment(p.tile0, p.nseg, g);
        const BucketSeg& sg = p.seg[s];
        const T* q = static_cast<const T*>(p.grad[(int)sg.t * n]) + sg.off;
        uint64_t head = (uint64_t)((L - phase_of(q, L)) & (L - 1));
        if (head > sg.len) head = sg.len;
        e = sg.off + head + (g - p.tile0[s]) * L;
        return true;
    };
    auto copy = [&](int s, int r) { return static_cast<T*>(p.grad[(int)p.seg[s].t * n + r]); };
    float a[R][L];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        int s;
        uint64_t e;
#pragma unroll
        for (int l = 0; l < L; ++l) a[j][l] = 0.0f;
        if (!locate(j, s, e)) continue;
        Ty::unpack(*reinterpret_cast<const uint4*>(copy(s, 0) + e), a[j]);
    }
    // the elements around the segments' whole vectors: at most 2 (L - 1) of each, one a thread of the last CTA
    static_assert(kParkSegsSmall * 2 * 8 <= kSmallThreads);
    const int es = (int)tid / (2 * L);
    uint64_t edge = 0;
    bool has_edge = false;
    float b[1] = {0.0f};
    if (me == kSmallCtas - 1 && es < p.nseg) {
        const BucketSeg& sg = p.seg[es];
        const T* q = static_cast<const T*>(p.grad[(int)sg.t * n]) + sg.off;
        uint64_t head = (uint64_t)((L - phase_of(q, L)) & (L - 1));
        if (head > sg.len) head = sg.len;
        const uint64_t nv = (sg.len - head) / L, k = tid % (2 * L);
        has_edge = k < sg.len - nv * L;
        edge = sg.off + (k < head ? k : nv * L + k);
        if (has_edge) b[0] = Ty::ld1(copy(es, 0) + edge);
    }
    double v = sum_squares(b);
    {
        float flat[R * L];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int l = 0; l < L; ++l) flat[j * L + l] = a[j][l];
        v += sum_squares(flat);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((tid & 31u) == 0) warps[tid >> 5] = v;
    __syncthreads();
    if (tid == 0) {
        double t = 0.0;
        for (int w = 0; w < kSmallThreads / 32; ++w) t += warps[w];
        mine = t;
    }
    __syncthreads();
    cluster_barrier();
    double sum = 0.0;
    for (uint32_t c = 0; c < kSmallCtas; ++c) {
        uint32_t at;
        double x;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&mine)), "r"(c));
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(x) : "r"(at) : "memory");
        sum += x;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA has read the others' sums
    const Coef c = coef_of(sp.clip, sum);
    if (sp.scale) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            int s;
            uint64_t e;
            if (!locate(j, s, e)) continue;
#pragma unroll
            for (int l = 0; l < L; ++l) a[j][l] = scaled(a[j][l], c);
            const uint4 out = Ty::pack(a[j]);
            for (int r = 0; r < n; ++r) *reinterpret_cast<uint4*>(copy(s, r) + e) = out;
        }
        if (has_edge)
            for (int r = 0; r < n; ++r) Ty::st1(copy(es, r) + edge, scaled(b[0], c));
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no CTA leaves before its sum was read
}

template <class Ty>
cudaError_t small_typed(const SmallParams& p, cudaStream_t s)
{
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSmallCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kSmallCtas);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, clip_small_kernel<Ty>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool clip_small_plan(int dtype, ParkSmallParams& p, int ntensors)
{
    const int L = dtype == kF32 ? 4 : 8;
    const uintptr_t es = dtype == kF32 ? 4 : 2;
    for (int t = 0; t < ntensors; ++t)
        for (int r = 1; r < p.n; ++r)
            if (((uintptr_t)p.grad[t * p.n + r] & 15u) != ((uintptr_t)p.grad[t * p.n] & 15u)) return false;
    p.tile0[0] = 0;
    for (int s = 0; s < p.nseg; ++s) {
        const BucketSeg& sg = p.seg[s];
        const uint64_t at = (uintptr_t)p.grad[(int)sg.t * p.n] / es + sg.off;
        uint64_t head = (uint64_t)((L - (int)(at % (uint64_t)L)) % L);
        if (head > sg.len) head = sg.len;
        p.tile0[s + 1] = p.tile0[s] + (sg.len - head) / (uint64_t)L;
    }
    return p.tile0[p.nseg] <= (uint64_t)kSmallCtas * kSmallThreads * (32 / L);
}

cudaError_t launch_clip_small(int dtype, bool scale, const ParkSmallParams& f, const ClipArgs& clip, cudaStream_t s)
{
    SmallParams p{};
    p.f = f;
    p.clip = clip;
    p.scale = scale;
    switch (dtype) {
    case kF32: return small_typed<F32T>(p, s);
    case kBF16: return small_typed<BF16T>(p, s);
    case kF16: return small_typed<F16T>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace rr
