// rr_clip.cuh -- device pieces shared by the kernels that sum squares and by
// those that clip: the exact range of a sum of squares, the CTA's fp64 sum,
// the coefficient.
//
// The norm is sqrt(sum x^2).  Squares of fp32 values leave fp32's range where
// the norm itself does not (x = 1e30 or 1e-30), so a thread sums a few dozen
// squares in fp32 -- at most 64 terms, a relative error below 64 * 2^-24 of a
// term that the next level averages out -- and checks that sum: if it is not
// finite, or so small that a square could have been lost below fp32's range
// while some value is not zero, the same values are summed again in fp64.
// Everything above a thread's few dozen is fp64.
#pragma once

#include "rr_device.cuh"
#include "rr_internal.h"

namespace rr {

// Bulk store (a multiple of 16 bytes, shared to global, in the thread's bulk
// group) of bytes that L2 should evict before those the pass will still read.
__device__ __forceinline__ uint64_t evict_first_policy()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

__device__ __forceinline__ void bulk_store_last(void* to, uint32_t from, uint32_t bytes, uint64_t pol)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;"
                 ::"l"(to), "r"(from), "r"(bytes), "l"(pol) : "memory");
}

// A sum of at most 64 squares in fp32 is taken as it is when it is finite and
// at least 2^-96: a square lost below fp32's smallest normal number is below
// 2^-126, so 64 of them are below 2^-120, 2^-24 of the sum.
__device__ __forceinline__ bool squares_in_range(float s)
{
    return s >= 0x1p-96f && s <= 0x1.fffffep127f;
}

// Sum of the squares of N values given in fp32, exact in range.
template <int N>
__device__ __forceinline__ double sum_squares(const float (&a)[N])
{
    static_assert(N <= 64, "squares_in_range counts at most 64 terms");
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i & 3] = __fmaf_rn(a[i], a[i], s[i & 3]);
        big = fmaxf(big, fabsf(a[i]));  // 0 exactly where every value is (or is NaN: then the sum is too)
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    if (squares_in_range(t) || (t == 0.0f && big == 0.0f)) return (double)t;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) d = __fma_rn((double)a[i], (double)a[i], d);
    return d;
}

// The same for U whole vectors of a type, kept packed until they are summed.
template <class Ty, int U>
__device__ __forceinline__ double sum_squares_of(const uint4 (&raw)[U])
{
    constexpr int L = Ty::L;
    static_assert(U * L <= 64, "squares_in_range counts at most 64 terms");
    constexpr uint32_t kMagnitude = L == 8 ? 0x7fff7fffu : 0x7fffffffu;  // every bit but the signs
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t any = 0u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float a[L];
        Ty::unpack(raw[u], a);
#pragma unroll
        for (int l = 0; l < L; ++l) s[l & 3] = __fmaf_rn(a[l], a[l], s[l & 3]);
        any |= raw[u].x | raw[u].y | raw[u].z | raw[u].w;
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    if (squares_in_range(t) || (any & kMagnitude) == 0u) return (double)t;
    double d = 0.0;
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
        float a[L];
        uint4 r = raw[0];
#pragma unroll
        for (int k = 1; k < U; ++k)
            if (k == u) r = raw[k];  // a register array takes no run-time index
        Ty::unpack(r, a);
#pragma unroll
        for (int l = 0; l < L; ++l) d = __fma_rn((double)a[l], (double)a[l], d);
    }
    return d;
}

// The sum of v over the CTA's kThreads threads, in a fixed order, in every
// thread.  sh: kThreads / 32 doubles; the CTA must not be using them.
__device__ __forceinline__ double cta_sum(double v, double* sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += sh[w];
    return t;
}

// Sum of `count` partial sums, in the same order in every CTA.
__device__ __forceinline__ double partials_sum(const double* p, int64_t count, double* sh)
{
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) v += p[i];
    return cta_sum(v, sh);
}

// The clipping's coefficient: the product of two factors, of which the second
// is 1 unless the coefficient is below fp32's smallest normal number (a norm
// above 2^126 clipped to 1, say).  There one fp32 would keep few of its bits;
// the first factor keeps 24 and the second is the power of two.
struct Coef {
    float a, b;
};

__device__ __forceinline__ float scaled(float x, const Coef& c)
{
    return __fmul_rn(__fmul_rn(x, c.a), c.b);
}

// The norm into its word: see ClipArgs::lost.
__device__ __forceinline__ void write_norm(const ClipArgs& a, float norm)
{
    if (a.lost) atomicMax(reinterpret_cast<unsigned int*>(a.norm), __float_as_uint(norm) & 0x7fffffffu);
    else *a.norm = norm;
}

// A tile of the scaling was skipped: the norm says that the step is lost.
__device__ __forceinline__ void tile_lost(const ClipArgs& a)
{
    if (a.lost) atomicMax(reinterpret_cast<unsigned int*>(a.lost), 0x7fffffffu);
}

// The coefficient for a sum of squares, 1 where the norm is within max_norm
// and max_norm / (norm + eps) otherwise: 0 for an infinite norm, NaN for NaN.
// The norm counts in fp64, also where it is above fp32's largest number.  One
// thread writes it, where the launch is asked to.
__device__ __forceinline__ Coef coef_of(const ClipArgs& a, double squares)
{
    const double norm = sqrt(squares);
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) write_norm(a, (float)norm);
    const double den = norm + (double)a.eps;
    if (den <= (double)a.max_norm) return {1.0f, 1.0f};
    const double c = (double)a.max_norm / den;
    if (c < 0x1p-126) return {(float)(c * 0x1p126), 0x1p-126f};
    return {(float)c, 1.0f};
}

__device__ __forceinline__ Coef clip_coef(const ClipArgs& a, double* sh)
{
    return coef_of(a, partials_sum(a.partial, a.npartial, sh));
}

}  // namespace rr
