// rr_muon.cu -- the elementwise passes of the orthogonalisation and the Muon
// step: momentum and norm, the normalised matrix as blocked halves, and the
// result into the outputs or every replica's weights.
//
//   M <- momentum * M + G        u = G + momentum * M (Nesterov) or M
//   X = u / (||u||_F + eps)      (orthogonalize: u is the matrix itself)
//   O = the products' result     W_r <- (1 - lr * decay) * W_0 - lr * f * O
//
// All bound by HBM, and short against the products: of 4 layers of width 2048
// (201 M elements) they move 12 + 4 bytes and more an element.  The norm is
// summed as the gradient norm is (rr_clip.cuh: right over fp32's range, fp64
// partial sums joined in a fixed order).
#include <algorithm>

#include <cuda_fp16.h>

#include "rr_clip.cuh"
#include "rr_launch.cuh"
#include "rr_muon.h"
#include "rr_muon_device.cuh"

namespace rr {

namespace {

// The last matrix that begins (a partial sum, or a tile) at `at` or before.
template <class P>
__device__ __forceinline__ int mat_at(const P& p, uint32_t MuonMat::*begin, uint32_t at)
{
    int low = 0, high = p.n;
    while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (p.mat[mid].*begin <= at) low = mid;
        else high = mid;
    }
    return low;
}

__device__ __forceinline__ float updated(float g, float m, const MuonPrepHead& p)
{
    return p.nesterov ? __fmaf_rn(p.momentum, m, g) : m;
}

// One CTA per partial sum: the tiles of its matrix part, part + parts, ...
template <class P>
__global__ void __launch_bounds__(kThreads) muon_squares_kernel(const __grid_constant__ P p)
{
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    if (blockIdx.x == 0 && threadIdx.x < kMuonCounters) p.counters[threadIdx.x] = 0;
    const MuonMat& t = p.mat[mat_at(p, &MuonMat::part0, blockIdx.x)];
    const uint64_t len = (uint64_t)t.rows * t.cols;
    double acc = 0.0;
    muon_with_type(t.dtype, [&]<class Ty>() {
        const auto* g = static_cast<const typename Ty::T*>(t.g);
        for (uint64_t at = (uint64_t)(blockIdx.x - t.part0) * kPrepTile; at < len; at += (uint64_t)t.parts * kPrepTile) {
#pragma unroll 1
            for (uint32_t u = 0; u < kPrepTile / (kThreads * 8); ++u) {
                const uint64_t e = at + ((uint64_t)u * kThreads + threadIdx.x) * 8;
                if (e >= len) break;
                const uint32_t left = (uint32_t)min((uint64_t)8, len - e);
                float v[8];
                muon_load8<Ty>(g + e, t.vec, left, v);
                if (t.m) {
                    float m[8];
                    muon_load8<F32T>(t.m + e, t.vec, left, m);
#pragma unroll
                    for (int l = 0; l < 8; ++l) {
                        m[l] = __fmaf_rn(p.momentum, m[l], v[l]);
                        v[l] = updated(v[l], m[l], p);
                    }
                    muon_store8<F32T>(t.m + e, t.vec, left, m);
                }
                acc += sum_squares(v);
            }
        }
    });
    acc = cta_sum(acc, sh);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = acc;
}

// 128 rows x 64 columns of X, split into halves.
template <class P>
__global__ void __launch_bounds__(kThreads) muon_pack_kernel(const __grid_constant__ P p)
{
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    const MuonMat& t = p.mat[mat_at(p, &MuonMat::tile0, blockIdx.x)];
    const uint32_t nbj = pad_up(t.cols) / kBlk;
    const uint32_t tile = blockIdx.x - t.tile0, ti = tile / nbj, tj = tile % nbj;
    const MuonScale f = muon_scale(sqrt(partials_sum(p.partial + t.part0, t.parts, sh)) + (double)p.eps, p.scale);
    muon_with_type(t.dtype, [&]<class Ty>() {
        const auto* g = static_cast<const typename Ty::T*>(t.g);
#pragma unroll 1
        for (uint32_t u = 0; u < 128 * 8 / kThreads; ++u) {
            const uint32_t k = u * kThreads + threadIdx.x;
            const uint32_t r = ti * 128 + k / 8, c = tj * kBlk + (k % 8) * 8;
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (r < t.rows && c < t.cols) {
                const uint64_t e = (uint64_t)r * t.cols + c;
                const uint32_t left = min(8u, t.cols - c);
                muon_load8<Ty>(g + e, t.vec, left, v);
                if (t.m) {
                    float m[8];
                    muon_load8<F32T>(t.m + e, t.vec, left, m);
#pragma unroll
                    for (int l = 0; l < 8; ++l) v[l] = (uint32_t)l < left ? updated(v[l], m[l], p) : 0.0f;
                }
            }
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const float a = v[2 * l] * f.a * f.b, b = v[2 * l + 1] * f.a * f.b;
                const __half ah = __float2half_rn(a), bh = __float2half_rn(b);
                hw[l] = F16T::pack2(a, b);
                lw[l] = F16T::pack2(a - __half2float(ah), b - __half2float(bh));
            }
            const uint64_t at = piece_at(r, c, nbj);
            *reinterpret_cast<uint4*>(t.x.hi + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(t.x.lo + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
    });
}

// 128 rows x 64 columns of the result.
template <class P>
__global__ void __launch_bounds__(kThreads) muon_finish_kernel(const __grid_constant__ P p)
{
    pdl_begin();
    const MuonMat& t = p.mat[mat_at(p, &MuonMat::tile0, blockIdx.x)];
    const uint32_t nbj = pad_up(t.cols) / kBlk;
    const uint32_t tile = blockIdx.x - t.tile0, ti = tile / nbj, tj = tile % nbj;
    muon_with_type(t.out_dtype, [&]<class Ty>() {
        using T = typename Ty::T;
#pragma unroll 1
        for (uint32_t u = 0; u < 128 * 8 / kThreads; ++u) {
            const uint32_t k = u * kThreads + threadIdx.x;
            const uint32_t r = ti * 128 + k / 8, c = tj * kBlk + (k % 8) * 8;
            if (r >= t.rows || c >= t.cols) continue;
            const uint64_t at = piece_at(r, c, nbj), e = (uint64_t)r * t.cols + c;
            const uint32_t left = min(8u, t.cols - c);
            float h[8], l8[8];
            F16T::unpack(*reinterpret_cast<const uint4*>(t.x.hi + at), h);
            F16T::unpack(*reinterpret_cast<const uint4*>(t.x.lo + at), l8);
#pragma unroll
            for (int l = 0; l < 8; ++l) h[l] = (h[l] + l8[l]) * p.inv;
            if (t.m) {  // weights: rank 0's, updated, to every rank
                float w[8];
                muon_load8<Ty>(static_cast<const T*>(p.out[t.out]) + e, t.out_vec, left, w);
#pragma unroll
                for (int l = 0; l < 8; ++l) h[l] = __fmaf_rn(-t.factor, h[l], p.keep * w[l]);
            }
            for (int o = 0; o < p.nranks; ++o) muon_store8<Ty>(static_cast<T*>(p.out[t.out + o]) + e, t.out_vec, left, h);
        }
    });
}

// f on the parameters of few matrices, or on all.
template <class F>
cudaError_t with_prep(const MuonPrepParams& p, F&& f)
{
    if (p.n > kMuonMatsSmall) return f(p);
    MuonPrepParamsT<kMuonMatsSmall> q;
    static_cast<MuonPrepHead&>(q) = p;
    std::copy_n(p.mat, p.n, q.mat);
    return f(q);
}

}  // namespace

cudaError_t launch_muon_squares(const MuonPrepParams& p, uint32_t parts, cudaStream_t s)
{
    return with_prep(p, [&]<class P>(const P& q) { return launch_pdl(muon_squares_kernel<P>, dim3(parts), kThreads, 0, s, q); });
}

cudaError_t launch_muon_pack(const MuonPrepParams& p, uint32_t tiles, cudaStream_t s)
{
    return with_prep(p, [&]<class P>(const P& q) { return launch_pdl(muon_pack_kernel<P>, dim3(tiles), kThreads, 0, s, q); });
}

cudaError_t launch_muon_finish(const MuonFinishParams& p, uint32_t tiles, cudaStream_t s)
{
    if (p.n > kMuonMatsSmall || p.n * p.nranks > kMuonPtrsSmall)
        return launch_pdl(muon_finish_kernel<MuonFinishParams>, dim3(tiles), kThreads, 0, s, p);
    using Few = MuonFinishParamsT<kMuonMatsSmall, kMuonPtrsSmall>;
    Few q;
    static_cast<MuonFinishHead&>(q) = p;
    std::copy_n(p.mat, p.n, q.mat);
    std::copy_n(p.out, p.n * p.nranks, q.out);
    return launch_pdl(muon_finish_kernel<Few>, dim3(tiles), kThreads, 0, s, q);
}

}  // namespace rr
