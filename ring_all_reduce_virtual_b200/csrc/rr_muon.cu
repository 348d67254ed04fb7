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

// A warp's 4 rows x 64 columns, where lanes have eight neighbours each on one side
// (a piece of the blocks) and a row's neighbours lie in neighbouring lanes on the
// other: rows that do not begin on 16 bytes are read and written so (five layers of
// width 850, bf16, eight replicas: 2045 us, 600 less than with eight a lane everywhere;
// one of 288 and odd sides, fp32: 297, 166 less).
struct Rows4 {
    float v[4 * kBlk];

    __device__ __forceinline__ void put(int lane, const float (&a)[8])
    {
        reinterpret_cast<float4*>(v)[2 * lane] = make_float4(a[0], a[1], a[2], a[3]);
        reinterpret_cast<float4*>(v)[2 * lane + 1] = make_float4(a[4], a[5], a[6], a[7]);
    }
    __device__ __forceinline__ void get(int lane, float (&a)[8]) const
    {
        const float4 x = reinterpret_cast<const float4*>(v)[2 * lane], y = reinterpret_cast<const float4*>(v)[2 * lane + 1];
        a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w, a[4] = y.x, a[5] = y.y, a[6] = y.z, a[7] = y.w;
    }
};

// The updates of a warp's rows from r0 and columns from c0, W neighbours a lane.
template <class Ty, int W>
__device__ __forceinline__ void read_rows(const MuonPrepHead& p, const MuonMat& t, uint32_t r0, uint32_t c0, int lane, Rows4& rows)
{
    constexpr int kAll = 4 * (int)kBlk / (32 * W);
    float v[kAll][W], m[kAll][W];
#pragma unroll
    for (int k = 0; k < kAll; ++k) {
        const uint32_t at = (k * 32 + lane) * W, r = r0 + at / kBlk, c = c0 + at % kBlk;
        const uint64_t e = (uint64_t)r * t.cols + c;
        const bool in = r < t.rows && c < t.cols;
#pragma unroll
        for (int l = 0; l < W; ++l) v[k][l] = m[k][l] = 0.0f;
        if (in) muon_load_few<Ty, W>(static_cast<const typename Ty::T*>(t.g) + e, v[k]);
        if (in && t.m) muon_load_few<F32T, W>(t.m + e, m[k]);
    }
#pragma unroll
    for (int k = 0; k < kAll; ++k)
#pragma unroll
        for (int l = 0; l < W; ++l) rows.v[(k * 32 + lane) * W + l] = t.m ? updated(v[k][l], m[k][l], p) : v[k][l];
}

// A warp's rows into the outputs, W neighbours a lane.
template <class Ty, int W, class P>
__device__ __forceinline__ void write_rows(const P& p, const MuonMat& t, uint32_t r0, uint32_t c0, int lane, const Rows4& rows)
{
    using T = typename Ty::T;
    constexpr int kAll = 4 * (int)kBlk / (32 * W);
    float w[kAll][W];
#pragma unroll
    for (int k = 0; k < kAll; ++k) {
        const uint32_t at = (k * 32 + lane) * W, r = r0 + at / kBlk, c = c0 + at % kBlk;
        if (t.m && r < t.rows && c < t.cols) muon_load_few<Ty, W>(static_cast<const T*>(p.out[t.out]) + (uint64_t)r * t.cols + c, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kAll; ++k) {
        const uint32_t at = (k * 32 + lane) * W, r = r0 + at / kBlk, c = c0 + at % kBlk;
        if (r >= t.rows || c >= t.cols) continue;
#pragma unroll
        for (int l = 0; l < W; ++l) {
            const float o = rows.v[at + l];
            w[k][l] = t.m ? __fmaf_rn(-t.factor, o, p.keep * w[k][l]) : o;
        }
        for (int o = 0; o < p.nranks; ++o) muon_store_few<Ty, W>(static_cast<T*>(p.out[t.out + o]) + (uint64_t)r * t.cols + c, w[k]);
    }
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
    const bool flat = (((uintptr_t)t.g | (uintptr_t)t.m) & 15u) == 0;  // as one row, the matrix begins on 16 bytes
    double acc = 0.0;
    muon_with_type(t.dtype, [&]<class Ty>() {
        const auto* g = static_cast<const typename Ty::T*>(t.g);
        for (uint64_t at = (uint64_t)(blockIdx.x - t.part0) * kPrepTile; at < len; at += (uint64_t)t.parts * kPrepTile) {
#pragma unroll 1
            for (uint32_t u = 0; u < kPrepTile / (kThreads * 8); ++u) {
                const uint64_t e0 = at + (uint64_t)u * kThreads * 8, e = e0 + threadIdx.x * 8;
                if (e0 >= len) break;
                const uint32_t left = e < len ? (uint32_t)min((uint64_t)8, len - e) : 0;
                float v[8], m[8];
                if (flat) {
                    muon_load8<Ty>(g + e, true, left, v);
                    if (t.m) muon_load8<F32T>(t.m + e, true, left, m);
                } else {  // neighbours in neighbouring lanes
#pragma unroll
                    for (int l = 0; l < 8; ++l) {
                        const uint64_t k = e0 + l * kThreads + threadIdx.x;
                        v[l] = k < len ? Ty::ld1(g + k) : 0.0f;
                        m[l] = t.m && k < len ? t.m[k] : 0.0f;
                    }
                }
                if (t.m) {
#pragma unroll
                    for (int l = 0; l < 8; ++l) {
                        m[l] = __fmaf_rn(p.momentum, m[l], v[l]);
                        v[l] = updated(v[l], m[l], p);
                    }
                    if (flat) {
                        muon_store8<F32T>(t.m + e, true, left, m);
                    } else {
#pragma unroll
                        for (int l = 0; l < 8; ++l) {
                            const uint64_t k = e0 + l * kThreads + threadIdx.x;
                            if (k < len) t.m[k] = m[l];
                        }
                    }
                }
                acc += sum_squares(v);
            }
        }
    });
    acc = cta_sum(acc, sh);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = acc;
}

// 128 rows x 64 columns of X, split into halves.  ALL: every matrix's rows begin on
// 16 bytes; without the other code it takes 32 registers instead of 39 (one layer of
// width 2048, bf16: 79 and 85 us).
template <class P, bool ALL>
__global__ void __launch_bounds__(kThreads) muon_pack_kernel(const __grid_constant__ P p)
{
    __shared__ double sh[kThreads / 32];
    pdl_begin();
    const MuonMat& t = p.mat[mat_at(p, &MuonMat::tile0, blockIdx.x)];
    const uint32_t nbj = pad_up(t.cols) / kBlk;
    const uint32_t tile = blockIdx.x - t.tile0, ti = tile / nbj, tj = tile % nbj;
    __shared__ Rows4 rows[kThreads / 32];
    const int lane = threadIdx.x & 31;
    Rows4& mine = rows[threadIdx.x >> 5];
    const MuonScale f = muon_scale(sqrt(partials_sum(p.partial + t.part0, t.parts, sh)) + (double)p.eps, p.scale);
    muon_with_type(t.dtype, [&]<class Ty>() {
        const auto* g = static_cast<const typename Ty::T*>(t.g);
#pragma unroll 1
        for (uint32_t u = 0; u < 128 * 8 / kThreads; ++u) {
            const uint32_t k = u * kThreads + threadIdx.x;
            const uint32_t r = ti * 128 + k / 8, c = tj * kBlk + (k % 8) * 8;
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (!ALL && t.vec < 8) {
                if (t.vec == 2) read_rows<Ty, 2>(p, t, r - lane / 8, tj * kBlk, lane, mine);
                else read_rows<Ty, 1>(p, t, r - lane / 8, tj * kBlk, lane, mine);
                __syncwarp();
                mine.get(lane, v);
                __syncwarp();
            } else if (r < t.rows && c < t.cols) {  // whole pieces of eight
                const uint64_t e = (uint64_t)r * t.cols + c;
                muon_load8<Ty>(g + e, true, 8, v);
                if (t.m) {
                    float m[8];
                    muon_load8<F32T>(t.m + e, true, 8, m);
#pragma unroll
                    for (int l = 0; l < 8; ++l) v[l] = updated(v[l], m[l], p);
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

// 128 rows x 64 columns of the result.  ALL as above (31 registers and 64; 78 and
// 101 us).
template <class P, bool ALL>
__global__ void __launch_bounds__(kThreads) muon_finish_kernel(const __grid_constant__ P p)
{
    pdl_begin();
    const MuonMat& t = p.mat[mat_at(p, &MuonMat::tile0, blockIdx.x)];
    const uint32_t nbj = pad_up(t.cols) / kBlk;
    const uint32_t tile = blockIdx.x - t.tile0, ti = tile / nbj, tj = tile % nbj;
    __shared__ Rows4 rows[kThreads / 32];
    const int lane = threadIdx.x & 31;
    Rows4& mine = rows[threadIdx.x >> 5];
    muon_with_type(t.out_dtype, [&]<class Ty>() {
        using T = typename Ty::T;
#pragma unroll 1
        for (uint32_t u = 0; u < 128 * 8 / kThreads; ++u) {
            const uint32_t k = u * kThreads + threadIdx.x;
            const uint32_t r = ti * 128 + k / 8, c = tj * kBlk + (k % 8) * 8;
            const uint64_t at = piece_at(r, c, nbj), e = (uint64_t)r * t.cols + c;  // X is padded: there for every lane
            float h[8], l8[8];
            F16T::unpack(*reinterpret_cast<const uint4*>(t.x.hi + at), h);
            F16T::unpack(*reinterpret_cast<const uint4*>(t.x.lo + at), l8);
#pragma unroll
            for (int l = 0; l < 8; ++l) h[l] = (h[l] + l8[l]) * p.inv;
            if (!ALL && t.out_vec < 8) {
                mine.put(lane, h);
                __syncwarp();
                if (t.out_vec == 2) write_rows<Ty, 2>(p, t, r - lane / 8, tj * kBlk, lane, mine);
                else write_rows<Ty, 1>(p, t, r - lane / 8, tj * kBlk, lane, mine);
                __syncwarp();
                continue;
            }
            if (r >= t.rows || c >= t.cols) continue;
            if (t.m) {  // weights: rank 0's, updated, to every rank
                float w[8];
                muon_load8<Ty>(static_cast<const T*>(p.out[t.out]) + e, true, 8, w);
#pragma unroll
                for (int l = 0; l < 8; ++l) h[l] = __fmaf_rn(-t.factor, h[l], p.keep * w[l]);
            }
            for (int o = 0; o < p.nranks; ++o) muon_store8<Ty>(static_cast<T*>(p.out[t.out + o]) + e, true, 8, h);
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
    const bool all = std::all_of(p.mat, p.mat + p.n, [](const MuonMat& t) { return t.vec == 8; });
    return with_prep(p, [&]<class P>(const P& q) {
        return launch_pdl(all ? muon_pack_kernel<P, true> : muon_pack_kernel<P, false>, dim3(tiles), kThreads, 0, s, q);
    });
}

cudaError_t launch_muon_finish(const MuonFinishParams& p, uint32_t tiles, cudaStream_t s)
{
    const bool all = std::all_of(p.mat, p.mat + p.n, [](const MuonMat& t) { return t.out_vec == 8; });
    const auto launch = [&]<class P>(const P& q) {
        return launch_pdl(all ? muon_finish_kernel<P, true> : muon_finish_kernel<P, false>, dim3(tiles), kThreads, 0, s, q);
    };
    if (p.n > kMuonMatsSmall || p.n * p.nranks > kMuonPtrsSmall) return launch(p);
    using Few = MuonFinishParamsT<kMuonMatsSmall, kMuonPtrsSmall>;
    Few q;
    static_cast<MuonFinishHead&>(q) = p;
    std::copy_n(p.mat, p.n, q.mat);
    std::copy_n(p.out, p.n * p.nranks, q.out);
    return launch(q);
}

}  // namespace rr
