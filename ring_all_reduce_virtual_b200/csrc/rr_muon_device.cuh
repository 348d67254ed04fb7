// rr_muon_device.cuh -- device pieces shared by the kernels of the
// orthogonalisation and the Muon step: rows of eight values of any type, the
// normalisation's factor, the tensor cores' descriptors and instructions.
#pragma once

#include <cuda_fp16.h>

#include "rr_device.cuh"
#include "rr_muon.h"

namespace rr {

template <class F>
__device__ __forceinline__ void muon_with_type(int dtype, F&& f)
{
    switch (dtype) {
    case kF32: f.template operator()<F32T>(); break;
    case kBF16: f.template operator()<BF16T>(); break;
    default: f.template operator()<F16T>(); break;
    }
}

// Eight neighbouring values, whole vectors where vec says that every piece of
// eight lies on 16 bytes; `left` of them exist.
template <class Ty>
__device__ __forceinline__ void muon_load8(const typename Ty::T* p, bool vec, uint32_t left, float (&v)[8])
{
    if (vec && left >= 8) {
#pragma unroll
        for (int h = 0; h < 8 / Ty::L; ++h) {
            float a[Ty::L];
            Ty::unpack(*reinterpret_cast<const uint4*>(p + h * Ty::L), a);
#pragma unroll
            for (int l = 0; l < Ty::L; ++l) v[h * Ty::L + l] = a[l];
        }
    } else {
#pragma unroll
        for (int l = 0; l < 8; ++l) v[l] = (uint32_t)l < left ? Ty::ld1(p + l) : 0.0f;
    }
}

template <class Ty>
__device__ __forceinline__ void muon_store8(typename Ty::T* p, bool vec, uint32_t left, const float (&v)[8])
{
    if (vec && left >= 8) {
#pragma unroll
        for (int h = 0; h < 8 / Ty::L; ++h) {
            float a[Ty::L];
#pragma unroll
            for (int l = 0; l < Ty::L; ++l) a[l] = v[h * Ty::L + l];
            stv(p + h * Ty::L, Ty::pack(a));
        }
    } else {
#pragma unroll
        for (int l = 0; l < 8; ++l)
            if ((uint32_t)l < left) Ty::st1(p + l, v[l]);
    }
}

// W neighbouring values that lie on their common size.
template <class Ty, int W>
__device__ __forceinline__ void muon_load_few(const typename Ty::T* p, float (&v)[W])
{
    if constexpr (W == 1) {
        v[0] = Ty::ld1(p);
    } else if constexpr (sizeof(typename Ty::T) == 2) {
        Ty::unpack2(*reinterpret_cast<const uint32_t*>(p), v[0], v[1]);
    } else {
        const float2 a = *reinterpret_cast<const float2*>(p);
        v[0] = a.x;
        v[1] = a.y;
    }
}

template <class Ty, int W>
__device__ __forceinline__ void muon_store_few(typename Ty::T* p, const float (&v)[W])
{
    if constexpr (W == 1) Ty::st1(p, v[0]);
    else if constexpr (sizeof(typename Ty::T) == 2) *reinterpret_cast<uint32_t*>(p) = Ty::pack2(v[0], v[1]);
    else *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}

// scale / den as two factors that multiply a value one after the other: a power of
// two and one of 1..2, so that neither product leaves fp32's range where the
// result does not.  den is infinite or NaN where a value is (norms of fp32 values are
// within fp64's range): NaN for all of the matrix, also for what den alone would take to 0.
struct MuonScale {
    float a, b;
};

__device__ __forceinline__ MuonScale muon_scale(double den, float scale)
{
    if (!isfinite(den)) return {NAN, NAN};
    int ex = 0;
    const double frac = frexp(den, &ex);  // den = frac * 2^ex, frac in [0.5, 1)
    if (ex > -100 && ex < 100) return {ldexpf(1.0f, -ex) * scale, (float)(1.0 / frac)};
    return {ldexpf(1.0f, -ex / 2), ldexpf((float)(1.0 / frac), -(ex - ex / 2)) * scale};
}

// ------------------------------------------------------------ tensor cores

__device__ __forceinline__ uint32_t muon_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ bool muon_try_wait(uint32_t bar, uint32_t parity)
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

// Shared-memory descriptor of an operand in 128-byte-swizzled blocks: K along a
// block's columns (groups of 8 rows are 1024 bytes apart), or along its rows
// (groups of 8 of K 1024 bytes apart, of 64 of M or N `apart` bytes).
__device__ __forceinline__ uint64_t muon_operand(uint32_t addr, bool mn, uint32_t apart)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(mn ? apart >> 4 : 1u) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp16 operands, fp32 accumulator, m x n.
__device__ __forceinline__ uint32_t muon_instruction(uint32_t m, uint32_t n, bool a_mn, bool b_mn)
{
    return 1u << 4 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (n >> 3) << 17 | (m >> 4) << 24;
}

// 16 of K, by one CTA or (in the first of them) two.
template <int CTAS>
__device__ __forceinline__ void muon_mma(uint32_t acc, uint64_t a, uint64_t b, uint32_t inst, bool add)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
            "l"(a), "l"(b), "r"(inst), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
            "l"(a), "l"(b), "r"(inst), "r"((uint32_t)add)
            : "memory");
}

// 32 columns of the warp's 32 rows of an accumulator; there after muon_acc_landed.
__device__ __forceinline__ void muon_load_acc(uint32_t addr, uint32_t (&r)[32])
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
}

__device__ __forceinline__ void muon_acc_landed() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

}  // namespace rr
