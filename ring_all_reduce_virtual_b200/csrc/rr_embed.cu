// rr_embed.cu -- the embedding's two data-parallel steps: the lookup of every
// rank's tokens, and the gradient of the table summed over all ranks' tokens.
//
//   lookup    out_r[t, :] = round(scale * W_r[id_r[t], :])
//   gradient  dW[v, :] = f * sum over (r, t) with id_r[t] = v of dout_r[t, :]
//             f = scale, over the rank count for AVG
//
// The gradient of a step is row-sparse: M = ranks x tokens rows land on at
// most M of V table rows.  It is summed without atomics: the positions (r, t)
// are sorted by token id (stable, so a token's rows stay in rank and token
// order), the sorted list is cut into blocks of K positions, a warp sums the
// runs of equal ids inside a block for a slice of the columns, and runs that
// cross blocks are joined from their partial sums in block order.  Which terms
// are added in which order depends on the ids alone, so the bits repeat.
//
// Ids outside [0, V) have no row: the lookup gives zeros, the gradient skips
// them (they sort behind every row, as id V).
//
// Both are bound by HBM.  Lookup: 8 x 2048 bf16 rows of 2048 (101 MB) in 17.9 us, 5.6
// TB/s.  Gradient: 8 x 2048 tokens into eight bf16 tables of 32000 x 2048 (1.11 GB)
// in 188 us, 5.9 TB/s: 14 for the sort, 47 for the sums, 127 (at 6.6 TB/s) for
// the rows without a token; 8 x 8192 tokens onto one fp32 table (470 MB) in 105
// us: 16, 77 and 11 for the joins.  A sort by a cluster of 8 CTAs in one launch,
// the keys in distributed shared memory, took 18 us for 16384 tokens and 37 for
// 65536, where the three launches take 14 and 16.
#include "rr_launch.cuh"
#include "rr_search.h"

namespace rr {

namespace {

// VEC consecutive elements of a type as one access (two for 32 bytes).
template <class Ty, int VEC>
struct Vec {
    using T = typename Ty::T;
    static constexpr int B = VEC * (int)sizeof(T), W = B < 4 ? 1 : B / 4;
    uint32_t r[W];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (B == 2) r[0] = *reinterpret_cast<const uint16_t*>(p);
        else if constexpr (B == 4) r[0] = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (B == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            r[0] = v.x;
            r[1] = v.y;
        } else {
#pragma unroll
            for (int k = 0; k < W; k += 4) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[k / 4];
                r[k] = v.x;
                r[k + 1] = v.y;
                r[k + 2] = v.z;
                r[k + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (B == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)r[0];
        else if constexpr (B == 4) *reinterpret_cast<uint32_t*>(p) = r[0];
        else if constexpr (B == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
        else {
#pragma unroll
            for (int k = 0; k < W; k += 4)
                reinterpret_cast<uint4*>(p)[k / 4] = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
        }
    }
    __device__ __forceinline__ void to_f(float (&a)[VEC]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int l = 0; l < VEC; ++l) a[l] = __uint_as_float(r[l]);
        } else if constexpr (VEC == 1) {
            float hi;
            Ty::unpack2(r[0], a[0], hi);
        } else {
#pragma unroll
            for (int l = 0; l < VEC; l += 2) Ty::unpack2(r[l / 2], a[l], a[l + 1]);
        }
    }
    __device__ __forceinline__ void from_f(const float (&a)[VEC])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int l = 0; l < VEC; ++l) r[l] = __float_as_uint(a[l]);
        } else if constexpr (VEC == 1) {
            r[0] = Ty::pack2(a[0], 0.0f);
        } else {
#pragma unroll
            for (int l = 0; l < VEC; l += 2) r[l / 2] = Ty::pack2(a[l], a[l + 1]);
        }
    }
};

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, uint32_t i)
{
    return ids64 ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
}

// ------------------------------------------------------------------ lookup

// Accesses per lane: 2 KB of a 16-byte aligned row per warp.  2 / 4 / 8: 8 x 2048
// rows of 4 KB in 18.2 / 18.1 / 18.0 us; 4 splits a single token's row over 2 warps.
constexpr int kLookupU = 4;

// A warp copies one slice of one token's row.
template <class Ty, int VEC>
__global__ void __launch_bounds__(kThreads) embed_lookup_kernel(const __grid_constant__ EmbedLookupParams p)
{
    using T = typename Ty::T;
    pdl_begin();
    const uint32_t row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31u;
    if (row >= p.M) return;
    const uint32_t r = row / p.T, t = row - r * p.T;
    const int64_t id = load_id(p.ids[r], p.ids64, t);
    const bool inside = id >= 0 && (uint64_t)id < p.V;
    const T* src = static_cast<const T*>(p.table[r]) + (inside ? (uint64_t)id * p.D : 0);
    T* dst = static_cast<T*>(p.out[r]) + (uint64_t)t * p.D;
    const uint32_t c0 = (blockIdx.y * 32u * kLookupU + lane) * VEC;
    Vec<Ty, VEC> v[kLookupU];
#pragma unroll
    for (int u = 0; u < kLookupU; ++u) {
        const uint32_t c = c0 + (uint32_t)u * 32u * VEC;
#pragma unroll
        for (int w = 0; w < Vec<Ty, VEC>::W; ++w) v[u].r[w] = 0u;
        if (inside && c < p.D) v[u].load(src + c);
    }
#pragma unroll
    for (int u = 0; u < kLookupU; ++u) {
        const uint32_t c = c0 + (uint32_t)u * 32u * VEC;
        float a[VEC];
        v[u].to_f(a);
#pragma unroll
        for (int l = 0; l < VEC; ++l) a[l] = inside ? __fmul_rn(a[l], p.scale) : 0.0f;
        v[u].from_f(a);
        if (c < p.D) v[u].store(dst + c);
    }
}

// -------------------------------------------------------------------- sort

// The sort key of position i: its token id, or V for an id without a row.
__device__ __forceinline__ uint32_t position_key(const EmbedGradParams& p, uint32_t i)
{
    const uint32_t r = i / p.T;
    const int64_t id = load_id(p.ids[r], p.ids64, i - r * p.T);
    return id >= 0 && (uint64_t)id < p.V && id != p.padding ? (uint32_t)id : (uint32_t)p.V;
}

constexpr int kWarps = kThreads / 32;

// Up to kRankMax tokens: every position's place is the number of positions
// with a smaller id, or the same id and an earlier place in the list.  Every
// CTA reads all the ids; kRankParts threads share a position's comparisons.
constexpr int kRankThreads = 128, kRankParts = 4;

__global__ void __launch_bounds__(kRankThreads) embed_rank_kernel(const __grid_constant__ EmbedGradParams p)
{
    __shared__ __align__(16) uint32_t keys[kRankMax];
    pdl_begin();
    const uint32_t M = p.M, padded = (M + 15u) & ~15u;
    if (blockIdx.x == 0)
        for (uint32_t c = threadIdx.x; c * kEmbedCols < p.D; c += kRankThreads) p.arrived[c] = 0u;
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < padded; i += kRankThreads) keys[i] = i < M ? position_key(p, i) : 0xffffffffu;
    __syncthreads();
    const uint32_t i = blockIdx.x * (kRankThreads / kRankParts) + threadIdx.x / kRankParts;
    const uint32_t key = i < M ? keys[i] : 0u;
    uint32_t place = 0;
    const uint4* v4 = reinterpret_cast<const uint4*>(keys);
#pragma unroll 4
    for (uint32_t v = threadIdx.x % kRankParts; v < padded / 4; v += kRankParts) {
        const uint4 k = v4[v];
        const uint32_t than = v < i / 4 ? key + 1u : key;  // equal ids in front count, equal ids behind do not
        place += (k.x < than) + (k.y < than) + (k.z < than) + (k.w < than);
    }
    place += __shfl_xor_sync(0xffffffffu, place, 1);
    place += __shfl_xor_sync(0xffffffffu, place, 2);
    if (i >= M || threadIdx.x % kRankParts) return;
    for (uint32_t e = i & ~3u; e < i; ++e) place += keys[e] == key;  // the vector that i is in
    p.key[0][place] = key;
    p.pos[0][place] = i;
}

// More tokens: least-significant-digit radix sort, a launch that counts the
// first digit and one per digit that places; pass k reads buffer
// (passes - k) & 1 and writes the other, so the last pass writes buffer 0.  A tile is kSortTile consecutive keys.
// The first launch counts every tile's keys per digit, tile by tile, writes
// the keys down, and clears the later digits' counts; each placing adds the
// next digit's counts of the tiles that it fills (whole numbers: any order of
// the atomics gives the same).
constexpr int kSortRounds = (int)kSortTile / kThreads;  // keys per thread

__global__ void __launch_bounds__(kThreads) embed_count_kernel(const __grid_constant__ EmbedGradParams p)
{
    __shared__ uint32_t hist[1 << kSortMaxBits];
    pdl_begin();
    const uint32_t digits = 1u << p.bits, from = (uint32_t)p.passes & 1u;
    const uint64_t table = (uint64_t)p.ntiles * digits;
    for (uint32_t d = threadIdx.x; d < digits; d += kThreads) hist[d] = 0;
    const uint32_t i0 = blockIdx.x * kSortTile + threadIdx.x;
    uint32_t key[kSortRounds];
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const uint32_t i = i0 + (uint32_t)j * kThreads;
        if (i < p.M) key[j] = position_key(p, i);
    }
    for (int later = 1; later < p.passes; ++later)
        for (uint32_t d = threadIdx.x; d < digits; d += kThreads)
            p.counts[(uint64_t)later * table + (uint64_t)blockIdx.x * digits + d] = 0u;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const uint32_t i = i0 + (uint32_t)j * kThreads;
        if (i >= p.M) continue;
        p.key[from][i] = key[j];
        atomicAdd(&hist[key[j] & (digits - 1)], 1u);
    }
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < digits; d += kThreads) p.counts[(uint64_t)blockIdx.x * digits + d] = hist[d];
}

// First place of every digit's keys: an exclusive scan over the digits of
// their totals, one digit per thread (digits <= blockDim.x * 2; a thread has
// the digits 2t and 2t + 1).
__device__ __forceinline__ void scan_digits(uint32_t (&v)[2], uint32_t* sums)
{
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    uint32_t x = v[0] + v[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= (uint32_t)o) x += y;
    }
    if (lane == 31u) sums[warp] = x;
    __syncthreads();
    uint32_t first = x - v[0] - v[1];
    for (uint32_t w = 0; w < warp; ++w) first += sums[w];
    v[1] = first + v[0];
    v[0] = first;
}

// Many tiles: one CTA turns the counts into every tile's first places.
__global__ void __launch_bounds__(kThreads) embed_scan_kernel(const __grid_constant__ EmbedGradParams p, int pass)
{
    __shared__ uint32_t sums[kWarps];
    pdl_begin();
    const uint32_t digits = 1u << p.bits, d = threadIdx.x * 2;
    uint32_t* counts = p.counts + (uint64_t)pass * p.ntiles * digits;
    uint32_t v[2] = {0, 0};
    if (d < digits)
#pragma unroll 8
        for (uint32_t t = 0; t < p.ntiles; ++t) {
            const uint2 c = *reinterpret_cast<const uint2*>(counts + (uint64_t)t * digits + d);
            v[0] += c.x;
            v[1] += c.y;
        }
    scan_digits(v, sums);
    if (d < digits)
#pragma unroll 8
        for (uint32_t t = 0; t < p.ntiles; ++t) {
            uint2* at = reinterpret_cast<uint2*>(counts + (uint64_t)t * digits + d);
            const uint2 c = *at;
            *at = make_uint2(v[0], v[1]);
            v[0] += c.x;
            v[1] += c.y;
        }
}

// Placing, stable: a warp takes consecutive keys, 32 at a time; lanes with
// the same digit rank themselves by lane, behind the warp's earlier ones, and
// the warps' counts stack in warp order.  A tile's first places come from the
// scan, or -- few tiles -- from the counts themselves, which every CTA sums.
template <bool SCANNED>
__global__ void __launch_bounds__(kThreads) embed_place_kernel(const __grid_constant__ EmbedGradParams p, int pass)
{
    __shared__ __align__(16) uint32_t cnt[kWarps][1 << kSortMaxBits];
    __shared__ __align__(16) uint32_t ahead_of[SCANNED ? 1 : kWarps][1 << kSortMaxBits];
    __shared__ uint32_t sums[kWarps];
    pdl_begin();
    const uint32_t digits = 1u << p.bits, shift = (uint32_t)(pass * p.bits), from = (uint32_t)(p.passes - pass) & 1u;
    const uint32_t* counts = p.counts + (uint64_t)pass * p.ntiles * digits;
    uint32_t* later = p.counts + (uint64_t)(pass + 1) * p.ntiles * digits;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t i0 = blockIdx.x * kSortTile + warp * (kSortTile / kWarps);
    uint32_t key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const uint32_t i = i0 + (uint32_t)j * 32u + lane;
        if (i < p.M) {
            key[j] = p.key[from][i];
            pos[j] = pass == 0 ? i : p.pos[from][i];
        }
    }
    // this tile's first place of the digits 2t and 2t + 1
    const uint32_t d2 = threadIdx.x * 2;
    uint32_t first[2] = {0, 0};
    if constexpr (SCANNED) {
        if (d2 < digits) {
            first[0] = counts[(uint64_t)blockIdx.x * digits + d2];
            first[1] = counts[(uint64_t)blockIdx.x * digits + d2 + 1];
        }
    } else {
        // a warp adds up every eighth tile's counts, four digits per lane and
        // access, four tiles in flight; the warps' sums meet in shared memory
        // (cnt is not in use yet)
        constexpr int Q = (1 << kSortMaxBits) / 128, U = 4;
        const uint32_t dl = min(lane * 4u, digits - 4u);  // fewer than 128 digits: the last lanes repeat and are not kept
        uint4 tot[Q], bef[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) tot[q] = bef[q] = make_uint4(0u, 0u, 0u, 0u);
        for (uint32_t t0 = warp; t0 < p.ntiles; t0 += kWarps * U) {
            uint4 c[U][Q];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t t = min(t0 + (uint32_t)u * kWarps, p.ntiles - 1u);
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    if ((uint32_t)q * 128u < digits)
                        c[u][q] = *reinterpret_cast<const uint4*>(counts + (uint64_t)t * digits + (uint32_t)q * 128u + dl);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t t = t0 + (uint32_t)u * kWarps;
                if (t >= p.ntiles) break;
                const bool before = t < blockIdx.x;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    if ((uint32_t)q * 128u >= digits) break;
                    const uint4 v = c[u][q];
                    tot[q] = make_uint4(tot[q].x + v.x, tot[q].y + v.y, tot[q].z + v.z, tot[q].w + v.w);
                    if (before) bef[q] = make_uint4(bef[q].x + v.x, bef[q].y + v.y, bef[q].z + v.z, bef[q].w + v.w);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint32_t d = (uint32_t)q * 128u + lane * 4u;
            if (d >= digits) continue;
            *reinterpret_cast<uint4*>(&cnt[warp][d]) = tot[q];
            *reinterpret_cast<uint4*>(&ahead_of[warp][d]) = bef[q];
        }
        __syncthreads();
        uint32_t total[2] = {0, 0}, ahead[2] = {0, 0};
        if (d2 < digits)
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    total[e] += cnt[w][d2 + e];
                    ahead[e] += ahead_of[w][d2 + e];
                }
        scan_digits(total, sums);
        first[0] = total[0] + ahead[0];
        first[1] = total[1] + ahead[1];
    }
    for (uint32_t d = threadIdx.x; d < kWarps << p.bits; d += kThreads) cnt[d >> p.bits][d & (digits - 1)] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const bool have = i0 + (uint32_t)j * 32u + lane < p.M;
        const uint32_t d = have ? (key[j] >> shift) & (digits - 1) : digits;  // lanes past the end match one another
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const uint32_t before = __popc(same & ((1u << lane) - 1u));
        if (have) rank[j] = cnt[warp][d] + before;
        __syncwarp();
        if (have && before == 0) cnt[warp][d] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    if (d2 < digits) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t c = cnt[w][d2 + e];
                cnt[w][d2 + e] = first[e];
                first[e] += c;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        if (i0 + (uint32_t)j * 32u + lane >= p.M) continue;
        const uint32_t to = cnt[warp][(key[j] >> shift) & (digits - 1)] + rank[j];
        p.key[from ^ 1u][to] = key[j];
        p.pos[from ^ 1u][to] = pos[j];
        if (pass + 1 < p.passes)
            atomicAdd(&later[(uint64_t)(to / kSortTile) * digits + ((key[j] >> (shift + (uint32_t)p.bits)) & (digits - 1))], 1u);
    }
}

// ------------------------------------------------------------------ reduce

// A lane's columns of a slice: NC chunks of VEC, 32 * VEC apart.
template <int VEC>
constexpr int kChunks = (int)kEmbedCols / 32 / VEC;

// The finished sum of row v (the lane's columns) into every replica.
template <class Out, int VEC>
__device__ __forceinline__ void write_row(const EmbedGradParams& p, uint64_t v, uint32_t c0,
                                          const float (&acc)[kChunks<VEC>][VEC])
{
    using T = typename Out::T;
    constexpr int NC = kChunks<VEC>;
#pragma unroll 1
    for (int o = 0; o < p.nout; ++o) {
        T* q = static_cast<T*>(p.grad[o]) + v * p.D;
        Vec<Out, VEC> x[NC];
        if (p.accumulate) {  // every load before the first store
#pragma unroll
            for (int k = 0; k < NC; ++k)
                if (c0 + (uint32_t)k * 32u * VEC < p.D) x[k].load(q + c0 + (uint32_t)k * 32u * VEC);
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float a[VEC];
            if (p.accumulate) {
                x[k].to_f(a);
#pragma unroll
                for (int l = 0; l < VEC; ++l) a[l] = __fadd_rn(a[l], __fmul_rn(acc[k][l], p.factor));
            } else {
#pragma unroll
                for (int l = 0; l < VEC; ++l) a[l] = __fmul_rn(acc[k][l], p.factor);
            }
            x[k].from_f(a);
            if (c0 + (uint32_t)k * 32u * VEC < p.D) x[k].store(q + c0 + (uint32_t)k * 32u * VEC);
        }
    }
}

// The same for a call that adds to one table, whose earlier values of the row
// (the lane's columns) have been brought to shared memory.
template <class Out, int VEC>
__device__ __forceinline__ void write_row_onto(const EmbedGradParams& p, uint64_t v, uint32_t c0,
                                               const float (&acc)[kChunks<VEC>][VEC], const typename Out::T* old)
{
    typename Out::T* q = static_cast<typename Out::T*>(p.grad[0]) + v * p.D;
#pragma unroll
    for (int k = 0; k < kChunks<VEC>; ++k) {
        if (kChunks<VEC> > 1 && c0 + (uint32_t)k * 32u * VEC >= p.D) continue;
        Vec<Out, VEC> x;
        float a[VEC];
        x.load(old + (k * 32 + (threadIdx.x & 31u)) * VEC);
        x.to_f(a);
#pragma unroll
        for (int l = 0; l < VEC; ++l) a[l] = __fadd_rn(a[l], __fmul_rn(acc[k][l], p.factor));
        x.from_f(a);
        if (c0 + (uint32_t)k * 32u * VEC < p.D) x.store(q + c0 + (uint32_t)k * 32u * VEC);
    }
}

// A run that crosses blocks: its partial sum, in fp32 (rows of Dp floats, on
// 16-byte boundaries).
template <int VEC>
__device__ __forceinline__ void write_part(float* q, uint32_t c0, uint32_t D,
                                           const float (&acc)[kChunks<VEC>][VEC])
{
#pragma unroll
    for (int k = 0; k < kChunks<VEC>; ++k) {
        const uint32_t c = c0 + (uint32_t)k * 32u * VEC;
        if (c >= D) continue;
        Vec<F32T, VEC> x;
        x.from_f(acc[k]);
        x.store(q + c);
    }
}

// The sorted list.
__device__ __forceinline__ const uint32_t* sorted_keys(const EmbedGradParams& p) { return p.key[0]; }
__device__ __forceinline__ const uint32_t* sorted_pos(const EmbedGradParams& p) { return p.pos[0]; }

// What a warp sums of the sorted list.  Block b covers positions [bK, (b+1)K)
// and owns the runs of equal ids that begin there: a run that goes on into the
// next block only is summed to its end by its owner, and that block's warp
// skips it.  A longer run (a frequent token) is cut at the blocks' ends: the
// block it begins in leaves its "last" partial sum, the others their "first"
// one, and the join adds them up.
struct Span {
    uint32_t from, to;  // positions
    uint32_t head;      // the id of a cut run that began earlier (V: none)
    bool cut;           // the last run goes on: it is cut at `to`
};

__device__ __forceinline__ Span block_span(const EmbedGradParams& p, uint32_t blk)
{
    const uint32_t* keys = sorted_keys(p);
    const uint32_t V = (uint32_t)p.V, K = p.K, lane = threadIdx.x & 31u;
    const uint32_t s = blk * K, e = s + K < p.M ? s + K : p.M;
    // six ids decide, loaded at once: before, first, last, after, one block back, one block on
    const uint32_t at = lane == 0 ? s - 1 : lane == 1 ? s : lane == 2 ? e - 1 : lane == 3 ? e : lane == 4 ? s - K - 1 : s + 2 * K;
    const bool there = lane == 0 ? s > 0 : lane == 3 ? e < p.M : lane == 4 ? s > K : lane == 5 ? (uint64_t)s + 2ull * K < p.M : true;
    const uint32_t k = lane < 6 && there ? keys[at] : 0xffffffffu;
    const uint32_t before = __shfl_sync(0xffffffffu, k, 0), first = __shfl_sync(0xffffffffu, k, 1);
    const uint32_t last = __shfl_sync(0xffffffffu, k, 2), after = __shfl_sync(0xffffffffu, k, 3);
    const uint32_t back = __shfl_sync(0xffffffffu, k, 4), on = __shfl_sync(0xffffffffu, k, 5);
    Span sp{s, e, V, false};
    if (first >= V) {  // nothing but ids without a row from here on
        sp.to = s;
        return sp;
    }
    const bool began_earlier = before == first;
    if (began_earlier) {
        if (back == first || after == first) {  // over three blocks or more: cut here
            sp.head = first;
        } else {  // the block before sums it: skip to its end
            for (uint32_t i = s; i < e; i += 32) {
                const uint32_t same = __ballot_sync(0xffffffffu, i + lane < e && keys[i + lane < e ? i + lane : s] == first);
                sp.from = i + __popc(same);
                if (same != 0xffffffffu) break;
            }
        }
    }
    if (last < V && after == last && !(began_earlier && last == first)) {  // begins here and goes on
        if (on == last) {
            sp.cut = true;
        } else {
            const uint32_t end = e + K < p.M ? e + K : p.M;
            for (uint32_t i = e; i < end; i += 32) {
                const uint32_t same = __ballot_sync(0xffffffffu, i + lane < end && keys[i + lane < end ? i + lane : e] == last);
                sp.to = i + __popc(same);
                if (same != 0xffffffffu) break;
            }
        }
    }
    return sp;
}

// Up to 32 positions of a span: a lane holds one position's id and row
// address, and three masks say after which of them a run ends, and where its
// sum goes.
template <class T>
struct Chunk {
    uint32_t n;       // positions with a row: the first n (ids are sorted)
    uint32_t ends;    // a run's last position in the span
    uint32_t first;   // ... of a cut run that began earlier: a partial sum
    uint32_t cut;     // ... of a cut run that goes on: a partial sum
    uint32_t key;
    const T* row;
};

template <class T>
__device__ __forceinline__ Chunk<T> load_chunk(const EmbedGradParams& p, uint32_t i0, const Span& sp)
{
    const uint32_t lane = threadIdx.x & 31u, i = i0 + lane, V = (uint32_t)p.V;
    Chunk<T> c;
    c.key = V;
    c.row = nullptr;
    uint32_t next = V;
    if (i < sp.to) {
        c.key = sorted_keys(p)[i];
        const uint32_t at = sorted_pos(p)[i], r = at / p.T;
        c.row = static_cast<const T*>(p.dout[r]) + (uint64_t)(at - r * p.T) * p.D;
        if (i + 1 < sp.to) next = sorted_keys(p)[i + 1];
    }
    const bool valid = c.key < V, end = valid && next != c.key;
    c.n = __popc(__ballot_sync(0xffffffffu, valid));
    c.ends = __ballot_sync(0xffffffffu, end);
    c.first = __ballot_sync(0xffffffffu, valid && c.key == sp.head);
    c.cut = __ballot_sync(0xffffffffu, end && sp.cut && i + 1 == sp.to);
    return c;
}

// Sum of the run that ends at position j of a chunk to where it belongs.
template <class Out, int VEC, class T>
__device__ __forceinline__ void close_run(const EmbedGradParams& p, const Chunk<T>& ch, uint32_t j, uint32_t blk,
                                          uint32_t c0, const float (&acc)[kChunks<VEC>][VEC])
{
    const uint32_t key = __shfl_sync(0xffffffffu, ch.key, j);
    const bool first = (ch.first >> j) & 1u;
    if (first || ((ch.cut >> j) & 1u))
        write_part<VEC>(p.part + ((first ? 0 : (uint64_t)p.nblk) + blk) * p.Dp, c0, p.D, acc);
    else
        write_row<Out, VEC>(p, key, c0, acc);
}

// The entries of the cut run that begins in block blk (its partial sums); 0:
// none begins there.
__device__ __forceinline__ uint32_t cut_entries(const EmbedGradParams& p, uint32_t blk)
{
    const uint32_t* keys = sorted_keys(p);
    const uint64_t on = ((uint64_t)blk + 2) * p.K;
    if (on >= p.M) return 0;
    const uint32_t end = (blk + 1) * p.K, key = keys[end - 1];
    const uint32_t before = blk > 0 ? keys[blk * p.K - 1] : 0xffffffffu;
    if (key >= (uint32_t)p.V || keys[on] != key || before == key) return 0;
    uint32_t lo = blk + 2, hi = p.nblk - 1;  // the last block whose first key is this one
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) / 2;
        if (keys[mid * p.K] == key) lo = mid;
        else hi = mid - 1;
    }
    return lo - blk + 1;
}

// Adds the partial sums of entries [a, b) of a run to acc, in order: entry 0
// is the last partial of block blk, entry i the first partial of block blk + i.
template <int VEC>
__device__ __forceinline__ void add_parts(const EmbedGradParams& p, uint32_t blk, uint32_t a, uint32_t b, uint32_t c0,
                                          float (&acc)[kChunks<VEC>][VEC])
{
    constexpr int NC = kChunks<VEC>, U = 1024 / (int)kEmbedCols;  // entries whose loads are in flight
    for (uint32_t i0 = a; i0 < b; i0 += U) {
        Vec<F32T, VEC> x[U][NC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u;
            const float* q = p.part + (i == 0 ? (uint64_t)p.nblk + blk : (uint64_t)blk + i) * p.Dp;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const uint32_t c = c0 + (uint32_t)k * 32u * VEC;
                if (i < b && c < p.D) x[u][k].load(q + c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= b) break;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                if (c0 + (uint32_t)k * 32u * VEC >= p.D) continue;
#pragma unroll
                for (int l = 0; l < VEC; ++l) acc[k][l] = __fadd_rn(acc[k][l], __uint_as_float(x[u][k].r[l]));
            }
        }
    }
}

// Few blocks (kJoinHere): the warp that comes last at a slice joins its cut runs
// itself, which saves the join's launch.  The count of those that came starts
// at zero with the sort's launch; a partial sum is in memory before its warp
// counts itself.
template <class Out, int VEC>
__device__ __forceinline__ void join_when_last(const EmbedGradParams& p, uint32_t slice, uint32_t c0)
{
    const uint32_t lane = threadIdx.x & 31u;
    __threadfence();
    __syncwarp();
    uint32_t came = 0;
    if (lane == 0) came = atomicAdd(&p.arrived[slice], 1u);
    if (__shfl_sync(0xffffffffu, came, 0) + 1 != p.nblk) return;
    __threadfence();
    for (uint32_t b0 = 0; b0 < p.nblk; b0 += 32) {
        const uint32_t mine = b0 + lane < p.nblk ? cut_entries(p, b0 + lane) : 0;
        for (uint32_t todo = __ballot_sync(0xffffffffu, mine > 0); todo; todo &= todo - 1) {
            const uint32_t l = __ffs(todo) - 1, n = __shfl_sync(0xffffffffu, mine, l);
            float acc[kChunks<VEC>][VEC];
#pragma unroll
            for (int k = 0; k < kChunks<VEC>; ++k)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[k][e] = 0.0f;
            add_parts<VEC>(p, b0 + l, 0, n, c0, acc);
            write_row<Out, VEC>(p, sorted_keys(p)[(b0 + l + 1) * p.K], c0, acc);
        }
    }
}

// Warps per CTA of the sums: with 8 / 4 / 2 / 1, 8 x 8192 tokens take 116.5 / 114.4 /
// 112.6 / 110.8 us, because a CTA keeps its shared memory until its slowest span ends.
constexpr int kReduceWarps = 1;
static_assert(kReduceWarps == 1, "join_when_last counts a warp per block");
constexpr uint32_t kRingBytes = 8192;  // of a warp

template <int B>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from)
{
    if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(B) : "memory");
}

template <class In, class Out, int VEC, bool ACC>
constexpr uint32_t kRingSlot =  // bytes of a warp's slot
    kEmbedCols * (ACC && sizeof(typename Out::T) > sizeof(typename In::T) ? sizeof(typename Out::T) : sizeof(typename In::T));

// A warp sums one slice of the columns over one block's span.
//
// The rows stream through a ring of slots in shared memory, kRingBytes a warp,
// by cp.async, one row's slice per slot, and where the call adds to one table
// the earlier values of a row follow the last position of its run through the
// same ring, so the sums wait only for loads that were issued several rows
// ago.  A lane reads only what it copied itself: no barrier.
//
// Bound by HBM, with instructions close behind (59 % of the issue slots taken):
// 8 x 8192 tokens of 2048 bf16 onto one fp32 table move 450 MB in 78 us (5.8
// TB/s).  With the loads of 8 rows held in registers instead (100 registers, 2
// CTAs per SM, 63 % of the warps' time waiting for memory) the kernel took 150
// us.  Slices of 512 columns halve the work per row but leave fewer warps (at 8
// warps per CTA the call took 121 us against 117, and 205 against 194 for 8 x 2048
// tokens into eight bf16 tables).
template <class In, class Out, int VEC, bool ACC, bool JOIN>
__global__ void __launch_bounds__(kReduceWarps * 32) embed_reduce_kernel(const __grid_constant__ EmbedGradParams p)
{
    using T = typename In::T;
    using TO = typename Out::T;
    constexpr int NC = kChunks<VEC>;
    constexpr uint32_t kSlot = kRingSlot<In, Out, VEC, ACC>;
    constexpr int kRing = (int)(kRingBytes / kSlot);
    static_assert(kRing >= 2 && (kRing & (kRing - 1)) == 0, "slots are counted modulo a power of two");
    constexpr int BI = VEC * (int)sizeof(T), BO = VEC * (int)sizeof(TO);
    extern __shared__ __align__(16) unsigned char ring_mem[];
    pdl_begin();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t blk = blockIdx.x * kReduceWarps + warp;
    if (blk >= p.nblk) return;
    unsigned char* ring = ring_mem + warp * kRingBytes;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    const Span sp = block_span(p, blk);
    const uint32_t c0 = blockIdx.y * kEmbedCols + lane * VEC;
    // one access per lane: a lane past the row's end copies the row's last
    // columns (and stores nothing), which saves a branch per row; several: it
    // copies nothing
    const uint32_t col = NC == 1 ? min(c0, p.D - VEC) : c0;
    auto inside = [&](int k) { return NC == 1 || c0 + (uint32_t)k * 32u * VEC < p.D; };
    float acc[NC][VEC];
    auto clear = [&] {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int l = 0; l < VEC; ++l) acc[k][l] = 0.0f;
    };
    clear();
    for (uint32_t i0 = sp.from; i0 < sp.to; i0 += 32) {
        const Chunk<T> ch = load_chunk<T>(p, i0, sp);
        const uint32_t fetch = ACC ? ch.ends & ~ch.first & ~ch.cut : 0u;  // rows whose earlier values are needed
        uint32_t made = 0;      // the next position to copy
        bool old_next = false;  // the earlier values of the one before it come first
        uint32_t in_slot = 0, out_slot = 0;
        auto issue = [&] {  // one item into the ring (an empty group where nothing is left)
            const uint32_t to = ring_at + in_slot * kSlot;
            if (ACC && old_next) {
                const TO* q = static_cast<const TO*>(p.grad[0]) + (uint64_t)__shfl_sync(0xffffffffu, ch.key, made - 1) * p.D;
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    constexpr int B = BO > 16 ? 16 : BO;
                    if (!inside(k)) continue;
#pragma unroll
                    for (int h = 0; h < BO; h += B)
                        copy_async<B < 4 ? 4 : B>(to + (uint32_t)(k * 32 + lane) * BO + h,
                                                  reinterpret_cast<const char*>(q + col + k * 32 * VEC) + h);
                }
                old_next = false;
            } else if (made < ch.n) {
                const T* q = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, (unsigned long long)ch.row, made));
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    if (inside(k)) copy_async<BI < 4 ? 4 : BI>(to + (uint32_t)(k * 32 + lane) * BI, q + col + k * 32 * VEC);
                if (ACC) old_next = (fetch >> made) & 1u;
                ++made;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            in_slot = (in_slot + 1) & (kRing - 1);
        };
        auto next_slot = [&]() -> const unsigned char* {  // the oldest item, landed
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            const unsigned char* q = ring + out_slot * kSlot;
            out_slot = (out_slot + 1) & (kRing - 1);
            return q;
        };
#pragma unroll 1
        for (int k = 0; k < kRing; ++k) issue();
#pragma unroll 1
        for (uint32_t j = 0; j < ch.n; ++j) {
            const T* x = reinterpret_cast<const T*>(next_slot());
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                if (!inside(k)) continue;
                Vec<In, VEC> v;
                float a[VEC];
                v.load(x + (k * 32 + lane) * VEC);
                v.to_f(a);
#pragma unroll
                for (int l = 0; l < VEC; ++l) acc[k][l] = __fadd_rn(acc[k][l], a[l]);
            }
            issue();
            if (!((ch.ends >> j) & 1u)) continue;
            if (ACC && ((fetch >> j) & 1u)) {
                write_row_onto<Out, VEC>(p, __shfl_sync(0xffffffffu, ch.key, j), c0, acc,
                                         reinterpret_cast<const TO*>(next_slot()));
                issue();
            } else {
                close_run<Out, VEC>(p, ch, j, blk, c0, acc);
            }
            clear();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");  // the ring is free for the next chunk
        if (ch.n < 32) break;
    }
    if constexpr (JOIN) join_when_last<Out, VEC>(p, blockIdx.y, c0);
}

// The same for rows in 2-byte pieces, which cp.async cannot copy: the loads of
// a few rows in flight in registers.
template <class In, class Out, int VEC>
__global__ void __launch_bounds__(kReduceWarps * 32) embed_reduce_narrow_kernel(const __grid_constant__ EmbedGradParams p)
{
    using T = typename In::T;
    constexpr int NC = kChunks<VEC>;
    constexpr int G = 4;  // rows whose loads are in flight
    pdl_begin();
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t blk = blockIdx.x * kReduceWarps + (threadIdx.x >> 5);
    if (blk >= p.nblk) return;
    const Span sp = block_span(p, blk);
    const uint32_t c0 = blockIdx.y * kEmbedCols + lane * VEC;
    float acc[NC][VEC];
    auto clear = [&] {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int l = 0; l < VEC; ++l) acc[k][l] = 0.0f;
    };
    clear();
    for (uint32_t i0 = sp.from; i0 < sp.to; i0 += 32) {
        const Chunk<T> ch = load_chunk<T>(p, i0, sp);
        for (uint32_t j0 = 0; j0 < ch.n; j0 += G) {
            Vec<In, VEC> x[G][NC];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const T* q = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, (unsigned long long)ch.row, j0 + g));
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const uint32_t c = c0 + (uint32_t)k * 32u * VEC;
                    if (j0 + g < ch.n && c < p.D) x[g][k].load(q + c);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t j = j0 + g;
                if (j >= ch.n) break;
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    if (c0 + (uint32_t)k * 32u * VEC >= p.D) continue;
                    float a[VEC];
                    x[g][k].to_f(a);
#pragma unroll
                    for (int l = 0; l < VEC; ++l) acc[k][l] = __fadd_rn(acc[k][l], a[l]);
                }
                if (!((ch.ends >> j) & 1u)) continue;
                close_run<Out, VEC>(p, ch, j, blk, c0, acc);
                clear();
            }
        }
        if (ch.n < 32) break;
    }
}

// Which of the 32 table rows from v0 on have a token, as bits: every lane
// looks its row up in the sorted list, the warp's 32 first steps together.
// Where a frequent token's run fills the range the lanes go on by themselves:
// going on together, a round moved an end of the range by one key, and 65536
// tokens of Zipf-like ids (width 2048, one table written) took 118 us instead of
// 97, 1048576 tokens (width 64, eight tables) 668 instead of 388.
__device__ __forceinline__ uint32_t touched_rows(const EmbedGradParams& p, uint64_t v0)
{
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t* keys = sorted_keys(p);
    const uint64_t v = v0 + lane;
    // the warp's range [lo, hi): keys before lo are below v0, keys from hi on are at least v0 + 32
    uint32_t lo = 0, hi = p.M;
    while (hi - lo > 64) {
        const uint32_t at = lo + lane * search_step(lo, hi);
        const uint32_t k = at < hi ? keys[at] : 0xffffffffu;
        const uint32_t below = __popc(__ballot_sync(0xffffffffu, at < hi && k < v0));
        const uint32_t within = __popc(__ballot_sync(0xffffffffu, at < hi && k < v0 + 32));
        if (!search_narrow(lo, hi, below, within)) break;  // a frequent token's run
    }
    while (lo < hi) {  // the first key that is at least v
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return __ballot_sync(0xffffffffu, lo < p.M && keys[lo] == v);
}

// Zeros into the rows that no token touched: a CTA takes 32 rows of one
// replica, run by run of untouched ones.
template <class Out>
__device__ __forceinline__ void zero_rows(const EmbedGradParams& p, uint32_t chunk, uint32_t replica)
{
    using T = typename Out::T;
    constexpr int L = Out::L;
    const uint64_t v0 = (uint64_t)chunk * 32u;
    const uint32_t rows = (uint32_t)(p.V - v0 < 32 ? p.V - v0 : 32);
    const uint32_t word = touched_rows(p, v0);
    T* base = static_cast<T*>(p.grad[replica]) + v0 * p.D;
    for (uint32_t i = 0; i < rows;) {
        if ((word >> i) & 1u) {
            ++i;
            continue;
        }
        uint32_t j = i + 1;
        while (j < rows && !((word >> j) & 1u)) ++j;
        T* q = base + (uint64_t)i * p.D;
        const uint64_t len = (uint64_t)(j - i) * p.D;
        uint64_t head = (uint64_t)((L - phase_of(q, L)) & (L - 1));
        if (head > len) head = len;
        const uint64_t nv = (len - head) / L, tail = len - head - nv * L;
        if (threadIdx.x < head + tail)
            Out::st1(q + (threadIdx.x < head ? threadIdx.x : head + nv * L + (threadIdx.x - head)), 0.0f);
        for (uint64_t v = threadIdx.x; v < nv; v += kThreads) stv(q + head + v * L, make_uint4(0u, 0u, 0u, 0u));
        i = j;
    }
}

// Joins the cut runs -- the block in which such a run begins adds its partial
// sums in block order and writes the row -- and, in the CTAs behind those
// (chunks of rows x replicas), clears the untouched rows: the joins wait for
// memory while the clearing fills it.  A warp looks at kJoinBlocks blocks, a
// lane at each, and joins a run for one slice; a run over many blocks is
// shared by the CTA's warps, each an eighth of the entries, and the eighths
// added in order.
constexpr uint32_t kLongRun = 8;     // entries from which a run is shared (32, with 8 blocks per warp: 1 us more)
constexpr uint32_t kJoinBlocks = 4;  // blocks per warp: fewer than a shared run's, so a warp meets at most one

template <class Out, int VEC>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const __grid_constant__ EmbedGradParams p, uint32_t joins,
                                                              uint32_t slices, uint32_t chunks)
{
    constexpr int NC = kChunks<VEC>;
    static_assert(kJoinBlocks < kLongRun);
    __shared__ uint32_t long_run[kWarps], long_blk[kWarps];
    __shared__ __align__(16) float eighth[kWarps][kEmbedCols];
    pdl_begin();
    if (blockIdx.x >= joins) {
        const uint32_t z = blockIdx.x - joins;
        zero_rows<Out>(p, z % chunks, z / chunks);
        return;
    }
    const uint32_t* keys = sorted_keys(p);
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t slice = blockIdx.x % slices, blk0 = (blockIdx.x / slices * kWarps + warp) * kJoinBlocks;
    const uint32_t c0 = slice * kEmbedCols + lane * VEC;
    float acc[NC][VEC];
    auto clear = [&] {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int l = 0; l < VEC; ++l) acc[k][l] = 0.0f;
    };
    const uint32_t mine = lane < kJoinBlocks ? cut_entries(p, blk0 + lane) : 0;
    const uint32_t shared_run = __ballot_sync(0xffffffffu, mine > kLongRun);
    if (lane == 0) long_run[warp] = 0;
    __syncwarp();
    if (mine > kLongRun) {
        long_run[warp] = mine;
        long_blk[warp] = blk0 + lane;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, mine > 0) & ~shared_run; todo; todo &= todo - 1) {
        const uint32_t l = __ffs(todo) - 1, blk = blk0 + l, n = __shfl_sync(0xffffffffu, mine, l);
        clear();
        add_parts<VEC>(p, blk, 0, n, c0, acc);
        write_row<Out, VEC>(p, keys[(blk + 1) * p.K], c0, acc);
    }
    __syncthreads();
    for (uint32_t w = 0; w < kWarps; ++w) {
        const uint32_t n = long_run[w];
        if (n == 0) continue;
        const uint32_t blk = long_blk[w];
        clear();
        add_parts<VEC>(p, blk, (uint32_t)((uint64_t)n * warp / kWarps), (uint32_t)((uint64_t)n * (warp + 1) / kWarps), c0,
                       acc);
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int l = 0; l < VEC; ++l) eighth[warp][(k * 32 + lane) * VEC + l] = acc[k][l];
        __syncthreads();
        if (warp == 0) {
            for (int e = 1; e < kWarps; ++e)
#pragma unroll
                for (int k = 0; k < NC; ++k)
#pragma unroll
                    for (int l = 0; l < VEC; ++l)
                        acc[k][l] = __fadd_rn(acc[k][l], eighth[e][(k * 32 + lane) * VEC + l]);
            write_row<Out, VEC>(p, keys[(blk + 1) * p.K], c0, acc);
        }
        __syncthreads();
    }
}

unsigned blocks_for(uint64_t items, uint64_t per) { return (unsigned)((items + per - 1) / per); }

template <class In, class Out, int VEC>
cudaError_t reduce_typed(const EmbedGradParams& p, int* launches, cudaStream_t s)
{
    const uint32_t slices = blocks_for(p.D, kEmbedCols);
    const dim3 grid(blocks_for(p.nblk, kReduceWarps), slices);
    constexpr uint32_t kRings = kReduceWarps * kRingBytes;
    static_assert(kRings <= 48 * 1024, "within the default dynamic shared memory of a CTA");
    cudaError_t e;
    if constexpr (VEC * sizeof(typename In::T) < 4) {
        e = launch_pdl(embed_reduce_narrow_kernel<In, Out, VEC>, grid, kReduceWarps * 32, 0, s, p);
    } else if (p.accumulate && p.nout == 1) {
        if (p.nblk > 2 && p.nblk <= kJoinHere && p.M <= kRankMax) {
            *launches += 1;
            return launch_pdl(embed_reduce_kernel<In, Out, VEC, true, true>, grid, kReduceWarps * 32, kRings, s, p);
        }
        e = launch_pdl(embed_reduce_kernel<In, Out, VEC, true, false>, grid, kReduceWarps * 32, kRings, s, p);
    } else {
        e = launch_pdl(embed_reduce_kernel<In, Out, VEC, false, false>, grid, kReduceWarps * 32, kRings, s, p);
    }
    if (e != cudaSuccess) return e;
    *launches += 1;
    const uint64_t joins = p.nblk > 2 ? (uint64_t)blocks_for(p.nblk, kWarps * kJoinBlocks) * slices : 0;  // a cut run covers three blocks
    const uint64_t chunks = p.accumulate ? 0 : (p.V + 31) / 32;
    const uint64_t work = joins + chunks * (uint64_t)p.nout;
    if (work == 0) return cudaSuccess;
    if (work > kMaxGrid) return cudaErrorInvalidValue;
    e = launch_pdl(embed_join_kernel<Out, VEC>, dim3((unsigned)work), kThreads, 0, s, p, (uint32_t)joins, slices,
                   (uint32_t)chunks);
    *launches += e == cudaSuccess;
    return e;
}

template <class In, class Out>
cudaError_t reduce_out(int vec, const EmbedGradParams& p, int* launches, cudaStream_t s)
{
    switch (vec) {
    case 8:
        if constexpr (sizeof(typename In::T) == 2) return reduce_typed<In, Out, 8>(p, launches, s);
        else return cudaErrorInvalidValue;
    case 4: return reduce_typed<In, Out, 4>(p, launches, s);
    case 2: return reduce_typed<In, Out, 2>(p, launches, s);
    case 1: return reduce_typed<In, Out, 1>(p, launches, s);
    }
    return cudaErrorInvalidValue;
}

template <class Ty>
cudaError_t lookup_typed(int vec, const EmbedLookupParams& p, cudaStream_t s)
{
    const dim3 grid(blocks_for(p.M, kWarps), blocks_for(p.D, (uint64_t)32 * kLookupU * vec));
    switch (vec) {
    case 8:
        if constexpr (sizeof(typename Ty::T) == 2) return launch_pdl(embed_lookup_kernel<Ty, 8>, grid, kThreads, 0, s, p);
        else return cudaErrorInvalidValue;
    case 4: return launch_pdl(embed_lookup_kernel<Ty, 4>, grid, kThreads, 0, s, p);
    case 2: return launch_pdl(embed_lookup_kernel<Ty, 2>, grid, kThreads, 0, s, p);
    case 1: return launch_pdl(embed_lookup_kernel<Ty, 1>, grid, kThreads, 0, s, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_embed_lookup(int dtype, int vec, const EmbedLookupParams& p, cudaStream_t s)
{
    switch (dtype) {
    case kF32: return lookup_typed<F32T>(vec, p, s);
    case kBF16: return lookup_typed<BF16T>(vec, p, s);
    case kF16: return lookup_typed<F16T>(vec, p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_embed_sort(const EmbedGradParams& p, int* launches, cudaStream_t s)
{
    if (p.M <= kRankMax) {
        *launches += 1;
        return launch_pdl(embed_rank_kernel, dim3(blocks_for(p.M, kRankThreads / kRankParts)), kRankThreads, 0, s, p);
    }
    const bool scan = p.ntiles > kScanTiles;
    cudaError_t e = launch_pdl(embed_count_kernel, dim3(p.ntiles), kThreads, 0, s, p);
    *launches += 1;
    for (int pass = 0; pass < p.passes && e == cudaSuccess; ++pass) {
        if (scan) e = launch_pdl(embed_scan_kernel, dim3(1), kThreads, 0, s, p, pass);
        if (e == cudaSuccess)
            e = scan ? launch_pdl(embed_place_kernel<true>, dim3(p.ntiles), kThreads, 0, s, p, pass)
                     : launch_pdl(embed_place_kernel<false>, dim3(p.ntiles), kThreads, 0, s, p, pass);
        *launches += scan ? 2 : 1;
    }
    return e;
}

cudaError_t launch_embed_reduce(int dtype, int out_dtype, int vec, const EmbedGradParams& p, int* launches,
                                cudaStream_t s)
{
    cudaError_t e = cudaErrorInvalidValue;
    if (dtype == kF32 && out_dtype == kF32) e = reduce_out<F32T, F32T>(vec, p, launches, s);
    else if (dtype == kBF16 && out_dtype == kBF16) e = reduce_out<BF16T, BF16T>(vec, p, launches, s);
    else if (dtype == kBF16 && out_dtype == kF32) e = reduce_out<BF16T, F32T>(vec, p, launches, s);
    else if (dtype == kF16 && out_dtype == kF16) e = reduce_out<F16T, F16T>(vec, p, launches, s);
    else if (dtype == kF16 && out_dtype == kF32) e = reduce_out<F16T, F32T>(vec, p, launches, s);
    return e;
}

}  // namespace rr
