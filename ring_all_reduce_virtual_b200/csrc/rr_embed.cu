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
#include "rr_device.cuh"
#include "rr_internal.h"

namespace rr {

namespace {

__device__ __forceinline__ void pdl_begin()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

constexpr int kLookupU = 4;  // accesses per lane: 2 KB of a 16-byte aligned row per warp

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
constexpr int kSortRounds = (int)kSortTile / kThreads;  // keys per thread

// Least-significant-digit radix sort, one digit per pass; pass k reads buffer
// k & 1 (pass 0 the ids) and writes the other.  Counting: a tile's keys per
// digit, digit-major, so one exclusive scan over all counts gives every tile's
// first place for every digit.  Pass 0 also clears the touched bits.
__global__ void __launch_bounds__(kThreads) embed_count_kernel(const __grid_constant__ EmbedGradParams p, int pass)
{
    __shared__ uint32_t hist[1 << kSortMaxBits];
    pdl_begin();
    const uint32_t digits = 1u << p.bits, shift = (uint32_t)(pass * p.bits);
    for (uint32_t d = threadIdx.x; d < digits; d += kThreads) hist[d] = 0;
    if (pass == 0)
        for (uint64_t w = (uint64_t)blockIdx.x * kThreads + threadIdx.x; w < (p.V + 31) / 32;
             w += (uint64_t)gridDim.x * kThreads)
            p.touched[w] = 0u;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * kSortTile;
    for (uint32_t k = threadIdx.x; k < kSortTile && k < p.M - i0; k += kThreads) {
        const uint32_t key = pass == 0 ? position_key(p, i0 + k) : p.key[pass & 1][i0 + k];
        atomicAdd(&hist[(key >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < digits; d += kThreads) p.counts[(uint64_t)d * p.ntiles + blockIdx.x] = hist[d];
}

// Exclusive scan of count values in place, by one CTA: every thread takes a
// run of consecutive ones.
__global__ void __launch_bounds__(1024) embed_scan_kernel(uint32_t* v, uint32_t count)
{
    __shared__ uint32_t sums[32];
    pdl_begin();
    const uint32_t per = (count + 1023) / 1024, tid = threadIdx.x, lane = tid & 31u;
    const uint32_t lo = tid * per < count ? tid * per : count, hi = lo + per < count ? lo + per : count;
    uint32_t s = 0;
    for (uint32_t i = lo; i < hi; ++i) s += v[i];
    uint32_t x = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= (uint32_t)o) x += y;
    }
    if (lane == 31u) sums[tid >> 5] = x;
    __syncthreads();
    uint32_t before = x - s;
    for (uint32_t w = 0; w < tid >> 5; ++w) before += sums[w];
    for (uint32_t i = lo; i < hi; ++i) {
        const uint32_t c = v[i];
        v[i] = before;
        before += c;
    }
}

// Placing, stable: a warp takes consecutive keys, 32 at a time; lanes with
// the same digit rank themselves by lane, behind the warp's earlier ones, and
// the warps' counts stack in warp order.  Pass 0 also marks the rows.
__global__ void __launch_bounds__(kThreads) embed_place_kernel(const __grid_constant__ EmbedGradParams p, int pass)
{
    __shared__ uint32_t cnt[kWarps][1 << kSortMaxBits];
    pdl_begin();
    const uint32_t digits = 1u << p.bits, shift = (uint32_t)(pass * p.bits);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    for (uint32_t d = threadIdx.x; d < kWarps << p.bits; d += kThreads) cnt[d >> p.bits][d & (digits - 1)] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * kSortTile + warp * (kSortTile / kWarps);
    uint32_t key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const uint32_t i = i0 + (uint32_t)j * 32u + lane;
        if (i < p.M) {
            key[j] = pass == 0 ? position_key(p, i) : p.key[pass & 1][i];
            pos[j] = pass == 0 ? i : p.pos[pass & 1][i];
            if (pass == 0 && key[j] < p.V) atomicOr(&p.touched[key[j] >> 5], 1u << (key[j] & 31u));
        }
    }
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
    for (uint32_t d = threadIdx.x; d < digits; d += kThreads) {
        uint32_t at = p.counts[(uint64_t)d * p.ntiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = cnt[w][d];
            cnt[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        if (i0 + (uint32_t)j * 32u + lane >= p.M) continue;
        const uint32_t to = cnt[warp][(key[j] >> shift) & (digits - 1)] + rank[j];
        p.key[(pass + 1) & 1][to] = key[j];
        p.pos[(pass + 1) & 1][to] = pos[j];
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
    for (int o = 0; o < p.nout; ++o) {
        T* q = static_cast<T*>(p.grad[o]) + v * p.D;
#pragma unroll
        for (int k = 0; k < kChunks<VEC>; ++k) {
            const uint32_t c = c0 + (uint32_t)k * 32u * VEC;
            if (c >= p.D) continue;
            Vec<Out, VEC> x;
            float a[VEC];
            if (p.accumulate) {
                x.load(q + c);
                x.to_f(a);
#pragma unroll
                for (int l = 0; l < VEC; ++l) a[l] = __fadd_rn(a[l], __fmul_rn(acc[k][l], p.factor));
            } else {
#pragma unroll
                for (int l = 0; l < VEC; ++l) a[l] = __fmul_rn(acc[k][l], p.factor);
            }
            x.from_f(a);
            x.store(q + c);
        }
    }
}

// A run that crosses blocks: its partial sum, in fp32.
template <int VEC>
__device__ __forceinline__ void write_part(float* q, uint32_t c0, uint32_t D,
                                           const float (&acc)[kChunks<VEC>][VEC])
{
#pragma unroll
    for (int k = 0; k < kChunks<VEC>; ++k) {
        const uint32_t c = c0 + (uint32_t)k * 32u * VEC;
        if (c >= D) continue;
#pragma unroll
        for (int l = 0; l < VEC; ++l) q[c + l] = acc[k][l];
    }
}

// Where the sorted keys are after the last pass.
__device__ __forceinline__ const uint32_t* sorted_keys(const EmbedGradParams& p) { return p.key[p.passes & 1]; }
__device__ __forceinline__ const uint32_t* sorted_pos(const EmbedGradParams& p) { return p.pos[p.passes & 1]; }

// A warp sums one slice of the columns over one block of K sorted positions:
// runs that lie inside it go to the table, the first and the last run's sums
// to the block's partials where they go on outside.
template <class In, class Out, int VEC>
__global__ void __launch_bounds__(kThreads) embed_reduce_kernel(const __grid_constant__ EmbedGradParams p)
{
    using T = typename In::T;
    constexpr int NC = kChunks<VEC>;
    constexpr int G = sizeof(T) * VEC * NC == 16 ? 8 : 4;  // rows whose loads are in flight
    pdl_begin();
    const uint32_t* keys = sorted_keys(p);
    const uint32_t* poss = sorted_pos(p);
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t blk = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (blk >= p.nblk) return;
    const uint32_t b0 = blk * p.K, b1 = b0 + p.K < p.M ? b0 + p.K : p.M;
    const uint32_t c0 = blockIdx.y * kEmbedCols + lane * VEC;
    const uint32_t V = (uint32_t)p.V;
    const uint32_t before = b0 > 0 ? keys[b0 - 1] : V, after = b1 < p.M ? keys[b1] : V;
    float acc[NC][VEC];
    uint32_t cur = V;      // the run being summed (V: none)
    bool from = false;     // it began in an earlier block
    auto clear = [&] {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int l = 0; l < VEC; ++l) acc[k][l] = 0.0f;
    };
    auto close = [&](bool goes_on) {
        if (cur >= V) return;
        if (from) write_part<VEC>(p.part + (uint64_t)blk * p.Dp, c0, p.D, acc);
        else if (goes_on) write_part<VEC>(p.part + ((uint64_t)p.nblk + blk) * p.Dp, c0, p.D, acc);
        else write_row<Out, VEC>(p, cur, c0, acc);
    };
    clear();
    for (uint32_t i0 = b0; i0 < b1; i0 += 32) {
        const uint32_t mine = i0 + lane;
        uint32_t key = V;
        const T* row = nullptr;
        if (mine < b1) {
            key = keys[mine];
            const uint32_t at = poss[mine], r = at / p.T;
            row = static_cast<const T*>(p.dout[r]) + (uint64_t)(at - r * p.T) * p.D;
        }
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, key < V));  // sorted: the valid ones come first
        for (uint32_t j0 = 0; j0 < n; j0 += G) {
            Vec<In, VEC> x[G][NC];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const T* q = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, (unsigned long long)row, j0 + g));
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const uint32_t c = c0 + (uint32_t)k * 32u * VEC;
                    if (j0 + g < n && c < p.D) x[g][k].load(q + c);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t next = __shfl_sync(0xffffffffu, key, j0 + g);
                if (j0 + g >= n) continue;
                if (next != cur) {
                    close(false);
                    clear();
                    from = cur >= V && next == before;  // only a block's first run can have begun earlier
                    cur = next;
                }
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    if (c0 + (uint32_t)k * 32u * VEC >= p.D) continue;
                    float a[VEC];
                    x[g][k].to_f(a);
#pragma unroll
                    for (int l = 0; l < VEC; ++l) acc[k][l] = __fadd_rn(acc[k][l], a[l]);
                }
            }
        }
        if (n < 32) break;
    }
    close(cur == after);
}

// Joins the runs that cross blocks: the block in which such a run begins adds
// its partial sums in block order and writes the row.
template <class Out, int VEC>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const __grid_constant__ EmbedGradParams p)
{
    constexpr int NC = kChunks<VEC>;
    pdl_begin();
    const uint32_t* keys = sorted_keys(p);
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t blk = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (blk + 1 >= p.nblk) return;
    const uint32_t end = (blk + 1) * p.K;  // < M
    const uint32_t key = keys[end - 1];
    if (key >= (uint32_t)p.V || keys[end] != key) return;
    if (blk > 0 && keys[blk * p.K - 1] == key) return;  // begun earlier (then the whole block is the run's)
    uint32_t lo = blk + 1, hi = p.nblk - 1;             // the last block whose first key is this one
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) / 2;
        if (keys[mid * p.K] == key) lo = mid;
        else hi = mid - 1;
    }
    const uint32_t c0 = blockIdx.y * kEmbedCols + lane * VEC;
    float acc[NC][VEC];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int l = 0; l < VEC; ++l) {
            const uint32_t c = c0 + (uint32_t)k * 32u * VEC + l;
            if (c >= p.D) continue;
            float s = p.part[((uint64_t)p.nblk + blk) * p.Dp + c];
            for (uint32_t b = blk + 1; b <= lo; ++b) s = __fadd_rn(s, p.part[(uint64_t)b * p.Dp + c]);
            acc[k][l] = s;
        }
    write_row<Out, VEC>(p, key, c0, acc);
}

// Zeros into the rows that no token touched: a CTA takes 32 rows of one
// replica, run by run of untouched ones.
template <class Out>
__global__ void __launch_bounds__(kThreads) embed_zero_kernel(const __grid_constant__ EmbedGradParams p)
{
    using T = typename Out::T;
    constexpr int L = Out::L;
    pdl_begin();
    const uint64_t v0 = (uint64_t)blockIdx.x * 32u;
    const uint32_t rows = (uint32_t)(p.V - v0 < 32 ? p.V - v0 : 32);
    const uint32_t word = p.touched[blockIdx.x];
    T* base = static_cast<T*>(p.grad[blockIdx.y]) + v0 * p.D;
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

template <class... A>
cudaError_t launch_pdl(void (*kernel)(A...), dim3 grid, unsigned threads, cudaStream_t s, const A&... a)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned blocks_for(uint64_t items, uint64_t per) { return (unsigned)((items + per - 1) / per); }

template <class In, class Out, int VEC>
cudaError_t reduce_typed(const EmbedGradParams& p, int* launches, cudaStream_t s)
{
    const dim3 grid(blocks_for(p.nblk, kWarps), blocks_for(p.D, kEmbedCols));
    cudaError_t e = launch_pdl(embed_reduce_kernel<In, Out, VEC>, grid, kThreads, s, p);
    if (e != cudaSuccess) return e;
    *launches += 1;
    if (p.nblk > 1) {
        e = launch_pdl(embed_join_kernel<Out, VEC>, grid, kThreads, s, p);
        if (e != cudaSuccess) return e;
        *launches += 1;
    }
    return cudaSuccess;
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

template <class Out>
cudaError_t zero_typed(const EmbedGradParams& p, int* launches, cudaStream_t s)
{
    const cudaError_t e =
        launch_pdl(embed_zero_kernel<Out>, dim3(blocks_for(p.V, 32), (unsigned)p.nout), kThreads, s, p);
    *launches += e == cudaSuccess;
    return e;
}

template <class Ty>
cudaError_t lookup_typed(int vec, const EmbedLookupParams& p, cudaStream_t s)
{
    const dim3 grid(blocks_for(p.M, kWarps), blocks_for(p.D, (uint64_t)32 * kLookupU * vec));
    switch (vec) {
    case 8:
        if constexpr (sizeof(typename Ty::T) == 2) return launch_pdl(embed_lookup_kernel<Ty, 8>, grid, kThreads, s, p);
        else return cudaErrorInvalidValue;
    case 4: return launch_pdl(embed_lookup_kernel<Ty, 4>, grid, kThreads, s, p);
    case 2: return launch_pdl(embed_lookup_kernel<Ty, 2>, grid, kThreads, s, p);
    case 1: return launch_pdl(embed_lookup_kernel<Ty, 1>, grid, kThreads, s, p);
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
    for (int pass = 0; pass < p.passes; ++pass) {
        cudaError_t e = launch_pdl(embed_count_kernel, dim3(p.ntiles), kThreads, s, p, pass);
        if (e == cudaSuccess) e = launch_pdl(embed_scan_kernel, dim3(1), 1024, s, p.counts, p.ntiles << p.bits);
        if (e == cudaSuccess) e = launch_pdl(embed_place_kernel, dim3(p.ntiles), kThreads, s, p, pass);
        if (e != cudaSuccess) return e;
        *launches += 3;
    }
    return cudaSuccess;
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
    if (e != cudaSuccess || p.accumulate) return e;
    return out_dtype == kF32 ? zero_typed<F32T>(p, launches, s) : zero_typed<BF16T>(p, launches, s);
}

}  // namespace rr
