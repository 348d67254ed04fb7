// rr_logprob.cu -- log probabilities of given tokens over all ranks' logits,
// with entropy and top alternatives, and their gradient.
//
// For a row x of V logits, z = scale * x, m = max x, y_j = scale * (x_j - m):
//     s = sum e^y_j       lse = scale * m + ln s       logprob = y_t - ln s
//     t = sum e^y_j y_j   entropy = ln s - t / s
// in one pass over the row: a thread keeps the running maximum of what it has
// read with s and t relative to it, and rescales them when the maximum grows
// (t / s shifts by the difference).  x_j - m is 0 at the maximum, so a row with
// one value left has the log probability 0 exactly, and a row whose every value
// is the type's lowest is uniform, as it should be.  Exponentials are powers of
// two (y in units of ln 2).
//
// Bound by HBM: 2 or 4 bytes an element against about 5 issue slots (packed
// fp32 pairs: one subtraction, one product, one sum) and one exponential, of
// which an SM does 16 a clock -- bf16 logits at full bandwidth need 12.
//
// The top alternatives cost the pass nothing but the maxima it has anyway.  A
// thread's maximum is an element of its own.  With tau the k-th largest of the
// eight warps' four largest maxima each, at least k elements are at or above
// tau, and every element that is belongs to a thread whose maximum is: a few
// more than k threads of 256.  Their elements alone are read
// once more, from L2, and go through a sorted list of 32 per warp; the lists are
// merged.  Where more threads tie at tau -- a mask that leaves fewer than k tokens, a
// constant row -- all of theirs are read again, up to the whole row, but a vector
// whose largest value could not get into its warp's list goes no further.  Elements
// are ordered by (value, lowest id first), so the outcome does not depend on who
// saw them first.
#include <type_traits>

#include "rr_device.cuh"
#include "rr_launch.cuh"
#include "rr_logprob.h"

namespace rr {

namespace {

constexpr int kU = 4;              // vectors a thread has on the way
constexpr int kMaxSplit = 8;       // portable cluster size
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------- small pieces

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void un2(F2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The largest of a vector's values, NaN where one is.
template <class Ty>
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b)
{
    uint32_t y;
    if constexpr (std::is_same_v<Ty, BF16T>) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else if constexpr (std::is_same_v<Ty, F16T>) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else y = __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    return y;
}

template <class Ty, int N>
__device__ __forceinline__ float max_of(const uint4 (&raw)[N])
{
    uint32_t w = max_words<Ty>(max_words<Ty>(raw[0].x, raw[0].y), max_words<Ty>(raw[0].z, raw[0].w));
#pragma unroll
    for (int u = 1; u < N; ++u)
        w = max_words<Ty>(w, max_words<Ty>(max_words<Ty>(raw[u].x, raw[u].y), max_words<Ty>(raw[u].z, raw[u].w)));
    if constexpr (Ty::L == 8) {
        float lo, hi;
        Ty::unpack2(w, lo, hi);
        return max_nan(lo, hi);
    } else {
        return __uint_as_float(w);
    }
}

// Every element -inf.
template <class Ty>
__device__ __forceinline__ uint4 lowest_vector()
{
    const uint32_t w = std::is_same_v<Ty, BF16T> ? 0xff80ff80u : std::is_same_v<Ty, F16T> ? 0xfc00fc00u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

__device__ __forceinline__ int64_t id_at(const void* ids, int ids64, uint64_t t)
{
    return ids64 ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}

// A whole number that orders fp32 values, NaN above all, both zeros alike.
__device__ __forceinline__ uint32_t order_of(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t order)
{
    return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);  // NaN's order gives a NaN
}

// z - the row's largest z, also where the logits' difference leaves fp32.
__device__ __forceinline__ float z_below(float x, float top, float scale)
{
    const float d = x - top;
    return d == -INFINITY ? x * scale - top * scale : d * scale;
}

// ------------------------------------------------------- softmax statistics

// A thread's sums relative to the largest value m that it has read: s of 2^y, t
// of 2^y y, y = (x - m) c with c = scale log2 e.  y is 0 at the maximum and never
// above, also for rows of the type's lowest value.
template <class Ty, bool ENT>
struct Running {
    float m = -INFINITY;
    F2 s = f2(0.0f, 0.0f), t = f2(0.0f, 0.0f);

    // Relative to a larger value.  -inf - -inf counts as -2000: no sums are there.
    __device__ __forceinline__ void move(float to, float c)
    {
        const float d = fmaxf((m - to) * c, -2000.0f), f = ex2(d);
        if (ENT) t = mul2(fma2(s, f2(d, d), t), f2(f, f));
        s = mul2(s, f2(f, f));
        m = to;
    }
    __device__ __forceinline__ void take(const uint4 (&raw)[kU], float c)
    {
        const float b = max_of<Ty, kU>(raw);
        if (!(b <= m)) move(max_nan(m, b), c);  // NaN comes in here too
        const float ref = m == -INFINITY ? 0.0f : m;
        const F2 neg = f2(-ref, -ref), cc = f2(c, c);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float a[Ty::L];
            Ty::unpack(raw[u], a);
#pragma unroll
            for (int l = 0; l < Ty::L; l += 2) {
                float lo, hi;
                un2(mul2(add2(f2(a[l], a[l + 1]), neg), cc), lo, hi);
                const F2 e = f2(ex2(lo), ex2(hi));
                s = add2(s, e);
                if (ENT) t = fma2(e, f2(fmaxf(lo, -2000.0f), fmaxf(hi, -2000.0f)), t);  // 0 * -inf is no 0
            }
        }
    }
    __device__ __forceinline__ void take_one(float x, float c)
    {
        if (!(x <= m)) move(max_nan(m, x), c);
        const float y = x == -INFINITY ? -2000.0f : (x - m) * c, e = ex2(y);
        s = add2(s, f2(e, 0.0f));
        if (ENT) t = add2(t, f2(e * fmaxf(y, -2000.0f), 0.0f));
    }
};

template <int N>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The sums of some threads relative to their largest value.
struct Stat {
    uint32_t order;  // of that value
    float s, t;
};

// Of N neighbouring lanes' Stats; o: the largest order.
template <int N>
__device__ __forceinline__ Stat lanes_joined(const Stat& st, uint32_t o, float c)
{
    const float d = st.order ? fmaxf((value_of(st.order) - value_of(o)) * c, -2000.0f) : -2000.0f, f = ex2(d);
    return {o, lanes_sum<N>(st.s * f), lanes_sum<N>((st.t + d * st.s) * f)};
}

// --------------------------------------------------------- top alternatives

// An element's rank among all: the value above, the lowest id first.  0: none.
__device__ __forceinline__ uint64_t entry_of(uint32_t order, uint32_t id) { return (uint64_t)order << 32 | (uint32_t)~id; }

template <class K>
__device__ __forceinline__ K larger(K a, K b) { return a > b ? a : b; }
template <class K>
__device__ __forceinline__ K smaller(K a, K b) { return a < b ? a : b; }

// The warp's values, largest in lane 0 (a bitonic network).
template <class K>
__device__ __forceinline__ K warp_sorted(K v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int o = size / 2; o > 0; o /= 2) {
            const K other = __shfl_xor_sync(kFull, v, o);
            const bool keep_large = ((lane & o) == 0) == ((lane & size) == 0);
            v = keep_large ? larger(v, other) : smaller(v, other);
        }
    return v;
}

// The 32 largest of two sorted lists, sorted.
template <class K>
__device__ __forceinline__ K warp_merged(K a, K b)
{
    const int lane = threadIdx.x & 31;
    a = larger(a, __shfl_sync(kFull, b, 31 - lane));  // the larger half, bitonic
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const K other = __shfl_xor_sync(kFull, a, o);
        a = (lane & o) == 0 ? larger(a, other) : smaller(a, other);
    }
    return a;
}

// A warp's sorted list of the largest entries it has been offered.
struct TopList {
    uint64_t mine = 0;   // lane i: the i-th largest
    uint64_t least = 0;  // entries must exceed it: the k-th of the list

    __device__ __forceinline__ void offer(uint64_t e, int k)
    {
        uint32_t want = __ballot_sync(kFull, e > least);
        if (want == 0) return;
        if (__popc(want) > 5) {
            mine = warp_merged(mine, warp_sorted(e > least ? e : 0));
        } else {
            const int lane = threadIdx.x & 31;
            while (want) {
                const uint64_t v = __shfl_sync(kFull, e, __ffs(want) - 1);
                want &= want - 1;
                const uint64_t up = __shfl_up_sync(kFull, mine, 1);
                if (mine < v) mine = lane > 0 && up < v ? up : v;
            }
        }
        least = __shfl_sync(kFull, mine, k - 1);
    }
};

// ---------------------------------------------------------------- the pass

struct Shared {
    uint32_t order[kThreads / 32], best[32];
    float2 sums[kThreads / 32];
    uint64_t list[kThreads / 32][32];
    uint8_t who[kThreads];
    uint32_t count[kThreads / 32];
    Stat all[kMaxSplit];               // cluster rank 0: of every CTA of the row
    uint64_t lists[kMaxSplit][32];
};

// TEAM threads (a CTA of kThreads, or a warp) of each of `split` CTAs read a
// row.  A warp per row is for short rows, whose sums a CTA would spend more
// time joining than reading.
template <class Ty, int TEAM, bool ENT, bool TOP>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const __grid_constant__ LogprobParams p)
{
    using T = typename Ty::T;
    constexpr int L = Ty::L;
    constexpr bool kWarp = TEAM == 32;
    __shared__ Shared sh;
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t split = kWarp ? 1u : (uint32_t)p.split;
    const uint32_t part = kWarp ? 0u : blockIdx.x % split;
    const uint64_t row = kWarp ? (uint64_t)blockIdx.x * (kThreads / 32) + warp : blockIdx.x / split;
    pdl_begin();
    if (row >= p.M) return;  // a whole warp, of a kernel without barriers then
    if (!kWarp && split > 1) cluster_arrive();  // this CTA runs: its shared memory may be written
    const uint32_t r = (uint32_t)row / p.T, tok = (uint32_t)row % p.T;
    const T* x = static_cast<const T*>(p.x[r]) + (uint64_t)tok * p.ld;
    const float c = p.scale * kLog2e;

    // head up to the first 16-byte boundary, whole vectors, tail
    uint32_t head = (uint32_t)((L - phase_of(x, L)) & (L - 1));
    if (head > p.V) head = p.V;
    const uint32_t nv = (p.V - head) / L, tail = p.V - head - nv * L;
    const uint32_t v0 = (uint32_t)((uint64_t)nv * part / split), v1 = (uint32_t)((uint64_t)nv * (part + 1) / split);
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);

    Running<Ty, ENT> run;
    const auto load = [&](uint4 (&raw)[kU], uint32_t v) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint64_t at = (uint64_t)v + u * TEAM;
            raw[u] = lowest_vector<Ty>();
            if (at < v1) raw[u] = TOP ? xv[at] : __ldcs(xv + at);  // read again by the alternatives
        }
    };
    // the next vectors are on their way while these are summed (16384 rows of 32000
    // bf16 with entropy: 181 -> 174 us; 20000 of 2000: 19.3 -> 17.7)
    uint4 raw[kU], next[kU];
    load(raw, v0 + tid);
    for (uint32_t v = v0 + tid; v < v1; v += TEAM * kU) {
        load(next, v + TEAM * kU);
        run.take(raw, c);
#pragma unroll
        for (int u = 0; u < kU; ++u) raw[u] = next[u];
    }
    const uint32_t order = v0 + tid < v1 ? order_of(run.m) : 0u;  // 0: a thread without vectors
    const bool edge = part == 0 && (uint32_t)tid < head + tail;
    const uint32_t edge_id = (uint32_t)tid < head ? (uint32_t)tid : head + nv * L + ((uint32_t)tid - head);
    float edge_x = -INFINITY;
    if (edge) {
        edge_x = Ty::ld1(x + edge_id);
        run.take_one(edge_x, c);
    }

    // the team's largest value, then its sums relative to that
    Stat st;
    st.order = __reduce_max_sync(kFull, edge || order ? order_of(run.m) : 0u);
    uint32_t tau = 0;
    if constexpr (TOP && kWarp) tau = warp_sorted(order);
    if constexpr (!kWarp) {
        if (lane == 0) sh.order[warp] = st.order;
        if constexpr (TOP) {  // the warp's four largest, one after the other
            constexpr int kBest = 32 / (kThreads / 32);
            uint32_t rest = order;
#pragma unroll
            for (int i = 0; i < kBest; ++i) {
                const uint32_t o = __reduce_max_sync(kFull, rest);
                if (lane == 0) sh.best[warp * kBest + i] = o;
                if (lane == __ffs(__ballot_sync(kFull, rest == o)) - 1) rest = 0;
            }
        }
        __syncthreads();
        st.order = __reduce_max_sync(kFull, sh.order[lane % (kThreads / 32)]);
        if constexpr (TOP) tau = warp_sorted(sh.best[lane]);  // every warp for itself
    }
    if constexpr (TOP) tau = __shfl_sync(kFull, tau, p.k - 1);
    run.move(value_of(st.order), c);
    float a, b;
    un2(run.s, a, b);
    st.s = lanes_sum<32>(a + b);
    st.t = 0.0f;
    if constexpr (ENT) {
        un2(run.t, a, b);
        st.t = lanes_sum<32>(a + b);
    }
    if constexpr (!kWarp) {
        if (lane == 0) sh.sums[warp] = make_float2(st.s, st.t);
        __syncthreads();
        const float2 of_warp = sh.sums[lane % (kThreads / 32)];
        st.s = lanes_sum<kThreads / 32>(of_warp.x);
        if constexpr (ENT) st.t = lanes_sum<kThreads / 32>(of_warp.y);
    }

    uint64_t best = 0;  // lane i of the team's first warp: the i-th largest entry
    if constexpr (TOP) {
        TopList list;
        // the head's and the tail's elements first
        if (warp == 0 || kWarp) list.offer(edge ? entry_of(order_of(edge_x), edge_id) : 0, p.k);
        const bool in = order != 0 && order >= tau;
        const uint32_t votes = __ballot_sync(kFull, in);
        uint32_t nwho;
        if constexpr (kWarp) {
            nwho = __popc(votes);
        } else {
            if (lane == 0) sh.count[warp] = __popc(votes);
            __syncthreads();
            uint32_t before = 0;
            nwho = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                before += w < warp ? sh.count[w] : 0;
                nwho += sh.count[w];
            }
            if (in) sh.who[before + __popc(votes & ((1u << lane) - 1))] = (uint8_t)tid;
            __syncthreads();
        }
        // Every vector of the threads in question, one a lane: the i-th of
        // each, then the next of each, so that ids rise and a tie is refused by
        // the list at once.
        const uint32_t items = (v1 - v0 + TEAM - 1) / TEAM * nwho;  // at most 2^29 + 2^8
        for (uint32_t base = kWarp ? 0 : warp * 32; base < items; base += TEAM) {
            const uint32_t item = base + lane;
            const uint32_t i = item / nwho, j = item - i * nwho;
            const uint32_t who = kWarp ? __fns(votes, 0, (int)j + 1) : sh.who[j];
            const uint32_t at = v0 + i * TEAM + who;
            uint4 raw[1] = {};
            uint32_t o = 0;
            if (item < items && at < v1) {
                raw[0] = xv[at];
                o = order_of(max_of<Ty, 1>(raw));
            }
            // a vector with one at or above tau: an element a lane
            for (uint32_t hots = __ballot_sync(kFull, item < items && at < v1 && o >= tau); hots; hots &= hots - 1) {
                // Many are ties, of which the first fill the list: one goes on if its largest
                // value with its lowest id could get in (64 rows of 128000 fp16 of which a
                // mask leaves 5, 20 alternatives: 17 us, 119 if all go on).
                if (__popc(hots) > 4) hots &= __ballot_sync(kFull, entry_of(o, head + at * L) > list.least);
                if (hots == 0) break;
                const int src = __ffs(hots) - 1;
                const uint4 v = make_uint4(__shfl_sync(kFull, raw[0].x, src), __shfl_sync(kFull, raw[0].y, src),
                                           __shfl_sync(kFull, raw[0].z, src), __shfl_sync(kFull, raw[0].w, src));
                const uint32_t id = __shfl_sync(kFull, head + at * L, src) + lane;
                const int word = lane / (L / 4) & 3;
                const uint32_t w = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
                float a = __uint_as_float(w);
                if constexpr (L == 8) {
                    float lo, hi;
                    Ty::unpack2(w, lo, hi);
                    a = lane & 1 ? hi : lo;
                }
                const uint32_t mine = order_of(a);
                list.offer(lane < L && mine >= tau ? entry_of(mine, id) : 0, p.k);
            }
        }
        best = list.mine;
        if constexpr (!kWarp) {
            sh.list[warp][lane] = best;
#pragma unroll
            for (int n = kThreads / 64; n > 0; n /= 2) {  // half of the lists into the other half
                __syncthreads();
                if (warp < n && sh.list[warp + n][0] != 0) {
                    best = warp_merged(best, sh.list[warp + n][lane]);
                    sh.list[warp][lane] = best;
                }
            }
        }
    }

    if (!kWarp && split > 1) {  // the other CTAs' results to the cluster's first
        cluster_wait();
        if (threadIdx.x == 0) *cluster_at(&sh.all[part], 0) = st;
        if (TOP && warp == 0) *cluster_at(&sh.lists[part][lane], 0) = best;
        cluster_arrive();
        cluster_wait();
        if (part != 0) return;
        if (warp != 0) return;
        st = lane % kMaxSplit < split ? sh.all[lane % kMaxSplit] : Stat{0u, 0.0f, 0.0f};
        st = lanes_joined<kMaxSplit>(st, __reduce_max_sync(kFull, st.order), c);
        if (TOP)
            for (uint32_t q = 1; q < split; ++q)
                if (sh.lists[q][0] > __shfl_sync(kFull, best, p.k - 1)) best = warp_merged(best, sh.lists[q][lane]);
    }
    if (!kWarp && warp != 0) return;

    // the row's results; a row whose every scaled value is -inf has no
    // distribution: lse and its log probabilities are -inf, its entropy 0.  One
    // whose largest is +inf, or with a NaN, is NaN.
    const float top = value_of(st.order), peak = top * p.scale;
    const bool empty = peak == -INFINITY;
    const float ln_s = peak == INFINITY ? NAN : logf(st.s);
    if (lane == 0) {
        const int64_t id = id_at(p.ids[r], p.ids64, tok);
        float lp = 0.0f;
        if (id >= 0 && id < (int64_t)p.V) lp = empty ? -INFINITY : z_below(Ty::ld1(x + id), top, p.scale) - ln_s;
        p.logprob[row] = lp;
        p.lse[row] = empty ? -INFINITY : __fmaf_rn(top, p.scale, ln_s);
        if (ENT) p.entropy[row] = empty ? 0.0f : ln_s - kLn2 * (st.t / st.s);
    }
    if (TOP && lane < p.k) {
        const float v = value_of((uint32_t)(best >> 32));
        p.top_logprob[row * p.k + lane] = empty ? -INFINITY : z_below(v, top, p.scale) - ln_s;
        p.top_id[row * p.k + lane] = (int32_t)~(uint32_t)best;
    }
}

// --------------------------------------------------------------- gradient
//
// dx_j = scale * (g (d_jt - p_j) - h p_j (ln p_j + H)), p_j = e^(z_j - lse):
// one pass, each logit read once, each gradient written once.  A warp takes
// kU vectors a lane of one row.  Rows of zero gradients (ignored tokens) and
// rows without a distribution are written as zeros without being read.

template <class Ty, bool ENT>
struct GradRow {
    float scale, lse, g, h, H, at_target;
    uint32_t target;

    // z - lse rounds once, at its own size, and lse came rounded at its: p is off by
    // (|ln p| + |lse|) 2^-24 of itself, beside the exponential's 2^-22
    __device__ __forceinline__ float at(float x) const
    {
        const float lp = __fmaf_rn(x, scale, -lse);
        const float e = ex2(lp * kLog2e);
        float d = g * e;
        if (ENT) d += h * e * (fmaxf(lp, -2000.0f) + H);  // 0 * -inf is no 0
        return d;
    }
};

// MIXED: some row's logits and gradients lie at different 16-byte phases.
template <class Ty, bool ENT, bool MIXED>
__global__ void __launch_bounds__(kThreads) logprob_grad_kernel(const __grid_constant__ LogprobGradParams p)
{
    using T = typename Ty::T;
    constexpr int L = Ty::L;
    constexpr uint32_t TV = 32 * kU;
    const int lane = threadIdx.x & 31;
    pdl_begin();
    const uint64_t w = p.first + (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint64_t row = w / p.tiles;
    const uint32_t tile = (uint32_t)(w % p.tiles);
    if (row >= p.M) return;
    const uint32_t r = (uint32_t)row / p.T, tok = (uint32_t)row % p.T;
    const T* x = static_cast<const T*>(p.x[r]) + (uint64_t)tok * p.ld;
    T* dx = static_cast<T*>(p.dx[r]) + (uint64_t)tok * p.gld;
    const int64_t id = id_at(p.ids[r], p.ids64, tok);
    const bool known = id >= 0 && id < (int64_t)p.V;
    const float lse = p.lse[row], dl = known ? p.dlogprob[row] : 0.0f;
    GradRow<Ty, ENT> q;
    q.scale = p.scale;
    q.lse = lse;
    q.g = -dl * p.scale;
    q.h = ENT ? -p.dentropy[row] * p.scale : 0.0f;
    q.H = ENT ? p.entropy[row] : 0.0f;
    q.at_target = dl * p.scale;
    q.target = known ? (uint32_t)id : 0xffffffffu;
    const bool zeros = lse == -INFINITY || (q.g == 0.0f && q.h == 0.0f);

    // head up to the gradient row's first 16-byte boundary, whole vectors, tail
    uint32_t head = (uint32_t)((L - phase_of(dx, L)) & (L - 1));
    if (head > p.V) head = p.V;
    const uint32_t nv = (p.V - head) / L, tail = p.V - head - nv * L;
    if (tile == 0 && (uint32_t)lane < head + tail) {
        const uint32_t e = (uint32_t)lane < head ? (uint32_t)lane : head + nv * L + ((uint32_t)lane - head);
        float d = 0.0f;
        if (!zeros) {
            d = q.at(Ty::ld1(x + e));
            if (e == q.target) d += q.at_target;
        }
        Ty::st1(dx + e, d);
    }
    // Where the logits' row lies at another phase, a vector of the gradient's needs
    // the two of the logits' that it straddles, its own lane's and the next one's
    // (4096 rows of 32001 bf16: 98 us; element by element 258; rows at one phase 80).
    const uint32_t off = MIXED ? (uint32_t)((uintptr_t)(x + head) & 15u) : 0u;
    const uint8_t* from = reinterpret_cast<const uint8_t*>(x + head) - off;
    uint4 raw[kU];
    uint32_t v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        v[u] = tile * TV + u * 32 + lane;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (v[u] < nv && !zeros) raw[u] = ldv(from + (uint64_t)v[u] * 16);
    }
    if (MIXED && off != 0 && !zeros) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            uint4 next;
            next.x = __shfl_down_sync(kFull, raw[u].x, 1);
            next.y = __shfl_down_sync(kFull, raw[u].y, 1);
            next.z = __shfl_down_sync(kFull, raw[u].z, 1);
            next.w = __shfl_down_sync(kFull, raw[u].w, 1);
            // its last elements lie there, so the aligned vector may be read
            if (v[u] < nv && (lane == 31 || v[u] + 1 == nv)) next = ldv(from + (uint64_t)v[u] * 16 + 16);
            raw[u] = shift_window(raw[u], next, (int)off);
        }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (v[u] >= nv) continue;
        const uint32_t e0 = head + v[u] * L;
        uint4 res = make_uint4(0u, 0u, 0u, 0u);
        if (!zeros) {
            float a[L];
            Ty::unpack(raw[u], a);
#pragma unroll
            for (int l = 0; l < L; ++l) a[l] = q.at(a[l]);
            if (q.target - e0 < (uint32_t)L) {
#pragma unroll
                for (int l = 0; l < L; ++l)
                    if (e0 + l == q.target) a[l] += q.at_target;
            }
            res = Ty::pack(a);
        }
        stv(dx + e0, res);
    }
}

template <class Ty, bool ENT, bool TOP>
cudaError_t launch_logprob_as(const LogprobParams& p, bool warp, cudaStream_t s)
{
    if (warp)
        return launch_pdl(logprob_kernel<Ty, 32, ENT, TOP>, dim3((unsigned)((p.M + kThreads / 32 - 1) / (kThreads / 32))), kThreads, 0, s, p);
    if (p.split == 1) return launch_pdl(logprob_kernel<Ty, kThreads, ENT, TOP>, dim3(p.M), kThreads, 0, s, p);
    return launch_pdl_clusters(logprob_kernel<Ty, kThreads, ENT, TOP>, p.M * (unsigned)p.split, kThreads, 0, (unsigned)p.split, s, p);
}

template <class F>
cudaError_t with_float(int dtype, F&& f)
{
    switch (dtype) {
    case kF32: return f.template operator()<F32T>();
    case kBF16: return f.template operator()<BF16T>();
    case kF16: return f.template operator()<F16T>();
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// CTAs per row.  Parts of a row want a cluster's barriers and merges, 2 us and
// more: a few rows are split as long as the parts of all still find an idle SM
// and have 8 KB (1 row of 256 KB with 20 alternatives in 1 / 2 / 4 / 8 parts: 21.3
// / 14.3 / 10.0 / 9.0 us, 64 rows of it 25.0 / 15.6 / 13.5 / 15.6), then as long
// as they find a free slot and have 64 KB (150 rows of 512 KB: 41.4 / 27.2 / 24.6 /
// 29.5); more rows are not (1500 of 64 KB: 34 / 46 / 73 / 141).
int logprob_split(uint64_t M, uint64_t V, int dtype)
{
    const uint64_t bytes = V * (dtype == kF32 ? 4 : 2);
    uint64_t split = 1;
    while (split < kMaxSplit) {
        const uint64_t ctas = 2 * split * M, part = bytes / (2 * split);
        if (!(ctas <= 148 * 2 && part >= 8192) && !(ctas <= 148 * 5 && part >= 65536)) break;
        split *= 2;
    }
    return (int)split;
}

cudaError_t launch_logprob(int dtype, const LogprobParams& p, cudaStream_t s)
{
    const uint64_t bytes = (uint64_t)p.V * (dtype == kF32 ? 4 : 2);
    const bool warp = p.split == 1 && bytes <= 8192 && p.M > 8 * 148;
    return with_float(dtype, [&]<class Ty>() -> cudaError_t {
        if (p.entropy) return p.k ? launch_logprob_as<Ty, true, true>(p, warp, s) : launch_logprob_as<Ty, true, false>(p, warp, s);
        return p.k ? launch_logprob_as<Ty, false, true>(p, warp, s) : launch_logprob_as<Ty, false, false>(p, warp, s);
    });
}

cudaError_t launch_logprob_grad(int dtype, LogprobGradParams p, int* launches, cudaStream_t s)
{
    const uint32_t L = dtype == kF32 ? 4 : 8;
    const uint32_t per = 32 * kU * L;
    p.tiles = (uint32_t)(((uint64_t)p.V + per - 1) / per);
    const uint64_t work = ((uint64_t)p.M * p.tiles + kThreads / 32 - 1) / (kThreads / 32);
    bool mixed = p.T > 1 && (p.ld - p.gld) % L != 0;
    for (uint32_t r = 0; r < p.M / p.T; ++r) mixed = mixed || ((uintptr_t)p.x[r] - (uintptr_t)p.dx[r]) % 16 != 0;
    for (uint64_t at = 0; at < work; at += kMaxGrid) {
        p.first = at * (kThreads / 32);
        const dim3 grid((unsigned)(work - at < kMaxGrid ? work - at : kMaxGrid));
        const cudaError_t e = with_float(dtype, [&]<class Ty>() -> cudaError_t {
            const auto as = [&]<bool ENT, bool MIXED>() {
                return launch_pdl(logprob_grad_kernel<Ty, ENT, MIXED>, grid, kThreads, 0, s, p);
            };
            if (p.dentropy) return mixed ? as.template operator()<true, true>() : as.template operator()<true, false>();
            return mixed ? as.template operator()<false, true>() : as.template operator()<false, false>();
        });
        if (e != cudaSuccess) return e;
        *launches += 1;
    }
    return cudaSuccess;
}

}  // namespace rr
