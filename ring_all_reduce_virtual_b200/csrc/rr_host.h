// rr_host.h -- host-side pieces shared by the C ABI's files (rr_api.cu,
// rr_clip_api.cu, rr_embed_api.cu): call statistics and the last error of a
// thread, argument checks, the bucket plan.  Not part of the C ABI.
#pragma once

#include <algorithm>
#include <chrono>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <string>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "rr.h"
#include "rr_internal.h"

struct rr_bucket_plan {
    int ntensors = 0;
    int grad_dtype = RR_BF16;
    size_t cap_bytes = 0;
    std::vector<uint64_t> numel;   // per tensor
    std::vector<uint64_t> offset;  // per tensor: element offset in its bucket
    std::vector<int> bucket_of;    // per tensor
    std::vector<int> first;        // per bucket: first tensor
    std::vector<int> count;        // per bucket: number of tensors
    std::vector<uint64_t> bnumel;  // per bucket: elements
};

namespace rr {

inline thread_local rr_stats_t t_stats{};
inline thread_local std::string t_error;


inline rr_status_t fail(rr_status_t st, const std::string& why)
{
    t_error = why;
    return st;
}

inline rr_status_t cuda_fail(cudaError_t e, const char* where)
{
    t_error = std::string(where) + ": " + cudaGetErrorString(e);
    return RR_ERR_CUDA;
}

inline bool env_flag(const char* name)
{
    const char* v = std::getenv(name);
    return v && *v && std::strcmp(v, "0") != 0;
}

inline size_t esize(rr_dtype_t d) { return d == RR_BF16 || d == RR_F16 ? 2u : 4u; }

inline bool dtype_ok(rr_dtype_t d) { return d == RR_F32 || d == RR_BF16 || d == RR_I32 || d == RR_F16; }
inline bool op_ok(rr_op_t o) { return o >= RR_SUM && o <= RR_PROD; }

inline const char* algo_name(int a)
{
    switch (a) {
    case RR_ALGO_AUTO: return "auto";
    case RR_ALGO_RING: return "ring";
    case RR_ALGO_ONESHOT: return "oneshot";
    case RR_ALGO_TREE: return "tree";
    case RR_ALGO_TREE_ONESHOT: return "tree_oneshot";
    case RR_ALGO_TWO_SHOT: return "two_shot";
    case RR_ALGO_DOUBLE_RING: return "double_ring";
    }
    return "?";
}

// Common checks of dtype, op and rank count.
inline rr_status_t check_basic(int n, rr_dtype_t dtype, rr_op_t op)
{
    if (n < 1 || n > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    if (!dtype_ok(dtype)) return fail(RR_ERR_INVALID_ARG, "unknown dtype");
    if (!op_ok(op)) return fail(RR_ERR_INVALID_ARG, "unknown op");
    if (dtype == RR_I32 && op == RR_AVG) return fail(RR_ERR_UNSUPPORTED, "AVG is not defined for int32");
    return RR_OK;
}

// Element counts above 2^48 (far beyond any device memory) are refused, so
// count * 64 ranks * 4 bytes stays below 2^56 and no byte range wraps.
inline constexpr uint64_t kMaxElems = 1ull << 48;

inline rr_status_t check_count(uint64_t count)
{
    if (count > kMaxElems) return fail(RR_ERR_INVALID_ARG, "element count above 2^48");
    return RR_OK;
}

struct Span {
    uintptr_t lo, hi;
    bool out;
};

// The spans of a call with one or two buffers per rank, kept on the stack so
// that a call allocates nothing on the host either.
struct SpanBuf {
    Span s[2 * RR_MAX_RANKS];
    size_t n = 0;
    void push_back(const Span& x) { s[n++] = x; }
    Span* begin() { return s; }
    Span* end() { return s + n; }
    size_t size() const { return n; }
    Span& operator[](size_t i) { return s[i]; }
};

// Every output span must be non-NULL and overlap no other span; inputs may
// overlap one another (they are only read).
template <class Spans>
inline rr_status_t check_spans(Spans& s)
{
    for (const Span& a : s)
        if (a.lo == 0) return fail(RR_ERR_INVALID_ARG, "NULL buffer pointer");
    const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    if (!std::is_sorted(s.begin(), s.end(), before)) std::sort(s.begin(), s.end(), before);
    for (size_t i = 0; i < s.size(); ++i)
        for (size_t j = i + 1; j < s.size() && s[j].lo < s[i].hi; ++j)
            if (s[i].out || s[j].out) return fail(RR_ERR_INVALID_ARG, "buffers overlap (or repeat)");
    return RR_OK;
}

// Every pointer on a boundary of its element size (a device access of an
// element at any other address faults).
inline rr_status_t check_elem_aligned(const void* const* p, int n, size_t es)
{
    for (int i = 0; i < n; ++i)
        if ((uintptr_t)p[i] % es != 0) return fail(RR_ERR_INVALID_ARG, "buffer not aligned to its element size");
    return RR_OK;
}

// True when all pointers agree modulo 16 bytes.
inline bool same_phase(const void* const* p, int n)
{
    for (int i = 1; i < n; ++i)
        if (((uintptr_t)p[i] & 15u) != ((uintptr_t)p[0] & 15u)) return false;
    return true;
}

// Optional (RR_DEBUG=1): reject pointers the driver does not know as device
// or managed memory, before any launch.
inline rr_status_t check_device_ptrs(const void* const* p, int n)
{
    static const bool debug = env_flag("RR_DEBUG");  // read once: getenv scans the environment
    if (!debug) return RR_OK;
    for (int i = 0; i < n; ++i) {
        cudaPointerAttributes a{};
        if (cudaPointerGetAttributes(&a, p[i]) != cudaSuccess ||
            (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)) {
            cudaGetLastError();
            return fail(RR_ERR_INVALID_ARG, "pointer is not device memory");
        }
    }
    return RR_OK;
}

// The same for a call's spans, which leave out tensors without elements.
inline rr_status_t check_device_spans(const std::vector<Span>& spans)
{
    for (const Span& s : spans) {
        const void* p = reinterpret_cast<const void*>(s.lo);
        const rr_status_t st = check_device_ptrs(&p, 1);
        if (st != RR_OK) return st;
    }
    return RR_OK;
}

// Optional (RR_DEBUG=1): after a call that enqueued work, synchronise its
// stream (unless the stream is being captured into a graph) and report a
// kernel fault, or a bounded device wait that ran out, at the call that
// caused it instead of at some later synchronisation.
inline rr_status_t debug_check(rr_status_t st, cudaStream_t stream)
{
    static const bool debug = env_flag("RR_DEBUG");
    if (!debug || st != RR_OK || t_stats.launches == 0) return st;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return st;
    }
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "RR_DEBUG: the call's kernels failed");
    unsigned int ran_out = 0, in_flight = 0;
    if ((e = take_bulk_timeouts(&ran_out, &in_flight)) != cudaSuccess) return cuda_fail(e, "RR_DEBUG: reading the wait counters");
    if (ran_out || in_flight)
        return fail(RR_ERR_TIMEOUT, "RR_DEBUG: bounded device waits ran out on " + std::to_string(ran_out) +
                                        " tiles during this call; copies not seen to land: " + std::to_string(in_flight));
    return st;
}

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return b ? (a + b - 1) / b : 0; }

inline void log_call(const char* what, int n, size_t count, rr_dtype_t dtype, int op, int algo)
{
    static const bool on = env_flag("RR_LOG");
    if (on)
        std::fprintf(stderr, "[rr] %s nranks=%d count=%zu dtype=%d op=%d algo=%s launches=%d\n", what, n,
                     count, (int)dtype, op, algo_name(algo), t_stats.launches);
}

inline void stats_begin(int algo, int n, uint64_t S)
{
    t_stats = rr_stats_t{};
    t_stats.algo = algo;
    t_stats.nranks = n;
    t_stats.bytes_per_rank = S;
}

inline uint64_t now_ns()
{
    return (uint64_t)std::chrono::duration_cast<std::chrono::nanoseconds>(
               std::chrono::steady_clock::now().time_since_epoch())
        .count();
}

// One API call: an NVTX range named for it (for timeline tools; a no-op
// when none is attached), and its host time, entry to return, into the
// call's statistics.
struct CallTimer {
    uint64_t t0;
    explicit CallTimer(const char* name)
    {
        nvtxRangePushA(name);
        t0 = now_ns();
    }
    ~CallTimer()
    {
        t_stats.host_ns = now_ns() - t0;
        nvtxRangePop();
    }
};

// A launch, its host time added to the call's statistics.
template <class F>
cudaError_t timed_launch(F&& f)
{
    const uint64_t t0 = now_ns();
    const cudaError_t e = f();
    t_stats.launch_ns += now_ns() - t0;
    return e;
}

// Checks buckets [b0, b0 + nb) of a plan and the gradients they cover, whose
// spans (every rank's copy of every tensor in the range) are added to
// `spans`; *t0 and *nt are the range's first tensor and tensor count.
inline rr_status_t bucket_range_spans(const rr_bucket_plan_t* plan, int b0, int nb, const void* const* grads, int nranks,
                                      int* t0, int* nt, std::vector<Span>& spans)
{
    if (!plan) return fail(RR_ERR_INVALID_ARG, "NULL plan");
    if (nranks < 1 || nranks > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    const int nbk = (int)plan->first.size();
    if (b0 < 0 || nb < 1 || b0 >= nbk || nb > nbk - b0) return fail(RR_ERR_INVALID_ARG, "bad bucket");
    if (!grads) return fail(RR_ERR_INVALID_ARG, "NULL gradient array");
    *t0 = plan->first[b0];
    *nt = plan->first[b0 + nb - 1] + plan->count[b0 + nb - 1] - *t0;
    const uint64_t es = esize((rr_dtype_t)plan->grad_dtype);
    spans.reserve(spans.size() + (size_t)nranks * *nt);
    for (int r = 0; r < nranks; ++r)
        for (int t = *t0; t < *t0 + *nt; ++t) {
            const void* g = grads[(size_t)r * plan->ntensors + t];
            if (plan->numel[t] == 0) continue;
            if (((uintptr_t)g & (es - 1)) != 0) return fail(RR_ERR_INVALID_ARG, "gradient not aligned to its element size");
            spans.push_back({(uintptr_t)g, (uintptr_t)g + plan->numel[t] * es, true});
        }
    return RR_OK;
}

// The same for a call without other buffers: the gradients pairwise disjoint.
inline rr_status_t bucket_range_check(const rr_bucket_plan_t* plan, int b0, int nb, const void* const* grads, int nranks,
                                      int* t0, int* nt)
{
    std::vector<Span> spans;
    const rr_status_t st = bucket_range_spans(plan, b0, nb, grads, nranks, t0, nt, spans);
    return st != RR_OK ? st : check_spans(spans);
}

// The segments of a fused sync of buckets [b0, b0 + nb) as launch tables:
// every bucket is chunked over its own flat index (chunk size ceil(bucket
// numel / N)) exactly as a sync of that bucket alone, and its tensors are
// split at its chunk boundaries into segments (tensor, chunk); segments of
// consecutive buckets share a launch until the parameter block is full, so a
// range costs a few launches instead of one per bucket, with the same bits.
// Fills p's pointers and segments and calls flush(tensors in p) for each
// launch that has any; grads may be NULL for a walk that only counts.
template <class Flush>
rr_status_t for_each_fold_launch(const rr_bucket_plan_t* plan, int b0, int nb, void* const* grads, int n,
                                 BucketFoldParams& p, Flush&& flush)
{
    rr_status_t st = RR_OK;
    int lt = 0;  // tensors in the current launch
    p.nseg = 0;
    for (int b = b0; b < b0 + nb && st == RR_OK; ++b) {
        const uint64_t C = ceil_div(plan->bnumel[b], (uint64_t)n);  // this bucket's chunk size
        for (int t = plan->first[b]; t < plan->first[b] + plan->count[b] && st == RR_OK; ++t) {
            const uint64_t lo = plan->offset[t], hi = lo + plan->numel[t];  // offsets are bucket-relative
            const int nsegs_t = hi > lo ? (int)((hi - 1) / C - lo / C + 1) : 0;
            if (lt + 1 > kMaxBucketTensors || (lt + 1) * n > kMaxBucketPtrs || p.nseg + nsegs_t > kMaxBucketSegs) {
                if (p.nseg > 0) st = flush(lt);
                p.nseg = 0;
                lt = 0;
            }
            for (int r = 0; grads && r < n; ++r) p.grad[lt * n + r] = grads[(size_t)r * plan->ntensors + t];
            for (uint64_t pos = lo; pos < hi;) {  // split the tensor at the bucket's chunk boundaries
                const uint64_t c = pos / C, end = std::min(hi, (c + 1) * C);
                p.seg[p.nseg++] = BucketSeg{(uint32_t)lt, (uint32_t)c, pos - lo, end - pos};
                pos = end;
            }
            ++lt;
        }
    }
    if (st == RR_OK && p.nseg > 0) st = flush(lt);
    return st;
}

// A C entry that lets no C++ exception out: the host's memory may be
// exhausted (the message fits a std::string's own storage).
template <class F>
rr_status_t guarded(F&& f)
{
    try {
        return f();
    } catch (const std::exception&) {
        return fail(RR_ERR_CUDA, "no host memory");
    }
}

}  // namespace rr
