// rr_clip_api.cu -- host side of the global norm and clipping calls
// (rr_grad_norm, rr_clip_grads, rr_bucket_allreduce_clip in include/rr.h):
// argument checks, launch tables, the order of the passes.
#include <cmath>
#include <memory>

#include "rr_host.h"

using namespace rr;

namespace {

bool grad_dtype_ok(rr_dtype_t d) { return d == RR_F32 || d == RR_BF16 || d == RR_F16; }

// A tensor list's own fields, and its elements in all.
rr_status_t check_list(const rr_tensor_list_t* l, uint64_t* total)
{
    *total = 0;
    if (!l) return fail(RR_ERR_INVALID_ARG, "NULL tensor list");
    if (l->nranks < 1 || l->nranks > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    if (l->ntensors < 0) return fail(RR_ERR_INVALID_ARG, "negative tensor count");
    if (l->ntensors > 0 && (!l->ptrs || !l->numels || !l->dtypes))
        return fail(RR_ERR_INVALID_ARG, "NULL array in the tensor list");
    for (int t = 0; t < l->ntensors; ++t) {
        if (!dtype_ok(l->dtypes[t])) return fail(RR_ERR_INVALID_ARG, "unknown dtype");
        if (!grad_dtype_ok(l->dtypes[t])) return fail(RR_ERR_UNSUPPORTED, "gradients must be bf16, fp16 or fp32");
        if (l->numels[t] > kMaxElems || *total + l->numels[t] > kMaxElems)
            return fail(RR_ERR_INVALID_ARG, "element count above 2^48");
        *total += l->numels[t];
        if (l->numels[t] == 0) continue;
        for (int r = 0; r < l->nranks; ++r) {
            const uintptr_t a = (uintptr_t)l->ptrs[(size_t)r * l->ntensors + t];
            if (a == 0) return fail(RR_ERR_INVALID_ARG, "NULL buffer pointer");
            if ((a & (esize(l->dtypes[t]) - 1)) != 0)
                return fail(RR_ERR_INVALID_ARG, "gradient not aligned to its element size");
        }
    }
    return RR_OK;
}

// The first `ranks` ranks' tensors of a list as spans.
void add_spans(const rr_tensor_list_t* l, int ranks, bool out, std::vector<Span>& spans)
{
    for (int r = 0; r < ranks; ++r)
        for (int t = 0; t < l->ntensors; ++t)
            if (l->numels[t]) {
                const uintptr_t a = (uintptr_t)l->ptrs[(size_t)r * l->ntensors + t];
                spans.push_back({a, a + l->numels[t] * esize(l->dtypes[t]), out});
            }
}

// Whether [lo, hi) meets one of the spans, which are sorted and disjoint where
// they are written (check_spans has passed).
bool meets(const std::vector<Span>& spans, uintptr_t lo, uintptr_t hi)
{
    // read-only spans may nest, so every span that begins before hi counts
    auto it = std::lower_bound(spans.begin(), spans.end(), hi, [](const Span& s, uintptr_t x) { return s.lo < x; });
    if (it == spans.begin()) return false;
    if (std::prev(it)->out) return std::prev(it)->hi > lo;
    return std::any_of(spans.begin(), it, [lo](const Span& s) { return s.hi > lo; });
}

// The gradients' spans, then the norm and the workspace against them: two
// more spans at the end of a sorted list would have it sorted anew.
rr_status_t check_scratch(float* norm, void* ws, size_t have, size_t need, std::vector<Span>& spans)
{
    if (!norm) return fail(RR_ERR_INVALID_ARG, "NULL norm pointer");
    if ((uintptr_t)norm % 4 != 0) return fail(RR_ERR_INVALID_ARG, "norm not aligned to 4 bytes");
    if (!ws || (uintptr_t)ws % 8 != 0) return fail(RR_ERR_INVALID_ARG, "workspace NULL or not aligned to 8 bytes");
    if (have < need)
        return fail(RR_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
    const rr_status_t st = check_spans(spans);
    if (st != RR_OK) return st;
    const uintptr_t a = (uintptr_t)norm, b = (uintptr_t)ws;
    if (meets(spans, a, a + 4) || meets(spans, b, b + need) || (a < b + need && b < a + 4))
        return fail(RR_ERR_INVALID_ARG, "buffers overlap (or repeat): the norm or the workspace");
    return check_device_spans(spans);
}

rr_status_t check_clip(float max_norm, float eps)
{
    if (!(max_norm >= 0.0f)) return fail(RR_ERR_INVALID_ARG, "max_norm must be 0 or more (not NaN)");
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(RR_ERR_INVALID_ARG, "eps must be finite and 0 or more");
    return RR_OK;
}

// Elements up to which a call tries the one launch of a small set (its
// vectors have to fit the cluster's registers too).
constexpr uint64_t kSmallElems = 8 * 1024 * 32;

constexpr rr_dtype_t kGradTypes[] = {RR_F32, RR_BF16, RR_F16};

// One call's passes: launches on its stream, and the fp64 partial sums they
// leave in the workspace.
struct Passes {
    double* partial;
    cudaStream_t stream;
    bool bulk = false;  // the scaling runs by bulk copies
    float* clear = nullptr;  // the norm's word where the first launch is to zero it (ClipArgs::lost)
    int64_t count = 0;  // partials so far

    float* take_clear()  // once: the first launch zeroes the word
    {
        float* w = clear;
        clear = nullptr;
        return w;
    }

    // The norm's launches over rank 0's tensors, one type at a time.
    rr_status_t norm(const rr_tensor_list_t* l)
    {
        NormParams p;  // as it comes: every field that counts is set
        p.nt = 0;
        p.tile0[0] = 0;
        for (rr_dtype_t d : kGradTypes) {
            const uint64_t te = norm_tile_elems(d);
            for (int t = 0; t <= l->ntensors; ++t) {
                const bool end = t == l->ntensors;
                if ((end || p.nt == kNormTensors) && p.nt > 0) {
                    int slots = 0;
                    p.partial = partial + count;
                    p.clear = take_clear();
                    const cudaError_t e = timed_launch([&] { return launch_norm(d, p, &slots, stream); });
                    if (e != cudaSuccess) return cuda_fail(e, "norm launch");
                    t_stats.launches += 1;
                    count += slots;
                    p.nt = 0;
                }
                if (end || l->dtypes[t] != d || l->numels[t] == 0) continue;
                p.ptr[p.nt] = l->ptrs[t];
                p.len[p.nt] = l->numels[t];
                p.tile0[p.nt + 1] = p.tile0[p.nt] + ceil_div(l->numels[t], te);
                p.nt += 1;
            }
        }
        return RR_OK;
    }

    // The partials as the next launches read them: at most kMaxPartials.
    rr_status_t join(ClipArgs* a)
    {
        a->partial = partial;
        a->npartial = (int)count;
        if (count <= kMaxPartials) return RR_OK;
        int slots = 0;
        const cudaError_t e =
            timed_launch([&] { return launch_norm_join(partial, count, partial + count, &slots, stream); });
        if (e != cudaSuccess) return cuda_fail(e, "norm join launch");
        t_stats.launches += 1;
        a->partial = partial + count;
        a->npartial = slots;
        return RR_OK;
    }

    // The norm alone, of a call that had nothing to scale.
    rr_status_t finish(ClipArgs a)
    {
        a.lost = nullptr;
        const cudaError_t e = timed_launch([&] { return launch_norm_finish(a, stream); });
        if (e != cudaSuccess) return cuda_fail(e, "norm launch");
        t_stats.launches += 1;
        return RR_OK;
    }

    // The scaling's launches over tensors of one type; ptr(t, r), numel(t).
    // The first launch of a call writes the norm (and clears a.norm).
    template <class Ptr, class Len>
    rr_status_t scale(rr_dtype_t d, bool parked, int n, int ntensors, Ptr&& ptr, Len&& numel, ClipArgs& a)
    {
        std::unique_ptr<ScaleParams> p(new ScaleParams);  // as it comes: every field that counts is set
        p->nt = 0;
        p->tile0[0] = 0;
        const uint64_t te = scale_tile_elems(d, parked, bulk);
        const int most = std::min(kScaleTensors, kScalePtrs / n);
        for (int t = 0; t <= ntensors; ++t) {
            const bool end = t == ntensors;
            if ((end || p->nt == most) && p->nt > 0) {
                p->n = n;
                p->clip = a;
                const cudaError_t e = timed_launch([&] { return launch_clip_scale(d, parked, bulk, *p, stream); });
                if (e != cudaSuccess) return cuda_fail(e, "clip launch");
                t_stats.launches += 1;
                a.norm = nullptr;
                p->nt = 0;
            }
            if (end || numel(t) == 0) continue;
            void** q = &p->ptr[p->nt * n];
            for (int r = 0; r < n; ++r) q[r] = ptr(t, r);
            p->len[p->nt] = numel(t);
            p->vec[p->nt] = same_phase(q, n);
            p->tile0[p->nt + 1] = p->tile0[p->nt] + ceil_div(numel(t), te);
            p->nt += 1;
        }
        return RR_OK;
    }

    rr_status_t scale_list(const rr_tensor_list_t* l, ClipArgs& a)
    {
        for (rr_dtype_t d : kGradTypes) {
            const rr_status_t st = scale(
                d, false, l->nranks, l->ntensors, [&](int t, int r) { return l->ptrs[(size_t)r * l->ntensors + t]; },
                [&](int t) { return l->dtypes[t] == d ? (uint64_t)l->numels[t] : 0; }, a);
            if (st != RR_OK) return st;
        }
        return RR_OK;
    }
};

// The first `ranks` ranks' tensors of a list in the one launch of a small set:
// *done says whether it was one (tensors of one type, few enough).
rr_status_t small_list(const rr_tensor_list_t* l, uint64_t total, int ranks, bool scale, const ClipArgs& a,
                       cudaStream_t stream, bool* done)
{
    *done = false;
    if (total == 0 || total > kSmallElems) return RR_OK;
    ParkSmallParams p{};
    p.n = ranks;
    p.divisor = 1.0f;
    rr_dtype_t d = RR_F32;
    for (int t = 0; t < l->ntensors; ++t) {
        if (l->numels[t] == 0) continue;
        if (p.nseg > 0 && l->dtypes[t] != d) return RR_OK;
        if (p.nseg == kParkSegsSmall || (p.nseg + 1) * ranks > kParkPtrsSmall) return RR_OK;
        d = l->dtypes[t];
        for (int r = 0; r < ranks; ++r) p.grad[p.nseg * ranks + r] = l->ptrs[(size_t)r * l->ntensors + t];
        p.seg[p.nseg] = BucketSeg{(uint32_t)p.nseg, 0, 0, l->numels[t]};
        ++p.nseg;
    }
    if (!clip_small_plan(d, p, p.nseg)) return RR_OK;
    const cudaError_t e = timed_launch([&] { return launch_clip_small(d, scale, p, a, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "clip launch");
    t_stats.launches += 1;
    *done = true;
    return RR_OK;
}

// Partial sums that the norm's launches over a list leave, at most.
uint64_t norm_slots(const rr_tensor_list_t* l)
{
    uint64_t slots = 0;
    for (rr_dtype_t d : kGradTypes) {
        int nt = 0;
        for (int t = 0; t < l->ntensors; ++t) nt += l->dtypes[t] == d && l->numels[t] ? 1 : 0;
        slots += ceil_div(nt, kNormTensors) * (uint64_t)kNormCtas;
    }
    return slots;
}

// Tiles of the first pass over a bucket range, one partial sum each: the tiles
// of every run of a tensor inside one of its bucket's chunks.
uint64_t park_tiles(const rr_bucket_plan_t* plan, int b0, int nb, int n)
{
    uint64_t tiles = 0;
    const uint64_t te = park_tile_elems(plan->grad_dtype, n);
    for (int b = b0; b < b0 + nb; ++b) {
        const uint64_t C = ceil_div(plan->bnumel[b], (uint64_t)n);
        for (int t = plan->first[b]; t < plan->first[b] + plan->count[b]; ++t) {
            const uint64_t hi = plan->offset[t] + plan->numel[t];
            for (uint64_t pos = plan->offset[t]; pos < hi;) {
                const uint64_t end = std::min(hi, (pos / C + 1) * C);
                tiles += ceil_div(end - pos, te);
                pos = end;
            }
        }
    }
    return tiles;
}

// Partial sums, and the joined ones.
size_t workspace_bytes(uint64_t partials) { return (size_t)(partials + kJoinCtas) * sizeof(double); }

rr_status_t bucket_range_ok(const rr_bucket_plan_t* plan, int b0, int nb, int nranks)
{
    if (!plan) return fail(RR_ERR_INVALID_ARG, "NULL plan");
    if (nranks < 1 || nranks > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    const int nbk = (int)plan->first.size();
    if (b0 < 0 || nb < 1 || b0 >= nbk || nb > nbk - b0) return fail(RR_ERR_INVALID_ARG, "bad bucket");
    return RR_OK;
}

// The tensors of a bucket range on one rank as a list (a sync of one rank).
struct RangeList {
    std::vector<size_t> numels;
    std::vector<rr_dtype_t> dtypes;
    rr_tensor_list_t list{};
    RangeList(const rr_bucket_plan_t* plan, int t0, int nt, void* const* grads)
        : numels(plan->numel.begin() + t0, plan->numel.begin() + t0 + nt), dtypes(nt, (rr_dtype_t)plan->grad_dtype)
    {
        list.ptrs = grads ? grads + t0 : nullptr;
        list.numels = numels.data();
        list.dtypes = dtypes.data();
        list.ntensors = nt;
        list.nranks = 1;
    }
};

rr_status_t range_tensors(const rr_bucket_plan_t* plan, int b0, int nb, int* t0, int* nt)
{
    *t0 = plan->first[b0];
    *nt = plan->first[b0 + nb - 1] + plan->count[b0 + nb - 1] - *t0;
    return RR_OK;
}

uint64_t clip_partials(const rr_bucket_plan_t* plan, int b0, int nb, int n, const rr_tensor_list_t* list)
{
    uint64_t slots = list ? norm_slots(list) : 0;
    if (plan && n == 1) {
        int t0 = 0, nt = 0;
        range_tensors(plan, b0, nb, &t0, &nt);
        const RangeList own(plan, t0, nt, nullptr);
        slots += norm_slots(&own.list);
    } else if (plan) {
        slots += park_tiles(plan, b0, nb, n);
    }
    return slots;
}

rr_status_t list_bytes(const rr_tensor_list_t* l, uint64_t* S)
{
    *S = 0;
    for (int t = 0; t < l->ntensors; ++t) *S += l->numels[t] * esize(l->dtypes[t]);
    return RR_OK;
}

rr_status_t grad_norm(const rr_tensor_list_t* grads, float* norm, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    CallTimer timer("rr_grad_norm");
    uint64_t total = 0, S = 0;
    rr_status_t st = check_list(grads, &total);
    if (st != RR_OK) return st;
    list_bytes(grads, &S);
    stats_begin(RR_ALGO_ONESHOT, grads->nranks, S);
    std::vector<Span> spans;
    add_spans(grads, 1, false, spans);
    if ((st = check_scratch(norm, ws, ws_bytes, workspace_bytes(norm_slots(grads)), spans)) != RR_OK) return st;
    Passes run{static_cast<double*>(ws), stream};
    ClipArgs a{};
    a.norm = norm;
    bool done = false;
    if ((st = small_list(grads, total, 1, false, a, stream, &done)) != RR_OK) return st;
    if (!done && ((st = run.norm(grads)) != RR_OK || (st = run.join(&a)) != RR_OK || (st = run.finish(a)) != RR_OK))
        return st;
    t_stats.hbm_bytes = S;
    log_call("grad_norm", grads->nranks, total, RR_F32, RR_SUM, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

rr_status_t clip_grads(const rr_tensor_list_t* grads, float max_norm, float eps, float* norm, void* ws,
                       size_t ws_bytes, cudaStream_t stream)
{
    CallTimer timer("rr_clip_grads");
    uint64_t total = 0, S = 0;
    rr_status_t st = check_list(grads, &total);
    if (st != RR_OK || (st = check_clip(max_norm, eps)) != RR_OK) return st;
    const int n = grads->nranks;
    list_bytes(grads, &S);
    stats_begin(RR_ALGO_ONESHOT, n, S);
    std::vector<Span> spans;
    add_spans(grads, n, true, spans);
    if ((st = check_scratch(norm, ws, ws_bytes, workspace_bytes(norm_slots(grads)), spans)) != RR_OK) return st;
    Passes run{static_cast<double*>(ws), stream, n * S >= kBulkClipBytes && bulk_wait_counters()};
    ClipArgs a{};
    a.in_l2 = S <= kKeepBytes;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    a.lost = run.clear = run.bulk ? norm : nullptr;
    bool done = false;
    if ((st = small_list(grads, total, n, true, a, stream, &done)) != RR_OK) return st;
    if (!done) {
        if ((st = run.norm(grads)) != RR_OK || (st = run.join(&a)) != RR_OK) return st;
        if ((st = run.scale_list(grads, a)) != RR_OK) return st;
        if (a.norm && (st = run.finish(a)) != RR_OK) return st;  // nothing to scale: the norm alone
    }
    t_stats.steps = n > 1 ? 1 : 0;
    t_stats.bytes_sent_max = (uint64_t)(n - 1) * S;  // rank 0 sends its copy to every other
    t_stats.bytes_sent_total = t_stats.bytes_sent_max;
    t_stats.hbm_bytes = (uint64_t)((done ? 1 : 2) + n) * S;
    log_call("clip_grads", n, total, RR_F32, RR_SUM, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

rr_status_t bucket_allreduce_clip(const rr_bucket_plan_t* plan, int b0, int nb, void* const* grads, int nranks,
                                  rr_op_t op, const rr_tensor_list_t* synced, float max_norm, float eps, float* norm,
                                  void* ws, size_t ws_bytes, cudaStream_t stream)
{
    CallTimer timer("rr_bucket_allreduce_clip");
    if (op != RR_SUM && op != RR_AVG) return fail(RR_ERR_UNSUPPORTED, "bucket all-reduce takes SUM or AVG");
    rr_status_t st = check_clip(max_norm, eps);
    if (st != RR_OK || (st = bucket_range_ok(plan, b0, nb, nranks)) != RR_OK) return st;
    const int n = nranks;
    int t0 = 0, nt = 0;
    uint64_t rest = 0, S = 0, R = 0;
    if (synced) {
        if ((st = check_list(synced, &rest)) != RR_OK) return st;
        if (synced->ntensors == 0) synced = nullptr;  // no tensors: any rank count
    }
    if (synced) {
        if (synced->nranks != n) return fail(RR_ERR_INVALID_ARG, "the synced list has another number of ranks");
        list_bytes(synced, &R);
    }
    std::vector<Span> spans;
    if ((st = bucket_range_spans(plan, b0, nb, grads, n, &t0, &nt, spans)) != RR_OK) return st;
    const rr_dtype_t d = (rr_dtype_t)plan->grad_dtype;
    const uint64_t es = esize(d);
    uint64_t total = 0;
    for (int t = t0; t < t0 + nt; ++t) total += plan->numel[t];
    S = total * es;
    stats_begin(RR_ALGO_ONESHOT, n, S + R);
    if (synced) add_spans(synced, n, true, spans);
    const size_t need = workspace_bytes(clip_partials(plan, b0, nb, n, synced));
    if ((st = check_scratch(norm, ws, ws_bytes, need, spans)) != RR_OK) return st;
    Passes run{static_cast<double*>(ws), stream, n * (S + R) >= kBulkClipBytes && bulk_wait_counters()};
    ClipArgs a{};
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    const RangeList own(plan, t0, nt, grads);
    const bool twice = n > 1 && clip_folds_twice(n, d);
    a.lost = run.clear = run.bulk || twice ? norm : nullptr;
    // the range's launches, a pass at a time
    std::unique_ptr<BucketFoldParams> p(new BucketFoldParams);  // as it comes: every field that counts is set
    auto pass = [&](auto&& launch) {
        return for_each_fold_launch(plan, b0, nb, grads, n, *p, [&](int ntens) -> rr_status_t {
            const uint64_t te = park_tile_elems(d, n);
            p->tile0[0] = 0;
            for (int s = 0; s < p->nseg; ++s) p->tile0[s + 1] = p->tile0[s] + ceil_div(p->seg[s].len, te);
            p->n = n;
            p->divisor = (float)n;
            bool v = true;
            for (int t = 0; t < ntens; ++t) v = v && same_phase(&p->grad[t * n], n);
            p->vec_ok = v;
            const cudaError_t e = timed_launch([&] { return launch(ntens); });
            if (e != cudaSuccess) return cuda_fail(e, "bucket all-reduce launch");
            t_stats.launches += 1;
            return RR_OK;
        });
    };
    if (n == 1) {
        st = run.norm(&own.list);  // one rank: nothing to fold
    } else {
        st = pass([&](int ntens) {
            double* slots = run.partial + run.count;
            run.count += (int64_t)p->tile0[p->nseg];
            return twice ? launch_bucket_squares(d, op, *p, ntens, slots, run.take_clear(), stream)
                         : launch_bucket_park(d, op, *p, ntens, slots, run.take_clear(), stream);
        });
    }
    if (st != RR_OK) return st;
    if (synced && (st = run.norm(synced)) != RR_OK) return st;
    if ((st = run.join(&a)) != RR_OK) return st;
    if (twice)
        st = pass([&](int ntens) {
            const ClipArgs now = a;
            a.norm = nullptr;
            return launch_bucket_scaled(d, op, *p, ntens, now, stream);
        });
    else
        st = run.scale(
            d, n > 1, n, nt, [&](int t, int r) { return grads[(size_t)r * plan->ntensors + t0 + t]; },
            [&](int t) { return plan->numel[t0 + t]; }, a);
    if (st != RR_OK) return st;
    if (synced && (st = run.scale_list(synced, a)) != RR_OK) return st;
    if (a.norm && (st = run.finish(a)) != RR_OK) return st;
    t_stats.steps = 1;
    t_stats.bytes_sent_max = (uint64_t)(n - 1) * (S + R);
    t_stats.bytes_sent_total = (uint64_t)n * (uint64_t)(n - 1) * S + (uint64_t)(n - 1) * R;
    const uint64_t parked = d == RR_F32 || n == 1 ? S : 2 * S;
    t_stats.hbm_bytes = n == 1 ? 3 * S : twice ? 3 * (uint64_t)n * S : 2 * (uint64_t)n * S + 2 * parked;
    t_stats.hbm_bytes += (uint64_t)(2 + n) * R;
    log_call("bucket_allreduce_clip", n, total, d, op, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

}  // namespace

extern "C" {

rr_status_t rr_clip_workspace(const rr_bucket_plan_t* plan, int first_bucket, int nbuckets, int nranks,
                              const rr_tensor_list_t* list, size_t* bytes)
{
    return guarded([&]() -> rr_status_t {
        if (!bytes) return fail(RR_ERR_INVALID_ARG, "NULL workspace size output");
        rr_status_t st = RR_OK;
        uint64_t total = 0;
        if (plan && (st = bucket_range_ok(plan, first_bucket, nbuckets, nranks)) != RR_OK) return st;
        if (list && (st = check_list(list, &total)) != RR_OK) return st;
        if (!plan && !list) return fail(RR_ERR_INVALID_ARG, "NULL plan and NULL list");
        *bytes = workspace_bytes(clip_partials(plan, first_bucket, nbuckets, nranks, list));
        return RR_OK;
    });
}

rr_status_t rr_grad_norm(const rr_tensor_list_t* grads, float* norm, void* workspace, size_t workspace_bytes_,
                         cudaStream_t stream)
{
    return guarded([&] { return grad_norm(grads, norm, workspace, workspace_bytes_, stream); });
}

rr_status_t rr_clip_grads(const rr_tensor_list_t* grads, float max_norm, float eps, float* norm, void* workspace,
                          size_t workspace_bytes_, cudaStream_t stream)
{
    return guarded([&] { return clip_grads(grads, max_norm, eps, norm, workspace, workspace_bytes_, stream); });
}

rr_status_t rr_bucket_allreduce_clip(const rr_bucket_plan_t* plan, int first_bucket, int nbuckets, void* const* grads,
                                     int nranks, rr_op_t op, const rr_tensor_list_t* synced, float max_norm,
                                     float eps, float* norm, void* workspace, size_t workspace_bytes_,
                                     cudaStream_t stream)
{
    return guarded([&] {
        return bucket_allreduce_clip(plan, first_bucket, nbuckets, grads, nranks, op, synced, max_norm, eps, norm,
                                     workspace, workspace_bytes_, stream);
    });
}

}  // extern "C"
