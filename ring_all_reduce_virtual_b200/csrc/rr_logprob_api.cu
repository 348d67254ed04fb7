// rr_logprob_api.cu -- host side of the token log probabilities
// (rr_token_logprobs, rr_token_logprobs_grad in include/rr.h): argument checks
// and the rows' split.
#include "rr_host.h"
#include "rr_logprob.h"

using namespace rr;

namespace {

constexpr uint64_t kMaxRows = 0x7fffffffull;   // rows of all ranks
constexpr uint64_t kMaxWidth = 0x7ffffffeull;  // vocabulary, and elements from row to row

// Factors of log2 e and more stay within fp32, and where two logits differ by more than
// fp32 holds (2^128), their z differ by more than an exponential can show.
constexpr float kLeastScale = 0x1p-64f, kMostScale = 0x1p64f;

struct Rows {
    int n;
    uint64_t T, V, ld;
    rr_id_type_t ids;
    rr_dtype_t dtype;
    float scale;
};

rr_status_t check_rows(const Rows& s)
{
    if (s.n < 1 || s.n > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    if (!dtype_ok(s.dtype)) return fail(RR_ERR_INVALID_ARG, "unknown dtype");
    if (s.dtype == RR_I32) return fail(RR_ERR_UNSUPPORTED, "logits must be bf16, fp16 or fp32");
    if (s.ids != RR_ID_I32 && s.ids != RR_ID_I64) return fail(RR_ERR_INVALID_ARG, "unknown id type");
    if (s.V < 1 || s.V > kMaxWidth) return fail(RR_ERR_INVALID_ARG, "the vocabulary must be in 1..2^31-2");
    if (s.ld < s.V || s.ld > kMaxWidth) return fail(RR_ERR_INVALID_ARG, "the row stride must be in vocab..2^31-2");
    if (s.T > kMaxRows || s.T * (uint64_t)s.n > kMaxRows) return fail(RR_ERR_INVALID_ARG, "more than 2^31-1 tokens in all");
    if (!(s.scale >= kLeastScale && s.scale <= kMostScale)) return fail(RR_ERR_INVALID_ARG, "scale must be in 2^-64..2^64");
    return RR_OK;
}

// n buffers of T rows of V elements, ld apart.
rr_status_t add_rows(const void* const* p, const Rows& s, uint64_t ld, bool out, const char* what, std::vector<Span>& spans)
{
    const uint64_t es = esize(s.dtype), bytes = ((s.T - 1) * ld + s.V) * es;
    if (!p) return fail(RR_ERR_INVALID_ARG, std::string("NULL pointer array: ") + what);
    for (int i = 0; i < s.n; ++i) {
        if (!p[i]) return fail(RR_ERR_INVALID_ARG, std::string("NULL buffer pointer: ") + what);
        if ((uintptr_t)p[i] % es != 0)
            return fail(RR_ERR_INVALID_ARG, std::string("buffer not aligned to its element size: ") + what);
        spans.push_back({(uintptr_t)p[i], (uintptr_t)p[i] + bytes, out});
    }
    return check_device_ptrs(p, s.n);
}

rr_status_t add_ids(const void* const* p, const Rows& s, std::vector<Span>& spans)
{
    const uint64_t ib = s.ids == RR_ID_I64 ? 8 : 4;
    if (!p) return fail(RR_ERR_INVALID_ARG, "NULL pointer array: ids");
    for (int i = 0; i < s.n; ++i) {
        if (!p[i]) return fail(RR_ERR_INVALID_ARG, "NULL buffer pointer: ids");
        if ((uintptr_t)p[i] % ib != 0) return fail(RR_ERR_INVALID_ARG, "buffer not aligned to its element size: ids");
        spans.push_back({(uintptr_t)p[i], (uintptr_t)p[i] + s.T * ib, false});
    }
    return check_device_ptrs(p, s.n);
}

// One array of 4-byte values, `per` for every row of every rank.
rr_status_t add_values(const void* p, const Rows& s, uint64_t per, bool out, const char* what, std::vector<Span>& spans)
{
    if (!p) return fail(RR_ERR_INVALID_ARG, std::string("NULL pointer: ") + what);
    if ((uintptr_t)p % 4 != 0) return fail(RR_ERR_INVALID_ARG, std::string("buffer not aligned to its element size: ") + what);
    spans.push_back({(uintptr_t)p, (uintptr_t)p + s.T * (uint64_t)s.n * per * 4, out});
    return check_device_ptrs(&p, 1);
}

rr_status_t token_logprobs(const void* const* logits, const Rows& s, const void* const* ids, float* logprob, float* lse,
                           float* entropy, int k, float* top_logprob, int32_t* top_id, cudaStream_t stream)
{
    CallTimer timer("rr_token_logprobs");
    rr_status_t st = check_rows(s);
    if (st != RR_OK) return st;
    if (k < 0 || k > kMaxTop || (uint64_t)k > s.V)
        return fail(RR_ERR_INVALID_ARG, "top_k must be in 0..32 and at most the vocabulary");
    const uint64_t es = esize(s.dtype), M = s.T * (uint64_t)s.n;
    stats_begin(RR_ALGO_ONESHOT, s.n, s.T * s.V * es);
    if (M == 0) return RR_OK;
    std::vector<Span> spans;
    spans.reserve(2 * (size_t)s.n + 5);
    if ((st = add_rows(logits, s, s.ld, false, "logits", spans)) != RR_OK) return st;
    if ((st = add_ids(ids, s, spans)) != RR_OK) return st;
    if ((st = add_values(logprob, s, 1, true, "logprob", spans)) != RR_OK) return st;
    if ((st = add_values(lse, s, 1, true, "lse", spans)) != RR_OK) return st;
    if (entropy && (st = add_values(entropy, s, 1, true, "entropy", spans)) != RR_OK) return st;
    if (k > 0) {
        if ((st = add_values(top_logprob, s, k, true, "top_logprob", spans)) != RR_OK) return st;
        if ((st = add_values(top_id, s, k, true, "top_id", spans)) != RR_OK) return st;
    }
    if ((st = check_spans(spans)) != RR_OK) return st;
    LogprobParams p{};
    for (int r = 0; r < s.n; ++r) {
        p.x[r] = logits[r];
        p.ids[r] = ids[r];
    }
    p.ld = s.ld;
    p.T = (uint32_t)s.T;
    p.M = (uint32_t)M;
    p.V = (uint32_t)s.V;
    p.ids64 = s.ids == RR_ID_I64;
    p.scale = s.scale;
    p.k = k;
    p.split = logprob_split(M, s.V, s.dtype);
    p.logprob = logprob;
    p.lse = lse;
    p.entropy = entropy;
    p.top_logprob = top_logprob;
    p.top_id = top_id;
    const cudaError_t e = timed_launch([&] { return launch_logprob(s.dtype, p, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "log probability launch");
    t_stats.launches = 1;
    t_stats.steps = 1;
    t_stats.hbm_bytes = M * (s.V * es + 8 + (entropy ? 4 : 0) + 8 * (uint64_t)k);
    log_call("token_logprobs", s.n, s.T * s.V, s.dtype, RR_SUM, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

rr_status_t token_logprobs_grad(const void* const* logits, const Rows& s, const void* const* ids, const float* lse,
                                const float* entropy, const float* dlogprob, const float* dentropy, void* const* dlogits,
                                uint64_t gld, cudaStream_t stream)
{
    CallTimer timer("rr_token_logprobs_grad");
    rr_status_t st = check_rows(s);
    if (st != RR_OK) return st;
    if (gld < s.V || gld > kMaxWidth) return fail(RR_ERR_INVALID_ARG, "the gradients' row stride must be in vocab..2^31-2");
    if (dentropy && !entropy) return fail(RR_ERR_INVALID_ARG, "the entropy's gradient needs the entropy");
    const uint64_t es = esize(s.dtype), M = s.T * (uint64_t)s.n;
    stats_begin(RR_ALGO_ONESHOT, s.n, s.T * s.V * es);
    if (M == 0) return RR_OK;
    std::vector<Span> spans;
    spans.reserve(3 * (size_t)s.n + 4);
    if ((st = add_rows(dlogits, s, gld, true, "logit gradients", spans)) != RR_OK) return st;
    if (!logits) return fail(RR_ERR_INVALID_ARG, "NULL pointer array: logits");
    // a rank's gradients may take its logits' place, element for element
    std::vector<Span> read;
    read.reserve(s.n);
    if ((st = add_rows(logits, s, s.ld, false, "logits", read)) != RR_OK) return st;
    for (int r = 0; r < s.n; ++r)
        if (logits[r] != dlogits[r] || (s.ld != gld && s.T > 1)) spans.push_back(read[r]);
    if ((st = add_ids(ids, s, spans)) != RR_OK) return st;
    if ((st = add_values(lse, s, 1, false, "lse", spans)) != RR_OK) return st;
    if ((st = add_values(dlogprob, s, 1, false, "dlogprob", spans)) != RR_OK) return st;
    if (dentropy) {
        if ((st = add_values(entropy, s, 1, false, "entropy", spans)) != RR_OK) return st;
        if ((st = add_values(dentropy, s, 1, false, "dentropy", spans)) != RR_OK) return st;
    }
    if ((st = check_spans(spans)) != RR_OK) return st;
    LogprobGradParams p{};
    for (int r = 0; r < s.n; ++r) {
        p.x[r] = logits[r];
        p.ids[r] = ids[r];
        p.dx[r] = dlogits[r];
    }
    p.ld = s.ld;
    p.gld = gld;
    p.T = (uint32_t)s.T;
    p.M = (uint32_t)M;
    p.V = (uint32_t)s.V;
    p.ids64 = s.ids == RR_ID_I64;
    p.scale = s.scale;
    p.lse = lse;
    p.entropy = entropy;
    p.dlogprob = dlogprob;
    p.dentropy = dentropy;
    int launches = 0;
    const cudaError_t e = timed_launch([&] { return launch_logprob_grad(s.dtype, p, &launches, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "log probability gradient launch");
    t_stats.launches = launches;
    t_stats.steps = 1;
    t_stats.hbm_bytes = 2 * M * s.V * es;
    log_call("token_logprobs_grad", s.n, s.T * s.V, s.dtype, RR_SUM, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

}  // namespace

extern "C" {

rr_status_t rr_token_logprobs(const void* const* logits, size_t row_stride, const void* const* ids, rr_id_type_t id_type,
                              int nranks, size_t ntokens, size_t vocab, rr_dtype_t dtype, float scale, float* logprob,
                              float* lse, float* entropy, int top_k, float* top_logprob, int32_t* top_id,
                              cudaStream_t stream)
{
    return guarded([&] {
        return token_logprobs(logits, {nranks, ntokens, vocab, row_stride, id_type, dtype, scale}, ids, logprob, lse, entropy,
                              top_k, top_logprob, top_id, stream);
    });
}

rr_status_t rr_token_logprobs_grad(const void* const* logits, size_t row_stride, const void* const* ids,
                                   rr_id_type_t id_type, int nranks, size_t ntokens, size_t vocab, rr_dtype_t dtype,
                                   float scale, const float* lse, const float* entropy, const float* dlogprob,
                                   const float* dentropy, void* const* dlogits, size_t grad_stride, cudaStream_t stream)
{
    return guarded([&] {
        return token_logprobs_grad(logits, {nranks, ntokens, vocab, row_stride, id_type, dtype, scale}, ids, lse, entropy,
                                   dlogprob, dentropy, dlogits, grad_stride, stream);
    });
}

}  // extern "C"
