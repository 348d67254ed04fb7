// rr_embed_api.cu -- host side of the embedding calls (rr_embedding,
// rr_embedding_grad in include/rr.h): argument checks, the access width, the
// workspace's layout.
#include <cmath>

#include "rr_host.h"

using namespace rr;

namespace {

constexpr uint64_t kMaxDim = 1ull << 20;       // row width
constexpr uint64_t kMaxTokens = 0x7fffffffull;  // tokens of all ranks: positions are 32 bits
constexpr uint64_t kMaxVocab = 0x7ffffffeull;   // id V itself must fit

struct Shape {
    int n;
    uint64_t T, V, D;
};

rr_status_t check_shape(const Shape& s, rr_id_type_t ids, rr_dtype_t dtype)
{
    if (s.n < 1 || s.n > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    if (!dtype_ok(dtype)) return fail(RR_ERR_INVALID_ARG, "unknown dtype");
    if (dtype == RR_I32) return fail(RR_ERR_UNSUPPORTED, "rows must be bf16, fp16 or fp32");
    if (ids != RR_ID_I32 && ids != RR_ID_I64) return fail(RR_ERR_INVALID_ARG, "unknown id type");
    if (s.D < 1 || s.D > kMaxDim) return fail(RR_ERR_INVALID_ARG, "the row width must be in 1..2^20");
    if (s.V < 1 || s.V > kMaxVocab) return fail(RR_ERR_INVALID_ARG, "the table must have 1..2^31-2 rows");
    if (s.T > kMaxTokens || s.T * (uint64_t)s.n > kMaxTokens)
        return fail(RR_ERR_INVALID_ARG, "more than 2^31-1 tokens in all");
    return RR_OK;
}

// n buffers of `bytes` each, on boundaries of `align` bytes, as spans.
rr_status_t add_buffers(const void* const* p, int n, uint64_t bytes, uint64_t align, bool out, const char* what,
                        std::vector<Span>& spans)
{
    if (!p) return fail(RR_ERR_INVALID_ARG, std::string("NULL pointer array: ") + what);
    for (int i = 0; i < n; ++i) {
        if (!p[i]) return fail(RR_ERR_INVALID_ARG, std::string("NULL buffer pointer: ") + what);
        if ((uintptr_t)p[i] % align != 0)
            return fail(RR_ERR_INVALID_ARG, std::string("buffer not aligned to its element size: ") + what);
        spans.push_back({(uintptr_t)p[i], (uintptr_t)p[i] + bytes, out});
    }
    return check_device_ptrs(p, n);
}

// Elements per access: the most, up to 16 bytes of es-byte elements, that
// divide the row width and on whose bytes (at most 16) every buffer starts.
int access_width(uint64_t D, size_t es, const void* const* a, int na, size_t es2, const void* const* b, int nb)
{
    for (int vec = (int)(16 / es); vec > 1; vec /= 2) {
        bool ok = D % (uint64_t)vec == 0;
        for (int i = 0; ok && i < na; ++i) ok = (uintptr_t)a[i] % std::min<size_t>(16, vec * es) == 0;
        for (int i = 0; ok && i < nb; ++i) ok = (uintptr_t)b[i] % std::min<size_t>(16, vec * es2) == 0;
        if (ok) return vec;
    }
    return 1;
}

rr_status_t embedding(const void* const* ids, rr_id_type_t id_type, const void* const* tables, void* const* outs, int n,
                      size_t T, size_t V, size_t D, rr_dtype_t dtype, float scale, cudaStream_t stream)
{
    CallTimer timer("rr_embedding");
    rr_status_t st = check_shape({n, T, V, D}, id_type, dtype);
    if (st != RR_OK) return st;
    const uint64_t es = esize(dtype), ib = id_type == RR_ID_I64 ? 8 : 4;
    stats_begin(RR_ALGO_ONESHOT, n, T * D * es);
    if (T == 0) return RR_OK;
    std::vector<Span> spans;
    spans.reserve(3 * (size_t)n);
    if ((st = add_buffers(ids, n, T * ib, ib, false, "ids", spans)) != RR_OK) return st;
    if ((st = add_buffers(tables, n, V * D * es, es, false, "tables", spans)) != RR_OK) return st;
    if ((st = add_buffers(outs, n, T * D * es, es, true, "outs", spans)) != RR_OK) return st;
    if ((st = check_spans(spans)) != RR_OK) return st;
    EmbedLookupParams p{};
    for (int r = 0; r < n; ++r) {
        p.ids[r] = ids[r];
        p.table[r] = tables[r];
        p.out[r] = outs[r];
    }
    p.T = (uint32_t)T;
    p.M = (uint32_t)(T * (uint64_t)n);
    p.V = V;
    p.D = (uint32_t)D;
    p.ids64 = id_type == RR_ID_I64;
    p.scale = scale;
    const int vec = access_width(D, es, tables, n, es, outs, n);
    const cudaError_t e = timed_launch([&] { return launch_embed_lookup(dtype, vec, p, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "embedding launch");
    t_stats.launches = 1;
    t_stats.hbm_bytes = (uint64_t)n * T * (ib + 2 * D * es);
    log_call("embedding", n, T * D, dtype, RR_SUM, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

// The gradient's workspace, in the order in which it is laid out; every part
// starts on a 256-byte boundary.
struct Layout {
    uint64_t key[2], pos[2], counts, part, arrived, bytes;
    uint32_t ntiles, K, nblk, Dp;
    int passes, bits;
};

uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

// Sorted positions per block: 32, fewer where that leaves a GPU of 148 SMs
// short of warps (one per block and slice of the columns), more where the
// partial sums would need more than 8192 rows.  With 8 / 16 / 32: 300 tokens of
// width 515 44 / 48 / 54 us waited for, 16384 of 2048 (16 here) 197 / 194 / 196;
// with 16 / 32 / 64, 65536 of 2048 111 / 105 / 108.
uint32_t block_positions(uint64_t M, uint64_t D)
{
    if (M > 32 * 4096) return (uint32_t)(32 * ceil_div(M, 32 * 4096));
    uint32_t k = 32;
    while (k > 8 && ceil_div(M, k) * ceil_div(D, kEmbedCols) < 148 * 32) k /= 2;
    return k;
}

Layout layout(uint64_t M, uint64_t V, uint64_t D)
{
    Layout l{};
    int total = 1;  // bits of the largest key, V
    while (V >> total) ++total;
    l.passes = (total + kSortMaxBits - 1) / kSortMaxBits;
    l.bits = std::max(2, (total + l.passes - 1) / l.passes);  // counts are read four digits at a time
    l.ntiles = (uint32_t)ceil_div(M, kSortTile);
    l.K = block_positions(M, D);
    l.nblk = (uint32_t)ceil_div(M, l.K);
    l.Dp = (uint32_t)up(D, 4);
    uint64_t at = 0;
    auto part = [&](uint64_t bytes) {
        const uint64_t here = at;
        at = up(at + bytes, 256);
        return here;
    };
    for (int k = 0; k < 2; ++k) l.key[k] = part(M * 4);
    for (int k = 0; k < 2; ++k) l.pos[k] = part(M * 4);
    l.counts = part(((uint64_t)l.passes * l.ntiles << l.bits) * 4);
    l.part = part(2ull * l.nblk * l.Dp * 4);
    l.arrived = part(ceil_div(D, kEmbedCols) * 4);
    l.bytes = at;
    return l;
}

rr_status_t embedding_grad(const void* const* ids, rr_id_type_t id_type, const void* const* grad_out, int n, size_t T,
                           size_t V, size_t D, rr_dtype_t dtype, rr_op_t op, float scale, int64_t padding,
                           void* const* grads, int nout, rr_dtype_t grad_dtype, int accumulate, void* ws,
                           size_t ws_bytes, cudaStream_t stream)
{
    CallTimer timer("rr_embedding_grad");
    rr_status_t st = check_shape({n, T, V, D}, id_type, dtype);
    if (st != RR_OK) return st;
    if (op != RR_SUM && op != RR_AVG) return fail(RR_ERR_UNSUPPORTED, "the embedding gradient takes SUM or AVG");
    if (nout < 1 || nout > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "the number of gradients must be in 1..64");
    if (grad_dtype != dtype && grad_dtype != RR_F32)
        return fail(RR_ERR_UNSUPPORTED, "the gradient has the rows' type or fp32");
    const uint64_t es = esize(dtype), gs = esize(grad_dtype), ib = id_type == RR_ID_I64 ? 8 : 4;
    stats_begin(RR_ALGO_ONESHOT, n, T * D * es);
    if (T == 0 && accumulate) return RR_OK;
    const uint64_t M = T * (uint64_t)n;
    const Layout l = layout(M, V, D);
    std::vector<Span> spans;
    spans.reserve(2 * (size_t)n + nout + 1);
    if (T > 0) {
        if ((st = add_buffers(ids, n, T * ib, ib, false, "ids", spans)) != RR_OK) return st;
        if ((st = add_buffers(grad_out, n, T * D * es, es, false, "output gradients", spans)) != RR_OK) return st;
    }
    if ((st = add_buffers(grads, nout, V * D * gs, gs, true, "table gradients", spans)) != RR_OK) return st;
    if (!ws || (uintptr_t)ws % 256 != 0)
        return fail(RR_ERR_INVALID_ARG, "workspace NULL or not aligned to 256 bytes");
    if (ws_bytes < l.bytes)
        return fail(RR_ERR_INVALID_ARG, "workspace too small: " + std::to_string(l.bytes) + " bytes are needed");
    spans.push_back({(uintptr_t)ws, (uintptr_t)ws + l.bytes, true});
    if ((st = check_spans(spans)) != RR_OK) return st;

    int launches = 0;
    cudaError_t e = cudaSuccess;
    if (T == 0) {  // no token: every row is zero
        for (int o = 0; o < nout && e == cudaSuccess; ++o) e = cudaMemsetAsync(grads[o], 0, V * D * gs, stream);
        if (e != cudaSuccess) return cuda_fail(e, "clearing the embedding gradient");
        return RR_OK;
    }
    EmbedGradParams p{};
    for (int r = 0; r < n; ++r) {
        p.ids[r] = ids[r];
        p.dout[r] = grad_out[r];
    }
    for (int o = 0; o < nout; ++o) p.grad[o] = grads[o];
    p.padding = padding;
    p.V = V;
    p.T = (uint32_t)T;
    p.M = (uint32_t)M;
    p.D = (uint32_t)D;
    p.ids64 = id_type == RR_ID_I64;
    p.nout = nout;
    p.accumulate = accumulate != 0;
    p.factor = op == RR_AVG ? (float)((double)scale / n) : scale;
    char* base = static_cast<char*>(ws);
    for (int k = 0; k < 2; ++k) {
        p.key[k] = reinterpret_cast<uint32_t*>(base + l.key[k]);
        p.pos[k] = reinterpret_cast<uint32_t*>(base + l.pos[k]);
    }
    p.counts = reinterpret_cast<uint32_t*>(base + l.counts);
    p.part = reinterpret_cast<float*>(base + l.part);
    p.arrived = reinterpret_cast<uint32_t*>(base + l.arrived);
    p.passes = l.passes;
    p.bits = l.bits;
    p.ntiles = l.ntiles;
    p.K = l.K;
    p.nblk = l.nblk;
    p.Dp = l.Dp;
    const int vec = access_width(D, es, grad_out, n, gs, grads, nout);
    e = timed_launch([&] { return launch_embed_sort(p, &launches, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "embedding gradient: sort launch");
    e = timed_launch([&] { return launch_embed_reduce(dtype, grad_dtype, vec, p, &launches, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "embedding gradient: sum launch");
    t_stats.launches = launches;
    t_stats.steps = 1;
    t_stats.bytes_sent_max = (uint64_t)(n - 1) * T * (ib + D * es);  // every rank's rows to every other
    t_stats.bytes_sent_total = (uint64_t)n * t_stats.bytes_sent_max;
    t_stats.hbm_bytes = M * (ib + D * es) + (accumulate ? 2 * std::min(M, (uint64_t)V) : (uint64_t)V) * D * gs * nout;
    log_call("embedding_grad", n, T * D, dtype, op, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

}  // namespace

extern "C" {

rr_status_t rr_embedding(const void* const* ids, rr_id_type_t id_type, const void* const* tables, void* const* outs,
                         int nranks, size_t ntokens, size_t vocab, size_t dim, rr_dtype_t dtype, float scale,
                         cudaStream_t stream)
{
    return guarded([&] {
        return embedding(ids, id_type, tables, outs, nranks, ntokens, vocab, dim, dtype, scale, stream);
    });
}

rr_status_t rr_embedding_grad_workspace(int nranks, size_t ntokens, size_t vocab, size_t dim, size_t* bytes)
{
    return guarded([&]() -> rr_status_t {
        if (!bytes) return fail(RR_ERR_INVALID_ARG, "NULL workspace size output");
        const rr_status_t st = check_shape({nranks, ntokens, vocab, dim}, RR_ID_I32, RR_F32);
        if (st == RR_OK) *bytes = (size_t)layout(ntokens * (uint64_t)nranks, vocab, dim).bytes;
        return st;
    });
}

rr_status_t rr_embedding_grad(const void* const* ids, rr_id_type_t id_type, const void* const* grad_out, int nranks,
                              size_t ntokens, size_t vocab, size_t dim, rr_dtype_t dtype, rr_op_t op, float scale,
                              int64_t padding_idx, void* const* grads, int ngrads, rr_dtype_t grad_dtype,
                              int accumulate, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return guarded([&] {
        return embedding_grad(ids, id_type, grad_out, nranks, ntokens, vocab, dim, dtype, op, scale, padding_idx, grads,
                              ngrads, grad_dtype, accumulate, workspace, workspace_bytes, stream);
    });
}

}  // extern "C"
