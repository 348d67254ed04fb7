// rr_muon_api.cu -- host side of the orthogonalisation and the Muon step
// (rr_orthogonalize, rr_muon_step in include/rr.h): argument checks, the
// iteration's scales, the order of the products, groups of matrices.
#include <cmath>
#include <memory>

#include "rr_host.h"
#include "rr_muon.h"

using namespace rr;

namespace {

constexpr uint64_t kMaxSide = 1ull << 20;    // rows and columns
constexpr int kMaxSteps = 64;
// Workspace of a group of matrices that run in the same launches, unless one
// alone needs more.
constexpr uint64_t kGroupBytes = 2ull << 30;

bool real_dtype(rr_dtype_t d) { return d == RR_F32 || d == RR_BF16 || d == RR_F16; }

struct Shape {
    uint32_t rows, cols;
    uint64_t numel() const { return (uint64_t)rows * cols; }
    uint32_t small() const { return std::min(rows, cols); }
};

rr_status_t check_list(const rr_matrix_list_t* l, const char* what)
{
    if (!l) return fail(RR_ERR_INVALID_ARG, std::string("NULL matrix list: ") + what);
    if (l->nranks < 1 || l->nranks > RR_MAX_RANKS) return fail(RR_ERR_INVALID_ARG, "nranks must be in 1..64");
    if (l->nmatrices < 0) return fail(RR_ERR_INVALID_ARG, "negative matrix count");
    if (l->nmatrices > 0 && (!l->ptrs || !l->rows || !l->cols || !l->dtypes))
        return fail(RR_ERR_INVALID_ARG, std::string("NULL array in the matrix list: ") + what);
    for (int t = 0; t < l->nmatrices; ++t) {
        if (!dtype_ok(l->dtypes[t])) return fail(RR_ERR_INVALID_ARG, "unknown dtype");
        if (!real_dtype(l->dtypes[t])) return fail(RR_ERR_UNSUPPORTED, "matrices must be bf16, fp16 or fp32");
        if (l->rows[t] > kMaxSide || l->cols[t] > kMaxSide)
            return fail(RR_ERR_INVALID_ARG, "a matrix has at most 2^20 rows and columns");
    }
    return RR_OK;
}

rr_status_t same_shapes(const rr_matrix_list_t* a, const rr_matrix_list_t* b)
{
    if (a->nmatrices != b->nmatrices) return fail(RR_ERR_INVALID_ARG, "the lists have different matrix counts");
    for (int t = 0; t < a->nmatrices; ++t)
        if (a->rows[t] != b->rows[t] || a->cols[t] != b->cols[t])
            return fail(RR_ERR_INVALID_ARG, "the lists have different shapes");
    return RR_OK;
}

// The first `ranks` ranks' matrices as spans.
rr_status_t add_spans(const rr_matrix_list_t* l, int ranks, bool out, std::vector<Span>& spans)
{
    for (int r = 0; r < ranks; ++r)
        for (int t = 0; t < l->nmatrices; ++t) {
            if (l->rows[t] == 0 || l->cols[t] == 0) continue;
            const uintptr_t a = (uintptr_t)l->ptrs[(size_t)r * l->nmatrices + t];
            const uint64_t es = esize(l->dtypes[t]);
            if (a == 0) return fail(RR_ERR_INVALID_ARG, "NULL buffer pointer");
            if (a % es != 0) return fail(RR_ERR_INVALID_ARG, "matrix not aligned to its element size");
            spans.push_back({a, a + l->rows[t] * l->cols[t] * es, out});
        }
    return RR_OK;
}

// The scales of the halves, a power of two for every step's X, A = X X^T and
// B = b A + c A^2.  No element exceeds the largest singular value, which starts
// at 1 at most (the Frobenius norm is 1) and is carried through the
// polynomials' extrema; the scale puts that just below fp16's largest.
struct Plan {
    int steps;
    float a, b, c;
    double x[kMaxSteps + 1], gram[kMaxSteps], poly[kMaxSteps];
};

double scale_for(double bound)
{
    if (!(bound > 0x1p-12)) bound = 0x1p-12;
    return std::exp2(std::floor(std::log2(60000.0 / bound)));
}

rr_status_t make_plan(const rr_newton_schulz_t* ns, Plan* p)
{
    if (!ns) return fail(RR_ERR_INVALID_ARG, "NULL Newton-Schulz parameters");
    if (ns->steps < 0 || ns->steps > kMaxSteps) return fail(RR_ERR_INVALID_ARG, "steps must be in 0..64");
    if (!(ns->eps > 0.0f) || std::isinf(ns->eps)) return fail(RR_ERR_INVALID_ARG, "eps must be finite and above 0");
    if (!std::isfinite(ns->a) || !std::isfinite(ns->b) || !std::isfinite(ns->c))
        return fail(RR_ERR_INVALID_ARG, "the coefficients must be finite");
    p->steps = ns->steps;
    p->a = ns->a;
    p->b = ns->b;
    p->c = ns->c;
    const double a = ns->a, b = ns->b, c = ns->c;
    double rho = 1.0 + 0x1p-10;  // what the norm's and the halves' roundings add
    for (int k = 0; k <= ns->steps; ++k) {
        if (rho > 1024.0)
            return fail(RR_ERR_UNSUPPORTED, "with these coefficients a step can take a singular value above 1024");
        p->x[k] = scale_for(rho);
        if (k == ns->steps) break;
        const double top = rho * rho;
        p->gram[k] = scale_for(top);
        const auto poly = [&](double l) { return std::fabs(b * l + c * l * l); };
        double most = poly(top);
        if (c != 0.0 && -b / (2 * c) > 0.0 && -b / (2 * c) < top) most = std::max(most, poly(-b / (2 * c)));
        p->poly[k] = scale_for(most);
        // extrema of |a s + b s^3 + c s^5| on [0, rho]: a + 3 b l + 5 c l^2 = 0, l = s^2
        const auto step = [&](double l) { return std::fabs(a + b * l + c * l * l) * std::sqrt(l); };
        double next = step(top);
        double roots[2] = {-1.0, -1.0};
        if (c != 0.0) {
            const double disc = 9 * b * b - 20 * a * c;
            if (disc >= 0.0) {
                roots[0] = (-3 * b + std::sqrt(disc)) / (10 * c);
                roots[1] = (-3 * b - std::sqrt(disc)) / (10 * c);
            }
        } else if (b != 0.0) {
            roots[0] = -a / (3 * b);
        }
        for (double l : roots)
            if (l > 0.0 && l < top) next = std::max(next, step(l));
        rho = next * (1.0 + 0x1p-10);
    }
    return RR_OK;
}

uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

// One matrix's part of the workspace: X twice (a product reads one and writes
// the other), A and B, two halves each.
struct Room {
    uint64_t x[2], gram, poly;  // bytes of one half
    uint64_t bytes() const { return 2 * (x[0] + x[1] + gram + poly); }
};

Room room_of(const Shape& s, int steps)
{
    Room r{};
    r.x[0] = (uint64_t)pad_up(s.rows) * pad_up(s.cols) * 2;
    if (steps > 0) {
        r.x[1] = r.x[0];
        r.gram = r.poly = (uint64_t)pad_up(s.small()) * pad_up(s.small()) * 2;
    }
    return r;
}

uint32_t parts_of(const Shape& s) { return (uint32_t)std::min<uint64_t>(kNormParts, ceil_div(s.numel(), kPrepTile)); }

constexpr uint64_t kPartialBytes = (uint64_t)kMuonMats * kNormParts * sizeof(double);

// The groups of a list's matrices (those with elements), in order.
std::vector<std::vector<int>> groups_of(const rr_matrix_list_t* l, int steps, uint64_t* bytes)
{
    std::vector<std::vector<int>> groups;
    uint64_t used = 0;
    *bytes = 256;
    for (int t = 0; t < l->nmatrices; ++t) {
        const Shape s{(uint32_t)l->rows[t], (uint32_t)l->cols[t]};
        if (s.numel() == 0) continue;
        const uint64_t need = room_of(s, steps).bytes();
        if (groups.empty() || groups.back().size() == kMuonMats || used + need > kGroupBytes) {
            groups.emplace_back();
            used = kPartialBytes;
        }
        groups.back().push_back(t);
        used += need;
        *bytes = std::max(*bytes, used);
    }
    return groups;
}

// What differs between the two calls.
struct Job {
    const rr_matrix_list_t* in;     // gradients, or the matrices
    const rr_matrix_list_t* mom;    // momenta; NULL: orthogonalize
    const rr_matrix_list_t* out;    // weights, or the results
    float momentum, keep, lr, eps;
    int nesterov, adjust;
};

float shape_factor(const Shape& s, int adjust)
{
    if (adjust == RR_MUON_RMS) return 0.2f * (float)std::sqrt((double)std::max(s.rows, s.cols));
    return (float)std::sqrt(std::max(1.0, (double)s.rows / s.cols));
}

bool on16(const void* p) { return (uintptr_t)p % 16 == 0; }

rr_status_t run_group(const Job& job, const Plan& plan, const std::vector<int>& group, char* ws, cudaStream_t stream)
{
    const int n = (int)group.size();
    std::unique_ptr<MuonPrepParams> prep(new MuonPrepParams{});
    std::unique_ptr<MuonGemmParams> gemm(new MuonGemmParams{});
    std::vector<Halves> x[2], gram(n), poly(n);
    x[0].resize(n);
    x[1].resize(n);
    uint64_t at = kPartialBytes;
    const auto take = [&](uint64_t half) {
        Halves h;
        h.hi = reinterpret_cast<uint16_t*>(ws + at);
        h.lo = reinterpret_cast<uint16_t*>(ws + at + half);
        at += 2 * half;
        return h;
    };
    prep->n = n;
    prep->partial = reinterpret_cast<double*>(ws);
    prep->momentum = job.momentum;
    prep->nesterov = job.nesterov;
    prep->eps = job.eps;
    prep->scale = (float)plan.x[0];
    uint32_t parts = 0, tiles = 0;
    std::vector<Shape> shape(n);
    for (int k = 0; k < n; ++k) {
        const int t = group[k];
        const Shape s = shape[k] = {(uint32_t)job.in->rows[t], (uint32_t)job.in->cols[t]};
        const Room room = room_of(s, plan.steps);
        x[0][k] = take(room.x[0]);
        x[1][k] = plan.steps > 0 ? take(room.x[1]) : x[0][k];
        gram[k] = take(room.gram);
        poly[k] = take(room.poly);
        MuonMat& m = prep->mat[k];
        m.g = job.in->ptrs[t];
        m.m = job.mom ? static_cast<float*>(job.mom->ptrs[t]) : nullptr;
        m.rows = s.rows;
        m.cols = s.cols;
        m.part0 = parts;
        m.parts = parts_of(s);
        m.x = x[0][k];
        m.tile0 = tiles;
        m.dtype = (uint8_t)job.in->dtypes[t];
        m.vec = s.cols % 8 == 0 && on16(m.g) && (!m.m || on16(m.m));
        parts += m.parts;
        tiles += pad_up(s.rows) / 128 * (pad_up(s.cols) / kBlk);
    }
    cudaError_t e = timed_launch([&] { return launch_muon_squares(*prep, parts, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "Muon norm launch");
    e = timed_launch([&] { return launch_muon_pack(*prep, tiles, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "Muon pack launch");
    t_stats.launches += 2;

    gemm->n = n;
    for (int step = 0; step < plan.steps; ++step) {
        const std::vector<Halves>& from = x[step & 1];
        const std::vector<Halves>& to = x[(step + 1) & 1];
        const double sx = plan.x[step], sg = plan.gram[step], sp = plan.poly[step];
        for (int product = 0; product < 3; ++product) {
            for (int k = 0; k < n; ++k) {
                const Shape& s = shape[k];
                const bool wide = s.rows <= s.cols;
                const uint32_t xb = pad_up(s.cols) / kBlk, mb = pad_up(s.small()) / kBlk;
                MuonProduct q{};
                if (product == 0) {  // A = X X^T, or X^T X
                    q.a = q.b = from[k];
                    q.out = gram[k];
                    q.a_nbj = q.b_nbj = xb;
                    q.o_nbj = mb;
                    q.a_mn = q.b_mn = !wide;
                    q.mt = q.nu = pad_up(s.small()) / 128;
                    q.kb = (uint32_t)ceil_div(std::max(s.rows, s.cols), kBlk);
                    q.sym = 1;
                    q.alpha = (float)(sg / (sx * sx));
                } else if (product == 1) {  // B = b A + c A A
                    q.a = q.b = q.c = gram[k];
                    q.out = poly[k];
                    q.a_nbj = q.b_nbj = q.o_nbj = mb;
                    q.mt = q.nu = pad_up(s.small()) / 128;
                    q.kb = (uint32_t)ceil_div(s.small(), kBlk);
                    q.sym = 1;
                    q.alpha = (float)(plan.c * sp / (sg * sg));
                    q.beta = (float)(plan.b * sp / sg);
                } else {  // X' = a X + B X, or a X + X B (B is symmetric)
                    q.a = wide ? poly[k] : from[k];
                    q.b = wide ? from[k] : poly[k];
                    q.c = from[k];
                    q.out = to[k];
                    q.a_nbj = wide ? mb : xb;
                    q.b_nbj = wide ? xb : mb;
                    q.o_nbj = xb;
                    q.b_mn = wide;
                    q.mt = pad_up(s.rows) / 128;
                    q.nu = pad_up(s.cols) / 128;
                    q.kb = (uint32_t)ceil_div(s.small(), kBlk);
                    q.alpha = (float)(plan.x[step + 1] / (sp * sx));
                    q.beta = (float)(plan.a * plan.x[step + 1] / sx);
                }
                gemm->q[k] = q;
            }
            e = timed_launch([&] { return launch_muon_gemm(*gemm, stream); });
            if (e != cudaSuccess) return cuda_fail(e, "Newton-Schulz product launch");
            t_stats.launches += 1;
        }
    }

    std::unique_ptr<MuonFinishParams> fin(new MuonFinishParams{});
    const int nr = job.out->nranks, most = std::max(1, kMuonPtrs / nr);
    fin->nranks = nr;
    fin->inv = (float)(1.0 / plan.x[plan.steps]);
    fin->keep = job.keep;
    for (int k0 = 0; k0 < n; k0 += most) {
        fin->n = std::min(most, n - k0);
        uint32_t todo = 0;
        for (int k = 0; k < fin->n; ++k) {
            const int t = group[k0 + k];
            MuonMat& m = fin->mat[k];
            m = prep->mat[k0 + k];
            m.x = x[plan.steps & 1][k0 + k];
            m.tile0 = todo;
            todo += pad_up(m.rows) / 128 * (pad_up(m.cols) / kBlk);
            m.out_dtype = (uint8_t)job.out->dtypes[t];
            m.out = (uint32_t)(k * nr);
            m.factor = job.lr * shape_factor(shape[k0 + k], job.adjust);
            m.vec = m.cols % 8 == 0;
            for (int r = 0; r < nr; ++r) {
                fin->out[k * nr + r] = job.out->ptrs[(size_t)r * job.out->nmatrices + t];
                m.vec = m.vec && on16(fin->out[k * nr + r]);
            }
        }
        e = timed_launch([&] { return launch_muon_finish(*fin, todo, stream); });
        if (e != cudaSuccess) return cuda_fail(e, "Muon update launch");
        t_stats.launches += 1;
    }
    return RR_OK;
}

rr_status_t run(const Job& job, const Plan& plan, std::vector<Span>& spans, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    uint64_t need = 0, S = 0, total = 0;
    const auto groups = groups_of(job.in, plan.steps, &need);
    for (int t = 0; t < job.in->nmatrices; ++t) {
        const uint64_t numel = job.in->rows[t] * job.in->cols[t];
        S += numel * esize(job.out->dtypes[t]);
        total += numel;
    }
    stats_begin(RR_ALGO_ONESHOT, job.out->nranks, S);
    if (groups.empty()) return RR_OK;
    if (!ws || (uintptr_t)ws % 256 != 0) return fail(RR_ERR_INVALID_ARG, "workspace NULL or not aligned to 256 bytes");
    if (ws_bytes < need)
        return fail(RR_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
    spans.push_back({(uintptr_t)ws, (uintptr_t)ws + need, true});
    rr_status_t st = check_spans(spans);
    if (st != RR_OK) return st;
    if ((st = check_device_spans(spans)) != RR_OK) return st;
    for (const auto& group : groups)
        if ((st = run_group(job, plan, group, static_cast<char*>(ws), stream)) != RR_OK) return st;
    t_stats.steps = plan.steps;
    for (int t = 0; t < job.in->nmatrices; ++t)
        t_stats.hbm_bytes += job.in->rows[t] * job.in->cols[t] *
                             (esize(job.in->dtypes[t]) + (job.mom ? 8 + esize(job.out->dtypes[t]) : 0) +
                              (uint64_t)job.out->nranks * esize(job.out->dtypes[t]));
    log_call(job.mom ? "muon_step" : "orthogonalize", job.out->nranks, total, job.out->dtypes[0], RR_SUM, RR_ALGO_ONESHOT);
    return debug_check(st, stream);
}

rr_status_t orthogonalize(const rr_matrix_list_t* in, const rr_matrix_list_t* out, const rr_newton_schulz_t* ns, void* ws,
                          size_t ws_bytes, cudaStream_t stream)
{
    CallTimer timer("rr_orthogonalize");
    Plan plan;
    rr_status_t st = make_plan(ns, &plan);
    if (st != RR_OK) return st;
    if ((st = check_list(in, "matrices")) != RR_OK) return st;
    if ((st = check_list(out, "results")) != RR_OK) return st;
    if ((st = same_shapes(in, out)) != RR_OK) return st;
    std::vector<Span> spans, read;
    spans.reserve((size_t)(out->nranks + 1) * out->nmatrices + 1);
    if ((st = add_spans(out, out->nranks, true, spans)) != RR_OK) return st;
    for (int t = 0; t < in->nmatrices; ++t) {  // a result of its type may take its matrix's place
        if (in->rows[t] == 0 || in->cols[t] == 0) continue;
        bool own = false;
        for (int r = 0; r < out->nranks; ++r)
            own = own || (out->ptrs[(size_t)r * out->nmatrices + t] == in->ptrs[t] && out->dtypes[t] == in->dtypes[t]);
        const uintptr_t a = (uintptr_t)in->ptrs[t];
        if (a == 0) return fail(RR_ERR_INVALID_ARG, "NULL buffer pointer");
        if (a % esize(in->dtypes[t]) != 0) return fail(RR_ERR_INVALID_ARG, "matrix not aligned to its element size");
        if (!own) spans.push_back({a, a + in->rows[t] * in->cols[t] * esize(in->dtypes[t]), false});
    }
    const Job job{in, nullptr, out, 0.0f, 0.0f, 0.0f, ns->eps, 0, 0};
    return run(job, plan, spans, ws, ws_bytes, stream);
}

rr_status_t muon_step(const rr_matrix_list_t* params, const rr_matrix_list_t* grads, const rr_matrix_list_t* momenta,
                      const rr_muon_t* cfg, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    CallTimer timer("rr_muon_step");
    if (!cfg) return fail(RR_ERR_INVALID_ARG, "NULL Muon parameters");
    Plan plan;
    rr_status_t st = make_plan(&cfg->ns, &plan);
    if (st != RR_OK) return st;
    if (!std::isfinite(cfg->lr) || !std::isfinite(cfg->weight_decay))
        return fail(RR_ERR_INVALID_ARG, "lr and weight_decay must be finite");
    if (!(cfg->momentum >= 0.0f) || std::isinf(cfg->momentum))
        return fail(RR_ERR_INVALID_ARG, "momentum must be finite and 0 or more");
    if (cfg->adjust != RR_MUON_SPECTRAL && cfg->adjust != RR_MUON_RMS)
        return fail(RR_ERR_INVALID_ARG, "unknown adjustment of the step to the shape");
    if ((st = check_list(params, "weights")) != RR_OK) return st;
    if ((st = check_list(grads, "gradients")) != RR_OK) return st;
    if ((st = check_list(momenta, "momenta")) != RR_OK) return st;
    if ((st = same_shapes(params, grads)) != RR_OK) return st;
    if ((st = same_shapes(params, momenta)) != RR_OK) return st;
    if (momenta->nranks != 1) return fail(RR_ERR_INVALID_ARG, "the momenta are kept once (one rank)");
    for (int t = 0; t < momenta->nmatrices; ++t)
        if (momenta->dtypes[t] != RR_F32) return fail(RR_ERR_UNSUPPORTED, "momenta must be fp32");
    std::vector<Span> spans;
    spans.reserve((size_t)(params->nranks + 2) * params->nmatrices + 1);
    if ((st = add_spans(params, params->nranks, true, spans)) != RR_OK) return st;
    if ((st = add_spans(momenta, 1, true, spans)) != RR_OK) return st;
    if ((st = add_spans(grads, 1, false, spans)) != RR_OK) return st;
    const Job job{grads,
                  momenta,
                  params,
                  cfg->momentum,
                  (float)(1.0 - (double)cfg->lr * cfg->weight_decay),
                  cfg->lr,
                  cfg->ns.eps,
                  cfg->nesterov != 0,
                  cfg->adjust};
    return run(job, plan, spans, ws, ws_bytes, stream);
}

}  // namespace

extern "C" {

rr_status_t rr_muon_workspace(const rr_matrix_list_t* matrices, const rr_newton_schulz_t* ns, size_t* bytes)
{
    return guarded([&]() -> rr_status_t {
        if (!bytes) return fail(RR_ERR_INVALID_ARG, "NULL workspace size output");
        Plan plan;
        rr_status_t st = make_plan(ns, &plan);
        if (st == RR_OK) st = check_list(matrices, "matrices");
        if (st != RR_OK) return st;
        uint64_t need = 0;
        groups_of(matrices, plan.steps, &need);
        *bytes = (size_t)need;
        return RR_OK;
    });
}

rr_status_t rr_orthogonalize(const rr_matrix_list_t* matrices, const rr_matrix_list_t* results, const rr_newton_schulz_t* ns,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return guarded([&] { return orthogonalize(matrices, results, ns, workspace, workspace_bytes, stream); });
}

rr_status_t rr_muon_step(const rr_matrix_list_t* params, const rr_matrix_list_t* grads, const rr_matrix_list_t* momenta,
                         const rr_muon_t* config, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return guarded([&] { return muon_step(params, grads, momenta, config, workspace, workspace_bytes, stream); });
}

}  // extern "C"
