// rr_muon_api.cu -- host side of the orthogonalisation and the Muon step
// (rr_orthogonalize, rr_muon_step in include/rr.h): argument checks, the
// iteration's scales, the order of the products, groups of matrices.
#include <cmath>
#include <memory>
#include <tuple>

#include "rr_host.h"
#include "rr_muon.h"

using namespace rr;

namespace {

constexpr uint64_t kMaxSide = 1ull << 20;    // rows and columns
constexpr int kMaxSteps = kMuonMaxSteps;
// Workspace of a group of matrices that run in the same launches, unless one
// alone needs more.
constexpr uint64_t kGroupBytes = 5ull << 30;

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

// What the iteration's values are bounded by.  No element exceeds the largest
// singular value, which starts at 1 at most (the Frobenius norm is 1) and is
// carried through the polynomials' extrema.
struct Plan {
    int steps;
    float a, b, c;
    double rho[kMaxSteps + 1];   // of X before step k
    double poly[kMaxSteps];      // of D = a + b A + c A^2
};

// The halves' scale, a power of two: the bound comes just below fp16's largest.
double scale_for(double bound)
{
    if (!(bound > 0x1p-12)) bound = 0x1p-12;
    return std::exp2(std::floor(std::log2(60000.0 / bound)));
}

rr_status_t make_plan(const rr_newton_schulz_t* ns, Plan* p)
{
    if (!ns) return fail(RR_ERR_INVALID_ARG, "NULL Newton-Schulz parameters");
    if (ns->steps < 0 || ns->steps > kMaxSteps) return fail(RR_ERR_INVALID_ARG, "steps must be in 0..50");
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
        p->rho[k] = rho;
        if (k == ns->steps) break;
        // the extrema of |d(l)| and of |d(l)| sqrt(l), d = a + b l + c l^2, on 0 <= l <= rho^2
        const double top = rho * rho;
        const auto d = [&](double l) { return std::fabs(a + b * l + c * l * l); };
        double most = std::max(d(0.0), d(top)), next = d(top) * rho;
        const double vertex = c != 0.0 ? -b / (2 * c) : -1.0;
        if (vertex > 0.0 && vertex < top) most = std::max(most, d(vertex));
        double roots[2] = {-1.0, -1.0};  // of a + 3 b l + 5 c l^2
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
            if (l > 0.0 && l < top) next = std::max(next, d(l) * std::sqrt(l));
        p->poly[k] = most * (1.0 + 0x1p-10);
        rho = next * (1.0 + 0x1p-10);
    }
    return RR_OK;
}

// The steps of a matrix run in segments.  A segment of s steps forms A = X X^T
// once and carries on in the smaller side's m x m space,
//     D = a + b A + c A^2    Q <- D Q    A <- D (D A)
// and ends with X <- Q X; with n = r m the longer side its products cost
// 1.5 r + 2 s - 1.5 times 2 m^3 operations (symmetric ones count half), the
// whole 1.5 (r - 1) a segment and 2 a step: the fewer segments the better, the
// more so the longer the matrix, and none for a square one.  But D (D A)
// multiplies what A was rounded by, up to a^2 a step, where its eigenvalues are
// small: five steps on one A of 2^-22 are off by up to 2e4 * 1.4 * 2^-22 = 7e-3 of a
// result that one strong direction dominates, more than bf16's own 1.7e-3.
// Measured error of five steps against 64 bits in segments of 3 + 2 (chunk 2) / 2 + 2
// + 1 / 1 each (chunk 1), from noise to one direction in 1 % of noise: 4e-6..4e-5 /
// 2e-6..2e-5 / 1e-6..1e-5, the same steps in plain fp32 2e-6..5e-5; of 5 steps
// (chunk 4) 4e-6..7e-3.  So A's errors may grow by 200 (3 steps of the usual
// coefficients) for bf16 and fp16 results, which are rounded by 1.7e-3 and 2e-4 (four
// layers of width 2048, bf16: 12.7 ms, on one A 10.4), and by 12.5 (2 steps) for
// fp32's from 512 rows on (0.2 to 1.4 times plain fp32's error; 4 layers of width 2048
// in 17.8 ms instead of 24), below which plain fp32 errs less than that (up to 2.1
// times; 192 x 288 to 384 x 1536: 172..276 us, one step each 165..295).  A polynomial
// of a small a takes many steps, and the roundings of Q, which has a's part in the
// tensor cores' sums, add up over those on one A: no more than three (two) share one
// there, either, and below a^2 = 2 fp32's none (40 steps of 1, 0.6, -0.55 in fp32, two
// on one A: 3e-5, plain fp32 5e-7; 50 of 1, -0.3, 0.1 in fp16, all on one A: 2e-4).
// Weights are treated as results of their type are: how large a part of a weight the
// update is depends on the caller's lr, factor and weights, which may begin at zero.
// (fp32 weights on 3 + 2 steps, their sums in chunks of 256 of K, were 3 to 11 times
// as far off as the same steps in plain fp32, up to 6e-5 of O; a layer of width 700 /
// 1024: 450 / 1500 us then, 600 / 2060 now.)
std::vector<int> segments_of(const Plan& plan, uint32_t m, uint32_t n, bool exact)
{
    const double grow = std::max(1.0, (double)plan.a * plan.a);
    const double limit = exact ? (m < 512 || grow < 2.0 ? 0.0 : 12.5) : 200.0;
    const int longest = std::min(exact ? 2 : 3, plan.steps);
    int most = 1;
    for (double g = grow; g <= limit && most < longest; g *= grow) ++most;
    // nearly square matrices would gain less than a twentieth
    if (1.5 * ((double)n / m - 1.0) * (plan.steps - 1) < 0.05 * 2.0 * plan.steps) most = 1;
    std::vector<int> parts;
    for (int left = plan.steps; left > 0; left -= most) parts.push_back(std::min(most, left));
    return parts;
}

// One matrix's part of the workspace: X twice (a segment reads one and writes
// the other) and up to five m x m matrices, two halves each.
struct Room {
    uint64_t x, square;  // bytes of one half
    int xs, squares;
    uint64_t bytes() const { return 2 * (x * xs + square * squares); }
};

Room room_of(const Shape& s, const std::vector<int>& segments)
{
    const int most = segments.empty() ? 0 : *std::max_element(segments.begin(), segments.end());
    return {(uint64_t)pad_up(s.rows) * pad_up(s.cols) * 2, (uint64_t)pad_up(s.small()) * pad_up(s.small()) * 2,
            most > 0 ? 2 : 1, most > 1 ? 5 : most > 0 ? 2 : 0};
}

uint32_t parts_of(const Shape& s) { return (uint32_t)std::min<uint64_t>(kNormParts, ceil_div(s.numel(), kPrepTile)); }

constexpr uint64_t kPartialBytes = (uint64_t)kMuonMats * kNormParts * sizeof(double);
constexpr uint64_t kHeadBytes = kPartialBytes + 1024;  // and the counters
static_assert(kMuonCounters * 4 <= 1024 && kMuonMats < (int)kMuonCounters, "a counter per matrix and one more");
static_assert(kMuonMats < 256 && kMuonOps <= 256, "fields of MuonGemmParams::seq");

// Products of a matrix.
int products_in(const std::vector<int>& segments)
{
    int n = 0;
    for (int len : segments) n += 2 + len + (len - 1) * 3;
    return n;
}

// fp32 results, and updates of fp32 weights, come out as exactly as fp32 holds them.
bool is_exact(rr_dtype_t type) { return type == RR_F32; }

// Whether a cluster takes the matrix whole (rr_muon_small.cu).
bool is_small(uint64_t rows, uint64_t cols)
{
    return std::min(rows, cols) <= kMuonSmallSide && std::max(rows, cols) <= kMuonSmallSide * kMuonSmallCtas;
}

// What a matrix's products follow from, beside its shape: lists of products are
// made once for every kind of a group.
struct Kind {
    std::vector<int> segments;
    bool exact;
    bool operator==(const Kind& o) const { return exact == o.exact && segments == o.segments; }
};

// Matrices of one shape and kind, whatever their types: they follow one another
// in the launches, and each of their products is listed once for all of them.
struct Alike {
    Shape shape;
    size_t kind;
    std::vector<int> matrices;
};

// Matrices that run in the same launches.
struct Group {
    std::vector<Kind> kinds;
    std::vector<Alike> alike;
    int matrices = 0;
    int ops = 0;     // different products: of every kind once
    int listed = 0;  // entries of MuonGemmParams::seq: of every Alike once
    uint64_t used = kHeadBytes;
};

// The groups of a list's other matrices (those with elements), in order.
std::vector<Group> groups_of(const rr_matrix_list_t* l, const Plan& plan, uint64_t* bytes)
{
    std::vector<Group> groups;
    *bytes = 256;
    for (int t = 0; t < l->nmatrices; ++t) {
        const Shape s{(uint32_t)l->rows[t], (uint32_t)l->cols[t]};
        if (s.numel() == 0 || is_small(s.rows, s.cols)) continue;
        const bool exact = is_exact(l->dtypes[t]);
        const Kind kind{segments_of(plan, s.small(), std::max(s.rows, s.cols), exact), exact};
        const uint64_t need = room_of(s, kind.segments).bytes();
        const int products = products_in(kind.segments);
        size_t k = 0, a = 0;  // its kind and its like in the last group
        const auto look = [&] {
            const Group& g = groups.back();
            k = (size_t)(std::find(g.kinds.begin(), g.kinds.end(), kind) - g.kinds.begin());
            a = (size_t)(std::find_if(g.alike.begin(), g.alike.end(), [&](const Alike& e) {
                             return e.shape.rows == s.rows && e.shape.cols == s.cols && e.kind == k;
                         }) - g.alike.begin());
        };
        const auto fits = [&] {
            const Group& g = groups.back();
            return g.matrices < kMuonMats && g.used + need <= kGroupBytes &&
                   (a < g.alike.size() || g.listed + products <= kMuonSeq) && (k < g.kinds.size() || g.ops + products <= kMuonOps);
        };
        if (!groups.empty()) look();
        if (groups.empty() || !fits()) {
            groups.emplace_back();
            look();
        }
        Group& g = groups.back();
        if (k == g.kinds.size()) {
            g.kinds.push_back(kind);
            g.ops += products;
        }
        if (a == g.alike.size()) {
            g.alike.push_back({s, k, {}});
            g.listed += products;
        }
        g.alike[a].matrices.push_back(t);
        g.matrices += 1;
        g.used += need;
        *bytes = std::max(*bytes, g.used);
    }
    // smaller matrices of a group first
    for (Group& g : groups)
        std::stable_sort(g.alike.begin(), g.alike.end(), [](const Alike& x, const Alike& y) {
            return std::tie(x.shape.rows, x.shape.cols) < std::tie(y.shape.rows, y.shape.cols);
        });
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

// How many neighbours of a row of `cols` elements of `es` bytes lie on 16 bytes (8 of
// them) or on their common size (2) in every row.
uint8_t neighbours(const void* p, uint64_t es, uint32_t cols)
{
    if (cols % 8 == 0 && (uintptr_t)p % 16 == 0) return 8;
    return cols % 2 == 0 && (uintptr_t)p % (2 * es) == 0 ? 2 : 1;
}

// Stages of 64 of K between the roundings of a sum, of exact results and of others.
// Error of five steps in fp32, chunks of 1 / 2 / 4, from 128 x 128 to 8192 x 2048:
// 0.7e-6..2.0e-6 / 1.2e-6..3.4e-6 / 1.3e-6..4.5e-6 (the same steps in plain fp32:
// 1.3e-6..6e-6); of three and two on one A 2e-6..2e-5 / 4e-6..4e-5 / 7e-6..7e-5.  Four
// layers of width 2048, bf16: 15.4 / 12.7 / 12.5 ms, 24 of 256: 475 / 453 / 461 us.
constexpr uint8_t kExactChunk = 1, kChunk = 2;

// The products of a matrix of m <= n sides, in the order of their levels; X
// begins in buffer 0.  *last: the result's buffer.
std::vector<MuonOp> products_of(const Plan& plan, const std::vector<int>& segments, bool exact, int* last)
{
    std::vector<MuonOp> ops;
    const uint8_t A = kSquares, Y = kSquares + 1, D = kSquares + 2;
    uint8_t cur = 0;
    int step = 0, level = 0;
    const auto add = [&](int kind, uint8_t a, uint8_t b, uint8_t out, int at, double alpha) -> MuonOp& {
        MuonOp q{};
        q.kind = (uint8_t)kind;
        q.a = a;
        q.b = b;
        q.c = kNoBuffer;
        q.out = out;
        q.level = (uint8_t)at;
        q.chunk = exact ? kExactChunk : kChunk;
        q.alpha = (float)alpha;
        ops.push_back(q);
        return ops.back();
    };
    for (int len : segments) {
        const double sx = scale_for(plan.rho[step]);
        double top = plan.rho[step] * plan.rho[step], sa = scale_for(top);
        add(kGram, cur, cur, A, level++, sa / (sx * sx));
        // A segment of one step keeps a X out of the products, X <- a X + (D - a) X:
        // as a term of the tensor cores' sums it would be cut off with them
        // (a step's error 4e-7 instead of 8e-8).
        const bool alone = len == 1;
        uint8_t Q = alone ? Y : kSquares + 3, Q2 = kSquares + 4;
        double bound = 1.0, scale_q = 1.0;  // of Q
        for (int k = 0; k < len; ++k) {
            const double most = plan.poly[step + k] + (alone ? std::fabs(plan.a) : 0.0), sd = scale_for(most);
            const uint8_t d = k == 0 ? Q : D;
            MuonOp& q = add(kSquare, A, A, d, level++, plan.c * sd / (sa * sa));
            q.c = A;
            q.beta = (float)(plan.b * sd / sa);
            q.diag = alone ? 0.0f : (float)(plan.a * sd);
            if (k == 0) {
                bound = most;
                scale_q = sd;
            }
            if (k > 0) {  // Q <- D Q, beside D A
                bound *= most;
                const double to = scale_for(bound);
                add(kSquare, d, Q, Q2, level, to / (sd * scale_q));
                scale_q = to;
                std::swap(Q, Q2);
            }
            if (k + 1 < len) {  // A <- D (D A)
                const double sy = scale_for(most * top);
                add(kSquare, d, A, Y, level++, sy / (sd * sa));
                top = plan.rho[step + k + 1] * plan.rho[step + k + 1];
                sa = scale_for(top);
                add(kSquare, d, Y, A, level++, sa / (sd * sy));
            } else if (k > 0) {
                ++level;
            }
        }
        step += len;
        const double to = scale_for(plan.rho[step]);
        MuonOp& q = add(kApply, Q, cur, cur ^ 1, level++, to / (scale_q * sx));
        if (alone) {
            q.c = cur;
            q.beta = (float)(plan.a * to / sx);
        }
        cur ^= 1;
    }
    *last = cur;
    return ops;
}

// A matrix's gradient and momentum, and its outputs from out[at] on.
void place_matrix(const Job& job, int t, MuonMat& m, void** out, uint32_t at)
{
    const Shape s{(uint32_t)job.in->rows[t], (uint32_t)job.in->cols[t]};
    m.g = job.in->ptrs[t];
    m.m = job.mom ? static_cast<float*>(job.mom->ptrs[t]) : nullptr;
    m.rows = s.rows;
    m.cols = s.cols;
    m.dtype = (uint8_t)job.in->dtypes[t];
    m.out_dtype = (uint8_t)job.out->dtypes[t];
    m.factor = job.lr * shape_factor(s, job.adjust);
    m.vec = neighbours(m.g, esize(job.in->dtypes[t]), s.cols);
    if (m.m) m.vec = std::min(m.vec, neighbours(m.m, 4, s.cols));
    m.out_vec = 8;
    m.out = at;
    for (int r = 0; out && r < job.out->nranks; ++r) {
        out[at + r] = job.out->ptrs[(size_t)r * job.out->nmatrices + t];
        m.out_vec = std::min(m.out_vec, neighbours(out[at + r], esize(job.out->dtypes[t]), s.cols));
    }
}

// Matrices that a cluster takes whole.
rr_status_t run_small(const Job& job, const Plan& plan, const std::vector<int>& list, cudaStream_t stream)
{
    std::unique_ptr<MuonSmallParams> p(new MuonSmallParams{});
    const int nr = job.out->nranks, most = std::min(kMuonMats, std::max(1, kMuonPtrs / nr));
    p->nranks = nr;
    p->steps = plan.steps;
    p->nesterov = job.nesterov;
    p->momentum = job.momentum;
    p->eps = job.eps;
    p->keep = job.keep;
    p->scale = (float)scale_for(plan.rho[0]);
    p->inv = (float)(1.0 / scale_for(plan.rho[plan.steps]));
    for (int k = 0; k < plan.steps; ++k) {
        const double top = plan.rho[k] * plan.rho[k], sx = scale_for(plan.rho[k]), sa = scale_for(top);
        const double sb = scale_for(plan.poly[k] + std::fabs(plan.a)), to = scale_for(plan.rho[k + 1]);
        p->step[k] = {(float)(sa / (sx * sx)), (float)(plan.c * sb / (sa * sa)), (float)(plan.b * sb / sa), (float)(to / (sb * sx)),
                      (float)(plan.a * to / sx)};
    }
    for (size_t k0 = 0; k0 < list.size(); k0 += most) {
        p->n = (int)std::min<size_t>(most, list.size() - k0);
        p->ctas = 1;
        for (int k = 0; k < p->n; ++k) {
            MuonMat& m = p->mat[k];
            place_matrix(job, list[k0 + k], m, p->out, (uint32_t)(k * nr));
            p->ctas = std::max(p->ctas, (uint32_t)ceil_div(std::max(m.rows, m.cols), kMuonSmallSide));
        }
        const cudaError_t e = timed_launch([&] { return launch_muon_small(*p, stream); });
        if (e != cudaSuccess) return cuda_fail(e, "Muon launch of small matrices");
        t_stats.launches += 1;
    }
    return RR_OK;
}

rr_status_t run_group(const Job& job, const Plan& plan, const Group& group, char* ws, cudaStream_t stream)
{
    const int n = group.matrices;
    // groups_of counts what is listed here; more would pass the ends of the parameters' arrays
    const auto too_many = [] { return fail(RR_ERR_UNSUPPORTED, "a group of matrices has more products than a launch takes"); };
    if (n > kMuonMats) return too_many();
    std::unique_ptr<MuonPrepParams> prep(new MuonPrepParams{});
    std::unique_ptr<MuonGemmParams> gemm(new MuonGemmParams);  // as it comes: every field that counts is set
    std::vector<Halves> result(n);
    std::vector<int> matrix(n);  // of the list, in the launches' order
    uint64_t at = kHeadBytes;
    const auto take = [&](uint64_t bytes) {
        uint16_t* const p = reinterpret_cast<uint16_t*>(ws + at);
        at += bytes;
        return p;
    };
    prep->n = n;
    prep->partial = reinterpret_cast<double*>(ws);
    prep->counters = gemm->counters = reinterpret_cast<uint32_t*>(ws + kPartialBytes);
    prep->momentum = job.momentum;
    prep->nesterov = job.nesterov;
    prep->eps = job.eps;
    prep->scale = (float)scale_for(plan.rho[0]);
    // every kind's products, and the buffer that their result is in
    std::vector<std::vector<MuonOp>> products;
    std::vector<uint16_t> op0;
    std::vector<int> last;
    int nops = 0;
    for (const Kind& kind : group.kinds) {
        last.push_back(0);
        products.push_back(products_of(plan, kind.segments, kind.exact, &last.back()));
        op0.push_back((uint16_t)nops);
        if (nops + products.back().size() > (size_t)kMuonOps) return too_many();
        std::copy(products.back().begin(), products.back().end(), gemm->op + nops);
        nops += (int)products.back().size();
    }
    // The list of products: level by level, in each the longest first, so that the
    // end of a level is short tiles.
    struct Item {
        int level;
        uint32_t depth, at;
    };
    std::vector<Item> list;
    list.reserve(group.listed);
    uint32_t parts = 0, tiles = 0;
    int k = 0;
    for (const Alike& like : group.alike) {
        const Shape& s = like.shape;
        const Room room = room_of(s, group.kinds[like.kind].segments);
        const std::vector<MuonOp>& ops = products[like.kind];
        for (size_t o = 0; o < ops.size(); ++o) {
            const uint32_t depth = ops[o].kind == kGram ? std::max(s.rows, s.cols) : s.small();
            list.push_back({ops[o].level, depth, (uint32_t)k | (uint32_t)like.matrices.size() << 8 | (uint32_t)o << 16});
        }
        for (const int t : like.matrices) {
            MuonWork& w = gemm->work[k];
            for (int i = 0; i < 2; ++i) w.x[i] = i < room.xs ? take(2 * room.x) : nullptr;
            w.squares = take(2 * room.square * room.squares);
            w.rows = s.rows;
            w.cols = s.cols;
            w.op0 = op0[like.kind];
            w.ops = (uint16_t)ops.size();
            uint16_t* const res = w.x[last[like.kind]];
            result[k] = {res, res + room.x / 2};
            matrix[k] = t;
            MuonMat& m = prep->mat[k];
            place_matrix(job, t, m, nullptr, 0);
            m.part0 = parts;
            m.parts = parts_of(s);
            m.x = {w.x[0], w.x[0] + room.x / 2};
            m.tile0 = tiles;
            parts += m.parts;
            tiles += pad_up(s.rows) / 128 * (pad_up(s.cols) / kBlk);
            ++k;
        }
    }
    if (list.size() > (size_t)kMuonSeq) return too_many();
    cudaError_t e = timed_launch([&] { return launch_muon_squares(*prep, parts, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "Muon norm launch");
    e = timed_launch([&] { return launch_muon_pack(*prep, tiles, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "Muon pack launch");
    t_stats.launches += 2;

    std::stable_sort(list.begin(), list.end(),
                     [](const Item& a, const Item& b) { return a.level != b.level ? a.level < b.level : a.depth > b.depth; });
    gemm->n = (uint32_t)n;
    gemm->nseq = (uint32_t)list.size();
    for (size_t k = 0; k < list.size(); ++k) gemm->seq[k] = list[k].at;
    e = timed_launch([&] { return launch_muon_gemm(*gemm, nops, stream); });
    if (e != cudaSuccess) return cuda_fail(e, "Newton-Schulz product launch");
    t_stats.launches += gemm->nseq > 0 ? 1 : 0;

    std::unique_ptr<MuonFinishParams> fin(new MuonFinishParams{});
    const int nr = job.out->nranks, most = std::max(1, kMuonPtrs / nr);
    fin->nranks = nr;
    fin->inv = (float)(1.0 / scale_for(plan.rho[plan.steps]));
    fin->keep = job.keep;
    for (int k0 = 0; k0 < n; k0 += most) {
        fin->n = std::min(most, n - k0);
        uint32_t todo = 0;
        for (int k = 0; k < fin->n; ++k) {
            MuonMat& m = fin->mat[k];
            place_matrix(job, matrix[k0 + k], m, fin->out, (uint32_t)(k * nr));
            m.x = result[k0 + k];
            m.tile0 = todo;
            todo += pad_up(m.rows) / 128 * (pad_up(m.cols) / kBlk);
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
    const auto groups = groups_of(job.out, plan, &need);
    for (int t = 0; t < job.in->nmatrices; ++t) {
        const uint64_t numel = job.in->rows[t] * job.in->cols[t];
        S += numel * esize(job.out->dtypes[t]);
        total += numel;
    }
    stats_begin(RR_ALGO_ONESHOT, job.out->nranks, S);
    std::vector<int> small;
    for (int t = 0; t < job.in->nmatrices; ++t)
        if (job.in->rows[t] * job.in->cols[t] != 0 && is_small(job.in->rows[t], job.in->cols[t])) small.push_back(t);
    if (groups.empty() && small.empty()) return RR_OK;
    if (!ws || (uintptr_t)ws % 256 != 0) return fail(RR_ERR_INVALID_ARG, "workspace NULL or not aligned to 256 bytes");
    if (ws_bytes < need)
        return fail(RR_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
    spans.push_back({(uintptr_t)ws, (uintptr_t)ws + need, true});
    rr_status_t st = check_spans(spans);
    if (st != RR_OK) return st;
    if ((st = check_device_spans(spans)) != RR_OK) return st;
    // long matrices of a group share a cluster size with long ones
    std::stable_sort(small.begin(), small.end(), [&](int a, int b) {
        return std::max(job.in->rows[a], job.in->cols[a]) > std::max(job.in->rows[b], job.in->cols[b]);
    });
    if ((st = run_small(job, plan, small, stream)) != RR_OK) return st;
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
    std::vector<Span> spans;
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

// Weights come out as exactly as results of their type: both calls need the same.
rr_status_t rr_muon_workspace(const rr_matrix_list_t* results, int /* weights */, const rr_newton_schulz_t* ns, size_t* bytes)
{
    return guarded([&]() -> rr_status_t {
        if (!bytes) return fail(RR_ERR_INVALID_ARG, "NULL workspace size output");
        Plan plan;
        rr_status_t st = make_plan(ns, &plan);
        if (st == RR_OK) st = check_list(results, "results");
        if (st != RR_OK) return st;
        uint64_t need = 0;
        groups_of(results, plan, &need);
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
