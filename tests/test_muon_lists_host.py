"""The host side of the orthogonalisation and the Muon step over long and mixed
lists, on the CPU: the C calls themselves, compiled with the address sanitizer
and with launches that look over the parameters they are given."""
import os
import subprocess

import pytest

import ring_all_reduce_virtual_b200 as rrv

PACKAGE = os.path.dirname(os.path.abspath(rrv.__file__))
QUIET = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")  # which wants to trace the process

PROGRAM = r"""
#include "rr_muon_api.cu"

#include <cstdio>
#include <map>
#include <random>
#include <set>

// ------------------------------------------------- launches that check

static int bad = 0;
static std::string what;
#define EXPECT(c) do { if (!(c) && bad++ < 20) std::printf("%s: line %d: %s\n", what.c_str(), __LINE__, #c); } while (0)

static uintptr_t ws_lo, ws_hi;
static std::multiset<const void*> summed, packed, written;  // first pointers of the matrices that the passes go over
static std::vector<int> seq_sizes;
static std::map<const void*, rr::Halves> first_x, last_x;   // by gradient
static uint32_t total_tiles(const MuonMat* m, int n)
{
    uint32_t at = 0;
    for (int k = 0; k < n; ++k) {
        EXPECT(m[k].tile0 == at);
        at += pad_up(m[k].rows) / 128 * (pad_up(m[k].cols) / kBlk);
    }
    return at;
}
static void in_workspace(const void* p, uint64_t bytes)
{
    EXPECT((uintptr_t)p >= ws_lo && (uintptr_t)p + bytes <= ws_hi);
}

namespace rr {
cudaError_t launch_muon_squares(const MuonPrepParams& p, uint32_t parts, cudaStream_t)
{
    EXPECT(p.n >= 1 && p.n <= kMuonMats);
    uint32_t at = 0;
    for (int k = 0; k < p.n; ++k) {
        EXPECT(p.mat[k].part0 == at && p.mat[k].parts >= 1 && p.mat[k].parts <= kNormParts);
        at += p.mat[k].parts;
        summed.insert(p.mat[k].g);
    }
    EXPECT(at == parts);
    in_workspace(p.partial, parts * 8ull);
    in_workspace(p.counters, kMuonCounters * 4ull);
    EXPECT((uintptr_t)p.counters >= (uintptr_t)(p.partial + parts));
    return cudaSuccess;
}
cudaError_t launch_muon_pack(const MuonPrepParams& p, uint32_t tiles, cudaStream_t)
{
    EXPECT(total_tiles(p.mat, p.n) == tiles);
    first_x.clear();
    for (int k = 0; k < p.n; ++k) {
        packed.insert(p.mat[k].g);
        first_x[p.mat[k].g] = p.mat[k].x;
        in_workspace(p.mat[k].x.lo, 2ull * pad_up(p.mat[k].rows) * pad_up(p.mat[k].cols));
    }
    return cudaSuccess;
}
cudaError_t launch_muon_gemm(MuonGemmParams& p, int nops, cudaStream_t)
{
    EXPECT(p.n <= (uint32_t)kMuonMats && nops <= kMuonOps && p.nseq <= (uint32_t)kMuonSeq);
    if (p.n > (uint32_t)kMuonMats || nops > kMuonOps || p.nseq > (uint32_t)kMuonSeq) return cudaSuccess;
    seq_sizes.push_back((int)p.nseq);
    std::vector<std::vector<int>> seen(p.n);  // levels of each matrix's products, in the list's order
    std::set<std::pair<uint32_t, uint32_t>> once;
    for (uint32_t k = 0; k < p.nseq; ++k) {
        const uint32_t e = p.seq[k], first = e & 255u, many = e >> 8 & 255u, o = e >> 16;
        EXPECT(many >= 1 && first + many <= p.n);
        for (uint32_t m = first; m < first + many && m < p.n; ++m) {
            const MuonWork &w = p.work[m], &w0 = p.work[first];
            EXPECT(w.rows == w0.rows && w.cols == w0.cols && w.op0 == w0.op0 && w.ops == w0.ops);
            EXPECT(o < w.ops && w.op0 + w.ops <= nops);
            EXPECT(once.insert({m, o}).second);
            seen[m].push_back(p.op[w.op0 + o].level);
        }
    }
    std::vector<std::pair<uintptr_t, uintptr_t>> mem;
    last_x.clear();
    for (uint32_t m = 0; m < p.n; ++m) {
        const MuonWork& w = p.work[m];
        EXPECT(seen[m].size() == w.ops && std::is_sorted(seen[m].begin(), seen[m].end()));
        const uint64_t xb = 4ull * pad_up(w.rows) * pad_up(w.cols), side = pad_up(std::min(w.rows, w.cols));
        uint32_t squares = 0, cur = 0;
        for (uint32_t o = 0; o < w.ops; ++o) {
            const MuonOp& q = p.op[w.op0 + o];
            EXPECT(q.chunk >= 1 && q.chunk <= 4);
            for (const uint8_t b : {q.a, q.b, q.c, q.out})
                if (b != kNoBuffer && b >= kSquares) squares = std::max(squares, b - kSquares + 1u);
            if (q.kind == kApply) {
                EXPECT(q.b == cur && q.out == (cur ^ 1));
                cur ^= 1;
            }
        }
        for (int i = 0; i < (w.ops ? 2 : 1); ++i) mem.push_back({(uintptr_t)w.x[i], (uintptr_t)w.x[i] + xb});
        if (squares) mem.push_back({(uintptr_t)w.squares, (uintptr_t)w.squares + 4 * side * side * squares});
        bool found = false;  // the matrix whose X this begins with, which the last pass has to read where it ends
        for (const auto& e : first_x)
            if (e.second.hi == w.x[0]) {
                found = true;
                last_x[e.first] = {w.x[cur], w.x[cur] + xb / 4};
            }
        EXPECT(found);
    }
    std::sort(mem.begin(), mem.end());
    for (size_t k = 0; k < mem.size(); ++k) {
        EXPECT(mem[k].first >= ws_lo && mem[k].second <= ws_hi);
        EXPECT(k == 0 || mem[k - 1].second <= mem[k].first);
    }
    return cudaSuccess;
}
cudaError_t launch_muon_finish(const MuonFinishParams& p, uint32_t tiles, cudaStream_t)
{
    EXPECT(p.n <= kMuonMats && p.n * p.nranks <= kMuonPtrs && total_tiles(p.mat, p.n) == tiles);
    for (int k = 0; k < p.n; ++k) {
        const MuonMat& m = p.mat[k];
        EXPECT(last_x.count(m.g) && last_x[m.g].hi == m.x.hi && last_x[m.g].lo == m.x.lo);
        EXPECT(m.out + p.nranks <= (uint32_t)kMuonPtrs);
        for (int r = 0; r < p.nranks; ++r) written.insert(p.out[m.out + r]);
    }
    return cudaSuccess;
}
cudaError_t launch_muon_small(MuonSmallParams& p, cudaStream_t)
{
    EXPECT(p.n <= kMuonMats && p.n * p.nranks <= kMuonPtrs && p.ctas >= 1 && p.ctas <= kMuonSmallCtas);
    for (int k = 0; k < p.n; ++k) {
        const MuonMat& m = p.mat[k];
        EXPECT(std::min(m.rows, m.cols) <= kMuonSmallSide && std::max(m.rows, m.cols) <= p.ctas * kMuonSmallSide);
        summed.insert(m.g);
        packed.insert(m.g);
        for (int r = 0; r < p.nranks; ++r) written.insert(p.out[m.out + r]);
    }
    return cudaSuccess;
}
cudaError_t take_bulk_timeouts(unsigned int*, unsigned int*) { return cudaSuccess; }
}  // namespace rr

extern "C" {
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus*) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes*, const void*) { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return ""; }
}

// ------------------------------------------------------------- calls

struct Shape2 {
    size_t r, c;
    rr_dtype_t d;
};

static void call(const std::string& name, const std::vector<Shape2>& list, int ranks, bool weights, const rr_newton_schulz_t& ns)
{
    what = name;
    const int n = (int)list.size();
    std::vector<size_t> r, c;
    std::vector<rr_dtype_t> d, f32(n, RR_F32);
    std::vector<void*> out, in, mom;
    const uint64_t gap = 1ull << 34;  // nothing is read or written there
    for (int t = 0; t < n; ++t) {
        r.push_back(list[t].r);
        c.push_back(list[t].c);
        d.push_back(list[t].d);
        in.push_back((void*)((1ull << 50) + t * gap));
        mom.push_back((void*)((1ull << 52) + t * gap));
    }
    for (int k = 0; k < n * ranks; ++k) out.push_back((void*)((1ull << 54) + k * gap));
    const rr_matrix_list_t O{out.data(), r.data(), c.data(), d.data(), n, ranks}, G{in.data(), r.data(), c.data(), d.data(), n, 1},
        M{mom.data(), r.data(), c.data(), f32.data(), n, 1};
    size_t need = 0;
    EXPECT(rr_muon_workspace(&O, weights, &ns, &need) == RR_OK);
    ws_lo = 1ull << 56;
    ws_hi = ws_lo + need;
    summed.clear();
    packed.clear();
    written.clear();
    rr_status_t st;
    if (weights) {
        const rr_muon_t cfg{0.1f, 0.9f, 0.0f, 1, 0, ns};
        st = rr_muon_step(&O, &G, &M, &cfg, (void*)ws_lo, need, nullptr);
    } else {
        st = rr_orthogonalize(&G, &O, &ns, (void*)ws_lo, need, nullptr);
    }
    EXPECT(st == RR_OK);
    std::multiset<const void*> want_in, want_out;
    for (int t = 0; t < n; ++t)
        if (r[t] * c[t] != 0) {
            want_in.insert(in[t]);
            for (int k = 0; k < ranks; ++k) want_out.insert(out[(size_t)k * n + t]);
        }
    EXPECT(summed == want_in && packed == want_in && written == want_out);
}

static std::vector<Shape2> every_type(int shapes, size_t rows)
{
    std::vector<Shape2> v;
    for (int k = 0; k < shapes; ++k)
        for (const rr_dtype_t d : {RR_F32, RR_BF16, RR_F16}) v.push_back({rows, 1024 + 8 * (size_t)k, d});
    return v;
}

int main(int argc, char** argv)
{
    const rr_newton_schulz_t usual{5, 3.4445f, -4.7750f, 2.0315f, 1e-7f};
    if (argc == 1) {  // lists whose every shape comes in all three types
        for (const int shapes : {1, 13, 14, 20, 43, 60})
            for (const size_t rows : {150, 300, 512, 1024})
                for (const bool weights : {false, true})
                    call("every type " + std::to_string(shapes) + " x " + std::to_string(rows), every_type(shapes, rows), 2, weights, usual);
        // one shape in three types: its products once for each kind of iteration, whatever types are of a kind
        seq_sizes.clear();
        call("one shape", every_type(1, 1024), 1, true, usual);
        EXPECT(seq_sizes.size() == 1);
        std::printf("one shape: %d products\n", seq_sizes.at(0));
    } else {
        std::mt19937 gen(7);
        const auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(gen); };
        const rr_dtype_t types[3] = {RR_F32, RR_BF16, RR_F16};
        for (int k = 0; k < 400; ++k) {
            rr_newton_schulz_t ns = usual;
            const int form = pick(0, 3);
            if (form == 1) ns = {pick(0, 50), 1.5f, -0.5f, 0.0f, 1e-7f};
            if (form == 2) ns = {pick(0, 50), 1.0f, 0.0f, 0.0f, 1e-3f};
            if (form == 3) ns = {pick(0, 8), 2.0f, -1.5f, 0.5f, 1e-7f};
            std::vector<Shape2> list;
            const int n = pick(1, 300), shapes = pick(1, 40);
            std::vector<std::pair<size_t, size_t>> pool;
            for (int s = 0; s < shapes; ++s) {
                const int side = 1 << pick(3, 12);
                pool.push_back({(size_t)pick(0, 20) == 0 ? 0 : (size_t)pick(1, side), (size_t)pick(1, side)});
            }
            for (int t = 0; t < n; ++t) {
                const auto& s = pool[pick(0, shapes - 1)];
                list.push_back({s.first, s.second, types[pick(0, 2)]});
            }
            call("list " + std::to_string(k), list, pick(0, 3) ? pick(1, 9) : 64, pick(0, 1), ns);
        }
    }
    std::printf("bad %d\n", bad);
    return bad != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("muon_lists")
    src, exe = where / "lists.cpp", where / "lists"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++20", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                    "-I", os.path.join(PACKAGE, "csrc"), "-I", os.path.join(os.path.dirname(PACKAGE), "include"),
                    "-I", "/usr/local/cuda/include", "-o", str(exe), str(src), "-ldl"], check=True)
    return str(exe)


def test_lists_that_have_every_shape_in_three_types(program):
    """Each product of each matrix is listed once, within the launch's parameters and in the order of its levels."""
    out = subprocess.run([program], env=QUIET, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout + out.stderr[:4000]


def test_any_list(program):
    """Lists of any shapes, types, replicas and iterations: every matrix once, workspaces apart and within what was asked for."""
    out = subprocess.run([program, "any"], env=QUIET, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout + out.stderr[:4000]
