"""Host-side checks of the embedding calls: every call here fails its argument
checks before anything is enqueued, or computes on the host only."""
import ctypes

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from ring_all_reduce_virtual_b200 import _lib
from ring_all_reduce_virtual_b200.build import build

INVALID, UNSUPPORTED = _lib.RR_ERR_INVALID_ARG, _lib.RR_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def ptrs(n, base, gap=1 << 30):
    return (ctypes.c_void_p * n)(*[base + i * gap for i in range(n)])


IDS, TABLES, OUTS, WS = 1 << 40, 1 << 42, 1 << 44, 1 << 46


def lookup(ids=ptrs(2, IDS), id_type=0, tables=ptrs(2, TABLES), outs=ptrs(2, OUTS), n=2, T=16, V=100, D=32, dtype=0):
    return _lib.lib().rr_embedding(ids, id_type, tables, outs, n, T, V, D, dtype, 1.0, None)


def grad(ids=ptrs(2, IDS), id_type=0, dout=ptrs(2, TABLES), n=2, T=16, V=100, D=32, dtype=1, op=1, grads=ptrs(2, OUTS),
         nout=2, grad_dtype=1, accumulate=0, ws=WS, size=1 << 30):
    return _lib.lib().rr_embedding_grad(ids, id_type, dout, n, T, V, D, dtype, op, 1.0, -1, grads, nout, grad_dtype,
                                        accumulate, ws, size, None)


@pytest.mark.parametrize("call", [lookup, grad])
def test_shapes_types_and_pointers_are_checked(call):
    for bad in (dict(n=0), dict(n=65), dict(dtype=9), dict(id_type=2), dict(D=0), dict(D=(1 << 20) + 1), dict(V=0),
                dict(V=(1 << 31) - 1), dict(T=1 << 31), dict(T=1 << 30), dict(T=1 << 63), dict(ids=None),
                dict(ids=ptrs(2, IDS + 2)), dict(ids=ptrs(2, IDS + 4), id_type=1), dict(ids=(ctypes.c_void_p * 2)(IDS, None))):
        assert call(**bad) == INVALID, bad
    assert call(dtype=2) == UNSUPPORTED
    assert b"bf16, fp16 or fp32" in _lib.lib().rr_last_error()


def test_lookup_refuses_bad_buffers():
    for bad in (dict(tables=None), dict(outs=None), dict(tables=ptrs(2, TABLES + 2)), dict(outs=ptrs(2, OUTS + 1)),
                dict(outs=ptrs(2, TABLES)), dict(outs=ptrs(2, OUTS, gap=64)), dict(outs=ptrs(2, IDS))):
        assert lookup(**bad) == INVALID, bad
    assert lookup(T=0) == 0  # no token: nothing is enqueued


def test_grad_refuses_bad_arguments():
    for bad in (dict(dout=None), dict(grads=None), dict(nout=0), dict(nout=65), dict(dout=ptrs(2, TABLES + 1)),
                dict(grads=ptrs(2, OUTS + 2), grad_dtype=0), dict(grads=ptrs(2, OUTS, gap=0)), dict(grads=ptrs(2, TABLES)),
                dict(ws=None), dict(ws=WS + 128), dict(size=1000), dict(ws=OUTS)):
        assert grad(**bad) == INVALID, bad
    for bad in (dict(op=2), dict(grad_dtype=3), dict(grad_dtype=2), dict(dtype=0, grad_dtype=1)):
        assert grad(**bad) == UNSUPPORTED, bad
    assert grad(T=0, accumulate=1) == 0


def test_grad_workspace():
    lib, b = _lib.lib(), ctypes.c_size_t()
    assert lib.rr_embedding_grad_workspace(2, 10, 100, 32, None) == INVALID
    assert lib.rr_embedding_grad_workspace(0, 10, 100, 32, ctypes.byref(b)) == INVALID
    sizes = []
    for n, T, V, D in ((1, 0, 1, 1), (1, 1, 1, 1), (2, 10, 100, 32), (8, 8192, 32000, 2048), (8, 65536, 32000, 2048)):
        assert lib.rr_embedding_grad_workspace(n, T, V, D, ctypes.byref(b)) == 0
        assert b.value % 256 == 0
        sizes.append(b.value)
    assert sizes == sorted(sizes) and sizes[-1] < 200 << 20  # the partial sums do not grow with the tokens


def test_python_calls_check_their_tensors():
    cpu = torch.zeros(2, 4)
    ids = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="alike"):
        rrv.embedding([ids], [cpu], [cpu])  # not on a GPU
    with pytest.raises(TypeError, match="int32 or int64"):
        rrv.embedding([ids.float()], [cpu], [cpu])
    with pytest.raises(ValueError, match="1..64"):
        rrv.embedding_grad([], [cpu], [cpu])


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class OnDevice1:  # what a stream of a second GPU is to the check, without one
        device = torch.device("cuda", 1)
        cuda_stream = 0

    monkeypatch.setattr(torch.cuda, "Stream", OnDevice1)
    with pytest.raises(ValueError, match="cuda:1, the tensors to cuda:0"):
        with rrv._placed(OnDevice1(), torch.device("cuda", 0)):
            pass


class Fake:
    """What the argument checks read of a CUDA tensor, without a GPU; its address is never used."""

    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 40


@pytest.mark.parametrize("as_set", [False, True])
@pytest.mark.parametrize("bad", ["tables", "outs", "grad_out", "grads"])
@pytest.mark.parametrize("shape", [(8, 6), (2, 24), (48,), (48, 1)])
def test_rows_of_another_width_on_another_rank_are_refused(as_set, bad, shape):
    """Rank 1's tensor has rank 0's element count (6 rows of 8) but not its rows."""
    ids = [Fake(6, dtype=torch.int32), Fake(6, dtype=torch.int32)]
    wrap = rrv.RankSet if as_set else list
    good, mixed = wrap([Fake(6, 8), Fake(6, 8)]), wrap([Fake(6, 8), Fake(*shape)])
    with pytest.raises(ValueError, match="one width on every rank"):
        if bad in ("tables", "outs"):
            rrv.embedding(ids, mixed if bad == "tables" else good, mixed if bad == "outs" else good)
        else:
            rrv.embedding_grad(ids, mixed if bad == "grad_out" else good, mixed if bad == "grads" else good)


def test_rows_may_be_grouped_differently():
    """Leading axes only group the rows: the same rows and width count as alike."""
    assert rrv._row_set([Fake(6, 8), Fake(2, 3, 8)], "rows")[1:4] == (2, 6, 8)


SEARCH = r"""
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>
#include <algorithm>
#include "rr_search.h"

// A warp's search for the rows [v0, v0 + 32): its rounds, and the range that it leaves.
static int follow(const std::vector<uint32_t>& keys, uint64_t v0, uint32_t& lo, uint32_t& hi)
{
    int rounds = 0;
    lo = 0;
    hi = (uint32_t)keys.size();
    while (hi - lo > 64) {
        uint32_t below = 0, within = 0;
        for (uint32_t lane = 0; lane < 32; ++lane) {
            const uint64_t at = lo + (uint64_t)lane * rr::search_step(lo, hi);
            if (at >= hi) continue;
            below += keys[at] < v0;
            within += keys[at] < v0 + 32;
        }
        ++rounds;
        if (rounds > 1000000 || !rr::search_narrow(lo, hi, below, within)) break;
    }
    return rounds;
}

int main()
{
    std::mt19937_64 gen(1);
    std::uniform_real_distribution<double> unit(0.0, 1.0);
    int bad = 0;
    for (const uint32_t V : {1u, 40u, 5000u})
        for (const uint32_t M : {1u, 64u, 65u, 2049u, 65536u, 1000003u})
            for (int kind = 0; kind < 5; ++kind) {
                std::vector<uint32_t> keys(M);
                for (uint32_t i = 0; i < M; ++i) {
                    const double u = unit(gen);
                    const uint32_t zipf = std::min(V, (uint32_t)(std::exp(u * std::log(V + 1.0)) - 1.0));
                    keys[i] = kind == 0 ? zipf                              // frequent tokens, first rows
                              : kind == 1 ? (zipf * 2654435761u) % V        // ... anywhere
                              : kind == 2 ? V / 2                           // one token
                              : kind == 3 ? (u < 0.9 ? V : (uint32_t)(unit(gen) * V))  // ids without a row behind
                                          : (uint32_t)(unit(gen) * V);
                }
                std::sort(keys.begin(), keys.end());
                const double most = std::ceil(std::log2((double)M)) + 3;
                for (uint64_t v0 = 0; v0 < V; v0 += 32) {
                    uint32_t lo, hi;
                    const int rounds = follow(keys, v0, lo, hi);
                    const double steps = rounds + std::ceil(std::log2(hi - lo + 1.0));
                    const bool lost = lo > hi || hi > M || (lo > 0 && keys[lo - 1] >= v0) || (hi < M && keys[hi] < v0 + 32);
                    if ((lost || steps > most) && bad++ < 5)
                        std::printf("V %u M %u kind %d v0 %llu: %d rounds to [%u, %u)\n", V, M, kind, (unsigned long long)v0,
                                    rounds, lo, hi);
                }
            }
    std::printf("bad %d\n", bad);
    return bad != 0;
}
"""


def test_a_frequent_token_does_not_lengthen_the_search_for_rows_without_one(tmp_path):
    """Every round but the last halves the range, so r rounds leave at most M / 2^(r - 1) positions, and the rounds and the
    binary search behind them are at most log2(M) + 3 steps; the range keeps all that a lane looks for."""
    import os
    import subprocess

    src, exe = tmp_path / "search.cpp", tmp_path / "search"
    src.write_text(SEARCH)
    csrc = os.path.join(os.path.dirname(os.path.abspath(rrv.__file__)), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", csrc, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout
