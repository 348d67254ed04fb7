"""Host-side checks of the global norm and clipping calls: every call here
fails its argument checks before anything is enqueued, or computes on the host
only, so no GPU is needed."""
import ctypes

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from ring_all_reduce_virtual_b200 import _lib
from ring_all_reduce_virtual_b200.build import build

INVALID, UNSUPPORTED = _lib.RR_ERR_INVALID_ARG, _lib.RR_ERR_UNSUPPORTED
BASE = 1 << 40  # addresses that no call gets as far as using


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


class List:
    """A tensor list with made-up addresses, `gap` bytes from one to the next."""

    def __init__(self, numels, dtypes, nranks=1, base=BASE, gap=1 << 24, ptrs=None):
        n = len(numels)
        self.ptrs = (ctypes.c_void_p * max(n * nranks, 1))(*(ptrs or [base + i * gap for i in range(n * nranks)]))
        self.numels = (ctypes.c_size_t * max(n, 1))(*numels)
        self.dtypes = (ctypes.c_int * max(n, 1))(*dtypes)
        self.c = _lib.TensorList(ctypes.cast(self.ptrs, ctypes.POINTER(ctypes.c_void_p)),
                                 ctypes.cast(self.numels, ctypes.POINTER(ctypes.c_size_t)),
                                 ctypes.cast(self.dtypes, ctypes.POINTER(ctypes.c_int)), n, nranks)
        self.ref = ctypes.byref(self.c)


NORM, WS, BIG = 1 << 44, 1 << 45, 1 << 20


def norm(l, norm=NORM, ws=WS, size=BIG):
    return _lib.lib().rr_grad_norm(l.ref if l else None, norm, ws, size, None)


def clip(l, max_norm=1.0, eps=1e-6, norm=NORM, ws=WS, size=BIG):
    return _lib.lib().rr_clip_grads(l.ref if l else None, max_norm, eps, norm, ws, size, None)


@pytest.mark.parametrize("call", [norm, clip])
def test_list_calls_refuse_bad_arguments(call):
    good = [100, 7], [0, 1]
    assert call(None) == INVALID
    assert call(List(*good, nranks=0, ptrs=[BASE])) == INVALID
    assert call(List(*good, nranks=65)) == INVALID
    assert call(List([100], [9])) == INVALID
    assert call(List([100], [2])) == UNSUPPORTED  # int32 is no gradient type
    assert b"bf16, fp16 or fp32" in _lib.lib().rr_last_error()
    assert call(List([1 << 49], [0])) == INVALID
    assert call(List([1 << 48, 1], [0, 0], gap=1 << 52)) == INVALID  # above 2^48 in all
    assert call(List(*good, ptrs=[BASE, None])) == INVALID
    assert call(List([100], [0], base=BASE + 2)) == INVALID  # an fp32 tensor off its element size
    assert b"element size" in _lib.lib().rr_last_error()
    assert call(List(*good), norm=None) == INVALID
    assert call(List(*good), norm=NORM + 2) == INVALID
    assert call(List(*good), ws=None) == INVALID
    assert call(List(*good), ws=WS + 4) == INVALID
    assert call(List(*good), size=64) == INVALID
    assert b"workspace too small" in _lib.lib().rr_last_error()
    assert call(List(*good), norm=BASE + 8) == INVALID  # the norm inside a gradient
    assert call(List(*good), ws=BASE + 8) == INVALID
    assert call(List(*good), norm=WS + 8) == INVALID
    broken = List(*good)
    broken.c.ntensors = -1
    assert call(broken) == INVALID


def test_clip_refuses_overlaps_and_bad_norms():
    assert clip(List([100, 100], [0, 0], gap=396)) == INVALID
    assert b"overlap" in _lib.lib().rr_last_error()
    assert clip(List([100], [0], nranks=2, gap=0)) == INVALID  # a replica given twice
    for bad in (-1.0, float("nan")):
        assert clip(List([100], [0]), max_norm=bad) == INVALID
    for bad in (-1e-6, float("nan"), float("inf")):
        assert clip(List([100], [0]), eps=bad) == INVALID


def test_workspace_sizes():
    lib, b = _lib.lib(), ctypes.c_size_t()
    assert lib.rr_clip_workspace(None, 0, 0, 0, None, ctypes.byref(b)) == INVALID
    assert lib.rr_clip_workspace(None, 0, 0, 0, List([5], [0]).ref, None) == INVALID
    assert lib.rr_clip_workspace(None, 0, 0, 0, List([5], [2]).ref, ctypes.byref(b)) == UNSUPPORTED
    sizes = []
    for l in (List([], []), List([5], [0]), List([5, 5], [0, 1]), List([5] * 1025, [0] * 1025)):
        assert lib.rr_clip_workspace(None, 0, 0, 0, l.ref, ctypes.byref(b)) == 0
        sizes.append(b.value)
    assert sizes == sorted(sizes) and sizes[2] == sizes[3]  # two types, or two launches of one
    plan = rrv.BucketPlan([1000, 3, 100000], "bf16", 4096)
    for args in ((plan._h, 0, 0, 4), (plan._h, 0, 9, 4), (plan._h, 0, 1, 0), (plan._h, 0, 1, 65)):
        assert lib.rr_clip_workspace(*args, None, ctypes.byref(b)) == INVALID
    assert lib.rr_clip_workspace(plan._h, 0, plan.num_buckets, 4, None, ctypes.byref(b)) == 0 and b.value > 0


def test_bucket_clip_refuses_bad_arguments():
    lib = _lib.lib()
    plan = rrv.BucketPlan([1000, 20], "bf16", 1 << 20)
    grads = (ctypes.c_void_p * 4)(*[BASE + (i << 24) for i in range(4)])

    def call(plan=plan._h, first=0, count=1, grads=grads, n=2, op=1, synced=None, max_norm=1.0, eps=1e-6, norm=NORM,
             ws=WS, size=BIG):
        return lib.rr_bucket_allreduce_clip(plan, first, count, grads, n, op, synced, max_norm, eps, norm, ws, size, None)

    assert call(plan=None) == INVALID
    assert call(first=1) == INVALID
    assert call(count=0) == INVALID
    assert call(grads=None) == INVALID
    assert call(n=0) == INVALID
    assert call(n=65) == INVALID
    assert call(op=2) == UNSUPPORTED
    assert call(max_norm=float("nan")) == INVALID
    assert call(eps=-1.0) == INVALID
    assert call(norm=None) == INVALID
    assert call(ws=None) == INVALID
    assert call(size=8) == INVALID
    assert call(grads=(ctypes.c_void_p * 4)(*[BASE] * 4)) == INVALID
    assert call(synced=List([5], [2], nranks=2, base=1 << 42).ref) == UNSUPPORTED
    assert call(synced=List([5], [0], nranks=1, base=1 << 42).ref) == INVALID  # another number of ranks
    assert b"number of ranks" in lib.rr_last_error()
    assert call(synced=List([5], [0], nranks=2).ref) == INVALID  # overlaps the buckets' gradients
    assert b"overlap" in lib.rr_last_error()


def test_grad_list_checks_its_tensors():
    cpu = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        rrv.GradList([cpu])
    with pytest.raises(ValueError, match="ranks"):
        rrv.GradList([[cpu]] * 65)
    with pytest.raises(ValueError, match="same number"):
        rrv.GradList([[], [cpu]])
    with pytest.raises(ValueError, match="CUDA"):
        rrv.grad_norm([cpu])
    with pytest.raises(ValueError, match="CUDA"):
        rrv.clip_grads([cpu], 1.0)


@pytest.mark.parametrize("nranks", [1, 2, 3])
def test_an_empty_synced_list_is_none(nranks):
    """Whatever its rank count: the call goes on to its later checks (here the workspace's) and is refused there."""
    plan = rrv.BucketPlan([1000, 20], "bf16", 1 << 20)
    grads = (ctypes.c_void_p * 4)(*[BASE + (i << 24) for i in range(4)])
    st = _lib.lib().rr_bucket_allreduce_clip(plan._h, 0, 1, grads, 2, 1, List([], [], nranks=nranks).ref, 1.0, 1e-6, NORM,
                                             WS, 8, None)
    assert st == INVALID and b"workspace too small" in _lib.lib().rr_last_error()


class Fake:
    """What the argument checks read of a CUDA tensor, without a GPU; its address is never used."""

    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, n, dtype=torch.bfloat16, at=BASE):
        self.n, self.dtype, self.at = n, dtype, at

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def test_bucket_calls_take_a_grad_list():
    plan = rrv.BucketPlan([1000, 20], "bf16", 1 << 20)
    for n in (1, 3):
        ranks = [[Fake(m, at=BASE + ((2 * r + t) << 24)) for t, m in enumerate((1000, 20))] for r in range(n)]
        want = plan._grads(rrv.GradSet(ranks))
        gl = rrv.GradList(ranks if n > 1 else ranks[0])
        got = plan._grads(gl)
        assert list(got[0]) == list(want[0]) and got[1:] == want[1:]
        assert plan._grads(gl)[0] is got[0]  # marshalled once
    assert list(plan._grads(ranks[0])[0]) == list(want[0])[:2]  # one rank's tensors as they are
    for wrong in (rrv.GradList([Fake(1000), Fake(21)]), rrv.GradList([Fake(1000), Fake(20, torch.float32)]),
                  rrv.GradList([])):
        with pytest.raises(ValueError):
            plan._grads(wrong)


def test_debug_mode_checks_the_pointers_of_tensors_with_elements():
    """RR_DEBUG=1: an empty tensor's NULL passes as it does without it (the call gets as far as a launch, which fails where
    no GPU is), and every gradient of every call is looked up."""
    import os
    import subprocess
    import sys

    script = """
import sys
sys.path[:0] = sys.argv[1:]
from test_clip_host import *
from ring_all_reduce_virtual_b200 import _lib
lib = _lib.lib()
empty = List([0, 0], [0, 1], nranks=2, ptrs=[None] * 4)
made_up = List([0, 8], [0, 1], nranks=2, ptrs=[None, BASE] * 2)
for call in (norm, clip):
    print("EMPTY", call(empty) == _lib.RR_ERR_CUDA, b"not device memory" not in lib.rr_last_error())
print("MADE UP", norm(made_up) == INVALID, b"not device memory" in lib.rr_last_error())
two = List([0, 8], [0, 1], nranks=2, ptrs=[None, BASE, None, BASE + 64])
print("MADE UP", clip(two) == INVALID, b"not device memory" in lib.rr_last_error())
plan = rrv.BucketPlan([1000, 0], "bf16", 1 << 20)
grads = (ctypes.c_void_p * 4)(BASE, None, BASE + (1 << 20), None)
st = lib.rr_bucket_allreduce_clip(plan._h, 0, plan.num_buckets, grads, 2, 1, None, 1.0, 1e-6, NORM, WS, BIG, None)
print("MADE UP", st == INVALID, b"not device memory" in lib.rr_last_error())
"""
    here = os.path.dirname(os.path.abspath(__file__))
    out = subprocess.run([sys.executable, "-c", script, here, os.path.dirname(here)], capture_output=True, text=True,
                         env=dict(os.environ, RR_DEBUG="1", CUDA_VISIBLE_DEVICES=""), timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("EMPTY True True") == 2 and out.stdout.count("MADE UP True True") == 3, out.stdout
