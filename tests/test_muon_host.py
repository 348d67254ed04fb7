"""Host-side checks of the orthogonalisation and the Muon step: every call here
fails its argument checks before anything is enqueued, or computes on the host
only."""
import ctypes

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from ring_all_reduce_virtual_b200 import _lib
from ring_all_reduce_virtual_b200.build import build

INVALID, UNSUPPORTED = _lib.RR_ERR_INVALID_ARG, _lib.RR_ERR_UNSUPPORTED
COEF = (3.4445, -4.7750, 2.0315)
PARAMS, GRADS, MOM, WS = 1 << 40, 1 << 42, 1 << 44, 1 << 46
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def mlist(base, shapes=((64, 32), (300, 300)), dtypes=(0, 1), ranks=1, gap=1 << 30, ptrs=None):
    n = len(shapes)
    arrays = ((ctypes.c_void_p * max(1, n * ranks))(*(ptrs or [base + i * gap for i in range(n * ranks)])),
              (ctypes.c_size_t * max(1, n))(*[s[0] for s in shapes]), (ctypes.c_size_t * max(1, n))(*[s[1] for s in shapes]),
              (ctypes.c_int * max(1, n))(*dtypes[:n]))
    c = _lib.MatrixListC(*[ctypes.cast(a, t) for a, (_, t) in zip(arrays, _lib.MatrixListC._fields_)], n, ranks)
    c.keep = arrays
    return c


def ns(steps=5, coef=COEF, eps=1e-7):
    return _lib.NewtonSchulz(steps, *coef, eps)


def ortho(a=None, b=None, n=None, ws=WS, size=1 << 34):
    a, b, n = a or mlist(GRADS), b or mlist(PARAMS), n or ns()
    return _lib.lib().rr_orthogonalize(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n), ws, size, None)


def step(w=None, g=None, m=None, ws=WS, size=1 << 34, lr=0.1, momentum=0.9, decay=0.0, nesterov=1, adjust=0, n=None):
    w, g, m = w or mlist(PARAMS, ranks=2), g or mlist(GRADS), m or mlist(MOM, dtypes=(0, 0))
    cfg = _lib.Muon(lr, momentum, decay, nesterov, adjust, n or ns())
    return _lib.lib().rr_muon_step(ctypes.byref(w), ctypes.byref(g), ctypes.byref(m), ctypes.byref(cfg), ws, size, None)


def test_lists_are_checked():
    for bad in (dict(a=mlist(GRADS, ranks=0)), dict(b=mlist(PARAMS, ranks=65)), dict(a=mlist(GRADS, dtypes=(0, 9))),
                dict(a=mlist(GRADS, shapes=((64, 32),))), dict(a=mlist(GRADS, shapes=((64, 32), (300, 301)))),
                dict(a=mlist(GRADS, shapes=((64, 32), (1 << 21, 2))), b=mlist(PARAMS, shapes=((64, 32), (1 << 21, 2)))),
                dict(a=mlist(GRADS + 2)), dict(b=mlist(PARAMS + 2)), dict(a=mlist(0, ptrs=[GRADS, 0])), dict(b=mlist(0, ptrs=[PARAMS, 0])),
                dict(b=mlist(PARAMS, gap=4096)), dict(b=mlist(GRADS + 4096)), dict(b=mlist(GRADS, dtypes=(1, 1))),
                dict(b=mlist(GRADS, gap=0)), dict(ws=None), dict(ws=WS + 128), dict(size=1000), dict(ws=PARAMS)):
        assert ortho(**bad) == INVALID, bad
    assert ortho(a=mlist(GRADS, dtypes=(2, 0))) == UNSUPPORTED
    for null in range(3):
        refs = [ctypes.byref(mlist(GRADS)), ctypes.byref(mlist(PARAMS)), ctypes.byref(ns())]
        refs[null] = None
        assert _lib.lib().rr_orthogonalize(*refs, WS, 1 << 34, None) == INVALID
    empty = mlist(GRADS, shapes=((0, 4), (5, 0)))
    assert ortho(a=empty, b=mlist(PARAMS, shapes=((0, 4), (5, 0))), ws=None, size=0) == 0  # nothing to do
    assert ortho(a=mlist(GRADS, shapes=()), b=mlist(PARAMS, shapes=()), ws=None, size=0) == 0


def test_iterations_are_checked():
    for bad in (ns(steps=-1), ns(steps=51), ns(eps=0.0), ns(eps=-1.0), ns(eps=INF), ns(eps=NAN), ns(coef=(NAN, 0, 0)), ns(coef=(1, INF, 0))):
        assert ortho(n=bad) == INVALID
        assert step(n=bad) == INVALID
    for bad in (ns(coef=(2.0, 0.0, 0.0), steps=11), ns(coef=(3.0, 1.0, 1.0)), ns(coef=(1e3, 1e3, 0.0), steps=2)):
        assert ortho(n=bad) == UNSUPPORTED
    assert b"above 1024" in _lib.lib().rr_last_error()


def test_step_is_checked():
    for bad in (dict(lr=INF), dict(lr=NAN), dict(decay=INF), dict(momentum=-0.5), dict(momentum=NAN), dict(momentum=INF), dict(adjust=2),
                dict(adjust=-1), dict(m=mlist(MOM, dtypes=(0, 0), ranks=2)), dict(m=mlist(MOM, dtypes=(0, 0), shapes=((64, 32), (300, 301)))),
                dict(g=mlist(GRADS, shapes=((64, 32),))), dict(w=mlist(PARAMS, ranks=2, gap=64)), dict(g=mlist(PARAMS)), dict(m=mlist(GRADS, dtypes=(0, 0))),
                dict(m=mlist(PARAMS, dtypes=(0, 0))), dict(ws=None), dict(size=5000), dict(ws=MOM)):
        assert step(**bad) == INVALID, bad
    assert step(m=mlist(MOM, dtypes=(0, 1))) == UNSUPPORTED
    assert step(w=mlist(PARAMS, ranks=2, dtypes=(2, 0))) == UNSUPPORTED
    assert _lib.lib().rr_muon_step(None, None, None, None, WS, 1, None) == INVALID


def test_workspace():
    lib, b = _lib.lib(), ctypes.c_size_t()

    def need(shapes, dtypes, weights=0, n=None):
        m = mlist(PARAMS, shapes=shapes, dtypes=dtypes)
        assert lib.rr_muon_workspace(ctypes.byref(m), weights, ctypes.byref(n or ns()), ctypes.byref(b)) == 0
        return b.value

    assert need((), ()) == need(((128, 1024), (1024, 1), (0, 7)), (0, 1, 1)) == 256  # a cluster's own memory is enough
    one = need(((2048, 2048),), (0,))
    assert one >= 4 * 2 * 2 * 2048 * 2048  # X twice, A and B
    # several steps on one A keep three more m x m matrices
    assert need(((150, 8192),), (1,)) - need(((150, 8192),), (0,)) == 3 * 2 * 2 * 256 * 256
    assert need(((2048, 8192),), (0,), weights=1) == need(((2048, 8192),), (1,))
    assert need(((2048, 2048),), (1,), n=ns(steps=0)) < one / 3
    # the workspace does not grow with the list beyond a group's
    many = [need(((4096, 4096),) * k, (1,) * k) for k in (1, 10, 24, 25, 200)]
    assert many == sorted(many) and many[3] == many[4] and many[4] <= 5 << 30
    assert need(((40000, 40000),), (1,)) > 5 << 30  # one matrix that needs more has it
    assert lib.rr_muon_workspace(None, 0, ctypes.byref(ns()), ctypes.byref(b)) == INVALID
    assert lib.rr_muon_workspace(ctypes.byref(mlist(PARAMS)), 0, ctypes.byref(ns()), None) == INVALID
    assert lib.rr_muon_workspace(ctypes.byref(mlist(PARAMS)), 0, ctypes.byref(ns(steps=99)), ctypes.byref(b)) == INVALID


def test_python_calls_check_their_tensors():
    x = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="CUDA tensors"):
        rrv.orthogonalize([x])
    with pytest.raises(ValueError, match="1..64 ranks"):
        rrv.MatrixList([[]] * 65)
    with pytest.raises(ValueError, match="same number"):
        rrv.MatrixList([[], [x]])
    assert rrv.orthogonalize([]) == []
    rrv.muon_step([], [], [], lr=0.1)  # nothing to do
