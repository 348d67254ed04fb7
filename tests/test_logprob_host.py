"""Host-side checks of the token log probability calls: every call here fails
its argument checks before anything is enqueued."""
import ctypes

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from ring_all_reduce_virtual_b200 import _lib
from ring_all_reduce_virtual_b200.build import build

INVALID, UNSUPPORTED = _lib.RR_ERR_INVALID_ARG, _lib.RR_ERR_UNSUPPORTED
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def ptrs(n, base, gap=1 << 30):
    return (ctypes.c_void_p * n)(*[base + i * gap for i in range(n)])


IDS, LOGITS, GRADS = 1 << 40, 1 << 42, 1 << 44
A, B, C, D, E = (1 << 46, 1 << 47, 3 << 46, 1 << 48, 5 << 46)


def forward(x=ptrs(2, LOGITS), stride=100, ids=ptrs(2, IDS), id_type=0, n=2, T=16, V=100, dtype=0, scale=1.0, logprob=A, lse=B,
            entropy=C, k=4, top=D, top_id=E):
    return _lib.lib().rr_token_logprobs(x, stride, ids, id_type, n, T, V, dtype, scale, logprob, lse, entropy, k, top, top_id, None)


def backward(x=ptrs(2, LOGITS), stride=100, ids=ptrs(2, IDS), id_type=0, n=2, T=16, V=100, dtype=0, scale=1.0, lse=A, entropy=B,
             dlogprob=C, dentropy=D, dx=ptrs(2, GRADS), gstride=100):
    return _lib.lib().rr_token_logprobs_grad(x, stride, ids, id_type, n, T, V, dtype, scale, lse, entropy, dlogprob, dentropy, dx,
                                             gstride, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_shapes_types_and_pointers_are_checked(call):
    for bad in (dict(n=0), dict(n=65), dict(dtype=9), dict(id_type=2), dict(V=0), dict(V=(1 << 31) - 1), dict(stride=99),
                dict(stride=1 << 31), dict(T=1 << 31), dict(T=1 << 30), dict(T=1 << 63), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=INF), dict(scale=float("nan")), dict(x=None), dict(ids=None), dict(x=ptrs(2, LOGITS + 2)),
                dict(ids=ptrs(2, IDS + 2)), dict(ids=ptrs(2, IDS + 4), id_type=1), dict(x=(ctypes.c_void_p * 2)(LOGITS, None)),
                dict(ids=(ctypes.c_void_p * 2)(None, IDS)), dict(lse=None), dict(lse=A + 2)):
        assert call(**bad) == INVALID, bad
    assert call(dtype=2) == UNSUPPORTED
    assert b"bf16, fp16 or fp32" in _lib.lib().rr_last_error()
    assert call(T=0) == 0  # no row: nothing is enqueued


def test_forward_refuses_bad_outputs():
    for bad in (dict(logprob=None), dict(logprob=A + 1), dict(k=-1), dict(k=33), dict(k=5, V=4, stride=4), dict(top=None),
                dict(top_id=None), dict(top=D + 2), dict(entropy=C + 2), dict(logprob=B), dict(lse=B, entropy=B + 4),
                dict(top=LOGITS), dict(top_id=IDS)):
        assert forward(**bad) == INVALID, bad


def test_backward_refuses_bad_buffers():
    for bad in (dict(dx=None), dict(dx=ptrs(2, GRADS + 2)), dict(gstride=99), dict(gstride=1 << 31), dict(entropy=None),
                dict(dlogprob=None), dict(dlogprob=C + 2), dict(dentropy=D + 1), dict(dx=ptrs(2, GRADS, gap=64)),
                dict(dx=ptrs(2, LOGITS + 4)),                # over the logits, an element on
                dict(dx=ptrs(2, LOGITS), gstride=101),       # in the logits' place with another stride
                dict(dx=ptrs(2, IDS)), dict(dx=ptrs(2, A))):
        assert backward(**bad) == INVALID, bad


def test_python_calls_check_their_tensors():
    ids, x = torch.zeros(2, dtype=torch.int64), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="alike"):
        rrv.token_logprobs([x], [ids])  # not on a GPU
    with pytest.raises(ValueError, match="need 1..64"):
        rrv.token_logprobs([], [])
    with pytest.raises(TypeError, match="int32 or int64"):
        rrv.token_logprobs([x], [x])


@pytest.mark.parametrize("call", [forward, backward])
def test_scales_outside_their_range_are_refused(call):
    for scale in (2.0 ** 65, 3e38, 2.0 ** -65, 1e-40):
        assert call(scale=scale) == INVALID, scale
    assert call(scale=2.0 ** 64, T=0) == 0 and call(scale=2.0 ** -64, T=0) == 0
