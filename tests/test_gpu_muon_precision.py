"""How near the orthogonalisation and the Muon step come to the exact polynomial,
on matrices whose singular values are far apart.

Tolerance for fp32.  A value has 22 bits, so that a product's operands are off by
matrices of norm 2^-23 to 2^-22 of theirs.  In a step X' = a X + (b A + c A^2) X
a direction of a small singular value is off by the error of A, times |b| / a =
1.4, and of X: by about 3 x 2^-22 of itself, in five steps by 15 x 2^-22.  Where
two steps share one A, the error of A has grown by a^2 = 11.9 in the second: twice
in five steps, 2 x 11.9 x 1.4 x 2^-22 more.  That is 1.2e-5, and
    ||O - exact|| <= 2e-5 ||O||
leaves 1.7 for what the sums round.  (Plain fp32 steps err by 2e-6 to 4e-5 here.)
Tolerance for bf16 and fp16.  Three steps may share one A, whose error of 2^-22 has
grown by a^4 = 141 in the third: 141 x 1.4 x 2^-22 = 4.7e-5, 6e-5 with what the
fp32 results' bound has for two steps on one A.  The rounding to the type is
independent of it: its own sum of squares R^2, of N elements each within half a
step, differs from that of the exact values' rounding by 4 / sqrt(N) of itself at
most (four standard deviations), so
    ||O - exact||^2 <= ((1 + 4 / sqrt(N)) R)^2 + (6e-5 ||O||)^2
A weight's momentum and update round in fp32: 2^-23 of each.
"""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from test_gpu_muon import COEF

pytestmark = pytest.mark.gpu
KINDS = ["noise", "rank+1", "rank+.05", "rank+.001", "rank1+.01"]


def matrix(r, c, kind, seed=0):
    """A few strong directions (rank 1/16 of the side, or 1) and noise of the given size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = 1 if kind.startswith("rank1") else max(1, min(r, c) // 16)
    strong = torch.randn(r, k, generator=g, device="cuda") @ torch.randn(k, c, generator=g, device="cuda") / math.sqrt(k)
    noise = torch.randn(r, c, generator=g, device="cuda")
    return (noise if kind == "noise" else strong + noise * float(kind.split("+")[1])) * 1e-3


def exact(x, steps=5, eps=1e-7):
    a, b, c = COEF
    x = x.double() / (x.double().norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.T if tall else x


@pytest.mark.parametrize("r,c", [(192, 768), (512, 2048), (2048, 512), (700, 2800), (1024, 8192), (600, 600), (96, 1000)])
@pytest.mark.parametrize("kind", KINDS)
def test_fp32_weights_that_begin_at_zero(r, c, kind):
    """The update is all of the weight, so its error is O's."""
    x = matrix(r, c, kind)
    w, m = torch.zeros_like(x), torch.zeros_like(x)
    rrv.muon_step([w], [x], [m], lr=1.0, momentum=0.0, nesterov=False)
    o = exact(x)
    got = w.double() / -math.sqrt(max(1.0, r / c))
    err = float((got - o).norm() / o.norm())
    assert err <= 2e-5 + 2.0 ** -22, err


@pytest.mark.parametrize("r,c", [(192, 768), (512, 2048), (2048, 512), (700, 2800), (1024, 8192), (600, 600), (96, 1000)])
@pytest.mark.parametrize("kind", KINDS)
def test_fp32_results(r, c, kind):
    x = matrix(r, c, kind, seed=1)
    o = exact(x)
    err = float((rrv.orthogonalize([x])[0].double() - o).norm() / o.norm())
    assert err <= 2e-5 + 2.0 ** -23, err


def check_rounded(got, o):
    R, n = float((o.to(got.dtype).double() - o).norm()), o.numel()
    err = float((got.double() - o).norm())
    assert err <= math.hypot((1 + 4 / math.sqrt(n)) * R, 6e-5 * float(o.norm())), (err, R, float(o.norm()))


@pytest.mark.parametrize("r,c", [(192, 768), (512, 2048), (2048, 512), (700, 2800), (1024, 8192), (600, 600), (96, 1000)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounded_results_and_weights(r, c, kind, dtype):
    x = matrix(r, c, kind, seed=2)
    out = torch.empty(r, c, dtype=dtype, device="cuda")
    rrv.orthogonalize([x], [out])
    o = exact(x)
    check_rounded(out, o)
    w, m = torch.zeros_like(out), torch.zeros_like(x)
    rrv.muon_step([w], [x], [m], lr=1.0, momentum=0.0, nesterov=False)
    check_rounded(w, o * -math.sqrt(max(1.0, r / c)))
