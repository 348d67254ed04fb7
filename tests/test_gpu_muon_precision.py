"""How near the orthogonalisation and the Muon step come to the exact polynomial,
on matrices whose singular values are far apart.

Tolerances, relative to ||O||, from each matrix's singular values s_k(i) before
step k.  An error of step k reaches the result through the later steps' slopes:
relative to the direction's size, by the product g of |1 + 2 l d'(l) / d(l)|, d =
a + b l + c l^2, l = s^2, of which at least 1 is counted.
(1) A value has 22 bits, so that a matrix of them is off by a matrix of 2^-23 of its
norm, without a direction of its own: each of the m directions gets 1 / sqrt(m) of it.
    2^-23 sum_k ||s_k|| rms_i(g_k s_n / s_k) / ||s_n||
This counts where directions differ in size: one of 99 % and noise of 1 % make it 100
x 2^-23 for k = 0.
(2) In a step X' = a X + (b A + c A^2) X a direction is off by the error of A, times
|b| / a, and by the sums' roundings: 3 x 2^-22 together, as for one step.
(3) Where L steps share one A, its error of 2^-22 has grown by a^2 in each of the
later ones: (a^2 + ... + a^(2 (L - 1))) |b| / a x 2^-22 in L steps; L is 2 for fp32 and
3 for bf16 and fp16, where steps are shared.
    ||O - exact|| <= (1) + sum_k ((2) + (3) / L) ||g_(k+1) s_n||, relative to ||s_n||
(Plain fp32 steps err by 0.2e-5 to 4e-5 here.)

The rounding to the type is
independent of it: its own sum of squares R^2, of N elements each within half a
step, differs from that of the exact values' rounding by 4 / sqrt(N) of itself at
most (four standard deviations), so
    ||O - exact||^2 <= ((1 + 4 / sqrt(N)) R)^2 + (the bound above)^2
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


def exact(x, steps=5, eps=1e-7, coef=COEF):
    a, b, c = coef
    x = x.double() / (x.double().norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.T if tall else x


def bound(x, L, steps=5, coef=COEF):
    a, b, c = coef
    s, slope = [torch.linalg.svdvals(x.double() / x.double().norm())], []
    for _ in range(steps):
        l = s[-1] ** 2
        d = a + b * l + c * l * l
        slope.append((1 + 2 * l * (b + 2 * c * l) / d).abs())
        s.append(s[-1] * d)
    g = [torch.ones_like(s[0])] * (steps + 1)
    for k in reversed(range(steps)):
        g[k] = g[k + 1] * slope[k]
    g = [v.clamp(min=1) for v in g]
    one = sum(float(s[k].norm() * (g[k] * s[-1] / s[k]).square().mean().sqrt() / s[-1].norm()) for k in range(steps))
    reach = sum(float((g[k + 1] * s[-1]).norm() / s[-1].norm()) for k in range(steps))
    shared = sum(a ** (2 * j) for j in range(1, L)) * abs(b) / a / L
    return 2.0 ** -23 * one + 2.0 ** -22 * (3 + shared) * reach


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
    assert err <= bound(x, 2) + 2.0 ** -22, err


@pytest.mark.parametrize("r,c", [(192, 768), (512, 2048), (2048, 512), (700, 2800), (1024, 8192), (600, 600), (96, 1000)])
@pytest.mark.parametrize("kind", KINDS)
def test_fp32_results(r, c, kind):
    x = matrix(r, c, kind, seed=1)
    o = exact(x)
    err = float((rrv.orthogonalize([x])[0].double() - o).norm() / o.norm())
    assert err <= bound(x, 2) + 2.0 ** -23, err


def check_rounded(got, o, off):
    R, n = float((o.to(got.dtype).double() - o).norm()), o.numel()
    err = float((got.double() - o).norm())
    assert err <= math.hypot((1 + 4 / math.sqrt(n)) * R, off * float(o.norm())), (err, R, float(o.norm()))


@pytest.mark.parametrize("r,c", [(192, 768), (512, 2048), (2048, 512), (700, 2800), (1024, 8192), (600, 600), (96, 1000)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounded_results_and_weights(r, c, kind, dtype):
    x = matrix(r, c, kind, seed=2)
    out = torch.empty(r, c, dtype=dtype, device="cuda")
    rrv.orthogonalize([x], [out])
    o = exact(x)
    off = bound(x, 3)
    check_rounded(out, o, off)
    w, m = torch.zeros_like(out), torch.zeros_like(x)
    rrv.muon_step([w], [x], [m], lr=1.0, momentum=0.0, nesterov=False)
    check_rounded(w, o * -math.sqrt(max(1.0, r / c)), off)


@pytest.mark.parametrize("r,c", [(100, 900), (300, 1500), (600, 2400), (2400, 600)])
@pytest.mark.parametrize("kind", ["noise", "rank+.05", "rank1+.01"])
@pytest.mark.parametrize("steps,coef", [(12, (1.5, -0.5, 0.0)), (6, (2.0, -1.5, 0.5)), (8, (1.875, -1.25, 0.375)), (20, (1.0, -0.3, 0.1)),
                                        (50, (1.0, -0.3, 0.1)), (40, (1.0, 0.6, -0.55))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_other_polynomials(r, c, kind, steps, coef, dtype):
    x = matrix(r, c, kind, seed=3)
    o = exact(x, steps=steps, coef=coef)
    out = torch.empty(r, c, dtype=dtype, device="cuda")
    rrv.orthogonalize([x], [out], steps=steps, coefficients=coef)
    if dtype == torch.float32:
        err = float((out.double() - o).norm() / o.norm())
        assert err <= bound(x, 2 if coef[0] ** 2 >= 2 else 1, steps, coef), err
    else:
        check_rounded(out, o, bound(x, 3, steps, coef))
