"""The orthogonalisation and the Muon step at the ends of their range, as tiles and
in a cluster's shared memory (tolerances: test_gpu_muon.py)."""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from test_gpu_muon import COEF, TYPES, check, gradient, iterate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(50, 70), (200, 300), (300, 140)])
@pytest.mark.parametrize("steps", [0, 1, 5])
def test_an_infinity_or_nan_makes_every_element_nan(shape, steps):
    for bad in (math.inf, -math.inf, math.nan):
        for dt in TYPES.values():
            x = gradient(*shape, dt)
            x[shape[0] // 2, 3] = bad
            good = gradient(*shape, dt, seed=1)
            o = rrv.orthogonalize([x, good], steps=steps)
            assert o[0].isnan().all(), (bad, dt)
            check(o[1], good, steps=steps)


@pytest.mark.parametrize("steps,coef", [(0, COEF), (1, COEF), (2, COEF), (3, COEF), (4, COEF), (6, COEF), (7, COEF), (8, COEF), (11, COEF),
                                        (5, (2.0, -1.5, 0.5)), (4, (1.5, -0.5, 0.0)), (3, (1.0, 0.0, 0.0)), (50, (1.0, 0.0, 0.0)),
                                        (6, (-1.5, 0.5, 0.0))])
def test_other_iterations_as_tiles(steps, coef):
    """Segments of one, two and three steps, with and without a shorter last one, and no product at all."""
    for r, c in ((200, 520), (520, 200), (513, 1600), (300, 300)):
        for dt in TYPES.values():
            x = gradient(r, c, dt, seed=steps)
            check(rrv.orthogonalize([x], steps=steps, coefficients=coef)[0], x, steps=steps, coef=coef)


@pytest.mark.parametrize("shape", [(100, 300), (600, 200), (512, 2048)])
@pytest.mark.parametrize("norm", [1e-8, 1e-10, 1e-12, 1e-14])
def test_matrices_whose_norm_is_below_eps(shape, norm):
    """X begins small against its bound of 1, for which its halves are scaled by 2^15: they end at 2^-24 / 2^15, so
    every element is off by 2^-40 at most, and by as much again in every step, which multiplies it by a = 3.4445."""
    x = gradient(*shape, torch.float32)
    x = x / x.norm() * norm
    for dt in TYPES.values():
        out = torch.empty(shape, dtype=dt, device="cuda")
        rrv.orthogonalize([x], [out], eps=1e-7)
        want, _ = iterate(x, eps=1e-7)
        N = math.sqrt(shape[0] * shape[1])
        lost = 2.0 ** -40 * N * sum(COEF[0] ** k for k in range(6))
        near = 2e-5 if dt == torch.float32 else 6e-5  # test_gpu_muon_precision.py
        step = float(((want.to(dt).double() - want).abs() * (1 + 4 / N)).norm())
        err = float((out.double() - want).norm())
        assert err <= lost + near * float(want.norm()) + step, (dt, err, lost, float(want.norm()))


@pytest.mark.parametrize("shape", [(1, 1 << 20), (1 << 20, 3), (5, 200003), (131, 70001)])
def test_the_longest_matrices(shape):
    """Up to 2^20 rows or columns, where X X^T goes through 16384 blocks of K."""
    for dt in (torch.float32, torch.bfloat16):
        x = gradient(*shape, dt, seed=4)
        check(rrv.orthogonalize([x])[0], x)
        rrv.check_timeouts()
    torch.cuda.empty_cache()
