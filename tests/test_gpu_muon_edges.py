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
