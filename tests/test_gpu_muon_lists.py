"""The Muon step and the orthogonalisation over lists that mix shapes with types,
against the iteration in 64 bits (tolerances: test_gpu_muon.py)."""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from test_gpu_muon import TYPES, gradient, iterate, rounding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shapes", [[(512, 576 + 8 * i) for i in range(15)], [(300, 140), (140, 300), (256, 256), (64, 40)]])
def test_weights_of_every_type_in_one_list(shapes):
    """Every shape as fp32, bf16 and fp16 weights, gradients of the other types beside them."""
    names = list(TYPES)
    gen = torch.Generator(device="cuda").manual_seed(len(shapes))
    ws, gs, ms = [[], []], [], []
    for i, s in enumerate(shapes):
        for k, name in enumerate(names):
            w = (torch.randn(s, generator=gen, device="cuda") * 0.02).to(TYPES[name])
            ws[0].append(w)
            ws[1].append(torch.full_like(w, 9.0))
            gs.append(gradient(*s, TYPES[names[(k + i) % 3]], seed=3 * i + k))
            ms.append(torch.randn(s, generator=gen, device="cuda") * 3e-2)
    w0, m0 = [w.double() for w in ws[0]], [m.double() for m in ms]
    lr, mu, decay = 0.03, 0.9, 0.1
    rrv.muon_step(ws, gs, ms, lr=lr, momentum=mu, weight_decay=decay)
    for t, w in enumerate(ws[0]):
        r, c = w.shape
        m = mu * m0[t] + gs[t].double()
        o, bound = iterate(gs[t].double() + mu * m)
        f = lr * math.sqrt(max(1.0, r / c))
        want = (1 - lr * decay) * w0[t] - f * o
        err = float((w.double() - want).norm())
        assert err <= f * 2 * bound + rounding(want, w.dtype) * 1.01 + 2.0 ** -22 * float(want.norm()), (t, r, c, err)
        assert torch.equal(ws[1][t], w)
    again = [[w.clone() for w in ws[0]] for _ in range(2)]
    more = [m.clone() for m in ms]
    rrv.muon_step(ws, gs, ms, lr=lr, momentum=mu, weight_decay=decay)
    rrv.muon_step(again, gs, more, lr=lr, momentum=mu, weight_decay=decay)
    assert all(torch.equal(a, b) for a, b in zip(ws[0], again[0]))  # the same call, the same bits
