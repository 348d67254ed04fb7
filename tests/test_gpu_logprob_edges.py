"""Token log probabilities and their gradient at the ends of their range
(tolerances: test_gpu_logprob.py)."""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from test_gpu_logprob import E24, TYPES, check_backward, check_forward, formulas, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-64, -40, 40, 64])
def test_scales_at_the_ends(power):
    """Logits that a scale of 2^power takes to ordinary z, the same as those z give with a scale of 1."""
    xs, ids = make(1, 6, 3001, torch.float32, seed=2)
    plain = rrv.token_logprobs(xs, ids, entropy=True, top_k=5)
    x = xs[0] * 2.0 ** -power
    got = check_forward([x], ids, 2.0 ** power, 5)
    check_backward([x], ids, 2.0 ** power, got, True)
    assert torch.equal(got.top_id, plain.top_id)
    equal = torch.full((3, 3001), 7.0 * 2.0 ** -power, device="cuda")
    got = rrv.token_logprobs([equal], [torch.zeros(3, dtype=torch.int64, device="cuda")], scale=2.0 ** power, entropy=True)
    assert ((got.logprob + math.log(3001)).abs() <= E24 * (3001 / 512 + 128 + 16)).all()


def test_scales_beyond_are_refused():
    xs, ids = make(1, 2, 10, torch.float32)
    for scale in (2.0 ** 65, 3e38, 2.0 ** -65, 1e-40):
        with pytest.raises(rrv.RRError):
            rrv.token_logprobs(xs, ids, scale=scale)
        with pytest.raises(rrv.RRError):
            rrv.token_logprobs_grad(xs, ids, torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda"), scale=scale)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 1.0])
def test_logits_further_apart_than_fp32_reaches(scale):
    """3e38 and -3e38 in one row: their difference leaves fp32, the log probability of a small scale does not."""
    V = 1500
    x = torch.randn(4, V, device="cuda")
    x[0, 3], x[0, 9] = 3e38, -3e38
    x[1, 3], x[1, 9], x[1, 10] = 3e38, 2.9e38, -3.4e38
    x[2, :] = -3e38
    x[2, 700] = 3.3e38
    t = torch.tensor([9, 10, 8, 1], device="cuda")
    got = rrv.token_logprobs([x], [t], scale=scale, entropy=True, top_k=3)
    z = x.double() * scale
    logp = torch.log_softmax(z, -1)
    want = logp[torch.arange(4, device="cuda"), t]
    reach = torch.where(want < -3.4e38, -math.inf, want)  # below fp32's range
    fine = reach.isinf() == got.logprob[0].isinf()
    near = (got.logprob[0].double() - want).abs() <= 1e-4 + 2.0 ** -21 * want.abs()
    assert (fine & (near | reach.isinf())).all(), (got.logprob, want)
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :3]
    assert torch.equal(got.top_id[0].long(), best)
    w = logp.gather(1, best)
    assert (((got.top_logprob[0].double() - w).abs() <= 1e-4 + 2.0 ** -21 * w.abs()) | (w < -3.4e38)).all()
    assert not got.entropy.isnan().any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("offset", [0.0, 40.0, -1000.0, 6e4])
def test_gradients_of_rows_with_a_common_offset(dtype, offset):
    """Against the 64-bit formula of the logits alone, lse included: half a step of the lse that the gradient is given
    (|lse| 2^-24), what the forward pass errs by (its ln s: 2^-24 (V / 512 + 128)) and the difference's own rounding
    are p's relative error."""
    if dtype == "bf16" and abs(offset) > 1000:
        offset = 8192.0
    T, V, dt = 5, 2000, TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(T, V, generator=gen, device="cuda") * 2 + offset).to(dt)
    x[2] = torch.finfo(torch.float16).min if dtype == "f16" else offset  # a uniform row
    t = torch.tensor([5, -1, 7, 8, 1999], device="cuda")
    g, h = torch.randn(2, T, generator=gen, device="cuda")
    fwd = rrv.token_logprobs([x], [t], entropy=True)
    _, lse, H, logp, p, known = formulas(x, t, 1.0)
    base = E24 * (V / 512 + 128)
    off = base + E24 * (lse.abs()[:, None] + logp.abs() + 16)
    for ent in (False, True):
        got = rrv.token_logprobs_grad([x], [t], fwd.lse, g[None], entropy=fwd.entropy if ent else None,
                                      dentropy=h[None] if ent else None)[0].double()
        gk = torch.where(known, g.double(), 0.0)[:, None]
        want = -gk * p
        want[known, t[known]] += gk[known, 0]
        tol = gk.abs() * p * off
        if ent:
            want -= h.double()[:, None] * p * (logp + H[:, None])
            # ln p and the entropy are off, too, the latter by up to ln V times ln s's error
            tol = tol + h.abs()[:, None] * p * (off * ((logp + H[:, None]).abs() + 1) + base * (2 + math.log(V)))
        step = torch.finfo(dt).eps / 2
        tiny = torch.finfo(dt).tiny * (torch.finfo(dt).eps if dt == torch.float16 else 1.0)
        # the target's element is the sum of two terms, of at most g each before its rounding
        tol = tol * (1 + 2 * off) + want.abs() * step * (1 + 1e-3) + gk.abs() * 2 * E24 + tiny
        bad = (got - want).abs() > tol
        assert not bad.any(), (ent, bad.nonzero()[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,V", [(3, 50003), (64, 20000), (1, 128000), (900, 4001), (1300, 1024)])
@pytest.mark.parametrize("left", [0, 1, 5, 19])
def test_masks_that_leave_fewer_tokens_than_alternatives(dtype, T, V, left):
    """-inf, or the type's lowest value, everywhere but at a few tokens, some of them alike: these first, then the lowest
    of the masked ids."""
    dt, k = TYPES[dtype], 20
    gen = torch.Generator(device="cuda").manual_seed(left)
    for low in (-math.inf, torch.finfo(dt).min, 1.5):  # 1.5: a constant row with a few larger values
        x = torch.full((T, V), low, dtype=dt, device="cuda")
        if left:
            at = torch.stack([torch.randperm(V, generator=gen, device="cuda")[:left] for _ in range(min(T, 8))]).repeat(-(-T // 8), 1)[:T]
            x.scatter_(1, at, (torch.randint(4, (T, left), generator=gen, device="cuda") + 2.0).to(dt))
        t = torch.randint(V, (T,), generator=gen, device="cuda")
        got = rrv.token_logprobs([x], [t], entropy=True, top_k=k)
        want = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(got.top_id[0].long(), want), low
        if left or low > -math.inf:
            w = torch.log_softmax(x.double(), -1).gather(1, want)
            tol = E24 * (V / 512 + 128) + E24 * 8 * w.abs()
            assert ((got.top_logprob[0] == w) | ((got.top_logprob[0] - w).abs() <= tol)).all(), low
        else:
            assert (got.top_logprob == -math.inf).all()
