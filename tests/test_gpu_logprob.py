"""Token log probabilities and their gradient on the GPU, against the formulas
in 64 bits.

Tolerances, with e = 2^-24: z_t - m takes two roundings and the final
difference one (4 e |logprob|, with what lse itself rounds); ln s errs by s's
relative error: 2^-22 of a power of two, two roundings of its exponent (24 e at
the ln V of a term that counts), a thread's run of at most 64 or V / 512 terms
and the joins -- e (V / 512 + 128).  The entropy has that error times its
terms, which reach ln V.  A gradient has p's relative error, e (|ln p| + 16),
in each of its terms, and the rounding to its type.
"""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = math.inf


def make(n, T, V, dtype, seed=0, pitch=0, offset=0, std=2.0):
    """Rank logits as views [T, V] whose rows are V + pitch apart, `offset` elements past a boundary; ids with some outside."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    xs, ids = [], []
    for _ in range(n):
        big = torch.full((offset + T * (V + pitch) + 8,), 7.0, dtype=dtype, device="cuda")
        x = big[offset:offset + T * (V + pitch)].view(T, V + pitch)[:, :V]
        x.copy_(torch.randn(T, V, generator=g, device="cuda") * std)
        t = torch.randint(V, (T,), generator=g, device="cuda")
        if T > 2:
            t[1], t[T - 1] = -1, V + 3
        xs.append(x)
        ids.append(t)
    return xs, ids


def formulas(x, ids, scale):
    z = x.double() * scale
    lse = torch.logsumexp(z, -1)
    logp = z - lse[:, None]
    p = logp.exp()
    h = -torch.special.xlogy(p, p).sum(-1)
    V = x.shape[1]
    known = (ids >= 0) & (ids < V)
    lp = torch.where(known, logp.gather(1, ids.clamp(0, V - 1)[:, None])[:, 0], 0.0)
    return lp, lse, h, logp, p, known


def check_forward(xs, ids, scale, k, entropy=True):
    got = rrv.token_logprobs(xs, ids, scale=scale, entropy=entropy, top_k=k)
    V = xs[0].shape[1]
    base = E24 * (V / 512 + 128)
    for r, (x, t) in enumerate(zip(xs, ids)):
        lp, lse, h, logp, _, _ = formulas(x, t, scale)
        assert ((got.logprob[r] - lp).abs() <= base + E24 * (4 * lp.abs() + lse.abs())).all()
        assert ((got.lse[r] - lse).abs() <= base + E24 * 4 * lse.abs()).all()
        if entropy:
            assert ((got.entropy[r] - h).abs() <= base * (2 + math.log(V))).all()
        if k:
            want = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :k]
            assert torch.equal(got.top_id[r].long(), want)
            w = logp.gather(1, want)
            assert ((got.top_logprob[r] - w).abs() <= base + E24 * (4 * w.abs() + lse.abs()[:, None])).all()
    if not entropy:
        assert got.entropy is None
    if not k:
        assert got.top_id is None and got.top_logprob is None
    return got


def check_backward(xs, ids, scale, got, entropy, outs=None, g=None, h=None):
    n, T, V = len(xs), *xs[0].shape
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = torch.randn(n, T, generator=gen, device="cuda") if g is None else g
    h = (torch.randn(n, T, generator=gen, device="cuda") if entropy else None) if h is None else h
    want, tol = [], []
    for r, (x, t) in enumerate(zip(xs, ids)):
        known = (t >= 0) & (t < V)
        gr = torch.where(known, g[r].double(), 0.0)[:, None]
        logp = x.double() * scale - got.lse[r].double()[:, None]
        p = logp.exp()
        d = -gr * p
        d[known, t[known]] += gr[known, 0]
        slack = gr.abs() * (p + (d.abs() > 0))
        if entropy:
            hr, H = h[r].double()[:, None], got.entropy[r].double()[:, None]
            d -= hr * torch.where(p > 0, p * (logp + H), 0.0)
            slack = slack + hr.abs() * p * (torch.where(p > 0, logp, 0.0).abs() + H.abs() + 1)
        d, slack = d * scale, slack * scale
        reach = torch.where(p > 0, logp, 0.0).abs() + 16
        dt = x.dtype
        step = 0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2
        tiny = torch.finfo(dt).tiny * (torch.finfo(dt).eps if dt == torch.float16 else 1.0)
        want.append(d)
        tol.append(E24 * reach * slack * 2 + d.abs() * step * (1 + 1e-3) + tiny)
    out = rrv.token_logprobs_grad(xs, ids, got.lse, g, entropy=got.entropy if entropy else None, dentropy=h, scale=scale, outs=outs)
    for r in range(n):
        assert out[r].dtype == xs[r].dtype
        bad = (out[r].double() - want[r]).abs() > tol[r]
        assert not bad.any(), (r, bad.nonzero()[:4], out[r][bad][:4], want[r][bad][:4])
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,T,V,pitch,offset,scale,k", [
    (1, 1, 1, 0, 0, 1.0, 1), (1, 3, 2, 1, 1, 1.0, 2), (2, 5, 7, 0, 3, 0.7, 7), (1, 4, 31, 2, 0, 1.0, 31),
    (1, 2, 33, 0, 1, 1.0, 32), (3, 4, 255, 0, 0, 1.0, 5), (1, 3, 1000, 24, 0, 2.0, 20), (2, 7, 4099, 0, 5, 1.0, 8),
    (1, 1, 32000, 0, 0, 1.0, 5), (1, 5, 50003, 0, 1, 1.25, 32), (4, 50, 8192, 64, 0, 1.0, 3), (1, 1, 150001, 7, 2, 1.0, 32),
    (2, 1500, 1001, 0, 0, 1.0, 4), (1, 1400, 2048, 0, 0, 0.5, 32), (1, 1300, 7, 0, 0, 1.0, 3), (64, 2, 300, 0, 0, 1.0, 2),
    (1, 700, 20000, 0, 0, 1.0, 16)])
def test_forward_and_backward(dtype, n, T, V, pitch, offset, scale, k):
    xs, ids = make(n, T, V, TYPES[dtype], seed=V + T, pitch=pitch, offset=offset)
    got = check_forward(xs, ids, scale, k)
    plain = check_forward(xs, ids, scale, 0, entropy=False)
    assert torch.equal(plain.lse, got.lse) and torch.equal(plain.logprob, got.logprob)
    check_backward(xs, ids, scale, got, True)
    check_backward(xs, ids, scale, got, False)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_with_masks(dtype):
    """-inf entries, whole rows of -inf, rows of the type's lowest value, one entry left."""
    V, dt = 1237, TYPES[dtype]
    xs, ids = make(1, 8, V, dt, seed=1)
    x, t = xs[0], torch.tensor([5, 6, 7, 8, 9, 10, 11, 12], device="cuda")
    low = torch.finfo(dt).min
    x[0, ::2] = -INF                    # the target is left
    x[1, ::2] = -INF                    # the target is masked
    x[2] = -INF                         # nothing is left
    x[3] = low                          # nothing but the lowest value
    x[4] = -INF
    x[4, 9] = 3.0                       # one entry, the target
    x[5] = low
    x[5, 700] = -2.0                    # the lowest value as a mask
    x[6] = -INF
    x[6, 1236] = -1.0                   # one entry, not the target
    got = rrv.token_logprobs([x], [t], entropy=True, top_k=4)
    lp, lse, h, logp, p, _ = formulas(x, t, 1.0)
    keep = [0, 4, 5, 6, 7]
    base = E24 * (V / 512 + 128)
    assert ((got.lse[0] - lse)[keep].abs() <= base + E24 * 4 * lse[keep].abs()).all()
    assert torch.equal(got.logprob[0, 1].isinf(), torch.tensor(True, device="cuda")) and float(got.logprob[0, 1]) < 0
    assert float(got.lse[0, 2]) == -INF and float(got.logprob[0, 2]) == -INF and float(got.entropy[0, 2]) == 0.0
    assert got.top_id[0, 2].tolist() == [0, 1, 2, 3] and (got.top_logprob[0, 2] == -INF).all()
    assert abs(float(got.logprob[0, 3]) + math.log(V)) <= base + 4 * E24 * 8  # uniform
    assert abs(float(got.entropy[0, 3]) - math.log(V)) <= base * 12
    assert got.top_id[0, 3].tolist() == [0, 1, 2, 3]
    assert float(got.logprob[0, 4]) == 0.0 and float(got.entropy[0, 4]) == 0.0
    assert got.top_id[0, 4].tolist() == [9, 0, 1, 2] and got.top_logprob[0, 4].tolist() == [0.0, -INF, -INF, -INF]
    assert float(got.logprob[0, 5]) <= -6e4 and abs(float(got.entropy[0, 5])) <= base * 12 and int(got.top_id[0, 5, 0]) == 700
    assert float(got.logprob[0, 6]) == -INF and int(got.top_id[0, 6, 0]) == 1236
    out = rrv.token_logprobs_grad([x], [t], got.lse, torch.ones(1, 8, device="cuda"), entropy=got.entropy,
                                  dentropy=torch.ones(1, 8, device="cuda"))[0]
    assert not out.isnan().any() and (out[2] == 0).all()  # nothing is left: no gradient
    assert (out[0, ::2] == 0).all() and (out[4].abs() <= 0).all()
    step = torch.finfo(dt).eps
    for r in (0, 1, 5, 6, 7):
        d = -p[r].clone()
        d[t[r]] += 1
        d -= torch.where(p[r] > 0, p[r] * (logp[r] + h[r]), 0.0)
        assert ((out[r].double() - d).abs() <= step * d.abs() + 2e-5).all(), r


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_with_nan_and_infinity(dtype):
    x = torch.randn(4, 5000, device="cuda").to(TYPES[dtype])
    x[0, 4321], x[1, 17], x[1, 4000] = math.nan, INF, INF
    t = torch.tensor([3, 17, 3, -1], device="cuda")
    got = rrv.token_logprobs([x], [t], entropy=True, top_k=3)
    assert got.lse[0, :2].isnan().all() and got.logprob[0, :2].isnan().all() and got.entropy[0, :2].isnan().all()
    assert not got.lse[0, 2:].isnan().any() and float(got.logprob[0, 3]) == 0.0
    assert int(got.top_id[0, 0, 0]) == 4321 and got.top_id[0, 1, :2].tolist() == [17, 4000]
    out = rrv.token_logprobs_grad([x], [t], got.lse, torch.ones(1, 4, device="cuda"))[0]
    assert out[:2].isnan().all() and not out[2:].isnan().any()
    assert (out[3] == 0).all()


@pytest.mark.parametrize("V,T", [(5000, 3), (1024, 1300), (64000, 2)])
@pytest.mark.parametrize("kind", ["constant", "rising", "falling", "two values", "zeros of both signs"])
def test_ties_and_orders_that_suit_the_search_least(V, T, kind):
    at = torch.arange(V, device="cuda")
    x = {"constant": torch.full((V,), 1.5, device="cuda"), "rising": at / 64.0, "falling": -at / 64.0,
         "two values": (at % 7 == 3).float(), "zeros of both signs": torch.where(at % 2 == 0, -0.0, 0.0)}[kind]
    for dt in (torch.float32, torch.bfloat16):
        xs = [x.to(dt).repeat(T, 1)]
        check_forward(xs, [torch.zeros(T, dtype=torch.int32, device="cuda")], 1.0, 32)


def test_in_place_strided_and_other_columns_left():
    xs, ids = make(2, 9, 1003, torch.bfloat16, pitch=13, offset=3)
    got = rrv.token_logprobs(xs, ids, entropy=True)
    want = check_backward(xs, ids, 1.0, got, True)
    gen = torch.Generator(device="cuda").manual_seed(5)
    g, h = torch.randn(2, 9, generator=gen, device="cuda"), torch.randn(2, 9, generator=gen, device="cuda")
    rest = [x._base.clone() for x in xs]
    back = rrv.token_logprobs_grad(xs, ids, got.lse, g, entropy=got.entropy, dentropy=h, outs=xs)
    assert back is xs
    for x, w, b in zip(xs, want, rest):
        assert torch.equal(x, w)
        x.copy_(b[3:3 + 9 * 1016].view(9, 1016)[:, :1003])
        assert torch.equal(x._base, b)  # nothing but the gradients was written


def test_rank_sets_shapes_and_id_types():
    x = [torch.randn(2, 3, 40, device="cuda") for _ in range(3)]
    ids = [torch.randint(40, (2, 3), device="cuda") for _ in range(3)]
    a = rrv.token_logprobs(x, ids, top_k=2)
    b = rrv.token_logprobs(rrv.RankSet(x), rrv.RankSet([t.int() for t in ids]), top_k=2)
    assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
    g = torch.randn(3, 6, device="cuda")
    da = rrv.token_logprobs_grad(x, ids, a.lse, g)
    db = rrv.token_logprobs_grad(rrv.RankSet(x), rrv.RankSet([t.int() for t in ids]), a.lse, g)
    assert all(torch.equal(p, q) and p.shape == (2, 3, 40) for p, q in zip(da, db))


def test_gradients_against_differences():
    """The loss sum g logprob + h entropy, differenced in 64 bits along random directions."""
    xs, ids = make(1, 6, 500, torch.float32, seed=3)
    x, t = xs[0], ids[0]
    gen = torch.Generator(device="cuda").manual_seed(9)
    g, h = torch.randn(1, 6, generator=gen, device="cuda"), torch.randn(1, 6, generator=gen, device="cuda")
    got = rrv.token_logprobs([x], [t], scale=0.8, entropy=True)
    d = rrv.token_logprobs_grad([x], [t], got.lse, g, entropy=got.entropy, dentropy=h, scale=0.8)[0].double()

    def loss(v):
        lp, _, ent, _, _, _ = formulas(v, t, 0.8)
        return float((g[0].double() * lp + h[0].double() * ent).sum())

    for _ in range(5):
        v = torch.randn(6, 500, generator=gen, device="cuda", dtype=torch.float64)
        step = 1e-5
        slope = (loss(x.double() + step * v) - loss(x.double() - step * v)) / (2 * step)
        # the difference errs by its third derivative (1e-10 x values of order 10) and 1e-16 / step
        assert abs(slope - float((d * v).sum())) <= 1e-6 + 500 * 6 * 2 ** -24 * 4


def test_captured_and_replayed_on_another_stream():
    xs, ids = make(2, 40, 9000, torch.float16, seed=4)
    want = rrv.token_logprobs(xs, ids, entropy=True, top_k=6)
    g = torch.randn(2, 40, device="cuda")
    dwant = rrv.token_logprobs_grad(xs, ids, want.lse, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = rrv.token_logprobs(xs, ids, entropy=True, top_k=6)
        dgot = rrv.token_logprobs_grad(xs, ids, got.lse, g)
    for _ in range(2):
        for t in (*got, *dgot):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(a, b) for a, b in zip(dwant, dgot))
    side.wait_stream(torch.cuda.current_stream())
    again = rrv.token_logprobs(xs, ids, entropy=True, top_k=6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_rows_far_into_a_large_buffer():
    """Offsets past 2^32 bytes and 2^31 elements."""
    T, V = 70000, 32768
    x = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")  # 4.6 GB, 2.3e9 elements
    x[T - 1].copy_(torch.randn(V, device="cuda"))
    t = torch.full((T,), 11, dtype=torch.int64, device="cuda")
    got = rrv.token_logprobs([x], [t], top_k=2)
    assert (got.logprob[0, :-1] + math.log(V)).abs().max() <= 1e-5
    check = rrv.token_logprobs([x[T - 1:].clone()], [t[:1]], top_k=2)
    assert torch.equal(got.lse[0, -1], check.lse[0, 0]) or abs(float(got.lse[0, -1] - check.lse[0, 0])) <= 1e-5
    assert torch.equal(got.top_id[0, -1], check.top_id[0, 0])
    g = torch.zeros(1, T, device="cuda")
    g[0, -1] = 1.0
    rrv.token_logprobs_grad([x], [t], got.lse, g, outs=[x])
    assert float(x[T - 1].double().sum().abs()) < 0.05 and (x[T - 2] == 0).all() and float(x[T - 1, 11]) > 0.5
    del x
    torch.cuda.empty_cache()


def test_refused_tensors():
    x, t = torch.randn(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (lambda: rrv.token_logprobs([x.T], [torch.zeros(8, dtype=torch.int64, device="cuda")]),
                lambda: rrv.token_logprobs([x[:, ::2]], [t]), lambda: rrv.token_logprobs([x, x], [t]),
                lambda: rrv.token_logprobs([x[:3]], [t]), lambda: rrv.token_logprobs([x], [t], top_k=9),
                lambda: rrv.token_logprobs([x], [t], top_k=-1),
                lambda: rrv.token_logprobs_grad([x], [t], torch.zeros(4, device="cuda").double(), torch.zeros(4, device="cuda")),
                lambda: rrv.token_logprobs_grad([x], [t], torch.zeros(4, device="cuda"), torch.zeros(3, device="cuda")),
                lambda: rrv.token_logprobs_grad([x], [t], torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"),
                                                dentropy=torch.zeros(4, device="cuda")),
                lambda: rrv.token_logprobs_grad([x], [t], torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"),
                                                outs=[torch.empty(4, 9, device="cuda")])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(rrv.RRError):
        rrv.token_logprobs([x], [t], scale=0.0)
    with pytest.raises(TypeError):
        rrv.token_logprobs([x.double()], [t])


def test_no_rows_and_first_calls_under_capture():
    x, t = torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    got = rrv.token_logprobs([x, x], [t, t], entropy=True, top_k=3)
    assert got.logprob.shape == (2, 0) and got.top_id.shape == (2, 0, 3)
    assert rrv.token_logprobs_grad([x], [t], torch.empty(1, 0, device="cuda"), torch.empty(1, 0, device="cuda"))[0].shape == (0, 50)
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = r"""
import torch
import ring_all_reduce_virtual_b200 as rrv
x = torch.randn(5, 40000, device="cuda")
t = torch.arange(5, device="cuda")
small, large = torch.randn(70, 200, device="cuda"), torch.randn(300, 200, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = rrv.token_logprobs([x], [t], entropy=True, top_k=4)
    d = rrv.token_logprobs_grad([x], [t], a.lse, a.lse)
    o = rrv.orthogonalize([small, large])
g.replay()
torch.cuda.synchronize()
b = rrv.token_logprobs([x], [t], entropy=True, top_k=4)
e = rrv.token_logprobs_grad([x], [t], b.lse, b.lse)
p = rrv.orthogonalize([small, large])
print("SAME", all(torch.equal(u, v) for u, v in zip((*a, *d, *o), (*b, *e, *p))))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "SAME True" in r.stdout, r.stdout + r.stderr


def test_gradient_rows_at_every_phase_beside_the_logits():
    """Logits and gradients at all pairs of offsets, row strides that change the phase from row to row; neighbours left alone."""
    for dt in (torch.bfloat16, torch.float32):
        L = 16 // torch.tensor([], dtype=dt).element_size()
        for off in range(L):
            xs, ids = make(1, 5, 333, dt, seed=off, pitch=off % 3, offset=off)
            got = rrv.token_logprobs(xs, ids, entropy=True)
            base = torch.full((6 * 340 + 16,), 7.0, dtype=dt, device="cuda")
            out = base[3:3 + 5 * 336].view(5, 336)[:, :333]
            check_backward(xs, ids, 1.0, got, True, outs=[out])
            keep = torch.ones_like(base, dtype=torch.bool)
            keep[3:3 + 5 * 336].view(5, 336)[:, :333] = False
            assert (base[keep] == 7).all()
