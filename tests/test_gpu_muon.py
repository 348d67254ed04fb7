"""Orthogonalisation and the Muon step on the GPU, against the iteration in 64
bits.

Tolerances.  A step X' = a X + (b A + c A^2) X rounds operands at 2^-22 and sums
in fp32; with singular values up to 1.25 the terms reach a, b 1.6, c 2.5 times X
and each of the up to five factors of a term errs by two such roundings: an
error of at most KAPPA * 2^-22 * ||X_k|| in Frobenius' norm, KAPPA = 2 * 2 *
(a + 1.6 * 3 |b| / 2 + 2.5 * 5 c / 2) < 60.  Later steps multiply an error by
their slope, at most a.  So after n steps
    ||O - exact|| <= 60 * 2^-22 * sum_k a^(n-1-k) ||X_k||
(of the normalised X_0 too), where ||X_k|| is the 64-bit iteration's, and the
rounding to the result's type is half a step of each element.
"""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COEF = (3.4445, -4.7750, 2.0315)
KAPPA = 60.0


def iterate(x, steps=5, coef=COEF, eps=1e-7):
    """The iteration in 64 bits, and the bound on a 22-bit one's error in Frobenius' norm."""
    a, b, c = coef
    x = x.double() / (x.double().norm() + eps)
    wide = x.shape[0] <= x.shape[1]
    norms = [float(x.norm())]
    for _ in range(steps):
        if wide:
            A = x @ x.T
            x = a * x + (b * A + c * (A @ A)) @ x
        else:
            A = x.T @ x
            x = a * x + x @ (b * A + c * (A @ A))
        norms.append(float(x.norm()))
    grow = max(abs(a), 1.0)
    bound = KAPPA * 2.0 ** -22 * sum(grow ** (steps - 1 - k) * n for k, n in enumerate(norms[:-1]))
    return x, bound + 2.0 ** -21 * norms[-1]


def rounding(x, dtype):
    """Half a step of every element, in Frobenius' norm, and below the type's normal numbers half the smallest."""
    if dtype == torch.float32:
        return 2.0 ** -23 * float(x.norm())
    info = torch.finfo(dtype)
    least = info.tiny * info.eps / 2
    return float((x.abs() * (info.eps / 2) + least).norm())


def gradient(r, c, dtype, seed=0, kind="noise"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(r, c, generator=g, device="cuda")
    if kind == "low rank":
        k = max(1, min(r, c) // 16)
        x = torch.randn(r, k, generator=g, device="cuda") @ torch.randn(k, c, generator=g, device="cuda") + 0.05 * x
    return (x * 1e-2).to(dtype)


def check(got, x, dtype=None, **kw):
    want, bound = iterate(x, **kw)
    err = float((got.double() - want).norm())
    assert err <= bound + rounding(want, got.dtype), (tuple(x.shape), err, bound, float(want.norm()))


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (64, 64), (65, 63), (128, 128), (129, 257), (200, 72), (130, 640), (640, 130),
          (300, 300), (384, 96), (515, 1023), (1023, 515), (768, 256), (257, 1), (1000, 136)]


@pytest.mark.parametrize("r,c", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_one_matrix(r, c, dtype):
    x = gradient(r, c, TYPES[dtype], seed=r + c)
    keep = x.clone()
    (got,) = rrv.orthogonalize([x])
    assert got.dtype == x.dtype and got.shape == x.shape and torch.equal(x, keep)
    check(got, x)


@pytest.mark.parametrize("kind", ["low rank", "noise"])
def test_a_list_of_mixed_shapes_and_types(kind):
    xs = [gradient(r, c, TYPES[t], seed=i, kind=kind) for i, ((r, c), t) in
          enumerate([((640, 256), "bf16"), ((256, 256), "f32"), ((256, 1024), "f16"), ((1024, 256), "f32"), ((77, 131), "bf16"),
                     ((1, 500), "f16"), ((2048, 384), "bf16"), ((384, 2048), "f32")])]
    got = rrv.orthogonalize(xs)
    for g, x in zip(got, xs):
        check(g, x)
    alone = [rrv.orthogonalize([x])[0] for x in xs]
    again = rrv.orthogonalize(xs)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same call, the same bits
    for a, x in zip(alone, xs):
        check(a, x)


@pytest.mark.parametrize("steps,coef", [(0, COEF), (1, COEF), (3, COEF), (8, COEF), (5, (2.0, -1.5, 0.5)), (4, (1.5, -0.5, 0.0)),
                                        (3, (1.0, 0.0, 0.0))])
def test_other_iterations(steps, coef):
    for r, c in ((96, 160), (160, 96)):
        x = gradient(r, c, torch.float32, seed=steps)
        check(rrv.orthogonalize([x], steps=steps, coefficients=coef)[0], x, steps=steps, coef=coef)


def test_scales_of_the_input():
    """The iteration does not see the matrix's scale, to the ends of fp32."""
    x = gradient(100, 140, torch.float32)
    for scale in (2.0 ** 100, 2.0 ** -100, 2.0 ** 126, 2.0 ** -120):
        y = x * scale
        check(rrv.orthogonalize([y], eps=1e-37)[0], y, eps=1e-37)
    check(rrv.orthogonalize([x * 1e-9], eps=1e-7)[0], x * 1e-9, eps=1e-7)  # eps counts


def test_zeros_nan_and_infinity():
    zero = torch.zeros(50, 70, device="cuda")
    nan = gradient(50, 70, torch.float32)
    nan[3, 5] = math.nan
    inf = gradient(70, 50, torch.bfloat16)
    inf[1, 1] = math.inf
    good = gradient(50, 70, torch.float32)
    o = rrv.orthogonalize([zero, nan, inf, good])
    assert (o[0] == 0).all() and o[1].isnan().all() and o[2].isnan().all()
    check(o[3], good)


def test_in_place_other_type_and_every_rank():
    x = gradient(96, 224, torch.float32)
    want = rrv.orthogonalize([x])[0]
    outs = [[torch.empty(96, 224, device="cuda")] for _ in range(3)]
    assert rrv.orthogonalize([x], outs) is outs
    assert all(torch.equal(o[0], want) for o in outs)
    half = torch.empty(96, 224, dtype=torch.bfloat16, device="cuda")
    rrv.orthogonalize([x], [half])
    check(half, x)
    rrv.orthogonalize([x], [x])
    assert torch.equal(x, want)
    assert rrv.orthogonalize([]) == []
    e = torch.empty(0, 5, device="cuda")
    assert rrv.orthogonalize([e])[0].shape == (0, 5)


def test_odd_offsets_leave_the_neighbours_alone():
    flat = torch.full((4000,), 7.0, dtype=torch.bfloat16, device="cuda")
    x = gradient(31, 37, torch.bfloat16)
    flat[3:3 + 31 * 37].copy_(x.view(-1))
    view = flat[3:3 + 31 * 37].view(31, 37)
    rrv.orthogonalize([view], [view])
    check(view, x)
    assert (flat[:3] == 7).all() and (flat[3 + 31 * 37:] == 7).all()


def step(ranks, shapes, dtype, gdtype, seed=0, offset=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def tensor(shape, dt, std):
        big = torch.empty(shape[0] * shape[1] + offset, dtype=dt, device="cuda")
        t = big[offset:].view(shape)
        t.copy_(torch.randn(shape, generator=g, device="cuda") * std)
        return t

    w = [[tensor(s, dtype, 0.02) for s in shapes]]
    w += [[torch.full_like(t, 9.0) for t in w[0]] for _ in range(ranks - 1)]
    grads = [tensor(s, gdtype, 1e-2) for s in shapes]
    mom = [tensor(s, torch.float32, 3e-2) for s in shapes]
    w0, m0 = [t.double() for t in w[0]], [t.double() for t in mom]
    cfg = dict(lr=0.03, momentum=0.9, nesterov=True, weight_decay=0.1, adjust="spectral")
    cfg.update(kw)
    rrv.muon_step(w, grads, mom, **cfg)
    for t, shape in enumerate(shapes):
        m = cfg["momentum"] * m0[t] + grads[t].double()
        assert ((mom[t].double() - m).abs() <= 2.0 ** -23 * (m0[t].abs() + grads[t].double().abs())).all()
        u = grads[t].double() + cfg["momentum"] * m if cfg["nesterov"] else m
        o, bound = iterate(u)
        # u is formed in fp32 from the rounded momentum: 2^-22 of it, in every later step as the operands' own roundings
        f = math.sqrt(max(1.0, shape[0] / shape[1])) if cfg["adjust"] == "spectral" else 0.2 * math.sqrt(max(shape))
        want = (1 - cfg["lr"] * cfg["weight_decay"]) * w0[t] - cfg["lr"] * f * o
        err = float((w[0][t].double() - want).norm())
        assert err <= cfg["lr"] * f * 2 * bound + rounding(want, dtype) * 1.01 + 2.0 ** -22 * float(want.norm()), (shape, err)
        assert all(torch.equal(w[r][t], w[0][t]) for r in range(ranks))


@pytest.mark.parametrize("ranks,dtype,gdtype,kw", [
    (1, "f32", "f32", {}), (4, "f32", "bf16", dict(nesterov=False)), (3, "bf16", "bf16", dict(adjust="rms")),
    (2, "f16", "f16", dict(weight_decay=0.0)), (8, "bf16", "f32", dict(momentum=0.0)), (64, "f32", "f32", {})])
def test_muon_step(ranks, dtype, gdtype, kw):
    step(ranks, [(384, 128), (128, 128), (512, 128), (128, 512), (1, 200), (77, 53)], TYPES[dtype], TYPES[gdtype], **kw)


def test_muon_step_of_odd_matrices_at_odd_offsets():
    step(3, [(301, 101), (101, 105), (33, 7)], torch.float16, torch.float16, offset=1)
    step(2, [(301, 101), (101, 105)], torch.float32, torch.bfloat16, offset=3)


def test_more_matrices_than_a_launch_takes():
    step(2, [(40 + i, 130 - i) for i in range(60)], torch.float32, torch.float32)


def test_large_matrices():
    step(2, [(1536, 512), (512, 2048), (1100, 1100)], torch.bfloat16, torch.bfloat16)


def test_groups_that_share_the_workspace():
    """Matrices whose workspace passes what one group takes: one after the other in the same memory."""
    from ring_all_reduce_virtual_b200 import _lib
    shapes = [(4096, 4096)] * 16 + [(64, 64)]
    xs = [gradient(r, c, torch.bfloat16, seed=i) for i, (r, c) in enumerate(shapes)]
    ml = rrv.MatrixList(xs)
    ns = _lib.NewtonSchulz(2, *COEF, 1e-7)
    assert ml._workspace(False, ns) <= (5 << 30)
    got = rrv.orthogonalize(ml, steps=2)
    for g, x in zip(got, xs):
        check(g, x, steps=2)


def test_captured_with_two_graphs_of_their_own_workspaces():
    xs = [gradient(200, 300, torch.float32, seed=1)], [gradient(300, 200, torch.float32, seed=2)]
    want = [rrv.orthogonalize(x)[0] for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rrv.orthogonalize(x)[0])
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_calls_on_two_streams():
    xs = [[gradient(256, 512, torch.bfloat16, seed=i)] for i in range(2)]
    want = [rrv.orthogonalize(x)[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got = [rrv.orthogonalize(x, stream=s)[0] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_step_of_all_operators():
    """Loss and gradient of every rank's logits, the LM head's gradient synced and clipped, the Muon step on every replica."""
    n, T, V, D = 4, 96, 1200, 128
    gen = torch.Generator(device="cuda").manual_seed(0)
    head = [(torch.randn(V, D, generator=gen, device="cuda") * 0.05)]
    head += [head[0].clone() for _ in range(n - 1)]
    hidden = [torch.randn(T, D, generator=gen, device="cuda") for _ in range(n)]
    ids = [torch.randint(V, (T,), generator=gen, device="cuda") for _ in range(n)]
    mom = [torch.zeros(V, D, device="cuda")]
    logits = [h @ w.T for h, w in zip(hidden, head)]
    fwd = rrv.token_logprobs(logits, ids)
    dl = rrv.token_logprobs_grad(logits, ids, fwd.lse, torch.full((n, T), -1.0 / T, device="cuda"))
    grads = [[d.T @ h] for d, h in zip(dl, hidden)]
    p = [torch.softmax(x.double(), -1) for x in logits]
    want = []
    for r in range(n):
        p[r][torch.arange(T, device="cuda"), ids[r]] -= 1.0
        want.append((p[r].T / T) @ hidden[r].double())
    avg = sum(want) / n
    norm = rrv.BucketPlan([V * D], "f32").all_reduce_clip(grads, 0.5, eps=0.0)
    assert abs(float(norm) - float(avg.norm())) <= 1e-4 * float(avg.norm())
    before = head[0].double()
    rrv.muon_step([[w] for w in head], grads[:1], mom, lr=0.1, momentum=0.95)
    o, bound = iterate(avg)
    update = (before - head[0].double()) / (0.1 * math.sqrt(V / D))
    assert float((update - o).norm()) <= 0.01 * float(o.norm())  # the gradient itself comes from fp32 products
    assert all(torch.equal(w, head[0]) for w in head)


def test_refused_tensors():
    x = torch.randn(4, 6, device="cuda")
    for bad in (lambda: rrv.orthogonalize([x.T]), lambda: rrv.orthogonalize([x[0]]), lambda: rrv.orthogonalize([x], [x.clone(), x.clone()]),
                lambda: rrv.orthogonalize([x], [torch.empty(6, 4, device="cuda")]), lambda: rrv.orthogonalize([x.cpu()]),
                lambda: rrv.muon_step([x], [x.clone()], [torch.zeros(6, 4, device="cuda")], lr=0.1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        rrv.orthogonalize([x.int()])
    for bad in (dict(steps=-1), dict(steps=51), dict(eps=0.0), dict(eps=math.nan), dict(coefficients=(math.nan, 0, 0)),
                dict(steps=40, coefficients=(3.0, 1.0, 1.0))):
        with pytest.raises(rrv.RRError):
            rrv.orthogonalize([x], **bad)
    for bad in (dict(lr=math.inf), dict(lr=0.1, momentum=-0.1), dict(lr=0.1, adjust=2), dict(lr=0.1, weight_decay=math.nan)):
        with pytest.raises(rrv.RRError):
            rrv.muon_step([x], [x.clone()], [torch.zeros(4, 6, device="cuda")], **bad)
    with pytest.raises(rrv.RRError):
        rrv.muon_step([x], [x], [torch.zeros(4, 6, device="cuda")], lr=0.1)  # the gradient in the weights' place
    with pytest.raises(rrv.RRError):
        rrv.muon_step([x], [x.clone()], [torch.zeros(4, 6, device="cuda").half()], lr=0.1)


def test_waits_that_run_out():
    """RR_DEBUG_BULK_TIMEOUT=1 makes the products' waits run out, in the launch of many tiles and in a cluster's own: the
    status says so, copies and products are seen to end, and the context still runs a call."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = r"""
import torch
import ring_all_reduce_virtual_b200 as rrv
for shapes in ([(64, 64), (128, 500), (100, 700)], [(300, 300)], [(1024, 512), (512, 2048), (100, 100), (700, 700)]):
    for dt in (torch.float32, torch.bfloat16):
        rrv.orthogonalize([torch.randn(s, device="cuda").to(dt) for s in shapes])
        try:
            rrv.check_timeouts()
            print("NO TIMEOUT")
        except rrv.RRError as e:
            print("RAN OUT", e.status, "not seen to land: 0" in str(e))
x = torch.randn(3, 500, device="cuda")
got = rrv.token_logprobs([x], [torch.zeros(3, dtype=torch.int64, device="cuda")])
print("CONTEXT OK", bool((got.lse[0] - torch.logsumexp(x, -1)).abs().max() < 1e-5))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, RR_DEBUG_BULK_TIMEOUT="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.count("RAN OUT 4 True") == 6 and "CONTEXT OK True" in r.stdout, r.stdout + r.stderr


def test_more_steps_and_mixed_kinds_than_a_small_block_holds():
    """Fifty steps of a polynomial that keeps singular values where they are, lists whose kinds of iteration differ."""
    coef = (1.5, -0.5, 0.0)
    xs = [gradient(300, 200, torch.float32, 1), gradient(200, 300, torch.bfloat16, 2), gradient(256, 520, torch.float16, 3),
          gradient(90, 90, torch.float32, 4)]
    for g, x in zip(rrv.orthogonalize(xs, steps=50, coefficients=coef), xs):
        check(g, x, steps=50, coef=coef)


def test_statistics_of_a_call():
    rrv.orthogonalize([gradient(64, 64, torch.float32)])
    assert rrv.last_stats()["launches"] == 1
    rrv.orthogonalize([gradient(300, 300, torch.float32)])
    s = rrv.last_stats()
    assert s["launches"] == 4 and s["steps"] == 5 and s["hbm_bytes"] == 2 * 300 * 300 * 4


@pytest.mark.parametrize("r,c", [(128, 1024), (1024, 128), (129, 129), (128, 1025), (1025, 100), (1, 1024), (64, 65), (100, 129)])
def test_shapes_around_what_a_cluster_takes(r, c):
    for dt in TYPES.values():
        x = gradient(r, c, dt, seed=r)
        check(rrv.orthogonalize([x])[0], x)


def test_offset_views_beside_aligned_ones():
    """Matrices whose rows are whole vectors but whose addresses are not."""
    for r, c in ((64, 64), (264, 512)):
        base = torch.zeros(r * c + 8, device="cuda")
        x = base[1:1 + r * c].view(r, c)
        x.copy_(gradient(r, c, torch.float32))
        outs = [[torch.empty(r, c, device="cuda")], [torch.empty(r * c + 4, device="cuda")[3:3 + r * c].view(r, c)]]
        rrv.orthogonalize([x], outs)
        check(outs[0][0], x)
        assert torch.equal(outs[0][0], outs[1][0])


@pytest.mark.parametrize("r,c", [(230, 920), (690, 230), (920, 230), (511, 1500), (512, 1500)])
def test_small_fp32_weights_keep_their_precision(r, c):
    """The result's share of a small weight is large: O errs by 2e-5 of its norm at
    most, and the update's two roundings are half a step of fp32 each."""
    gen = torch.Generator(device="cuda").manual_seed(r + c)
    k = min(r, c) // 16
    noise = torch.randn(r, c, generator=gen, device="cuda")
    strong = torch.randn(r, k, generator=gen, device="cuda") @ torch.randn(k, c, generator=gen, device="cuda")
    g = (noise + strong / math.sqrt(k)) * 1e-3
    w = torch.randn(r, c, generator=gen, device="cuda") * 0.02
    m = torch.zeros(r, c, device="cuda")
    o, _ = iterate(g.double() * 1.95)
    f = 0.02 * math.sqrt(max(1.0, r / c))
    want = w.double() * (1.0 - 0.02 * 0.01) - f * o
    rrv.muon_step([w], [g], [m], lr=0.02, weight_decay=0.01)
    err = float((w.double() - want).norm())
    assert err <= f * 2e-5 * float(o.norm()) + 2.0 ** -23 * float(want.norm()), (err, float(o.norm()), float(want.norm()))


@pytest.mark.parametrize("count", [25, 128, 150])
def test_many_matrices_some_of_them_alike(count):
    """More than a small parameter block and a group hold; shapes and types that come again, in no order."""
    xs = [gradient(130 + i * i % 5, 140 + i % 3 * 130, TYPES[("f32", "bf16", "f16")[i % 7 % 3]], seed=i) for i in range(count)]
    got = rrv.orthogonalize(xs)
    for g, x in zip(got, xs):
        check(g, x)
    again = rrv.orthogonalize(xs)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("ranks,count,side", [(64, 20, 40), (64, 20, 140), (9, 130, 20), (9, 130, 130)])
def test_more_replicas_than_a_launch_writes(ranks, count, side):
    step(ranks, [(side + i % 2, side + i % 3) for i in range(count)], torch.float32, torch.float32)


@pytest.mark.parametrize("ranks", [2, 6])
@pytest.mark.parametrize("offset", [0, 1, 2, 8])
def test_rows_on_no_common_boundary(ranks, offset):
    """Columns that 8, 2 or nothing divides, from addresses that are and are not on 16 bytes."""
    shapes = [(270, 90), (91, 93), (258, 130), (257, 131), (140, 264), (1, 301), (299, 2)]
    for dt, gdt in (("f32", "bf16"), ("bf16", "f32"), ("f16", "f16")):
        step(ranks, shapes, TYPES[dt], TYPES[gdt], offset=offset)


@pytest.mark.parametrize("r,c", [(131, 260), (260, 131), (140, 8192), (150, 134), (33, 18)])
def test_results_at_odd_places_leave_the_neighbours_alone(r, c):
    for dt in TYPES.values():
        x = gradient(r, c, dt, seed=r)
        want = rrv.orthogonalize([x])[0]
        for at in (1, 2, 3):
            flats = [torch.full((r * c + 16,), 7.0, dtype=dt, device="cuda") for _ in range(6)]
            outs = [[f[at:at + r * c].view(r, c)] for f in flats]
            rrv.orthogonalize([x], outs)
            for f in flats:
                assert torch.equal(f[at:at + r * c].view(r, c), want)
                assert (f[:at] == 7).all() and (f[at + r * c:] == 7).all()


@pytest.mark.parametrize("side", [30, 150])
def test_many_matrices_captured(side):
    """Launches with large parameter blocks in a graph, replayed after the inputs changed."""
    xs = [gradient(side + i % 4, side + i % 3 * 50, torch.float32, seed=i) for i in range(60)]
    first = [x.clone() for x in xs]
    outs = [[torch.empty_like(x) for x in xs] for _ in range(5)]
    rrv.orthogonalize(xs, outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rrv.orthogonalize(xs, outs)
    for inputs in ([x.flip(0) for x in first], first):
        for x, v in zip(xs, inputs):
            x.copy_(v)
        graph.replay()
        want = rrv.orthogonalize(xs)
        assert all(torch.equal(a, b) for rank in outs for a, b in zip(rank, want))
