"""The embedding lookup and its gradient over all ranks.

The lookup is one fp32 product and one rounding: bits.  The gradient is
compared with the formula in 64 bits.  Tolerance of a row that sums c rows of
output gradients: each of its at most c additions is off by at most 2^-24 of
the partial sum, so by 2^-24 of the sum of magnitudes; the factor and its
product add one rounding each: (c + 2) * 2^-24 of f * sum |x|; adding to what
is there one more of the result; then the rounding to the gradient's type,
u = torch.finfo(t).eps / 2 of the value, or half the smallest subnormal step.
"""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv
from test_gpu_clip import DT, E, SUB, U, Guarded, near_norm, near_scaled, norm64, values

pytestmark = pytest.mark.gpu


def rows(seed, n, d, dtype, off=0, std=1.0):
    g = Guarded(values(seed, n * d, dtype, std), off)
    g.m = g.t.view(n, d)
    return g


def draw_ids(seed, t, v, dtype, kind="zipf"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "zipf":
        u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(v + 1)) - 1).long().clamp(0, v - 1)
    elif kind == "same":
        ids = torch.full((t,), v // 2, device="cuda")
    elif kind == "runs":  # neighbours alike, in falling order
        ids = (torch.arange(t, device="cuda") // 3).flip(0) % v
    elif kind == "none":
        ids = torch.where(torch.arange(t, device="cuda") % 2 == 0, -5, v + 3)
    else:  # spread, with ids that have no row among them
        ids = torch.randint(-v // 4 - 1, v + v // 4 + 1, (t,), generator=g, device="cuda")
    return ids.to(dtype)


# ------------------------------------------------------------------ lookup

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [1, 2, 3, 8, 36, 257, 515, 1030, 2048])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_lookup_bits(dtype, d, off):
    n, v = 3, 211
    for t, id_dtype in ((1, torch.int64), (37, torch.int32)):
        ids = [draw_ids(10 * r + t, t, v, id_dtype, "spread") for r in range(n)]
        ids[0][0] = v - 1
        tables = [rows(r, v, d, DT[dtype], off) for r in range(n)]
        outs = [rows(50 + r, t, d, DT[dtype], (off * r) % 8) for r in range(n)]
        scale = 1.7
        rrv.embedding(ids, [w.m for w in tables], [o.m for o in outs], scale)
        for r in range(n):
            i = ids[r].long()
            inside = (i >= 0) & (i < v)
            want = (tables[r].m[i.clamp(0, v - 1)].float() * torch.tensor(scale)).to(DT[dtype])
            want[~inside] = 0
            assert torch.equal(outs[r].m, want)
            outs[r].check()


def test_lookup_shares_a_table_and_keeps_bits_at_scale_1():
    v, d, t = 100, 64, 20
    table = rows(1, v, d, torch.bfloat16)
    ids = [draw_ids(r, t, v, torch.int32) for r in range(4)]
    outs = [torch.empty(t, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    sets = [rrv.RankSet(ids), rrv.RankSet([table.m] * 4), rrv.RankSet(outs)]
    for _ in range(2):
        rrv.embedding(*sets)
        for i, o in zip(ids, outs):
            assert torch.equal(o, table.m[i.long()])
            o.zero_()
    three = torch.empty(4, 5, d, dtype=torch.bfloat16, device="cuda")  # ids and rows of any leading shape
    rrv.embedding([ids[0].view(4, 5)], [table.m], [three])
    assert torch.equal(three, table.m[ids[0].long()].view(4, 5, d))


# ---------------------------------------------------------------- gradient

def check_grad(ids, dout, grads, before, v, f, accumulate, padding=-1):
    """Every table of `grads` against the 64-bit sum; `before`: their earlier values."""
    d = dout[0].shape[-1]
    flat = torch.cat([i.reshape(-1).long() for i in ids])
    x = torch.cat([g.reshape(-1, d) for g in dout]).double()
    inside = (flat >= 0) & (flat < v) & (flat != padding)
    flat, x = flat[inside], x[inside]
    total = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, flat, x)
    mag = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, flat, x.abs())
    cnt = torch.zeros(v, dtype=torch.float64, device="cuda").index_add_(0, flat, torch.ones_like(flat, dtype=torch.float64))
    for g, old in zip(grads, before):
        dt = g.dtype
        want = f * total + (old.double() if accumulate else 0.0)
        tol = abs(f) * (cnt[:, None] + 2) * E * mag + want.abs() * (U[dt] * 1.001 + 2 * E) + SUB[dt]
        touched = cnt > 0
        err = (g.double() - want).abs()
        assert not bool((err > tol)[touched].any()), float((err - tol)[touched].max())
        rest = old if accumulate else torch.zeros_like(old)
        assert torch.equal(g[~touched], rest[~touched])


def run_grad(n, t, v, d, dtype, kind, *, grad_dtype=None, nout=None, accumulate=False, op="avg", scale=1.0, padding=None,
             off=0, id_dtype=torch.int32):
    gd = grad_dtype or dtype
    ids = [draw_ids(31 * r + t, t, v, id_dtype, kind) for r in range(n)]
    dout = [rows(100 + r, t, d, dtype, (off * (r + 1)) % 8) for r in range(n)]
    grads = [rows(200 + o, v, d, gd, (off * o) % 8) for o in range(nout or n)]
    before = [g.m.clone() for g in grads]
    rrv.embedding_grad(ids, [g.m for g in dout], [g.m for g in grads], op, scale, accumulate, padding)
    check_grad(ids, [g.m for g in dout], [g.m for g in grads], before, v, scale / n if op == "avg" else scale, accumulate,
               -1 if padding is None else padding)
    for g in grads + dout:
        g.check()
    return grads


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", ["zipf", "same", "runs", "spread", "none"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_types_and_id_patterns(dtype, kind, accumulate):
    for n, t, d in ((1, 1, 40), (1, 33, 256), (3, 700, 264), (2, 2049, 17)):
        run_grad(n, t, 97, d, DT[dtype], kind, accumulate=accumulate, scale=1.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_grad_in_fp32_beside_16_bit_rows(dtype):
    for accumulate in (False, True):
        for d in (64, 515, 1026):
            run_grad(4, 300, 411, d, DT[dtype], "zipf", grad_dtype=torch.float32, nout=1, accumulate=accumulate, op="sum")


@pytest.mark.parametrize("d", [1, 2, 3, 4, 6, 8, 12, 31, 255, 256, 257, 512, 515, 1032])
@pytest.mark.parametrize("off", [0, 1, 2, 4])
def test_grad_widths_and_alignments(d, off):
    for dtype in (torch.bfloat16, torch.float32):
        run_grad(2, 150, 60, d, dtype, "zipf", off=off, id_dtype=torch.int64)


@pytest.mark.parametrize("t", [1, 2, 31, 32, 33, 63, 64, 65, 2047, 2048, 2049, 5000])
@pytest.mark.parametrize("v", [1, 2, 511, 513, 70001, 300007])
def test_grad_tokens_and_table_rows(t, v):
    for kind in ("zipf", "spread"):
        run_grad(1, t, v, 9, torch.float32, kind)


def test_grad_of_many_tokens():
    run_grad(2, 140_001, 5000, 8, torch.bfloat16, "zipf", nout=1)  # blocks of more than 32 positions
    run_grad(1, 200_000, 300_000, 8, torch.float32, "same")
    run_grad(3, 400_001, 40_000, 4, torch.float32, "zipf", nout=1)  # more tiles than a CTA sums
    run_grad(64, 11, 50, 16, torch.float16, "zipf", nout=2)
    for kind in ("zipf", "runs", "same"):  # blocks of 16 and of 32 positions
        run_grad(2, 5_003, 2000, 2048, torch.bfloat16, kind, nout=1)
        run_grad(2, 12_000, 2000, 2048, torch.bfloat16, kind, nout=1, accumulate=True, grad_dtype=torch.float32)


@pytest.mark.parametrize("length", [1, 7, 8, 9, 15, 16, 17, 24, 25, 63, 64, 65, 300])
def test_grad_runs_that_end_at_block_bounds(length):
    """Runs of one length shifted against the blocks of positions by 0..7."""
    for shift in range(8):
        t = length * 5 + shift
        ids = torch.cat([torch.zeros(shift, dtype=torch.int64), 1 + torch.arange(5).repeat_interleave(length)]).cuda()
        x = values(length + shift, t * 40, torch.bfloat16).view(t, 40)
        for accumulate in (False, True):
            g = values(3, 8 * 40, torch.float32).view(8, 40)
            old = g.clone()
            rrv.embedding_grad([ids], [x], [g], "sum", accumulate=accumulate)
            check_grad([ids], [x], [g], [old], 8, 1.0, accumulate)


def test_grad_padding_and_no_tokens():
    run_grad(2, 400, 30, 24, torch.bfloat16, "zipf", padding=0)
    run_grad(2, 400, 30, 24, torch.bfloat16, "same", padding=15)  # nothing is left
    none = [torch.empty(0, dtype=torch.int32, device="cuda")]
    g = rows(5, 20, 16, torch.float32)
    old = g.m.clone()
    rrv.embedding_grad(none, [torch.empty(0, 16, device="cuda")], [g.m], accumulate=True)
    assert torch.equal(g.m, old)
    rrv.embedding_grad(none, [torch.empty(0, 16, device="cuda")], [g.m])
    assert not bool(g.m.any())
    g.check()


def test_grad_bits_repeat_and_replicas_agree():
    first = run_grad(4, 3000, 500, 136, torch.bfloat16, "zipf", nout=4)
    again = run_grad(4, 3000, 500, 136, torch.bfloat16, "zipf", nout=4)
    for a, b in zip(first, again):
        assert torch.equal(a.m, b.m) and torch.equal(a.m, first[0].m)


def test_grad_with_infinities_and_nans():
    ids = [torch.tensor([3, 1, 3, -1, 2], dtype=torch.int32, device="cuda")]
    x = torch.ones(5, 8, device="cuda")
    x[0, 1], x[2, 1], x[1, 2] = math.inf, -math.inf, math.nan
    x[3] = math.nan  # a padded token's
    g = torch.full((5, 8), 7.0, device="cuda")
    rrv.embedding_grad(ids, [x], [g], "sum")
    assert math.isnan(float(g[3, 1])) and math.isnan(float(g[1, 2])) and int(g.isnan().sum()) == 2
    assert float(g[3, 0]) == 2.0 and float(g[2, 0]) == 1.0 and not bool(g[0].any()) and not bool(g[4].any())


def test_gradient_is_the_lookups_adjoint():
    """sum(dout * lookup(W)) is linear in W, so its difference along any
    direction P is sum(dW * P) exactly; both sums in 64 bits over fp32 values."""
    n, t, v, d, scale = 3, 257, 50, 40, 2.5
    ids = [draw_ids(r, t, v, torch.int64, "spread") for r in range(n)]
    dout = [values(r, t * d, torch.float32).view(t, d) for r in range(n)]
    P = values(9, v * d, torch.float32).view(v, d)
    W = values(10, v * d, torch.float32).view(v, d)

    def loss(table):
        outs = [torch.empty(t, d, device="cuda") for _ in range(n)]
        rrv.embedding(ids, [table] * n, outs, scale)
        return sum(float((o.double() * g.double()).sum()) for o, g in zip(outs, dout))

    dW = torch.empty(v, d, device="cuda")
    rrv.embedding_grad(ids, dout, [dW], "sum", scale)
    along = float((dW.double() * P.double()).sum())
    size = float((dW.double() * P.double()).abs().sum()) + sum(float(g.double().abs().sum()) for g in dout) * 8 * scale
    # W + P and W - P are rounded to fp32, as are the products: 4 roundings of values below 8 * scale * |dout|
    assert abs((loss(W + P) - loss(W - P)) / 2 - along) <= 300 * E * size


def test_offsets_past_32_bits():
    v, d = 140_001, 32768
    table = torch.zeros(v, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([v - 1, 0, 131_073, v - 1], dtype=torch.int32, device="cuda")
    for k, i in enumerate((v - 1, 0, 131_073)):
        table[i] = k + 1
    out = torch.empty(4, d, dtype=torch.bfloat16, device="cuda")
    rrv.embedding([ids], [table], [out], 2.0)
    assert torch.equal(out, torch.tensor([2.0, 4.0, 6.0, 2.0], device="cuda").bfloat16()[:, None].expand(4, d))
    rrv.embedding_grad([ids], [out], [table], "sum", accumulate=True)
    want = {v - 1: 1 + 4.0, 0: 2 + 4.0, 131_073: 3 + 6.0}
    for i, x in want.items():
        assert bool((table[i] == x).all())
    assert int(torch.count_nonzero(table)) == 3 * d
    rrv.embedding_grad([ids], [out], [table], "sum")
    assert int(torch.count_nonzero(table)) == 3 * d and bool((table[v - 1] == 4.0).all())


def test_embed_refusals_on_the_gpu():
    ids = [torch.zeros(4, dtype=torch.int32, device="cuda")]
    w, o = torch.zeros(10, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    for bad in ((ids * 2, [w], [o]), (ids, [w], [o[:3]]), (ids, [w], [o.bfloat16()]), (ids, [w], [o[:, :4].contiguous()]),
                (ids, [w.view(-1)], [o])):
        with pytest.raises(ValueError):
            rrv.embedding(*bad)
    with pytest.raises(rrv.RRError):
        rrv.embedding(ids, [w], [w[:4]])  # the output inside the table
    with pytest.raises(TypeError):
        rrv.embedding(rrv.RankSet([o[0]]), [w], [o])
    for bad in ((ids, [o[:3]], [w]), (ids, [o], [w[:, :4].contiguous()]), (ids, [o.view(-1)], [w])):
        with pytest.raises(ValueError):
            rrv.embedding_grad(*bad)
    with pytest.raises(rrv.RRError):
        rrv.embedding_grad(ids, [o], [w.bfloat16()])  # fp32 rows into a bf16 gradient
    with pytest.raises(rrv.RRError):
        rrv.embedding_grad(ids, [o], [w], op="max")
    with pytest.raises(rrv.RRError):
        rrv.embedding_grad(ids, [o], [w, w])  # the same replica twice


def test_wide_rows_many_ranks_and_far_ids():
    run_grad(2, 5, 3, 1 << 20, torch.bfloat16, "zipf", nout=1)
    run_grad(1, 40, 3, (1 << 18) + 1, torch.float16, "runs", accumulate=True)
    far = torch.tensor([1 << 40, -(1 << 40), 2, (1 << 31) - 1, 1 << 31, -1, 2, (1 << 63) - 1, -(1 << 63)], device="cuda")
    n, v, d = 64, 5, 24
    tables = [values(r, v * d, torch.float32).view(v, d) for r in range(n)]
    outs = [torch.full((len(far), d), 7.0, device="cuda") for _ in range(n)]
    rrv.embedding([far] * n, tables, outs, 3.0)
    for w, o in zip(tables, outs):
        want = torch.zeros(len(far), d, device="cuda")
        want[[2, 6]] = w[2] * 3.0
        assert torch.equal(o, want)
    g = [torch.full((v, d), 7.0, device="cuda") for _ in range(n)]
    rrv.embedding_grad([far] * n, outs, g, "sum")
    check_grad([far] * n, outs, g, g, v, 1.0, False)


def test_calls_on_two_streams_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    n, t, v, d = 2, 3000, 900, 136
    work = []
    for k in range(2):
        ids = [draw_ids(9 * k + r, t, v, torch.int32) for r in range(n)]
        x = [values(50 * k + r, t * d, torch.bfloat16).view(t, d) for r in range(n)]
        work.append((ids, x, [torch.empty(v, d, dtype=torch.bfloat16, device="cuda") for _ in range(n)]))
    torch.cuda.synchronize()
    for _ in range(5):
        for (ids, x, g), s in zip(work, streams):
            rrv.embedding_grad(ids, x, g, "avg", stream=s)
    torch.cuda.synchronize()
    for ids, x, g in work:
        check_grad(ids, x, g, g, v, 1.0 / n, False)


# ------------------------------------------------------- a step, as it is used

def step_inputs(n=4, t=300, v=700, d=72):
    ids = [torch.empty(t, dtype=torch.int32, device="cuda") for _ in range(n)]
    x = [torch.empty(t, d, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
    sizes = [d * d, d, 1001]
    grads = [[torch.empty(m, dtype=torch.bfloat16, device="cuda") for m in sizes] for _ in range(n)]
    table = values(1, v * d, torch.bfloat16).view(v, d)
    rest = [torch.empty(v, d, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
    return ids, x, grads, table, rest, rrv.BucketPlan(sizes, "bf16")


def fill(ids, grads, rest, v, seed):
    for r, i in enumerate(ids):
        i.copy_(draw_ids(seed + r, i.numel(), v, torch.int32))
        for k, g in enumerate(grads[r]):
            g.copy_(values(seed + 50 * r + k, g.numel(), torch.bfloat16))
        rest[r].fill_(float("nan"))  # written by the step


def one_step(ids, x, grads, table, rest, plan, out, limit=0.5):
    """Lookup; the rows themselves stand for what the backward pass hands back; the embedding's gradient into rank
    0's table; sync and clipping of everything."""
    rrv.embedding(ids, [table] * len(ids), x, scale=3.0)
    rrv.embedding_grad(ids, x, rest[:1], "avg", scale=3.0)
    return plan.all_reduce_clip(grads, limit, synced=[[w] for w in rest], eps=0.0, out=out)


def check_step(ids, x, before, grads, table, rest, out, limit=0.5):
    n, (v, d) = len(ids), table.shape
    flat = torch.cat([i.long() for i in ids])
    rows64 = torch.cat(x).double()
    total = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, flat, rows64) * (3.0 / n)
    mag = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, flat, rows64.abs()) * (3.0 / n)
    cnt = float(torch.bincount(flat).max())
    avg = [sum(rank[t].double() for rank in before) / n for t in range(len(before[0]))]
    want = norm64([total] + avg)
    # the embedding's gradient is rounded to bf16 once before the norm is taken: at most 2^-8 of its own norm
    assert abs(float(out) - want) <= (2.0 ** -8 * 1.01 + 40 * E) * want
    c = limit / float(out)
    for rank in grads:
        for g, a in zip(rank, avg):
            near_scaled(g, c * a, extra=c * 4 * E * 20)
    for w in rest:
        near_scaled(w, c * total, extra=c * (total.abs() * 2.0 ** -8 * 1.01 + (cnt + 2) * E * mag))
        assert torch.equal(w, rest[0])


def test_a_step_of_all_operators():
    ids, x, grads, table, rest, plan = step_inputs()
    fill(ids, grads, rest, table.shape[0], 7)
    before = [[g.clone() for g in rank] for rank in grads]
    out = torch.zeros((), device="cuda")
    one_step(ids, x, grads, table, rest, plan, out)
    check_step(ids, x, before, grads, table, rest, out)


def test_a_captured_step_replays_on_new_values():
    ids, x, grads, table, rest, plan = step_inputs()
    out = torch.zeros((), device="cuda")
    fill(ids, grads, rest, table.shape[0], 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one_step(ids, x, grads, table, rest, plan, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_step(ids, x, grads, table, rest, plan, out)
    for seed in (100, 200, 300):
        fill(ids, grads, rest, table.shape[0], seed)
        before = [[g.clone() for g in rank] for rank in grads]
        graph.replay()
        torch.cuda.synchronize()
        check_step(ids, x, before, grads, table, rest, out)


def test_embedding_calls_on_another_stream():
    s = torch.cuda.Stream()
    n, t, v, d = 2, 500, 300, 64
    ids = [draw_ids(r, t, v, torch.int64) for r in range(n)]
    table = values(1, v * d, torch.float32).view(v, d)
    outs = [torch.empty(t, d, device="cuda") for _ in range(n)]
    g = [torch.empty(v, d, device="cuda")]
    torch.cuda.synchronize()
    rrv.embedding(ids, [table] * n, outs, 0.5, stream=s)
    rrv.embedding_grad(ids, outs, g, "sum", stream=s.cuda_stream)
    s.synchronize()
    for i, o in zip(ids, outs):
        assert torch.equal(o, table[i] * 0.5)
    check_grad(ids, outs, g, g, v, 1.0, False)
