"""The global norm, clipping and the clipped bucket sync against their formulas
in 64 bits.

Tolerances, for values of type t with half a step u_t = torch.finfo(t).eps / 2
(fp32 2^-24, bf16 2^-8, fp16 2^-11):

* norm: a thread sums at most 64 squares in fp32 in four chains of at most 16
  fused steps and two joins, each off by at most 2^-24 of a sum of positive
  terms: 18 * 2^-24 of the sum of squares, half of that of its root, and one
  rounding to fp32: 10 * 2^-24.
* coefficient: the norm's 9 * 2^-24 and its own rounding: 10 * 2^-24; the
  product with an fp32 value one more: 11 * 2^-24; then the rounding to t, u_t
  (an fp32 result has only the product's), or half the smallest subnormal
  step where that is more.
* a fold of N ranks: N - 1 roundings, each at most 2^-24 of the sum of the
  magnitudes, and AVG's division one of the quotient.
"""
import math

import pytest
import torch

import ring_all_reduce_virtual_b200 as rrv

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SUB = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
GUARD = 64


class Guarded:
    """A tensor `off` elements past a 256-byte boundary between canaries."""

    def __init__(self, values, off=0):
        n = values.numel()
        self.big = torch.empty(GUARD * 2 + off + n, dtype=values.dtype, device="cuda")
        self.raw = self.big.view(torch.uint8)
        self.raw.fill_(0xA5)
        self.t = self.big[GUARD + off:GUARD + off + n]
        self.t.copy_(values)
        es = values.element_size()
        self.lo, self.hi = (GUARD + off) * es, (GUARD + off + n) * es

    def check(self):
        assert bool((self.raw[:self.lo] == 0xA5).all()) and bool((self.raw[self.hi:] == 0xA5).all())


def values(seed, n, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def near_norm(got, want):
    assert got.dtype == torch.float32 and abs(float(got) - want) <= 10 * E * want, (float(got), want)


def near_scaled(got, want, extra=0.0):
    """`got` is round(c * a) where want = c * a in 64 bits; extra: bound on c * (a's own error)."""
    dt = got.dtype
    tol = want.abs() * (11 * E + U[dt] * (1 + 2.0 ** -10)) + SUB[dt] + extra
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst {float((got.double() - want).abs().max())}"


# -------------------------------------------------------------------- norm

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("sizes", [[1], [0], [], [0, 1, 0], [7, 8, 9], [16384], [16385, 3], [70001, 5, 200003]])
@pytest.mark.parametrize("off", [0, 1, 5])
def test_norm_sizes_types_phases(dtype, sizes, off):
    ts = [Guarded(values(i, n, DT[dtype], 0.5), off * (i + 1) % 9) for i, n in enumerate(sizes)]
    got = rrv.grad_norm([g.t for g in ts], out=torch.full((), 7.0, device="cuda"))
    near_norm(got, norm64([g.t for g in ts]))
    for g in ts:
        g.check()


def test_norm_mixed_types_and_many_tensors():
    sizes = [(i * 37) % 301 for i in range(2500)]
    ts = [values(i, n, list(DT.values())[i % 3]) for i, n in enumerate(sizes)]
    got = rrv.grad_norm(ts)
    near_norm(got, norm64(ts))
    assert torch.equal(got, rrv.grad_norm(rrv.GradList(ts)))  # the same bits again


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-20, 1e18, 1e30])
def test_norm_over_the_whole_range(dtype, scale):
    t = (values(3, 5000, torch.float32).double() * scale).to(DT[dtype])
    near_norm(rrv.grad_norm([t]), norm64([t]))
    mixed = torch.cat([t, values(4, 5000, DT[dtype])])
    near_norm(rrv.grad_norm([mixed]), norm64([mixed]))


def test_norm_of_zeros_infinities_and_nans():
    z = torch.zeros(100003, device="cuda")
    assert float(rrv.grad_norm([z, -z])) == 0.0
    for dt in DT.values():
        t = values(5, 40000, dt)
        t[12345] = float("inf")
        assert float(rrv.grad_norm([t])) == math.inf
        t[20001] = float("nan")
        assert math.isnan(float(rrv.grad_norm([t])))
    huge = torch.full((4,), 3e38, device="cuda")  # the norm itself is above fp32's largest
    assert float(rrv.grad_norm([huge])) == math.inf


def test_norm_counts_repeated_tensors():
    t = values(6, 1001, torch.float32)
    near_norm(rrv.grad_norm([t, t]), math.sqrt(2) * norm64([t]))


# -------------------------------------------------------------------- clip

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n", [1, 2, 5])
@pytest.mark.parametrize("layout", ["aligned", "same", "mixed"])
@pytest.mark.parametrize("sizes", [[1, 40003, 8, 0, 5000], [260_000, 3, 2100], [1, 40003, 8, 0, 300_011], [5] * 49])
def test_clip_scales_rank_0s_copy_into_every_rank(dtype, n, layout, sizes):
    off = {"aligned": lambda r, t: 0, "same": lambda r, t: 3 * t + 1, "mixed": lambda r, t: r + t}[layout]
    ranks = [[Guarded(values(100 * r + t, m, DT[dtype], 0.1), off(r, t)) for t, m in enumerate(sizes)] for r in range(n)]
    src = [g.t.clone() for g in ranks[0]]
    want = norm64(src)
    got = rrv.clip_grads([[g.t for g in rank] for rank in ranks], 0.3 * want, eps=1e-3)
    near_norm(got, want)
    c = 0.3 * want / (want + 1e-3)
    for rank in ranks:
        for g, a in zip(rank, src):
            near_scaled(g.t, a.double() * c)
            assert torch.equal(g.t, ranks[0][rank.index(g)].t)
            g.check()


def test_clip_below_the_limit_changes_nothing():
    ts = [values(i, 3001, dt) for i, dt in enumerate(DT.values())]
    before = [t.clone() for t in ts]
    want = norm64(ts)
    for limit in (want * 1.001, math.inf):
        near_norm(rrv.clip_grads(ts, limit, eps=0.0), want)
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    rrv.clip_grads(ts, 0.0)
    assert all(not bool(t.any()) for t in ts)
    near_norm(rrv.clip_grads(ts, 1.0), 0.0)  # all zeros now
    near_norm(rrv.clip_grads([], 1.0), 0.0)


def test_clip_with_infinities_and_nans():
    t = values(8, 999, torch.float32)
    t[5] = -math.inf
    assert float(rrv.clip_grads([t], 1.0)) == math.inf
    assert math.isnan(float(t[5])) and int(torch.count_nonzero(t)) == 1  # 0 * inf; the finite values are 0
    t = values(8, 999, torch.bfloat16)
    t[5] = math.nan
    assert math.isnan(float(rrv.clip_grads([t], math.inf))) and bool(t.isnan().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[7, 1000], [300_001], [20_000_003]])  # one launch, two, by bulk copies
@pytest.mark.parametrize("limit", [1.0, 1e-3])
def test_clip_of_norms_near_and_above_the_largest_fp32(dtype, sizes, limit):
    """The coefficient is then below fp32's smallest normal number, where one
    fp32 would keep 2^-149 of it; the clipped values are ordinary ones."""
    ts = [(values(i, m, torch.float32).clamp(-3, 3).double() * 1e38).to(DT[dtype]) for i, m in enumerate(sizes)]
    src = [t.clone() for t in ts]
    want = norm64(src)
    got = rrv.clip_grads(ts, limit, eps=0.0)
    assert limit / want < 2.0 ** -126
    assert float(got) == math.inf if want > 1.01 * torch.finfo(torch.float32).max else abs(float(got) - want) <= 10 * E * want
    c = float(torch.tensor(limit)) / want
    for t, a in zip(ts, src):
        near_scaled(t, a.double() * c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 3, 4])
def test_clipped_sync_of_a_norm_above_the_largest_fp32(n, dtype):
    sizes = [5003, 900]
    ranks = [[(values(10 * r + t, m, torch.float32).clamp(-3, 3).double() * 2e37).to(DT[dtype]) for t, m in enumerate(sizes)]
             for r in range(n)]
    terms = [[rank[t].double() for rank in ranks] for t in range(len(sizes))]
    avg = [sum(x) / n for x in terms]
    mag = [sum(v.abs() for v in x) / n for x in terms]
    want = norm64(avg)
    assert want > torch.finfo(torch.float32).max
    assert float(rrv.BucketPlan(sizes, dtype).all_reduce_clip(ranks, 1.0, eps=0.0)) == math.inf
    # the norm's own error through the folds: at most the folds' share of the values
    fold = math.sqrt(sum(float((n * E * v).square().sum()) for v in mag)) / want
    for rank in ranks:
        for t, a, m in zip(rank, avg, mag):
            near_scaled(t, a / want, extra=m / want * n * E + a.abs() / want * fold)


def test_clip_many_tensors_in_several_launches():
    sizes = [(i * 53) % 97 + 1 for i in range(1200)]
    ranks = [[values(i + 7 * r, m, torch.bfloat16 if i % 4 else torch.float32) for i, m in enumerate(sizes)] for r in range(3)]
    src = [t.clone() for t in ranks[0]]
    want = norm64(src)
    near_norm(rrv.clip_grads(rrv.GradList(ranks), 0.5 * want, eps=0.0), want)
    for rank in ranks:
        for t, a in zip(rank, src):
            near_scaled(t, a.double() * 0.5)


def test_clip_offsets_past_32_bits():
    n = (1 << 32) + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 5, (1 << 31) + 1, (1 << 32) - 1, 1 << 32, n - 1], device="cuda")
    t[at] = 3.0
    want = 3.0 * math.sqrt(len(at))
    near_norm(rrv.clip_grads([t], 0.5 * want, eps=0.0), want)
    near_scaled(t[at], torch.full((len(at),), 1.5, dtype=torch.float64, device="cuda"))
    assert int(torch.count_nonzero(t)) == len(at)


# ------------------------------------------------------ the clipped bucket sync

SIZES = [100, 5000, 3, 777, 40001, 1, 16, 0, 9000]  # a small set: one launch where the phases allow it
MORE = SIZES + [300_007]  # above what one launch holds


def rank_grads(n, sizes, dtype, std=0.1, off=lambda r, t: 0):
    return [[Guarded(values(1000 * r + t, m, dtype, std), off(r, t)) for t, m in enumerate(sizes)] for r in range(n)]


def tensors(ranks):
    return [[g.t for g in rank] for rank in ranks]


LAYOUTS = {"aligned": lambda r, t: 0, "same": lambda r, t: t % 8, "mixed": lambda r, t: (r + 2 * t) % 7}


@pytest.mark.parametrize("n", [1, 2, 3, 4, 8, 16, 24])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("op", ["avg", "sum"])
@pytest.mark.parametrize("sizes", [SIZES, MORE])
def test_clipped_sync_without_a_limit_has_the_syncs_bits(n, dtype, op, sizes):
    for layout, off in LAYOUTS.items():
        a, b = rank_grads(n, sizes, DT[dtype], off=off), rank_grads(n, sizes, DT[dtype], off=off)
        plan = rrv.BucketPlan(sizes, dtype, 16384)
        plan.all_reduce_range(0, plan.num_buckets, tensors(a), op)
        plan.all_reduce_clip(tensors(b), math.inf, op)
        for r in range(n):
            for x, y in zip(a[r], b[r]):
                assert torch.equal(x.t, y.t), (layout, r)
                y.check()
    rrv.check_timeouts()


@pytest.mark.parametrize("n", [1, 2, 3, 8, 13])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("op", ["avg", "sum"])
@pytest.mark.parametrize("sizes,synced", [(SIZES, True), (SIZES, False), (MORE, True), (MORE, False)])
def test_clipped_sync_against_64_bits(n, dtype, op, sizes, synced):
    for layout, off in LAYOUTS.items():
        ranks = rank_grads(n, sizes, DT[dtype], off=off)
        rest = [[]] * n if not synced else rank_grads(1, [2000, 33], torch.float32) + rank_grads(n - 1, [2000, 33], torch.float32, std=9.0)
        div = n if op == "avg" and n > 1 else 1
        avg = [sum(rank[t].t.double() for rank in ranks) / div for t in range(len(sizes))]
        mag = [sum(rank[t].t.double().abs() for rank in ranks) / div for t in range(len(sizes))]
        src = [g.t.clone() for g in rest[0]]
        want = norm64(avg + src)
        plan = rrv.BucketPlan(sizes, dtype, 16384)
        got = plan.all_reduce_clip(rrv.GradSet(tensors(ranks)), 0.6 * want, op, synced=tensors(rest) if synced else None,
                                   eps=0.0)
        # the folds' errors are a share of the magnitudes; the norm's of them at most n * 2^-24 of their norm
        assert abs(float(got) - want) <= 10 * E * want + n * E * norm64(mag)
        for rank in ranks:
            for g, a, m in zip(rank, avg, mag):
                near_scaled(g.t, 0.6 * a, extra=n * E * (m + a.abs() * norm64(mag) / want))
                g.check()
        for rank in rest:
            for g, a in zip(rank, src):
                near_scaled(g.t, 0.6 * a.double(), extra=n * E * a.double().abs() * norm64(mag) / want)
                g.check()
    rrv.check_timeouts()


@pytest.mark.parametrize("n", [48, 64])
@pytest.mark.parametrize("dtype", list(DT))
def test_clipped_sync_of_many_ranks(n, dtype):
    sizes = [9000, 70_001, 5]
    a, b = rank_grads(n, sizes, DT[dtype]), rank_grads(n, sizes, DT[dtype])
    plan = rrv.BucketPlan(sizes, dtype, 16384)
    plan.all_reduce_range(0, plan.num_buckets, tensors(a), "avg")
    got = plan.all_reduce_clip(tensors(b), math.inf, "avg")
    assert abs(float(got) - norm64([g.t for g in a[0]])) <= 2.0 ** -8 * float(got)  # a is rounded to its type
    for ra, rb in zip(a, b):
        for x, y in zip(ra, rb):
            assert torch.equal(x.t, y.t)
            y.check()
    rrv.check_timeouts()


def test_clipped_sync_of_a_range_and_of_many_tensors():
    n, sizes = 8, [(i * 31) % 500 + 1 for i in range(700)]
    ranks = rank_grads(n, sizes, torch.bfloat16)
    before = [[g.t.clone() for g in rank] for rank in ranks]
    plan = rrv.BucketPlan(sizes, "bf16", 20000)
    first, count = 2, plan.num_buckets - 4
    t0, t1 = plan.info(first)[0], plan.info(first + count)[0]
    avg = [sum(rank[t].double() for rank in before) / n for t in range(t0, t1)]
    want = norm64(avg)
    got = plan.all_reduce_clip(tensors(ranks), 0.5 * want, first=first, count=count, eps=0.0)
    assert abs(float(got) - want) <= 30 * E * want
    for r in range(n):
        for t in range(len(sizes)):
            if t0 <= t < t1:
                near_scaled(ranks[r][t].t, 0.5 * avg[t - t0], extra=40 * E * 0.5)
            else:
                assert torch.equal(ranks[r][t].t, before[r][t])
            ranks[r][t].check()


@pytest.mark.parametrize("n", [1, 2, 3, 8])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_large_sets(n, dtype, layout):
    """Sets whose scaling runs by bulk copies: bits without a limit, values with one."""
    sizes = [40_000_003 // n, 17, 70_001, 0, 8192]
    off = LAYOUTS[layout]
    plan = rrv.BucketPlan(sizes, dtype)
    ranks = rank_grads(n, sizes, DT[dtype], off=off)
    other = [[g.t.clone() for g in rank] for rank in ranks]
    div = n if n > 1 else 1
    avg = [sum(rank[t].t.double() for rank in ranks) / div for t in range(len(sizes))]
    plan.all_reduce_range(0, plan.num_buckets, other, "avg")
    keep = [[g.t.clone() for g in rank] for rank in ranks]
    plan.all_reduce_clip(tensors(ranks), math.inf)
    for rank, want in zip(ranks, other):
        for g, w in zip(rank, want):
            assert torch.equal(g.t, w)
            g.check()
    for rank, k in zip(ranks, keep):
        for g, v in zip(rank, k):
            g.t.copy_(v)
    norm = norm64(avg)
    got = plan.all_reduce_clip(tensors(ranks), 0.3 * norm, eps=0.0)
    assert abs(float(got) - norm) <= (10 + 3 * n) * E * norm
    for rank in ranks:
        for g, a in zip(rank, avg):
            near_scaled(g.t, 0.3 * a, extra=0.3 * 0.1 * 6 * n * E)
            g.check()
    src = [g.t.clone() for g in ranks[0]]
    norm = norm64(src)
    near_norm(rrv.clip_grads(tensors(ranks), 0.7 * norm, eps=0.0), norm)
    for rank in ranks:
        for g, a in zip(rank, src):
            near_scaled(g.t, 0.7 * a.double())
            g.check()
    rrv.check_timeouts()


def test_clipped_sync_with_a_nan_and_with_a_large_sum():
    sizes = [500, 60]
    ranks = tensors(rank_grads(4, sizes, torch.float16))
    ranks[2][1][7] = math.nan
    plan = rrv.BucketPlan(sizes, "f16")
    assert math.isnan(float(plan.all_reduce_clip(ranks, 1.0)))
    assert all(bool(t.isnan().all()) for rank in ranks for t in rank)
    big = [[torch.full((m,), 6e4, dtype=torch.float16, device="cuda") for m in sizes] for _ in range(4)]
    got = plan.all_reduce_clip(big, 100.0, op="sum", eps=0.0)  # the sum leaves fp16's range, its clipped value does not
    want = 4 * float(torch.tensor(6e4, dtype=torch.float16)) * math.sqrt(560)
    near_norm(got, want)
    for rank in big:
        for t in rank:
            near_scaled(t, torch.full_like(t, 100.0 / math.sqrt(560), dtype=torch.float64))


# ------------------------------------------------- streams, graphs, arguments

def test_calls_on_another_stream_and_with_out():
    s = torch.cuda.Stream()
    ts = [values(i, 100003, torch.float32) for i in range(3)]
    want = norm64(ts)
    torch.cuda.synchronize()
    out = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    assert rrv.grad_norm(ts, out=out, stream=s) is out
    s.synchronize()
    near_norm(out[0], want)
    got = rrv.clip_grads(ts, 0.5 * want, eps=0.0, stream=s.cuda_stream)
    s.synchronize()
    near_norm(got, want)
    assert abs(norm64(ts) - 0.5 * want) <= 30 * E * want
    with pytest.raises(ValueError, match="out must be"):
        rrv.grad_norm(ts, out=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="out must be"):
        rrv.clip_grads(ts, 1.0, out=torch.zeros(1, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError):
        rrv.GradList([torch.zeros(3, dtype=torch.int32, device="cuda")])
    with pytest.raises(rrv.RRError):
        rrv.clip_grads([ts[0], ts[0]], 1.0)  # the same tensor twice


def test_captured_steps_replay_and_do_not_share_workspaces():
    n, sizes = 4, [3000, 70001, 12]
    plan = rrv.BucketPlan(sizes, "bf16", 1 << 20)
    sets = [tensors(rank_grads(n, sizes, torch.bfloat16)) for _ in range(2)]
    lists = [rrv.GradSet(s) for s in sets]
    outs = [torch.zeros((), device="cuda") for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    plan.all_reduce_clip(lists[0], math.inf)  # first use outside of a capture
    torch.cuda.synchronize()
    graphs = []
    for ls, out, s in zip(lists, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            plan.all_reduce_clip(ls, 0.25, out=out, eps=0.0)
        graphs.append(g)
    for step in range(3):
        want = []
        for k, ranks in enumerate(sets):
            new = rank_grads(n, sizes, torch.bfloat16, std=0.1 * (1 + step + 3 * k))
            for rank, src in zip(ranks, new):
                for t, g in zip(rank, src):
                    t.copy_(g.t + step)
            want.append([sum(rank[t].double() for rank in ranks) / n for t in range(len(sizes))])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for ranks, avg, out in zip(sets, want, outs):
            norm = norm64(avg)
            assert abs(float(out) - norm) <= 30 * E * norm
            for rank in ranks:
                for t, a in zip(rank, avg):
                    near_scaled(t, 0.25 / norm * a, extra=40 * E * 0.25 / norm * (step + 3.0))


def test_reducer_clips_when_its_step_ends():
    n, sizes = 4, [4096, 5, 30000, 64]
    plan = rrv.BucketPlan(sizes, "bf16", 8192)
    ranks = tensors(rank_grads(n, sizes, torch.bfloat16))
    synced = [[t.clone() for t in rank] for rank in ranks]
    plan.all_reduce_range(0, plan.num_buckets, synced, "avg")
    red = rrv.Reducer(plan, ranks, "avg")
    for limit in (None, 0.5):
        for rank, s in zip(ranks, synced):  # alike on every rank: their average is what they are
            for t, v in zip(rank, s):
                t.copy_(v)
        for t in range(len(sizes)):
            red.ready(t)
        got = red.finish() if limit is None else red.finish(max_norm=limit, eps=0.0)
        if limit is None:
            assert got is None
            continue
        want = norm64(synced[0])
        near_norm(got, want)
        for rank in ranks:
            for t, v in zip(rank, synced[0]):
                near_scaled(t, v.double() * (limit / want))


def run_child(script, **env):
    import os
    import subprocess
    import sys

    out = subprocess.run([sys.executable, "-c", script], env=dict(os.environ, **env), capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    return out.stdout


def test_first_calls_of_a_process_may_be_captured():
    """A fresh process whose first calls of these operators are captured into a graph."""
    out = run_child(r"""
import torch
import ring_all_reduce_virtual_b200 as rrv
g = [[torch.full((m,), float(r + 1), device="cuda").bfloat16() for m in (300_000, 7)] for r in range(4)]
plan = rrv.BucketPlan([300_000, 7], "bf16")
ids = [torch.tensor([1, 3, 1], dtype=torch.int32, device="cuda")]
w, o, dw = torch.ones(5, 64, device="cuda"), torch.zeros(3, 64, device="cuda"), torch.zeros(5, 64, device="cuda")
norm = torch.zeros((), device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    rrv.embedding(ids, [w], [o], 2.0)
    rrv.embedding_grad(ids, [o], [dw], "sum")
    rrv.grad_norm([dw], out=norm)
    plan.all_reduce_clip(g, 1.0)
    rrv.clip_grads([dw], 1.0)
graph.replay()
torch.cuda.synchronize()
want = (64 * (4.0 ** 2 + 2.0 ** 2)) ** 0.5
assert abs(float(norm) - want) < 1e-5 * want, float(norm)
assert abs(float(dw.double().norm()) - 1.0) < 1e-5
total = sum(float(t.double().square().sum()) for t in g[0]) ** 0.5
assert abs(total - 1.0) < 1e-2, total
rrv.check_timeouts()
print("CAPTURED")
""")
    assert "CAPTURED" in out


def test_timeouts_of_the_clipping_are_reported_and_the_context_survives():
    """RR_DEBUG_BULK_TIMEOUT=1 makes every first bounded wait run out: the tiles are skipped, the norm is NaN, the status
    says so, nothing partly folded is stored (a scaling without such waits makes every value NaN, as a NaN norm does),
    and the context still runs a call."""
    out = run_child(r"""
import torch
import ring_all_reduce_virtual_b200 as rrv
def report():
    try:
        rrv.check_timeouts()
        print("NO TIMEOUT")
    except rrv.RRError as e:
        print("TIMEOUT", e.status, "not seen to land: 0" in str(e))
for n, m in ((8, 1 << 20), (2, 1 << 23)):  # parked and folded twice, scaled by bulk copies
    plan = rrv.BucketPlan([m], "bf16")
    g = [[torch.full((m,), float(r + 1), device="cuda").bfloat16()] for r in range(n)]
    norm = plan.all_reduce_clip(g, 1.0)
    report()
    assert bool(norm.isnan())
    assert all(bool(((t[0] == r + 1) | t[0].isnan()).all()) for r, t in enumerate(g)), "a skipped tile was stored"
x = [torch.ones(1000, device="cuda")]
print("CONTEXT OK", float(rrv.grad_norm(x)) == 1000 ** 0.5 or abs(float(rrv.grad_norm(x)) - 1000 ** 0.5) < 1e-4)
""", RR_DEBUG_BULK_TIMEOUT="1")
    assert out.count("TIMEOUT 4 True") == 2 and "CONTEXT OK True" in out, out


def test_timeouts_of_the_second_pass_alone_make_the_norm_nan():
    """RR_DEBUG_BULK_TIMEOUT=2 makes only the scaling's bounded waits run out: every partial sum is whole, and the norm says
    all the same that the step is lost, also where a later launch of the call skips the tile; a call without such waits
    (the norm, a small clipping, a scaling by the threads) is as ever."""
    out = run_child(r"""
import torch
import ring_all_reduce_virtual_b200 as rrv
def report():
    try:
        rrv.check_timeouts()
        print("NO TIMEOUT")
    except rrv.RRError as e:
        print("RAN OUT", e.status, "not seen to land: 0" in str(e))
def ranks(n, m, dtype=torch.bfloat16):
    return [[torch.full((m,), float(r + 1), device="cuda").to(dtype)] for r in range(n)]
for n, m, d in ((8, 1 << 23, "bf16"), (2, 1 << 23, "bf16"), (3, 1 << 12, "f16"), (4, 1 << 23, "f32")):
    g = ranks(n, m, {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[d])
    norm = rrv.BucketPlan([m], d).all_reduce_clip(g, 1.0)  # parked, folded twice, the same with one tile's few, fp32
    assert bool(norm.isnan()), (n, m, float(norm))
    report()
big = ranks(2, 1 << 24, torch.float32)
assert bool(rrv.clip_grads(big, 1.0).isnan())
report()
# the buckets' scaling runs by the threads, or not at all; the synced list's by bulk copies
big = ranks(4, 1 << 24, torch.float32)
norm = rrv.BucketPlan([0], "f32").all_reduce_clip([[torch.empty(0, device="cuda")] for _ in range(4)], 1.0, synced=big)
assert bool(norm.isnan())
report()
one = [torch.ones(1000, device="cuda")]
assert abs(float(rrv.grad_norm(one)) - 1000 ** 0.5) < 1e-4 and abs(float(rrv.clip_grads(one, 1.0)) - 1000 ** 0.5) < 1e-4
g = ranks(4, 1 << 19, torch.float32)
assert abs(float(rrv.BucketPlan([1 << 19], "f32").all_reduce_clip(g, 1.0)) - 2.5 * 2 ** 9.5) < 1e-2
report()
""", RR_DEBUG_BULK_TIMEOUT="2")
    assert out.count("RAN OUT 4 True") == 6 and out.count("NO TIMEOUT") == 1, out


@pytest.mark.parametrize("n", [1, 2, 4])
def test_clipped_sync_with_an_empty_synced_list(n):
    plan = rrv.BucketPlan([5000, 3], "bf16")
    for empty in ([], [[]] * n, rrv.GradList([])):
        a = [[values(10 * r + t, m, torch.bfloat16) for t, m in enumerate((5000, 3))] for r in range(n)]
        b = [[t.clone() for t in rank] for rank in a]
        want, got = plan.all_reduce_clip(a, 0.5), plan.all_reduce_clip(b, 0.5, synced=empty)
        assert torch.equal(want, got) and all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


@pytest.mark.parametrize("n", [1, 2, 4])
def test_clipped_sync_of_a_grad_list(n):
    plan = rrv.BucketPlan([5000, 3], "bf16")
    a = [[values(10 * r + t, m, torch.bfloat16) for t, m in enumerate((5000, 3))] for r in range(n)]
    b = [[t.clone() for t in rank] for rank in a]
    gl = rrv.GradList(b if n > 1 else b[0])
    for limit in (0.5, 0.25):
        want, got = plan.all_reduce_clip(a, limit, "avg"), plan.all_reduce_clip(gl, limit, "avg")
        assert torch.equal(want, got) and all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))
    assert torch.equal(rrv.grad_norm(gl), rrv.grad_norm(b))


def test_debug_mode_takes_lists_with_empty_tensors():
    """RR_DEBUG=1 with tensors whose own pointer is NULL, in every call."""
    out = run_child(r"""
import torch
import ring_all_reduce_virtual_b200 as rrv
def grads(n):
    return [[torch.empty(0, device="cuda"), torch.full((500,), 2.0, device="cuda"), torch.empty(0, device="cuda")] for _ in range(n)]
assert grads(1)[0][0].data_ptr() == 0
want = 2.0 * 500 ** 0.5
print("NORM", abs(float(rrv.grad_norm(grads(1))) - want) < 1e-5 * want)
g = grads(2)
print("CLIP", abs(float(rrv.clip_grads(g, 1.0)) - want) < 1e-5 * want, abs(float(g[1][1].norm()) - 1.0) < 1e-5)
g, s = grads(3), grads(3)
norm = rrv.BucketPlan([0, 500, 0], "f32").all_reduce_clip(g, 1.0, synced=s)
print("SYNC", abs(float(norm) - want * 2 ** 0.5) < 1e-5 * want, abs(float(g[2][1].norm()) - 0.5 ** 0.5) < 1e-5)
""", RR_DEBUG="1")
    assert "NORM True" in out and "CLIP True True" in out and "SYNC True True" in out, out


def test_a_kept_norm_keeps_four_bytes():
    """Norms of calls without `out` have a storage of their own, not a piece of the call's workspace."""
    g = [[torch.ones(5000, device="cuda")] for _ in range(2)]
    kept = [rrv.grad_norm(g), rrv.clip_grads(g, 1.0), rrv.BucketPlan([5000], "f32").all_reduce_clip(g, 1.0)]
    for norm in kept:
        assert norm.shape == () and norm.dtype == torch.float32 and norm.untyped_storage().nbytes() == 4
    near_norm(kept[0], 5000 ** 0.5)  # as they were, with later calls' workspaces beside them
    near_norm(kept[1], 5000 ** 0.5)
