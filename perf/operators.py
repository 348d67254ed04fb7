"""The operators around the gradient sync that are measured: the global
gradient norm, clipping, the bucket sync with clipping, the embedding lookup
and the embedding's gradient over all ranks.

``listed()`` and ``draw()`` give the cases, ``prepare()`` a case's inputs on
the GPU, ``run()`` one pass -- the plain form in elementary torch operations, or
with ``own`` set the library's calls -- and ``exact()`` the same from the
definitions in 64 bits.

Gradients are laid out as one flat buffer per rank whose views are the
tensors, in the order in which a backward pass produces them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IDS = {"i32": torch.int32, "i64": torch.int64}
PAD_SHARE = 0.05  # of each rank's tokens: the padded end of a batch, id -1
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the norm of one small layer's gradients: a launch's latency
        dict(name="norm-layer64-f32", op="norm", dtype="f32", ranks=1, layers=1, width=64, vocab=0, odd=False),
        # a quarter of the 24-layer GPT-like model and its LM head, one rank, bf16
        dict(name="norm-6x2048-bf16", op="norm", dtype="bf16", ranks=1, layers=6, width=2048, vocab=32000, odd=False),
        # clipping a small model's fp32 gradients in place: fits in the L2 cache
        dict(name="clip-4x512-f32", op="clip", dtype="f32", ranks=1, layers=4, width=512, vocab=0, odd=False),
        # clipping four replicas of loss-scaled fp16 gradients of ragged sizes
        dict(name="clip-4r-3x1200-f16", op="clip", dtype="f16", ranks=4, layers=3, width=1200, vocab=0, odd=True),
        # the sync and clipping of a test-sized model on four ranks: latency
        dict(name="sync-clip-4r-1x128-f32", op="sync", dtype="f32", ranks=4, layers=1, width=128, vocab=0, odd=False),
        # three ranks, tensors of odd sizes at odd offsets
        dict(name="sync-clip-3r-2x1000-f16", op="sync", dtype="f16", ranks=3, layers=2, width=1000, vocab=0, odd=True),
        # eight ranks, four layers of the GPT-like model in buckets, the token embedding's gradient synced apart
        dict(name="sync-clip-8r-4x2048-bf16", op="sync", dtype="bf16", ranks=8, layers=4, width=2048, vocab=32000, odd=False),
        # one token's row, as a generating model asks for it
        dict(name="lookup-1-bf16", op="lookup", dtype="bf16", ids="i64", ranks=1, tokens=1, width=2048, vocab=32000),
        # one training sequence on each of eight ranks
        dict(name="lookup-8x2048-bf16", op="lookup", dtype="bf16", ids="i32", ranks=8, tokens=2048, width=2048, vocab=32000),
        # a short batch of an odd-sized fp32 model, added to the gradients that are there
        dict(name="embgrad-1x300-f32", op="embgrad", dtype="f32", grad_dtype="f32", ids="i64", ranks=1, outs=1, tokens=300,
             width=515, vocab=5003, accumulate=True, padding=3),
        # one sequence on each of eight ranks, the dense gradient of every replica written
        dict(name="embgrad-8x2048-bf16", op="embgrad", dtype="bf16", grad_dtype="bf16", ids="i32", ranks=8, outs=8, tokens=2048,
             width=2048, vocab=32000, accumulate=False, padding=-1),
        # a long batch on each of eight ranks, added to one fp32 main gradient
        dict(name="embgrad-8x8192-bf16", op="embgrad", dtype="bf16", grad_dtype="f32", ids="i32", ranks=8, outs=1, tokens=8192,
             width=2048, vocab=32000, accumulate=True, padding=-1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "clip", "sync", "sync", "lookup", "embgrad", "embgrad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("norm", "clip", "sync"):
        most = _total(listed()[6]) * (8 if op == "sync" else 4)
        while True:
            c = dict(op=op, dtype=dtype, ranks=1 if op == "norm" else rng.choice([1, 2, 4] if op == "clip" else [2, 3, 4, 6, 8]),
                     layers=_log(rng, 1, 24), width=_log(rng, 64, 2048), vocab=rng.choice([0, 0, _log(rng, 1000, 32000)]),
                     odd=rng.random() < 0.5)
            if _total(c) * c["ranks"] * (2 if dtype == "f32" else 1) <= most:
                return c
    while True:
        c = dict(op=op, dtype=dtype, ids=rng.choice(["i32", "i64"]), ranks=rng.choice([1, 1, 2, 3, 4, 8]), tokens=_log(rng, 1, 8192),
                 width=_log(rng, 64, 4096), vocab=_log(rng, 1000, 150000))
        if op == "embgrad":
            c.update(grad_dtype=rng.choice([dtype, "f32"]), outs=rng.choice([1, c["ranks"]]), accumulate=rng.random() < 0.5,
                     padding=rng.choice([-1, rng.randrange(50)]))
        tables = c["ranks"] if op == "lookup" else c["outs"]
        if tables * c["vocab"] * c["width"] <= 8 * 32000 * 2048 and c["ranks"] * c["tokens"] * c["width"] <= 8 * 8192 * 2048:
            return c


def _numels(c):
    """The gradient sizes of a GPT-like model's layers, last layer first; with a vocabulary the LM head in front."""
    d = c["width"]
    layer = [d, 4 * d * d, 4 * d, 4 * d * d, d, d, d, d * d, 3 * d, 3 * d * d, d, d]
    sizes = ([c["vocab"] * d] if c["vocab"] else []) + [d, d] + layer * c["layers"]
    return [m + 2 * i + 1 for i, m in enumerate(sizes)] if c["odd"] else sizes


def _synced(c):
    """Elements of the token embedding's gradient, which a step with a vocabulary syncs apart from the buckets."""
    return c["vocab"] * c["width"] if c["op"] == "sync" else 0


def _total(c):
    return sum(_numels(c)) + _synced(c)


def _std(c):
    return 0.1 if c["dtype"] == "f16" else 1e-3  # fp16 gradients come with a loss scale


def _max_norm(c):
    """0.7 of the norm that the gradients come to: the clipping clips."""
    return 0.7 * _std(c) * math.sqrt(_total(c) / (c["ranks"] if c["op"] == "sync" else 1))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed % (1 << 62))


def _rows(n, total, dtype, gen, std):
    """n rows of `total` normal values, each row starting on a 256-byte boundary."""
    stride = -(-total // 128) * 128
    rows = torch.empty(n, stride, dtype=dtype, device="cuda")
    return rows.normal_(0.0, std, generator=gen)[:, :total]


def _tokens(c, gen):
    """[ranks, tokens] ids whose frequency falls with their rank among the words, as text's does; the padded end is -1."""
    u = torch.rand(c["ranks"], c["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    word = (torch.exp(u * math.log(c["vocab"] + 1)) - 1).long().clamp_(0, c["vocab"] - 1)
    ids = torch.randperm(c["vocab"], generator=gen, device="cuda")[word]
    pad = int(PAD_SHARE * c["tokens"])
    if pad:
        ids[:, c["tokens"] - pad:] = -1
    return ids.to(IDS[c["ids"]])


def _views(flat, numels):
    return list(flat[: sum(numels)].split(numels))


def prepare(case, seed):
    c, gen = dict(case), _generator(seed)
    s = {"case": c}
    if c["op"] in ("norm", "clip", "sync"):
        numels = _numels(c)
        s["grads"] = _rows(c["ranks"], sum(numels), DTYPES[c["dtype"]], gen, _std(c))
        if c["op"] == "sync" and _synced(c):
            row = _rows(1, _synced(c), DTYPES[c["dtype"]], gen, _std(c) / math.sqrt(c["ranks"]))
            s["synced"] = row.repeat(c["ranks"], 1)
        if own:
            import ring_all_reduce_virtual_b200 as rrv

            views = [_views(g, numels) for g in s["grads"]]
            if c["op"] == "sync":  # a step's program keeps the plan and the marshalled gradients
                s["plan"] = rrv.BucketPlan(numels, c["dtype"])
                s["set"] = rrv.GradSet(views)
                s["rest"] = rrv.GradList([[r] for r in s["synced"]]) if "synced" in s else None
            else:
                s["set"] = rrv.GradList(views)
        return s
    s["tokens"] = _tokens(c, gen)
    V, D, dt = c["vocab"], c["width"], DTYPES[c["dtype"]]
    if c["op"] == "lookup":
        table = torch.empty(V, D, dtype=dt, device="cuda").normal_(0.0, 0.02, generator=gen)
        s["weights"] = table.repeat(c["ranks"], 1, 1)
        s["out"] = torch.empty(c["ranks"], c["tokens"], D, dtype=dt, device="cuda")
        names = ["tokens", "weights", "out"]
    else:
        s["dout"] = torch.empty(c["ranks"], c["tokens"], D, dtype=dt, device="cuda").normal_(0.0, _std(c), generator=gen)
        s["grads"] = torch.empty(c["outs"], V, D, dtype=DTYPES[c["grad_dtype"]], device="cuda").normal_(0.0, _std(c), generator=gen)
        names = ["tokens", "dout", "grads"]
    if own:
        import ring_all_reduce_virtual_b200 as rrv

        # int32 ids, tables and activations live in buffers that a program marshals once; int64 ids come anew
        s["sets"] = [list(s[n]) if s[n].dtype == torch.int64 else rrv.RankSet(list(s[n])) for n in names]
    return s


# --------------------------------------------------------------------- run

def _scale(c):
    return math.sqrt(c["width"])


def _norm(*parts):
    return torch.stack([p.float().square().sum(dtype=torch.float64) for p in parts]).sum().sqrt().float()


def _coef(norm, max_norm):
    return torch.clamp(max_norm / (norm + EPS), max=1.0)


def run(s):
    c = s["case"]
    return globals()[("_own_" if own else "_plain_") + c["op"]](s, c)


def _plain_norm(s, c):
    return {"norm": _norm(s["grads"][0])}


def _plain_clip(s, c):
    norm = _norm(s["grads"][0])
    s["grads"].copy_(s["grads"][0].float() * _coef(norm, _max_norm(c)))
    return {"grads": s["grads"], "norm": norm}


def _plain_sync(s, c):
    avg = s["grads"].sum(0, dtype=torch.float32) / c["ranks"]
    rest = [s["synced"]] if "synced" in s else []
    norm = _norm(avg, *[r[0] for r in rest])
    coef = _coef(norm, _max_norm(c))
    s["grads"].copy_(avg * coef)
    out = {"grads": s["grads"], "norm": norm}
    if rest:
        rest[0].copy_(rest[0][0].float() * coef)
        out["synced"] = rest[0]
    return out


def _plain_lookup(s, c):
    ids = s["tokens"].long()
    inside = (ids >= 0) & (ids < c["vocab"])
    at = torch.arange(c["ranks"], device="cuda")[:, None]
    rows = s["weights"][at, ids.clamp(0, c["vocab"] - 1)].float() * _scale(c)
    s["out"].copy_(torch.where(inside[..., None], rows, 0.0))
    return {"out": s["out"]}


def _plain_embgrad(s, c):
    ids = s["tokens"].long().reshape(-1)
    inside = (ids >= 0) & (ids < c["vocab"]) & (ids != c["padding"])
    sums = torch.zeros(c["vocab"] + 1, c["width"], device="cuda")
    sums.index_add_(0, torch.where(inside, ids, c["vocab"]), s["dout"].reshape(-1, c["width"]).float())
    grad = sums[:-1] * (_scale(c) / c["ranks"])
    s["grads"].copy_(s["grads"].float() + grad if c["accumulate"] else grad.expand(s["grads"].shape))
    return {"grads": s["grads"]}


def _own_norm(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    return {"norm": rrv.grad_norm(s["set"])}


def _own_clip(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    norm = rrv.clip_grads(s["set"], _max_norm(c), eps=EPS)
    return {"grads": s["grads"], "norm": norm}


def _own_sync(s, c):
    norm = s["plan"].all_reduce_clip(s["set"], _max_norm(c), op="avg", synced=s["rest"], eps=EPS)
    out = {"grads": s["grads"], "norm": norm}
    if "synced" in s:
        out["synced"] = s["synced"]
    return out


def _own_lookup(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    rrv.embedding(*s["sets"], scale=_scale(c))
    return {"out": s["out"]}


def _own_embgrad(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    rrv.embedding_grad(*s["sets"], op="avg", scale=_scale(c), accumulate=c["accumulate"], padding_idx=c["padding"])
    return {"grads": s["grads"]}


# -------------------------------------------------------------------- work

def _distinct(c, tokens):
    """The expected number of distinct ids among `tokens` unpadded ones."""
    edge = np.log(np.arange(1, c["vocab"] + 2)) / math.log(c["vocab"] + 1)
    return float(-np.expm1(tokens * np.log1p(-np.diff(edge))).sum())


def work(case):
    c = dict(case)
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("norm", "clip", "sync"):
        S, N, rest = sum(_numels(c)), c["ranks"], _synced(c)
        if c["op"] == "norm":
            return {"bytes": S * es + 4, "flops": 2 * S}
        if c["op"] == "clip":  # rank 0's copy in, every rank's out
            return {"bytes": (1 + N) * S * es + 4, "flops": 3 * S}
        return {"bytes": 2 * N * S * es + (1 + N) * rest * es + 4, "flops": (N + 4) * S + 3 * rest}
    D, V, ids = c["width"], c["vocab"], 4 if c["ids"] == "i32" else 8
    T = c["tokens"] - int(PAD_SHARE * c["tokens"])
    M = c["ranks"] * c["tokens"]
    if c["op"] == "lookup":
        return {"bytes": M * ids + c["ranks"] * _distinct(c, T) * D * es + M * D * es, "flops": M * D}
    rows, gs = c["ranks"] * T, 4 if c["grad_dtype"] == "f32" else 2
    wrote = 2 * _distinct(c, rows) if c["accumulate"] else V
    return {"bytes": M * ids + rows * D * es + c["outs"] * wrote * D * gs, "flops": rows * D}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] in ("norm", "clip", "sync"):
        parts = {"grads": s["grads"].double().mean(0) if c["op"] == "sync" else s["grads"][0].double()}
        if "synced" in s:
            parts["synced"] = s["synced"][0].double()
        norm = math.sqrt(sum(float(torch.dot(p, p)) for p in parts.values()))
        out = {"norm": torch.tensor(norm, dtype=torch.float64)}
        if c["op"] != "norm":
            shrink = min(1.0, _max_norm(c) / (norm + EPS))
            out.update({k: (p * shrink).expand(c["ranks"], -1) for k, p in parts.items()})
        return out
    D, V = c["width"], c["vocab"]
    ids = s["tokens"].cpu().numpy().astype(np.int64)
    if c["op"] == "lookup":
        table = torch.cat([s["weights"][0].double() * math.sqrt(D), torch.zeros(1, D, dtype=torch.float64, device="cuda")])
        return {"out": table[torch.from_numpy(np.where((ids < 0) | (ids >= V), V, ids)).cuda()]}
    flat = ids.reshape(-1)
    keep = np.flatnonzero((flat >= 0) & (flat < V) & (flat != c["padding"]))
    order = keep[np.argsort(flat[keep], kind="stable")]
    tokens, first = np.unique(flat[order], return_index=True)
    grad = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    if len(order):
        run = torch.zeros(len(order) + 1, D, dtype=torch.float64, device="cuda")
        torch.cumsum(s["dout"].reshape(-1, D)[torch.from_numpy(order).cuda()].double(), 0, out=run[1:])
        ends = torch.from_numpy(np.append(first, len(order))).cuda()
        grad[torch.from_numpy(tokens).cuda()] = run[ends[1:]] - run[ends[:-1]]
    grad *= math.sqrt(D) / c["ranks"]
    return {"grads": s["grads"].double() + grad if c["accumulate"] else grad.expand(c["outs"], -1, -1)}
