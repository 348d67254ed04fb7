"""The operators at the two ends of a data-parallel step that are measured:
the log probabilities of given tokens over all ranks' logits (with entropy and
top alternatives), their gradient, the orthogonalisation of matrices by
Newton-Schulz products, and the Muon step that updates every replica with it.

``listed()`` and ``draw()`` give the cases, ``prepare()`` a case's inputs on
the GPU, ``run()`` one pass -- the plain form in elementary torch operations, or
with ``own`` set the library's calls -- and ``exact()`` the same from the
definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IDS = {"i32": torch.int32, "i64": torch.int64}
PAD_SHARE = 0.05  # of each rank's tokens: the padded end of a batch, id -1
MASKED = 0.3      # of the vocabulary, where a grammar rules words out
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one generated token's logits, with what a chat service reports of it
        dict(name="logprob-1-bf16", op="logprob", dtype="bf16", ids="i64", ranks=1, tokens=1, vocab=32000, pitch=0, scale=1.0,
             entropy=True, top=5, masked=False),
        # one step of 64 generating requests under a grammar's mask, at a temperature
        dict(name="logprob-64-f16", op="logprob", dtype="f16", ids="i64", ranks=1, tokens=64, vocab=128000, pitch=0, scale=1.25,
             entropy=True, top=20, masked=True),
        # scoring short texts on three ranks: odd vocabulary, rows not on 16-byte boundaries
        dict(name="logprob-3x333-f32", op="logprob", dtype="f32", ids="i32", ranks=3, tokens=333, vocab=50003, pitch=0, scale=1.0,
             entropy=True, top=8, masked=False),
        # the loss of one training sequence on each of eight ranks
        dict(name="logprob-8x2048-bf16", op="logprob", dtype="bf16", ids="i32", ranks=8, tokens=2048, vocab=32000, pitch=0,
             scale=1.0, entropy=False, top=0, masked=False),
        # a short batch of an odd-sized fp32 model with an entropy bonus, the LM head's rows padded
        dict(name="logprob-grad-1x300-f32", op="logprob_grad", dtype="f32", ids="i64", ranks=1, tokens=300, vocab=5003, pitch=5,
             scale=0.5, entropy=True, top=0, masked=False),
        # the start of the backward pass of one sequence on each of eight ranks
        dict(name="logprob-grad-8x2048-bf16", op="logprob_grad", dtype="bf16", ids="i32", ranks=8, tokens=2048, vocab=32000,
             pitch=0, scale=1.0, entropy=False, top=0, masked=False),
        # one small layer's matrices: latency
        dict(name="ortho-1x128-f32", op="ortho", dtype="f32", ranks=1, layers=1, width=128, odd=False),
        # ragged fp16 matrices
        dict(name="ortho-2x1000-f16", op="ortho", dtype="f16", ranks=1, layers=2, width=1000, odd=True),
        # four layers of the GPT-like model
        dict(name="ortho-4x2048-bf16", op="ortho", dtype="bf16", ranks=1, layers=4, width=2048, odd=False),
        # the update of a test-sized model on four ranks: latency
        dict(name="muon-4r-1x128-f32", op="muon", dtype="f32", ranks=4, layers=1, width=128, odd=False),
        # three ranks, matrices of odd sizes at odd offsets
        dict(name="muon-3r-1x700-f32", op="muon", dtype="f32", ranks=3, layers=1, width=700, odd=True),
        # eight ranks, four layers of the GPT-like model
        dict(name="muon-8r-4x2048-bf16", op="muon", dtype="bf16", ranks=8, layers=4, width=2048, odd=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprob", "logprob", "logprob_grad", "ortho", "muon"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("ortho", "muon"):
        most = work(listed()[8])["flops"]
        while True:
            c = dict(op=op, dtype=dtype, ranks=1 if op == "ortho" else rng.choice([1, 2, 3, 4, 8]), layers=_log(rng, 1, 24),
                     width=_log(rng, 64, 2048), odd=rng.random() < 0.5)
            if work(c)["flops"] <= most:
                return c
    while True:
        c = dict(op=op, dtype=dtype, ids=rng.choice(["i32", "i64"]), ranks=rng.choice([1, 1, 2, 3, 4, 8]), tokens=_log(rng, 1, 2048),
                 vocab=_log(rng, 1000, 150000), pitch=rng.choice([0, 0, rng.randrange(1, 64)]),
                 scale=rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.0), 3)]), entropy=rng.random() < 0.5,
                 top=rng.choice([0, 0, rng.randrange(1, 33)]) if op == "logprob" else 0, masked=rng.random() < 0.25)
        size = c["ranks"] * c["tokens"] * (c["vocab"] + c["pitch"]) * (2 if dtype == "f32" else 1)
        if size <= 8 * 2048 * 32000 // (4 if c["top"] else 1):
            return c


def _shapes(c):
    """The matrices of a GPT-like layer as they are kept, (rows, columns) each: QKV, projection, and the MLP's two."""
    d = c["width"]
    shapes = [(3 * d, d), (d, d), (4 * d, d), (d, 4 * d)]
    return [(r + 2 * i + 1, q + (3 * i) % 5) for i, (r, q) in enumerate(shapes)] if c["odd"] else shapes


def _total(c):
    return c["layers"] * sum(r * q for r, q in _shapes(c))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed % (1 << 62))


def _flat(n, total, dtype):
    """n rows of `total` values, each row starting on a 256-byte boundary."""
    return torch.empty(n, -(-total // 128) * 128, dtype=dtype, device="cuda")[:, :total]


def _stacks(flat, c):
    """One flat buffer as its layers' matrices, stacked by kind: a view [layers, rows, columns] of each."""
    sizes = [c["layers"] * r * q for r, q in _shapes(c)]
    return [p.view(c["layers"], r, q) for p, (r, q) in zip(flat[: sum(sizes)].split(sizes), _shapes(c))]


def _fill(flat, c, gen, std):
    """Gradients as they are: a few strong directions over the noise of a batch."""
    for stack in _stacks(flat, c):
        layers, r, q = stack.shape
        k = max(1, min(r, q) // 16)
        left = torch.randn(layers, r, k, generator=gen, device="cuda")
        right = torch.randn(layers, k, q, generator=gen, device="cuda")
        stack.copy_((torch.randn(layers, r, q, generator=gen, device="cuda") + left @ right / math.sqrt(k)) * std)


def prepare(case, seed):
    c, gen = dict(case), _generator(seed)
    s = {"case": c}
    if c["op"] in ("ortho", "muon"):
        total = _total(c)
        s["grads"] = _flat(1, total, DTYPES[c["dtype"]])
        _fill(s["grads"][0], c, gen, 1e-3)
        s["out"] = torch.empty_like(s["grads"]) if c["op"] == "ortho" else None
        if c["op"] == "muon":
            s["momenta"] = _flat(1, total, torch.float32)
            _fill(s["momenta"][0], c, gen, 3e-3)
            s["params"] = _flat(c["ranks"], total, DTYPES[c["dtype"]])
            s["params"][0].copy_(torch.randn(total, generator=gen, device="cuda") * 0.02)
            s["params"][1:] = s["params"][0]
        if own:  # a step's program keeps its tensors' lists
            import ring_all_reduce_virtual_b200 as rrv

            lists = {k: [[m for stack in _stacks(row, c) for m in stack] for row in s[k]]
                     for k in ("grads", "out", "momenta", "params") if s.get(k) is not None}
            s["lists"] = {k: rrv.MatrixList(v) for k, v in lists.items()}
        return s
    n, T, V = c["ranks"], c["tokens"], c["vocab"]
    wide = torch.empty(n, T, V + c["pitch"], dtype=DTYPES[c["dtype"]], device="cuda").normal_(0.0, 2.0, generator=gen)
    s["logits"] = wide[:, :, :V]  # columns that pad the LM head hold what they hold
    ids = torch.randint(V, (n, T), generator=gen, device="cuda")
    s["logits"].scatter_add_(2, ids[..., None], torch.rand(n, T, 1, generator=gen, device="cuda").mul_(12.0).to(wide.dtype))
    if c["masked"]:
        out = torch.rand(n, T, V, generator=gen, device="cuda") < MASKED
        out.scatter_(2, ids[..., None], False)
        s["logits"].masked_fill_(out, -math.inf)
    pad = int(PAD_SHARE * T)
    if pad:
        ids[:, T - pad:] = -1
    s["tokens"] = ids.to(IDS[c["ids"]])
    if c["op"] == "logprob_grad":
        count = n * (T - pad)
        s["dlogprob"] = torch.rand(n, T, generator=gen, device="cuda").add_(0.5).mul_(-1.0 / count)
        s["dentropy"] = torch.rand(n, T, generator=gen, device="cuda").mul_(-0.1 / count) if c["entropy"] else None
        s["out"] = torch.empty(n, T, V, dtype=wide.dtype, device="cuda")
        x = s["logits"].double() * c["scale"] if n * T * V < 1 << 27 else None
        rows = [x[r] if x is not None else s["logits"][r].double() * c["scale"] for r in range(n)]
        s["lse"] = torch.stack([torch.logsumexp(r, -1) for r in rows]).float()
        s["entropy"] = None
        if c["entropy"]:
            s["entropy"] = torch.stack([-(torch.special.xlogy(p, p)).sum(-1) for p in (torch.softmax(r, -1) for r in rows)]).float()
        del x, rows
    if own:
        s["logits_list"], s["tokens_list"] = list(s["logits"]), list(s["tokens"])
        if c["op"] == "logprob_grad":
            s["out_list"] = list(s["out"])
    return s


# --------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    return globals()[("_own_" if own else "_plain_") + c["op"]](s, c)


def _target(s, c):
    """The tokens' ids, 0 in the place of those outside the vocabulary, and which are inside."""
    ids = s["tokens"].long()
    inside = (ids >= 0) & (ids < c["vocab"])
    return torch.where(inside, ids, 0), inside


def _plain_logprob(s, c):
    z = s["logits"].float() * c["scale"]
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1)
    lse = m[..., 0] + torch.log(total)
    ids, inside = _target(s, c)
    out = {"logprob": torch.where(inside, z.gather(2, ids[..., None])[..., 0] - lse, 0.0), "lse": lse}
    if c["entropy"]:
        out["entropy"] = torch.log(total) - (e * torch.where(e > 0, z - m, 0.0)).sum(-1) / total
    if c["top"]:  # ties go to the lowest id: the value's order above, the id's below it in one whole number
        bits = s["logits"].float().add(0.0).view(torch.int32).long()
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32) - torch.arange(c["vocab"], device="cuda")
        top = torch.topk(order, c["top"], -1).indices
        out["top_id"] = top.int()
        out["top_logprob"] = z.gather(2, top) - lse[..., None]
    return out


def _plain_logprob_grad(s, c):
    z = s["logits"].float() * c["scale"]
    logp = z - s["lse"][..., None]
    p = torch.exp(logp)
    ids, inside = _target(s, c)
    g = torch.where(inside, s["dlogprob"], 0.0)
    d = -g[..., None] * p
    d.scatter_add_(2, ids[..., None], g[..., None])
    if c["entropy"]:
        d -= s["dentropy"][..., None] * p * torch.where(p > 0, logp + s["entropy"][..., None], 0.0)
    s["out"].copy_(d * c["scale"])
    return {"dlogits": s["out"]}


def _newton_schulz(g):
    """The polynomial's steps on a stack of matrices [layers, rows, columns] in fp32."""
    x = g.float()
    x = x / (x.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt().float() + EPS)
    if x.shape[1] > x.shape[2]:
        return _iterate(x.transpose(1, 2)).transpose(1, 2)
    return _iterate(x)


def _iterate(x):
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


def _plain_ortho(s, c):
    for g, o in zip(_stacks(s["grads"][0], c), _stacks(s["out"][0], c)):
        o.copy_(_newton_schulz(g))
    return {"out": s["out"]}


def _factor(rows, cols):
    return LR * math.sqrt(max(1.0, rows / cols))


def _plain_muon(s, c):
    g = s["grads"][0].float()
    s["momenta"][0].mul_(MOMENTUM).add_(g)
    u = g + MOMENTUM * s["momenta"][0]
    w = s["params"][0].float() * (1.0 - LR * DECAY)
    for uk, wk, (rows, cols) in zip(_stacks(u, c), _stacks(w, c), _shapes(c)):
        wk.sub_(_newton_schulz(uk), alpha=_factor(rows, cols))
    s["params"].copy_(w.expand(c["ranks"], -1))
    return {"params": s["params"], "momenta": s["momenta"]}


def _own_logprob(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    r = rrv.token_logprobs(s["logits_list"], s["tokens_list"], scale=c["scale"], entropy=c["entropy"], top_k=c["top"])
    out = {"logprob": r.logprob, "lse": r.lse}
    if c["entropy"]:
        out["entropy"] = r.entropy
    if c["top"]:
        out["top_id"], out["top_logprob"] = r.top_id, r.top_logprob
    return out


def _own_logprob_grad(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    rrv.token_logprobs_grad(s["logits_list"], s["tokens_list"], s["lse"], s["dlogprob"], entropy=s["entropy"],
                            dentropy=s["dentropy"], scale=c["scale"], outs=s["out_list"])
    return {"dlogits": s["out"]}


def _own_ortho(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    rrv.orthogonalize(s["lists"]["grads"], s["lists"]["out"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    return {"out": s["out"]}


def _own_muon(s, c):
    import ring_all_reduce_virtual_b200 as rrv

    rrv.muon_step(s["lists"]["params"], s["lists"]["grads"], s["lists"]["momenta"], lr=LR, momentum=MOMENTUM, nesterov=True,
                  weight_decay=DECAY, steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    return {"params": s["params"], "momenta": s["momenta"]}


# -------------------------------------------------------------------- work

def work(case):
    c = dict(case)
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("ortho", "muon"):
        total, flops = _total(c), 0
        for r, q in _shapes(c):
            m, n = min(r, q), max(r, q)
            # symmetric products by half; the cheaper of the iteration on the matrix and the one on its Gram matrix
            each = min(STEPS * (3 * m * m * n + m**3), 3 * m * m * n + (4 * STEPS - 3) * m**3)
            flops += c["layers"] * each
        if c["op"] == "ortho":
            return {"bytes": 2 * total * es, "flops": flops}
        return {"bytes": total * (es + 8 + es + c["ranks"] * es), "flops": flops}
    M, V = c["ranks"] * c["tokens"], c["vocab"]
    small = M * ((4 if c["ids"] == "i32" else 8) + 8 + (4 if c["entropy"] else 0) + 8 * c["top"])
    if c["op"] == "logprob":
        return {"bytes": M * V * es + small, "flops": M * V * (5 if c["entropy"] else 3)}
    return {"bytes": 2 * M * V * es + small, "flops": M * V * (7 if c["entropy"] else 4)}


# ------------------------------------------------------------------- exact

def _exact_row(x, ids, c):
    """One rank's rows in 64 bits: (logprob, lse, entropy, probabilities, log probabilities)."""
    logp = torch.log_softmax(x, -1)
    lse = torch.logsumexp(x, -1)
    p = torch.softmax(x, -1)
    known = (ids >= 0) & (ids < c["vocab"])
    mine = torch.zeros(len(ids), dtype=torch.float64, device="cuda")
    mine[known] = logp[known].gather(1, ids[known][:, None])[:, 0]
    return mine, lse, -torch.special.xlogy(p, p).sum(-1), p, logp


def _polar(g):
    """The same polynomial as a matrix Q of the smaller Gram matrix's side, X Q or Q X: every step multiplies the singular
    values s by a + b s^2 + c s^4, a polynomial of the Gram matrix, which the step takes from L to L (a + b L + c L^2)^2."""
    a, b, c = COEFFICIENTS
    x = g / (torch.linalg.matrix_norm(g, keepdim=True) + EPS)
    tall = x.shape[1] >= x.shape[2]
    lam = x.mT @ x if tall else x @ x.mT
    eye = torch.eye(lam.shape[-1], dtype=torch.float64, device="cuda")
    q = eye
    for _ in range(STEPS):
        step = a * eye + b * lam + c * torch.linalg.matrix_power(lam, 2)
        q = step @ q
        lam = step @ lam @ step
    return x @ q if tall else q @ x


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] in ("ortho", "muon"):
        g = s["grads"][0].double()
        out = {}
        if c["op"] == "muon":
            m = MOMENTUM * s["momenta"][0].double() + g
            g = g + MOMENTUM * m
            out["momenta"] = m[None]
        o = torch.cat([_polar(stack).reshape(-1) for stack in _stacks(g, c)])
        if c["op"] == "ortho":
            return {"out": o[None]}
        shares = torch.cat([torch.full((c["layers"] * r * q,), _factor(r, q), dtype=torch.float64, device="cuda") for r, q in _shapes(c)])
        w = s["params"][0].double() * (1.0 - LR * DECAY) - shares * o
        return {"params": w.expand(c["ranks"], -1), **out}
    ids = s["tokens"].long()
    rows = {"logprob": [], "lse": [], "entropy": [], "top_id": [], "top_logprob": [], "dlogits": []}
    for r in range(c["ranks"]):
        raw = s["logits"][r].double()
        mine, lse, entropy, p, logp = _exact_row(raw * c["scale"], ids[r], c)
        rows["logprob"].append(mine)
        rows["lse"].append(lse)
        rows["entropy"].append(entropy)
        if c["top"]:
            host = raw.cpu().numpy()
            best = torch.from_numpy(np.argsort(-host, axis=-1, kind="stable")[:, : c["top"]].copy()).cuda()
            rows["top_id"].append(best.int())
            rows["top_logprob"].append(logp.gather(1, best))
        if c["op"] == "logprob_grad":
            known = (ids[r] >= 0) & (ids[r] < c["vocab"])
            g = s["dlogprob"][r].double() * known
            d = -g[:, None] * p
            d[known, ids[r][known]] += g[known]
            if c["entropy"]:
                d -= s["dentropy"][r].double()[:, None] * (torch.special.xlogy(p, p) + p * entropy[:, None])
            rows["dlogits"].append(d * c["scale"])
    if c["op"] == "logprob_grad":
        return {"dlogits": torch.stack(rows["dlogits"])}
    names = ["logprob", "lse"] + (["entropy"] if c["entropy"] else []) + (["top_id", "top_logprob"] if c["top"] else [])
    return {k: torch.stack(rows[k]) for k in names}
