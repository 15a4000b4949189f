"""The sampling and distillation operators over grammar-masked logits: cases, inputs, plain forms and exact values.

Three operators read rows of vocabulary logits under the packed token bitmask:
  sample   a draw with temperature, top-k, top-p and min-p from a given uniform number per row
  top      the K largest logits of a row and its log-normaliser (what a teacher records, or a reply's top log-probabilities)
  distill  the loss against a teacher's recorded top logits, and its gradient
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one interactive stream of the decision-schema workload: latency is all that counts
        {"name": "sample f32 1x32000", "op": "sample", "dtype": "f32", "rows": 1, "vocab": 32000, "pad": 0, "mask": "none",
         "sigma": 2.0, "filters": "top-k"},
        # a batch of the decision-schema workload, each request with settings of its own
        {"name": "sample f32 64x32000", "op": "sample", "dtype": "f32", "rows": 64, "vocab": 32000, "pad": 0, "mask": "grammar",
         "sigma": 2.0, "filters": "mixed"},
        # the tool-call workload's decode step
        {"name": "sample bf16 256x128256", "op": "sample", "dtype": "bf16", "rows": 256, "vocab": 128256, "pad": 0,
         "mask": "grammar", "sigma": 3.0, "filters": "mixed"},
        # the largest vocabulary, nothing masked, a flat distribution cut by its mass alone
        {"name": "sample bf16 512x256000", "op": "sample", "dtype": "bf16", "rows": 512, "vocab": 256000, "pad": 0,
         "mask": "none", "sigma": 1.0, "filters": "top-p"},
        # a few streams that ask for the top log-probabilities of each token
        {"name": "top20 bf16 4x128256", "op": "top", "dtype": "bf16", "rows": 4, "vocab": 128256, "pad": 0, "mask": "grammar",
         "sigma": 3.0, "k": 20},
        # an odd vocabulary in padded float32 rows
        {"name": "top5 f32 48x50021", "op": "top", "dtype": "f32", "rows": 48, "vocab": 50021, "pad": 11, "mask": "none",
         "sigma": 2.0, "k": 5},
        # a teacher's pass over recorded answers: its top logits at every position
        {"name": "top64 bf16 1024x151936", "op": "top", "dtype": "bf16", "rows": 1024, "vocab": 151936, "pad": 0,
         "mask": "grammar", "sigma": 3.0, "k": 64},
        # a short answer, both directions at once
        {"name": "distill both f32 24x32000", "op": "distill", "dtype": "f32", "rows": 24, "vocab": 32000, "pad": 0,
         "mask": "none", "sigma": 2.0, "k": 16, "tau": 2.0, "way": "both"},
        # validation: the loss alone
        {"name": "distill loss bf16 1024x256000", "op": "distill", "dtype": "bf16", "rows": 1024, "vocab": 256000, "pad": 0,
         "mask": "none", "sigma": 2.0, "k": 32, "tau": 1.0, "way": "loss"},
        # a backward pass after other work: the normalisers are in hand
        {"name": "distill grad f32 700x50021", "op": "distill", "dtype": "f32", "rows": 700, "vocab": 50021, "pad": 0,
         "mask": "none", "sigma": 2.0, "k": 100, "tau": 1.5, "way": "grad"},
        # a training step over the tool-call vocabulary under the grammar's masks
        {"name": "distill both bf16 2048x128256", "op": "distill", "dtype": "bf16", "rows": 2048, "vocab": 128256, "pad": 0,
         "mask": "grammar", "sigma": 3.0, "k": 64, "tau": 2.0, "way": "both"},
    ]


def draw(rng):
    op = rng.choice(["sample", "top", "distill"])
    vocab = int(round(math.exp(rng.uniform(math.log(512), math.log(256000)))))
    most = {"sample": 1024, "top": 2048, "distill": 4096}[op]
    rows = int(round(math.exp(rng.uniform(0.0, math.log(most)))))
    rows = max(1, min(rows, (2048 * 128256 if op == "distill" else 512 * 256000) // vocab))
    case = {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16"]), "rows": rows, "vocab": vocab,
            "pad": rng.choice([0, 0, rng.randrange(1, 40)]), "mask": rng.choice(["none", "grammar"]),
            "sigma": round(rng.uniform(0.5, 4.0), 3)}
    if case["dtype"] == "f32":
        case["rows"] = max(1, rows // 2)
    if op == "sample":
        case["filters"] = rng.choice(["top-k", "top-p", "min-p", "mixed", "mixed", "none"])
    elif op == "top":
        case["k"] = int(round(math.exp(rng.uniform(0.0, math.log(min(512, vocab))))))
    else:
        case["k"] = int(round(math.exp(rng.uniform(0.0, math.log(min(256, vocab))))))
        case["tau"] = round(rng.uniform(0.7, 4.0), 3)
        case["way"] = rng.choice(["loss", "grad", "both", "both"])
    return case


def _blocks(rows, vocab, most=1 << 27):
    """Row ranges of at most `most` logits: what the plain forms hold in 64 bits at a time."""
    step = max(1, most // vocab)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _grammar_masks(rows, vocab, gen):
    """Bitmask rows as a grammar leaves them: string interiors that allow nearly everything, keys that allow a part, structural
    positions that allow a few ids; the last row of a larger batch is finished and allows nothing."""
    words = (vocab + 63) // 64
    out = torch.empty((rows, words), dtype=torch.int64, device="cuda")
    share = torch.tensor([0.97, 0.97, 0.2, 0.001], device="cuda")
    keep = share[torch.randint(0, 4, (rows,), generator=gen, device="cuda")]
    if rows > 8:
        keep[-1] = -1.0
    shift = torch.arange(64, device="cuda", dtype=torch.int64)
    for a, b in _blocks(rows, words * 64, 1 << 25):
        bits = torch.rand((b - a, words * 64), generator=gen, device="cuda") < keep[a:b, None]
        bits[:, vocab:] = False
        first = torch.randint(0, vocab, (b - a,), generator=gen, device="cuda")
        bits[torch.arange(b - a, device="cuda"), first] |= keep[a:b] > 0
        out[a:b] = (bits.view(b - a, words, 64).to(torch.int64) << shift).sum(-1)
    return out


def _settings(kind, rows, gen):
    """Each row's temperature, top-k, top-p and min-p, as requests bring them; None where no row asks."""
    def rand():
        return torch.rand(rows, generator=gen, device="cuda")

    temperature = 0.4 + 0.9 * rand()
    top_k = torch.randint(1, 101, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    top_p = 0.7 + 0.29 * rand()
    min_p = 0.01 + 0.1 * rand()
    if kind == "mixed":
        on = torch.rand((4, rows), generator=gen, device="cuda")
        temperature = torch.where(on[0] < 0.1, torch.zeros_like(temperature), temperature)
        top_k = torch.where(on[1] < 0.5, torch.zeros_like(top_k), top_k)
        top_p = torch.where(on[2] < 0.4, torch.ones_like(top_p), top_p)
        min_p = torch.where(on[3] < 0.5, torch.zeros_like(min_p), min_p)
        return temperature, top_k, top_p, min_p
    return (temperature, top_k if kind == "top-k" else None, top_p if kind in ("top-p", "top-k") else None,
            min_p if kind == "min-p" else None)


def _allowed(mask, a, b, vocab):
    shift = torch.arange(64, device=mask.device, dtype=torch.int64)
    return ((mask[a:b, :, None] >> shift) & 1).view(b - a, -1)[:, :vocab].bool()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows, vocab = case["rows"], case["vocab"]
    dtype = _DTYPES[case["dtype"]]
    logits = torch.empty((rows, vocab + case["pad"]), dtype=dtype, device="cuda")
    for a, b in _blocks(rows, vocab + case["pad"]):
        logits[a:b] = torch.randn((b - a, vocab + case["pad"]), generator=gen, device="cuda") * case["sigma"]
    mask = _grammar_masks(rows, vocab, gen) if case["mask"] == "grammar" else None
    state = {"case": case, "logits": logits, "mask": mask}
    if case["op"] == "sample":
        state["settings"] = _settings(case["filters"], rows, gen)
        state["uniform"] = torch.rand(rows, generator=gen, device="cuda")
        state["ids"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        state["logprob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    elif case["op"] == "top":
        state["ids"] = torch.empty((rows, case["k"]), dtype=torch.int32, device="cuda")
        state["top"] = torch.empty((rows, case["k"]), dtype=torch.float32, device="cuda")
        state["lse"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    else:
        k, tau = case["k"], case["tau"]
        ids = torch.empty((rows, k), dtype=torch.int32, device="cuda")
        top = torch.empty((rows, k), dtype=torch.float32, device="cuda")
        lse = torch.empty(rows, dtype=torch.float32, device="cuda")
        for a, b in _blocks(rows, vocab, 1 << 26):
            x = logits[a:b, :vocab].float()
            t = 0.8 * x + 0.6 * case["sigma"] * torch.randn((b - a, vocab), generator=gen, device="cuda")
            if mask is not None:
                off = ~_allowed(mask, a, b, vocab)
                x.masked_fill_(off, -math.inf)
                t.masked_fill_(off, -math.inf)
            v, i = t.topk(k, dim=1)
            top[a:b] = v
            ids[a:b] = torch.where(v > -math.inf, i, -1).to(torch.int32)
            lse[a:b] = torch.logsumexp(x.double() / tau, dim=1).float()
        if rows > 8:  # a position behind the answer's end: nothing was recorded
            ids[rows // 2] = -1
        state["teacher_ids"], state["teacher"] = ids, top
        weight = torch.rand(rows, generator=gen, device="cuda") / rows
        if case["way"] == "grad":
            state["lse_in"], state["weight"] = lse, weight
        elif case["way"] == "both":
            state["weight"] = weight
        state["loss"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        state["lse"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        state["grad"] = torch.empty((rows, vocab), dtype=dtype, device="cuda") if case["way"] != "loss" else None
    if own:
        import logit_masking_amd as cg
        if case["op"] == "sample":
            state["workspace"] = cg.new_filter_workspace(rows, vocab)
        elif case["op"] == "top":
            state["workspace"] = cg.new_top_workspace(rows, vocab, case["k"])
    return state


def run(state):
    case = state["case"]
    return {"sample": _sample, "top": _top, "distill": _distill}[case["op"]](state, case)


def work(case):
    rows, vocab = case["rows"], case["vocab"]
    size = 2 if case["dtype"] == "bf16" else 4
    read = rows * vocab * size + (rows * ((vocab + 63) // 64) * 8 if case["mask"] != "none" else 0)
    if case["op"] == "sample":
        return {"bytes": read + rows * 28, "flops": 4 * rows * vocab}
    if case["op"] == "top":
        return {"bytes": read + rows * (8 * case["k"] + 4), "flops": 4 * rows * vocab}
    teacher = rows * case["k"] * 8
    if case["way"] == "loss":
        return {"bytes": read + teacher + rows * 8, "flops": 4 * rows * vocab}
    return {"bytes": read + teacher + rows * vocab * size + rows * 12, "flops": (4 if case["way"] == "grad" else 7) * rows * vocab}


# ---------------------------------------------------------------------------
# One pass of each operator.
# ---------------------------------------------------------------------------

def _masked(state, a, b, dtype):
    """Rows a..b of the logits, -inf where nothing may be drawn; both zeros are one value."""
    vocab = state["case"]["vocab"]
    x = state["logits"][a:b, :vocab].to(dtype) + 0.0
    if state["mask"] is not None:
        x = x.masked_fill(~_allowed(state["mask"], a, b, vocab), -math.inf)
    return x.masked_fill(x.isnan(), -math.inf)


def _sample(state, case):
    temperature, top_k, top_p, min_p = state["settings"]
    if own:
        import logit_masking_amd as cg
        cg.filter_sample(state["logits"], state["mask"], temperature, top_k, top_p, min_p, state["uniform"],
                         state["workspace"], state["ids"], state["logprob"], vocab=case["vocab"])
        return {"ids": state["ids"], "logprob": state["logprob"]}
    rows, vocab = case["rows"], case["vocab"]
    ids, logprob = [], []
    for a, b in _blocks(rows, vocab):
        x, order = torch.sort(_masked(state, a, b, torch.float64), dim=1, descending=True, stable=True)
        best = x[:, :1]
        t = temperature[a:b, None].double()
        greedy = ~(t > 0)
        t = torch.where(greedy, torch.ones_like(t), t)
        y = torch.where(x == best, torch.zeros_like(x), (x - best) / t)
        w = torch.where(x > -math.inf, y.exp(), torch.zeros_like(y))
        total = w.sum(1)
        rank = torch.arange(vocab, device=x.device)[None]
        keep = torch.ones_like(x, dtype=torch.bool)
        if top_k is not None:
            k = top_k[a:b, None]
            keep &= (rank < k) | (k <= 0)
        if top_p is not None:
            p = top_p[a:b, None].double()
            cut = w * keep
            upto = cut.cumsum(1)
            before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
            keep &= (before < p * cut.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
        if min_p is not None:
            keep &= (w >= min_p[a:b, None].double()) | (rank == 0)
        w = w * (keep & (~greedy | (rank == 0)))
        upto = w.cumsum(1)
        mass = upto[:, -1:]
        at = (upto <= state["uniform"][a:b, None].double() * mass).sum(1, keepdim=True)
        at = torch.minimum(at, (w > 0).sum(1, keepdim=True) - 1).clamp(min=0)
        none = ~(best > -math.inf)
        value = torch.where(greedy, -total[:, None].log(), y.gather(1, at) - mass.log())
        ids.append(torch.where(none, torch.full_like(at, -1), order.gather(1, at))[:, 0].to(torch.int32))
        logprob.append(torch.where(none, torch.zeros_like(value), value)[:, 0].float())
    return {"ids": torch.cat(ids), "logprob": torch.cat(logprob)}


def _top(state, case):
    if own:
        import logit_masking_amd as cg
        cg.top_logits(state["logits"], state["mask"], state["workspace"], state["ids"], state["top"], state["lse"],
                      vocab=case["vocab"])
        return {"ids": state["ids"], "logits": state["top"], "lse": state["lse"]}
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    ids, top, lse = [], [], []
    for a, b in _blocks(rows, vocab):
        x, order = torch.sort(_masked(state, a, b, torch.float32), dim=1, descending=True, stable=True)
        best = x[:, :1]
        some = best > -math.inf
        shift = torch.where(some, best, torch.zeros_like(best))
        total = (x - shift).exp().sum(1, keepdim=True)
        lse.append((shift + total.log())[:, 0])
        top.append(x[:, :k].clone())
        ids.append(torch.where(x[:, :k] > -math.inf, order[:, :k], -1).to(torch.int32))
    return {"ids": torch.cat(ids), "logits": torch.cat(top), "lse": torch.cat(lse)}


def _distill(state, case):
    way, tau, vocab = case["way"], case["tau"], case["vocab"]
    if own:
        import logit_masking_amd as cg
        if way == "grad":
            cg.distill_topk_grad(state["logits"], state["mask"], state["teacher_ids"], state["teacher"], tau, state["lse_in"],
                                 state["weight"], state["grad"], vocab=vocab)
            return {"grad": state["grad"]}
        if way == "loss":
            cg.distill_topk(state["logits"], state["mask"], state["teacher_ids"], state["teacher"], tau, state["loss"],
                            state["lse"], vocab=vocab)
            return {"loss": state["loss"], "lse": state["lse"]}
        cg.distill_topk(state["logits"], state["mask"], state["teacher_ids"], state["teacher"], tau, state["loss"], state["lse"],
                        weight=state["weight"], out_grad=state["grad"], vocab=vocab)
        return {"loss": state["loss"], "lse": state["lse"], "grad": state["grad"]}
    losses, lses = [], []
    grad = torch.empty_like(state["grad"]) if way != "loss" else None
    for a, b in _blocks(case["rows"], vocab):
        x = _masked(state, a, b, torch.float32) / tau
        ids = state["teacher_ids"][a:b].long()
        at = ids.clamp(0, vocab - 1)
        student = x.gather(1, at)
        t = torch.where((ids >= 0) & (ids < vocab) & (student > -math.inf), state["teacher"][a:b] / tau, -math.inf)
        high = t.max(1, keepdim=True).values
        some = high > -math.inf
        e = (t - torch.where(some, high, torch.zeros_like(high))).exp()
        p = e / torch.where(some, e.sum(1, keepdim=True), torch.ones_like(high))
        if way == "grad":
            lse = state["lse_in"][a:b, None]
        else:
            best = x.max(1, keepdim=True).values
            shift = torch.where(best > -math.inf, best, torch.zeros_like(best))
            lse = shift + (x - shift).exp().sum(1, keepdim=True).log()
            terms = torch.where(p > 0, p * (p.log() - student + lse), torch.zeros_like(p))
            losses.append(tau * tau * terms.sum(1))
            lses.append(lse[:, 0])
        if way != "loss":
            q = torch.where(some & (x > -math.inf), (x - lse).exp(), torch.zeros_like(x))
            q.scatter_add_(1, at, -p)
            grad[a:b] = (q * (tau * state["weight"][a:b, None])).to(grad.dtype)
    if way == "grad":
        return {"grad": grad}
    out = {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    return out if way == "loss" else {**out, "grad": grad}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, row by row.
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    rows, vocab = case["rows"], case["vocab"]

    def row(r):
        """Row r's logits in 64 bits and the ids that may be used, in rising order."""
        x = state["logits"][r, :vocab].double()
        ok = ~(x.isnan() | (x == -math.inf))
        if state["mask"] is not None:
            at = torch.arange(vocab, device=x.device)
            ok &= ((state["mask"][r][at // 64] >> (at % 64)) & 1) == 1
        return x, ok.nonzero()[:, 0]

    if case["op"] == "sample":
        temperature, top_k, top_p, min_p = (None if s is None else s.double().tolist() for s in state["settings"])
        uniform = state["uniform"].double().tolist()
        ids = torch.full((rows,), -1, dtype=torch.int32)
        logprob = torch.zeros(rows, dtype=torch.float64)
        for r in range(rows):
            x, use = row(r)
            if not len(use):
                continue
            v = x[use]
            if not temperature[r] > 0:
                ids[r] = int(use[v.argmax()]) if int((v == v.max()).sum()) == 1 else int(use[(v == v.max()).nonzero()[0, 0]])
                logprob[r] = float(v.max() - torch.logsumexp(v, 0))
                continue
            # the candidates from the best downwards; equal logits keep their ids' order
            by = torch.sort(0.0 - v, stable=True).indices
            z = v[by] / temperature[r]
            n = len(z)
            if top_k is not None and top_k[r] > 0:
                n = min(n, int(top_k[r]))
            mass = (z[:n] - z[0]).exp()
            if top_p is not None and top_p[r] < 1:
                goal = top_p[r] * float(mass.sum())
                n = max(1, 1 + int((mass.cumsum(0)[:-1] < goal).sum()))
                mass = mass[:n]
            if min_p is not None:
                n = max(1, int((mass >= min_p[r]).sum()))
                mass = mass[:n]
            run_ = mass.cumsum(0)
            j = int(torch.searchsorted(run_, uniform[r] * run_[-1], right=True))
            j = min(j, n - 1)
            ids[r] = int(use[by[j]])
            logprob[r] = float(z[j] - torch.logsumexp(z[:n], 0))
        return {"ids": ids, "logprob": logprob}
    if case["op"] == "top":
        k = case["k"]
        ids = torch.full((rows, k), -1, dtype=torch.int32, device="cuda")
        top = torch.full((rows, k), -math.inf, dtype=torch.float64, device="cuda")
        lse = torch.full((rows,), -math.inf, dtype=torch.float64, device="cuda")
        for r in range(rows):
            x, use = row(r)
            v = x[use]
            by = torch.sort(0.0 - v, stable=True).indices[:k]
            ids[r, :len(by)] = use[by].to(torch.int32)
            top[r, :len(by)] = v[by]
            lse[r] = torch.logsumexp(v, 0)
        return {"ids": ids, "logits": top, "lse": lse}
    tau, way = case["tau"], case["way"]
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    lse = torch.full((rows,), -math.inf, dtype=torch.float64, device="cuda")
    grad = torch.zeros((rows, vocab), dtype=torch.float64, device="cuda") if way != "loss" else None
    for r in range(rows):
        x, use = row(r)
        lse[r] = torch.logsumexp(x[use] / tau, 0)
        norm = state["lse_in"][r].double() if way == "grad" else lse[r]
        logq = torch.full((vocab,), -math.inf, dtype=torch.float64, device="cuda")
        logq[use] = x[use] / tau - norm
        ids = state["teacher_ids"][r].long()
        has = (ids >= 0) & (ids < vocab)
        has &= logq[ids.clamp(0, vocab - 1)] > -math.inf
        ids, t = ids[has], state["teacher"][r][has].double() / tau
        if not len(ids):
            continue
        logp = torch.log_softmax(t, 0)
        loss[r] = tau ** 2 * (logp.exp() * (logp - logq[ids])).sum()
        if way != "loss":
            g = logq.exp()
            g.index_add_(0, ids, -logp.exp())
            grad[r] = tau * float(state["weight"][r]) * g
    if way == "grad":
        return {"grad": grad}
    return {"loss": loss, "lse": lse} if way == "loss" else {"loss": loss, "lse": lse, "grad": grad}
