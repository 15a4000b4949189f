"""GPU: the filtered draw (cg_filter_sample) against the float64 oracle.

Picks are compared exactly.  A row whose nearest comparison of masses is
within 1e-8 of a tie may fall either way (a weight is held to 2^-41, a row of
2^17 of them to 2^-24 of its largest weight, and a sum of that many roundings
spreads as its root: 2^-32); such a row is not compared, and no more than one
row in 64 of a case may be one.
"""
import math

import numpy as np
import pytest

import logit_masking_amd as cg
from logit_masking_amd import workloads as W
from oracle import oracle as O
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
INF = math.inf
# a log-probability: half a float32 step, and the mass's relative error above
LP_REL, LP_ABS = 2.0 ** -24, 2.0 ** -28


def pack(allowed):
    """bool [B, V] -> int64 words [B, ceil(V / 64)]."""
    import torch
    B, V = allowed.shape
    pad = np.zeros((B, (V + 63) // 64 * 64), dtype=bool)
    pad[:, :V] = allowed
    w = np.packbits(pad, axis=1, bitorder="little").view(np.int64)
    return torch.from_numpy(np.ascontiguousarray(w)).cuda()


def run(x, mask, T, k, p, mp, u, vocab=None, stream=None):
    import torch
    B = x.shape[0]

    def dev(v, dt):
        return None if v is None else torch.tensor(np.asarray(v), dtype=dt).cuda()
    ids = torch.full((B + 1,), -77, dtype=torch.int32, device="cuda")
    lp = torch.full((B + 1,), -77.0, dtype=torch.float32, device="cuda")
    V = x.shape[1] if vocab is None else vocab
    cg.filter_sample(x, mask, dev(T, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(mp, torch.float32),
                     dev(u, torch.float32), cg.new_filter_workspace(B, V), ids, lp, vocab=vocab, stream=stream)
    torch.cuda.synchronize()
    assert int(ids[B]) == -77 and float(lp[B]) == -77.0  # nothing behind the last row
    return ids[:B].cpu().numpy(), lp[:B].cpu().numpy().astype(np.float64)


def check(x, allowed, T, k, p, mp, u, ids, lp, vocab=None, ties=None):
    B = x.shape[0]
    V = x.shape[1] if vocab is None else vocab
    xs = x[:, :V].float().cpu().numpy().astype(np.float64)
    near = 0
    for r in range(B):
        i, l, margin = O.filter_sample_row(xs[r], None if allowed is None else allowed[r], T[r], None if k is None else k[r],
                                           None if p is None else p[r], None if mp is None else mp[r], u[r])
        if margin < 1e-8:
            near += 1
            continue
        assert ids[r] == i, f"row {r}: {ids[r]} for {i} (margin {margin:.3g}, T {T[r]}, u {u[r]})"
        assert abs(lp[r] - l) <= LP_REL * abs(l) + LP_ABS, f"row {r}: logprob {lp[r]} for {l}"
    assert near <= (max(1, B // 64) if ties is None else ties), near


def settings(rng, B, kind):
    T = rng.uniform(0.3, 1.5, B).astype(np.float32)
    k = rng.integers(1, 120, B)
    p = rng.uniform(0.3, 0.99, B).astype(np.float32)
    mp = rng.uniform(0.001, 0.3, B).astype(np.float32)
    u = rng.random(B).astype(np.float32)
    u[u >= 1] = 0.5
    if kind == "mixed":
        T[rng.random(B) < 0.15] = 0
        k[rng.random(B) < 0.5] = rng.choice([0, -3, 1 << 30])
        p[rng.random(B) < 0.3] = rng.choice([1.0, 2.0])
        mp[rng.random(B) < 0.4] = rng.choice([0.0, -1.0])
        u[0] = 0.0
        return T, k, p, mp, u
    return (T, k if kind == "k" else None, p if kind == "p" else None, mp if kind == "minp" else None, u)


def make(rng, B, V, dtype, sigma=2.5, pad=0):
    import torch
    x = torch.from_numpy((rng.normal(size=(B, V + pad)) * sigma).astype(np.float32)).cuda()
    return x.to(getattr(torch, dtype))


def masks(rng, B, V):
    allowed = rng.random((B, V)) < rng.choice([0.9, 0.3, 0.02], size=(B, 1))
    if B > 2:
        allowed[1] = False
        allowed[2] = False
        allowed[2, rng.integers(V)] = True
    return allowed


SIZES = [1, 2, 63, 64, 65, 511, 1000, 2048, 4099, 8191, 32000, 50021]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", SIZES)
def test_sizes_and_filters(V, dtype):
    say("filter_sample", dtype, V)
    rng = np.random.default_rng(V)
    B = 12
    for kind in ("none", "k", "p", "minp", "mixed"):
        x = make(rng, B, V, dtype)
        s = settings(rng, B, kind)
        check(x, None, *s, *run(x, None, *s))
        allowed = masks(rng, B, V)
        s = settings(rng, B, kind)
        check(x, allowed, *s, *run(x, pack(allowed), *s))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [65536, 65537, 128256, 131072, 131080, 151936, 256000, 262144 + 9])
def test_large_vocabularies(V, dtype):
    say("filter_sample large", dtype, V)
    rng = np.random.default_rng(V + 1)
    B = 6
    for sigma, kind in ((3.0, "mixed"), (0.3, "p"), (1.0, "none")):
        x = make(rng, B, V, dtype, sigma)
        allowed = masks(rng, B, V)
        s = settings(rng, B, kind)
        check(x, None, *s, *run(x, None, *s))
        check(x, allowed, *s, *run(x, pack(allowed), *s))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V,pad,off", [(1000, 0, 1), (1001, 6, 3), (4096, 1, 0), (32000, 24, 5), (129, 0, 0)])
def test_strides_and_alignment(V, pad, off, dtype):
    """Rows whose storage starts anywhere and is longer than the vocabulary; what lies past it is never read as a logit."""
    import torch
    say("filter_sample stride", dtype, V, pad, off)
    rng = np.random.default_rng(V + pad)
    B = 7
    flat = torch.full((B * (V + pad) + off + 64,), INF, dtype=getattr(torch, dtype), device="cuda")
    x = flat[off:off + B * (V + pad)].view(B, V + pad)
    x[:, :V] = make(rng, B, V, dtype)
    allowed = masks(rng, B, V)
    words = pack(allowed)
    wide = torch.full((B, words.shape[1] + 3), -1, dtype=torch.int64, device="cuda")
    wide[:, :words.shape[1]] = words
    s = settings(rng, B, "mixed")
    check(x, allowed, *s, *run(x, wide, *s, vocab=V), vocab=V)
    s = settings(rng, B, "p")
    check(x, None, *s, *run(x, None, *s, vocab=V), vocab=V)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_ties(dtype):
    """Logits of few values: cuts and picks inside runs of equal candidates go by the lowest id."""
    import torch
    say("filter_sample ties", dtype)
    rng = np.random.default_rng(5)
    B = 48
    for V in (9, 300, 5000, 70001, 140000):
        x = torch.from_numpy(rng.integers(-3, 4, size=(B, V)).astype(np.float32) * 0.5)
        x[::5] = 1.25  # one value throughout
        x[1::5][x[1::5] == 0] = -0.0
        x[1::5, ::3] = 0.0
        x = x.cuda().to(getattr(torch, dtype))
        for kind in ("k", "p", "mixed", "none"):
            s = settings(rng, B, kind)
            if s[1] is not None:
                s[1][::2] = rng.integers(1, V + 2, size=s[1][::2].shape)
            allowed = masks(rng, B, V)
            check(x, allowed, *s, *run(x, pack(allowed), *s))
            check(x, None, *s, *run(x, None, *s))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_special_values(dtype):
    """-inf and NaN carry nothing, masked places may hold anything, the type's lowest value is a value, +inf takes all."""
    import torch
    say("filter_sample specials", dtype)
    rng = np.random.default_rng(11)
    B, V = 24, 3001
    x = make(rng, B, V, dtype)
    allowed = masks(rng, B, V)
    junk = torch.tensor(rng.choice([np.nan, np.inf, -np.inf], size=(B, V)).astype(np.float32)).cuda().to(x.dtype)
    off = torch.from_numpy(~allowed).cuda()
    low = torch.finfo(x.dtype).min
    x[off] = junk[off]
    x[3, ::2] = -INF
    x[4] = -INF
    x[5] = low
    x[6, 10:] = low
    x[7, ::3] = math.nan
    x[8] = math.nan
    x[9, 100] = INF
    x[9, 200] = INF
    x[10, :] = torch.finfo(x.dtype).max
    x[11, :] = torch.finfo(x.dtype).tiny / 2  # subnormal
    x[12, ::2] = -torch.finfo(x.dtype).tiny / 4
    for kind in ("none", "p", "k", "mixed"):
        s = settings(rng, B, kind)
        check(x, allowed, *s, *run(x, pack(allowed), *s))
        y = x.nan_to_num(nan=-INF, posinf=1.0, neginf=-INF)
        check(y, None, *s, *run(y, None, *s))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_settings_at_their_ends(dtype):
    say("filter_sample ends", dtype)
    rng = np.random.default_rng(13)
    V = 2500
    last = np.float32(1 - 2.0 ** -24)
    rows = []
    for T in (1e-3, 0.02, 1.0, 50.0, 1e30, INF, 0.0, -1.0, math.nan):
        for k, p, mp, u in ((0, 1.0, 0.0, 0.0), (0, 1.0, 0.0, last), (1, 1.0, 0.0, 0.7), (2, 0.999, 0.0, last), (V, 0.5, 0.0, last),
                            (V + 1, 1.0, 1.0, 0.9), (0, 1.0, 1.5, 0.9), (0, 0.0, 0.0, 0.9), (0, -1.0, 0.0, 0.9), (7, 1e-30, 0.0, last),
                            (0, math.nan, math.nan, 0.25), (V - 1, 1.0, 1e-30, last), (0, 1.0, 0.0, -0.5)):
            rows.append((T, k, p, mp, u))
    T, k, p, mp, u = (np.array(c) for c in zip(*rows))
    x = make(rng, len(rows), V, dtype)
    ids, lp = run(x, None, T, k, p, mp, u)
    # six of these rows compare masses within 1e-8 of a tie: equal weights (T = 1e30 and inf) cut at p = 0.5, V / 2 of them
    # exactly, or drawn at u = 0.25, V / 4 of them; and u = 1 - 2^-24 at T = 1, where the last 6e-8 of the mass is many ids'
    check(x, None, T, k, p, mp, u, ids, lp, ties=6)
    # 1 and above, and NaN, are numbers a caller should not give: the last candidate that has weight, and the first
    ids, _ = run(x[:3], None, [1.0] * 3, [5] * 3, None, None, [1.0, 7.0, math.nan])
    order = [O.ranked(x[r].float().cpu().numpy()) for r in range(3)]
    assert list(ids) == [order[0][4], order[1][4], order[2][0]]


def test_draws_follow_the_distribution():
    """An even grid of uniform numbers over one row: each id as often as its probability says, to one a border."""
    import torch
    say("filter_sample grid")
    rng = np.random.default_rng(17)
    B, V = 4096, 600
    row = make(rng, 1, V, "float32", 1.5)
    x = row.expand(B, V).contiguous()
    u = ((np.arange(B) + 0.5) / B).astype(np.float32)
    ids, _ = run(x, None, np.full(B, 0.9), np.full(B, 60), np.full(B, 0.95), np.full(B, 0.01), u)
    got = np.bincount(ids, minlength=V)
    v = row[0].cpu().numpy().astype(np.float64)
    w = np.exp((v - v.max()) / np.float32(0.9))
    keep = np.argsort(-v)[:60]
    before = np.cumsum(w[keep]) - w[keep]
    keep = keep[(before < np.float32(0.95) * w[keep].sum()) & (w[keep] >= np.float32(0.01))]
    want = np.zeros(V)
    want[keep] = w[keep] / w[keep].sum() * B
    assert np.all(np.abs(got - want) <= 1.001)


@pytest.mark.parametrize("cfg", [2, 3])
def test_workload_rows(cfg):
    """The decision-schema and tool-call workloads' logits under their own grammars' masks, then the walk of the picks."""
    import torch
    say("filter_sample workload", cfg)
    V0 = 20000
    blob, off = W.make_vocab(cfg, V0)
    g = cg.Grammar(W.spec_json(cfg), blob, off)
    V, B = g.V, 16
    st = g.new_states(B)
    g.init_state(st)
    steps = torch.zeros(B, dtype=torch.int32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    mask = torch.empty((B, g.W), dtype=torch.int64, device="cuda")
    ids = torch.empty(B, dtype=torch.int32, device="cuda")
    lp = torch.empty(B, dtype=torch.float32, device="cuda")
    rng = np.random.default_rng(cfg)
    for step in range(12):
        g.fill_bitmask(st, mask)
        x = W.make_logits(cfg, step, B, V, "cuda")
        T, k, p, mp, u = settings(rng, B, "mixed")
        f = lambda v: torch.tensor(v, dtype=torch.float32).cuda()  # noqa: E731
        cg.filter_sample(x, mask, f(T), torch.tensor(k, dtype=torch.int32).cuda(), f(p), f(mp), f(u), None, ids, lp)
        allowed = np.stack([O.unpack_mask(w, V) for w in mask.cpu().numpy().view(np.uint64)])
        check(x, allowed, T, k, p, mp, u, ids.cpu().numpy(), lp.cpu().numpy().astype(np.float64))
        picked = ids.cpu().numpy()
        g.advance(st, ids, steps, status)
        s = status.cpu().numpy()
        for r in range(B):
            assert (s[r] == cg.ROW_NOOP) == (picked[r] == -1)
            assert s[r] != cg.ROW_REJECTED  # a masked pick is always legal


def test_streams_graph_and_repeats():
    """The same bits on another stream, in a captured graph replayed with eager work between, and call after call."""
    import torch
    say("filter_sample streams and graph")
    rng = np.random.default_rng(23)
    B, V = 40, 32000
    xs = [make(rng, B, V, d) for d in ("bfloat16", "float32", "bfloat16")]
    allowed = masks(rng, B, V)
    words = pack(allowed)
    sets = [settings(rng, B, "mixed") for _ in xs]
    want = [run(x, words, *s) for x, s in zip(xs, sets)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, s, (i, l) in zip(xs, sets, want):
        got = run(x, words, *s, stream=side)
        assert np.array_equal(got[0], i) and np.array_equal(got[1], l)
    f = lambda v, d=torch.float32: torch.tensor(v, dtype=d).cuda()  # noqa: E731
    for dt in ("bfloat16", "float32"):
        x = torch.empty((B, V), dtype=getattr(torch, dt), device="cuda")
        T, p, mp, u = f(sets[0][0]), f(sets[0][2]), f(sets[0][3]), f(sets[0][4])
        k = f(sets[0][1], torch.int32)
        ws = cg.new_filter_workspace(B, V)
        ids = torch.empty(B, dtype=torch.int32, device="cuda")
        lp = torch.empty(B, dtype=torch.float32, device="cuda")
        x.copy_(xs[0])
        cg.filter_sample(x, words, T, k, p, mp, u, ws, ids, lp)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cg.filter_sample(x, words, T, k, p, mp, u, ws, ids, lp)
        for n in range(4):
            x.copy_(xs[n % 3])
            u.copy_(torch.rand(B, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            a, b = ids.clone(), lp.clone()
            ids.fill_(-9)
            cg.filter_sample(x, words, T, k, p, mp, u, ws, ids, lp)
            torch.cuda.synchronize()
            assert torch.equal(a, ids) and torch.equal(b, lp)


def test_binding_refusals():
    import torch
    say("filter_sample refusals")
    x = torch.zeros((4, 128), device="cuda", dtype=torch.bfloat16)
    m = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = [x, m, f, i, f, f, f, None, i, f.clone()]
    cg.filter_sample(*ok)
    for at, bad in ((0, x.half()), (0, x.t()), (0, x[0]), (1, m[:3]), (1, m[:, :1]), (1, m.int()), (2, f[:3]), (2, f.double()),
                    (3, i.long()), (4, f.cpu()), (5, f.repeat(2)[::2]), (6, f[:1]), (8, i[:2]), (8, i.long()), (9, f.half())):
        args = list(ok)
        args[at] = bad
        with pytest.raises(ValueError):
            cg.filter_sample(*args)
    for v in (0, 129, -1):
        with pytest.raises(ValueError):
            cg.filter_sample(*ok, vocab=v)
    torch.cuda.synchronize()
