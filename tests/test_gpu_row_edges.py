"""GPU: the row operators at the ends of their ranges: rows masked by the
type's lowest value, denormals, runs of neighbours, more rows than the device
has units, the longest vocabulary, rows more than 2^31 elements apart, two
streams at once.  Tolerances are those of the operators' own tests."""
import math

import numpy as np
import pytest

import logit_masking_amd as cg
from oracle import oracle as O
from tests import test_gpu_distill as D
from tests import test_gpu_filter_sample as F
from tests import test_gpu_top_logits as T
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
INF = math.inf
DTYPES = ["bfloat16", "float32"]


def top(x, allowed, k, **kw):
    T.check(x, allowed, k, T.run(x, None if allowed is None else F.pack(allowed), k, **kw), **kw)


def draw(x, allowed, s, **kw):
    F.check(x, allowed, *s, *F.run(x, None if allowed is None else F.pack(allowed), *s, **kw), **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [40, 5000, 70001, 140000, 270000])
def test_rows_masked_by_the_lowest_value(V, dtype):
    """Programs mask by writing the lowest value: few others, one, none; all of them are still candidates, in their order."""
    import torch
    say("lowest value", dtype, V)
    rng = np.random.default_rng(V)
    B = 8
    x = F.make(rng, B, V, dtype)
    low = torch.finfo(x.dtype).min
    for r, n in enumerate((0, 1, 2, 3, 7, 15, 30, V - 1)):
        drop = rng.permutation(V)[:V - n]
        x[r, torch.from_numpy(drop).cuda()] = low
    allowed = F.masks(rng, B, V)
    for k in (1, 5, 20, 1024):
        top(x, None, k)
        top(x, allowed, k)
    for kind in ("none", "k", "p", "minp", "mixed"):
        s = F.settings(rng, B, kind)
        if s[1] is not None:
            s[1][::2] = V  # more than the others
        draw(x, None, s)
        draw(x, allowed, s)
    # at these temperatures the lowest values weigh as much as the others
    hot = np.array([1e30, 3e38, INF, 1e38, 2e30, INF, 1e35, 1e37])
    u = rng.random(B).astype(np.float32) * np.float32(0.999)
    draw(x, None, (hot, None, None, None, u))
    draw(x, allowed, (hot, np.full(B, 9), np.full(B, 0.7), np.full(B, 0.001), u))


def test_denormals():
    """Float32 logits around zero: denormals keep their order, and the two zeros are one value."""
    import torch
    say("denormals")
    rng = np.random.default_rng(3)
    B, V = 9, 4001
    tiny = rng.choice([0.0, -0.0, 1.0, -1.0, 2.0, -2.0, 3.0, 30000.0, -30000.0, 65536.0, -65536.0, -65535.0, 131072.0, -131072.0],
                      size=(B, V))
    x = np.ldexp(tiny, -149).astype(np.float32)
    assert np.array_equal(x.astype(np.float64), np.ldexp(tiny, -149))
    x[3] = -np.abs(x[3])
    x[4][x[4] > 0] = 0
    x[5, ::2] = rng.normal(size=(V + 1) // 2)
    x[6] = np.ldexp(rng.integers(-200, 200, V).astype(np.float64), -149).astype(np.float32)
    x[7] = np.ldexp(rng.integers(-200, -1, V).astype(np.float64), -149).astype(np.float32)
    x = torch.from_numpy(x).cuda()
    allowed = F.masks(rng, B, V)
    for k in (1, 3, 64, 1000):
        top(x, None, k)
        top(x, allowed, k)
    for kind in ("k", "none", "mixed", "p"):
        s = F.settings(rng, B, kind)
        draw(x, None, s)
        draw(x, allowed, s)


def test_neighbours_in_float32():
    """Float32 logits that agree in their upper bits, or hold bfloat16 values: cuts and picks among many in one bin."""
    import torch
    say("neighbours")
    rng = np.random.default_rng(4)
    B = 10
    for V in (900, 5000, 66000):
        x = torch.from_numpy((1.0 + rng.integers(0, 60000, size=(B, V)) * 2.0 ** -23).astype(np.float32)).cuda()
        x[1] = -x[1]
        x[2, 5:] = 1.0
        x[3] = F.make(rng, 1, V, "bfloat16")[0].float()
        x[4] = F.make(rng, 1, V, "bfloat16", 0.05)[0].float()
        x[5, ::2] = F.make(rng, 1, V, "float32")[0, ::2]
        x[6] = 1.0 + F.make(rng, 1, V, "float32", 0.001)[0]
        x[7] = 1e4 + F.make(rng, 1, V, "float32", 0.001)[0]
        allowed = F.masks(rng, B, V)
        for kind in ("none", "k", "p", "minp", "mixed"):
            s = F.settings(rng, B, kind)
            if s[1] is not None:
                s[1][::2] = rng.integers(1, V + 2, size=s[1][::2].shape)
            draw(x, None, s)
            draw(x, allowed, s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,B", [(700, 1500), (32000, 601), (50021, 420), (128256, 140), (151936, 120), (256000, 70)])
def test_rows_do_not_know_each_other(V, B, dtype):
    """Many rows give the bits that a few of them give; some of them against the oracle."""
    import torch
    say("many rows", dtype, V, B)
    rng = np.random.default_rng(B)
    x = F.make(rng, 40, V, dtype)
    x = x[torch.arange(B, device="cuda") % 40].contiguous()  # rows come again under other settings
    allowed = F.masks(rng, 40, V)[np.arange(B) % 40]
    words = F.pack(allowed)
    s = F.settings(rng, B, "mixed")
    few = 17
    for mask in (None, words):
        whole = F.run(x, mask, *s)
        for at in range(0, B, few * 7):
            to = min(at + few, B)
            part = F.run(x[at:to], None if mask is None else mask[at:to], *(v[at:to] for v in s))
            assert np.array_equal(part[0], whole[0][at:to]) and np.array_equal(part[1], whole[1][at:to])
        n = min(B, 6)
        F.check(x[:n], None if mask is None else allowed[:n], *(v[:n] for v in s), whole[0][:n], whole[1][:n])
        whole = T.run(x, mask, 9)
        for at in range(0, B, few * 7):
            to = min(at + few, B)
            part = T.run(x[at:to], None if mask is None else mask[at:to], 9)
            assert all(np.array_equal(a, b[at:to]) for a, b in zip(part, whole))
        T.check(x[:n], None if mask is None else allowed[:n], 9, tuple(v[:n] for v in whole))
    ids, t = D.teacher(rng, x, None, 8, V)
    w = rng.uniform(0.1, 2, B).astype(np.float32)
    for way in ("loss", "both", "grad"):
        got = D.run(x, words, ids, t, 1.5, way, w)
        # few rows may take another kernel than many, whose float32 sums are in another order: both are held to the oracle
        for n in (3, B):
            part = got if n == B else D.run(x[:n], words[:n], ids[:n], t[:n], 1.5, way, w[:n])
            D.check(x[:3].double().cpu().numpy(), allowed[:3], ids[:3], t[:3], 1.5, w[:3],
                    [None if g is None else g[:3] for g in part], dtype, way == "grad")


@pytest.mark.parametrize("dtype,V", [(d, v + n) for d, limits in (("float32", (16381, 32765, 65533)),
                                                                  ("bfloat16", (32761, 65529, 131065, 163833)))
                                     for v in limits for n in (0, 1)])
def test_at_the_variants_limits(dtype, V):
    """Rows as long as a variant takes them, and one id longer, starting as far off 16 bytes as they can and on them."""
    import torch
    say("limits", dtype, V)
    rng = np.random.default_rng(V)
    B = 3
    for off, pad in ((3 if dtype == "float32" else 7, 0), (0, -V % 8), (1, 2)):
        flat = torch.full((B * (V + pad) + off + 64,), INF, dtype=getattr(torch, dtype), device="cuda")
        x = flat[off:off + B * (V + pad)].view(B, V + pad)
        x[:, :V] = F.make(rng, B, V, dtype)
        x[:, V - 1] = 9.5  # the last id is one that counts
        allowed = F.masks(rng, B, V)
        allowed[0, V - 1] = True
        s = F.settings(rng, B, "p")
        draw(x, allowed, s, vocab=V)
        top(x, allowed, 6, vocab=V)
        draw(x, None, s, vocab=V)
        top(x, None, 6, vocab=V)
        ids, t = D.teacher(rng, x, None, 8, V)
        ids[0, 4] = V - 1
        w = np.array([0.5, 1.0, 2.0], dtype=np.float32)
        xs = x[:, :V].double().cpu().numpy()
        for way in ("both", "grad"):
            D.check(xs, allowed, ids, t, 1.0, w, D.run(x, F.pack(allowed), ids, t, 1.0, way, w, vocab=V), dtype, way == "grad")


@pytest.mark.parametrize("dtype", DTYPES)
def test_longest_vocabulary(dtype):
    import torch
    say("longest vocabulary", dtype)
    rng = np.random.default_rng(9)
    B, V = 3, cg.MAX_ROW_VOCAB
    x = F.make(rng, B, V, dtype, 3.0)
    x[1, ::3] = torch.finfo(x.dtype).min
    x[2] = 0.5
    allowed = rng.random((B, V)) < 0.6
    s = F.settings(rng, B, "p")
    draw(x, allowed, s)
    draw(x, None, (s[0], np.array([50, V - 1, V]), s[2], None, s[4]))
    top(x, None, 1024)
    top(x, allowed, 33)
    ids, t = D.teacher(rng, x, None, 8, V)
    w = np.array([0.5, 1.0, 2.0], dtype=np.float32)
    xs = x.double().cpu().numpy()
    for way in ("both", "grad"):
        D.check(xs, allowed, ids, t, 1.0, w, D.run(x, F.pack(allowed), ids, t, 1.0, way, w), dtype, way == "grad")
    for call in (lambda v: F.run(v, None, *s), lambda v: T.run(v, None, 4),
                 lambda v: D.run(v, None, ids, t, 1.0, "loss")):
        with pytest.raises(ValueError):
            call(torch.zeros((B, V + 1), dtype=x.dtype, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_far_apart(dtype):
    """Rows of a tensor whose later ones start past 2^31 elements."""
    import torch
    say("rows far apart", dtype)
    rng = np.random.default_rng(10)
    B, V, step = 3, 1203, 1_100_000_001
    store = torch.empty(2 * step + V + 64, dtype=getattr(torch, dtype), device="cuda")
    x = store.as_strided((B, V), (step, 1))
    x.copy_(F.make(rng, B, V, dtype))
    allowed = rng.random((B, V)) < 0.5
    s = F.settings(rng, B, "p")
    draw(x, allowed, s)
    top(x, allowed, 12)
    ids, t = D.teacher(rng, x, None, 8, V)
    w = np.array([0.5, 1.0, 2.0], dtype=np.float32)
    xs = x.double().cpu().numpy()
    got = D.run(x, F.pack(allowed), ids, t, 1.0, "both", w)
    D.check(xs, allowed, ids, t, 1.0, w, got, dtype)
    # the gradient in the student's place
    D.check(xs, allowed, ids, t, 1.0, w, D.run(x, F.pack(allowed), ids, t, 1.0, "both", w, inplace=True), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("way", ["both", "grad"])
def test_gradient_in_place(way, dtype):
    """The gradient over the student's logits, of few long rows and of more than a row per unit."""
    say("gradient in place", way, dtype)
    rng = np.random.default_rng(13)
    for B, V in ((2, 131075), (5, 50021), (300, 9000)):
        x = F.make(rng, B, V, dtype)
        allowed = F.masks(rng, B, V)
        ids, t = D.teacher(rng, x, None, 40, V)
        w = rng.uniform(0.1, 2, B).astype(np.float32)
        xs = x.double().cpu().numpy()
        apart = D.run(x, F.pack(allowed), ids, t, 1.5, way, w)
        D.check(xs, allowed, ids, t, 1.5, w, apart, dtype, way == "grad")
        same = D.run(x, F.pack(allowed), ids, t, 1.5, way, w, inplace=True)
        assert all(np.array_equal(a, b) for a, b in zip(apart, same))


@pytest.mark.parametrize("dtype", DTYPES)
def test_two_streams_at_once(dtype):
    """Calls that run beside each other, on rows and outputs of their own, give what they give alone."""
    import torch
    say("two streams", dtype)
    rng = np.random.default_rng(12)
    B, V, k = 90, 32000, 10
    f = lambda v, d=torch.float32: torch.tensor(v, dtype=d).cuda()  # noqa: E731
    sets = []
    for _ in range(2):
        x = F.make(rng, B, V, dtype)
        s = F.settings(rng, B, "mixed")
        ids, t = D.teacher(rng, x, None, 8, V)
        sets.append((x, F.pack(F.masks(rng, B, V)), (f(s[0]), f(s[1], torch.int32), f(s[2]), f(s[3]), f(s[4])),
                     torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda()))

    def outs():
        i32 = lambda *n: torch.full(n, -9, dtype=torch.int32, device="cuda")  # noqa: E731
        f32 = lambda *n: torch.full(n, -9.0, device="cuda")  # noqa: E731
        return [i32(B), f32(B), i32(B, k), f32(B, k), f32(B), f32(B), f32(B), torch.zeros(B, V, dtype=sets[0][0].dtype, device="cuda")]

    def calls(a, o, stream):
        x, m, s, ids, t = a
        cg.filter_sample(x, m, *s, None, o[0], o[1], stream=stream)
        cg.top_logits(x, m, None, o[2], o[3], o[4], stream=stream)
        cg.distill_topk(x, m, ids, t, 2.0, o[5], o[6], weight=s[0], out_grad=o[7], stream=stream)
    want = []
    for a in sets:
        o = outs()
        calls(a, o, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append(o)
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[outs() for _ in range(4)] for _ in sets]
    torch.cuda.synchronize()
    for n in range(4):
        for a, st, o in zip(sets, streams, got):
            calls(a, o[n], st)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o in g:
            assert all(torch.equal(p, q) for p, q in zip(w, o))


@pytest.mark.parametrize("dtype", DTYPES)
def test_mask_bits_past_the_vocabulary(dtype):
    """Ones in a mask's last word behind the vocabulary are no candidates; logits there are not read."""
    import torch
    say("mask bits past the vocabulary", dtype)
    rng = np.random.default_rng(14)
    B = 5
    for V in (1, 65, 1003, 8200):
        wide = torch.full((B, V + 70), INF, dtype=getattr(torch, dtype), device="cuda")
        wide[:, :V] = F.make(rng, B, V, dtype)
        ones = torch.full((B, (V + 63) // 64), -1, dtype=torch.int64, device="cuda")
        s = F.settings(rng, B, "none")
        F.check(wide, None, *s, *F.run(wide, ones, *s, vocab=V), vocab=V)
        T.check(wide, None, 70, T.run(wide, ones, 70, vocab=V), vocab=V)
        ids, t = D.teacher(rng, wide, None, 6, V)
        D.check(wide[:, :V].double().cpu().numpy(), None, ids, t, 1.0, s[0],
                D.run(wide, ones, ids, t, 1.0, "both", s[0], vocab=V), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_rows_between_the_logits_rows(dtype):
    """One tensor holds each row's logits and, behind them, its gradient."""
    import torch
    say("gradient between", dtype)
    rng = np.random.default_rng(15)
    B, V = 6, 2003
    both = torch.zeros((B, 2 * V + 3), dtype=getattr(torch, dtype), device="cuda")
    x, g = both[:, :V], both[:, V:2 * V]
    x.copy_(F.make(rng, B, V, dtype))
    kept = x.clone()
    ids, t = D.teacher(rng, x, None, 8, V)
    i, t2 = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda()
    w = torch.full((B,), 0.75, device="cuda")
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    cg.distill_topk(x, None, i, t2, 2.0, loss, lse, weight=w, out_grad=g)
    want = torch.empty((B, V), dtype=x.dtype, device="cuda")
    cg.distill_topk(kept, None, i, t2, 2.0, loss, lse, weight=w, out_grad=want)
    torch.cuda.synchronize()
    assert torch.equal(x, kept) and torch.equal(g, want) and not both[:, 2 * V:].any()
    with pytest.raises(ValueError, match="overlap"):
        cg.distill_topk(x, None, i, t2, 2.0, loss, lse, weight=w, out_grad=both[:, V - 1:2 * V - 1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_temperatures_at_their_ends(dtype):
    """Distillation at the smallest and largest temperatures: all on the largest logit, and all alike."""
    import torch
    say("distill temperatures", dtype)
    rng = np.random.default_rng(16)
    B, V, k = 4, 1500, 6
    x = F.make(rng, B, V, dtype)
    ids, t = D.teacher(rng, x, None, k, V)
    w = np.full(B, 1.0, dtype=np.float32)
    xs = x.double().cpu().numpy()
    for tau in (1e-30, 1e30):
        loss, lse, grad = D.run(x, None, ids, t, tau, "both", w)
        assert np.isfinite(grad).all()
        if tau > 1:  # q = 1 / V everywhere, p alike over a row's entries: tau (q - p) to float32's precision
            assert np.abs(lse - math.log(V)).max() <= 2.0 ** -24 * (math.log(V) + 6) + 1e-6
        else:
            assert np.allclose(lse, xs.max(1) / float(np.float32(tau)), rtol=2.0 ** -23)
            # w tau (q - p) of the largest logit's id: within tau of nothing, and nothing anywhere else but at entries
            rest = xs < xs.max(1, keepdims=True)
            for r in range(B):
                rest[r, ids[r][(ids[r] >= 0) & (ids[r] < V)]] = False
            assert not grad[rest].any() and np.abs(grad).max() <= 1.01e-30


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [INF, math.nan])
def test_distillation_of_what_is_no_number(value, dtype):
    """An allowed NaN or +inf spreads over its row's allowed places, in every variant, and over no other row."""
    import torch
    say("no number", value, dtype)
    rng = np.random.default_rng(17)
    for B, V in ((3, 900), (300, 2500), (2, 70001)):
        x = F.make(rng, B, V, dtype)
        allowed = rng.random((B, V)) < 0.7
        ids, t = D.teacher(rng, x, None, 6, V)
        allowed[1, ids[1, 0]] = True  # an entry that the student can take
        w = np.ones(B, dtype=np.float32)
        at = int(np.flatnonzero(allowed[1])[5])
        for way in ("both", "grad"):
            clean = D.run(x, F.pack(allowed), ids, t, 1.0, way, w)
            y = x.clone()
            y[1, at] = value
            loss, lse, grad = D.run(y, F.pack(allowed), ids, t, 1.0, way, w)
            assert math.isnan(loss[1]) and math.isnan(lse[1])
            assert np.isnan(grad[1][allowed[1]]).all() and not grad[1][~allowed[1]].any()
            rest = np.arange(B) != 1
            assert all(np.array_equal(a[rest], b[rest]) for a, b in zip((loss, lse, grad), clean))


def test_rows_that_share_storage_are_refused():
    import torch
    say("shared rows")
    x = torch.zeros((1, 500), device="cuda").expand(4, 500)
    f = torch.zeros(4, device="cuda")
    i = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    for call in (lambda: cg.filter_sample(x, None, f, None, None, None, f, None, i[:, 0].contiguous(), f.clone()),
                 lambda: cg.top_logits(x, None, None, i, torch.zeros(4, 3, device="cuda"), f.clone()),
                 lambda: cg.distill_topk(x, None, i, torch.zeros(4, 3, device="cuda"), 1.0, f.clone(), f.clone())):
        with pytest.raises(ValueError):
            call()
