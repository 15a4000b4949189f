"""GPU: distillation from a teacher's top logits (cg_distill_topk,
cg_distill_topk_grad, distill_topk_loss) against the float64 oracle.

Tolerances, with e = 2^-24 (half a float32 step of one):
  lse   half a step of itself, and the exponentials' error (2 ln V + 6) e (an
        exponent d below the largest is rounded to d e twice, the exponential
        to two units; the mean of d under the softmax is at most ln V);
  loss  tau^2 times that normaliser's error, and half a step of itself; its
        own terms are summed in 64 bits;
  grad  tau w q times the relative error of q = 2^((x - m) kk - log2 s), s the
        sum, in float32: (2 |x - m| / tau + 2 ln V + 6) 2 e (kk, the
        difference and the fma round once each, log2 s once) and the
        normaliser's; from a saved normaliser, q = 2^(x kk - L log2 e) and
        (2 |x| / tau + 3 |L|) 2 e more, unless |L| > 1024, where it is summed
        again; and half a float32 step of p, half a step of the output type.
"""
import math

import numpy as np
import pytest

import logit_masking_amd as cg
from oracle import oracle as O
from tests.gpu_util import say
from tests.test_gpu_filter_sample import make, masks, pack

pytestmark = pytest.mark.gpu
INF, E = math.inf, 2.0 ** -24


def teacher(rng, x, allowed, k, V):
    """A record as a teacher leaves it: its top ids, some of them none, one of them twice, some masked for the student."""
    B = x.shape[0]
    ids = np.stack([rng.permutation(V)[:k] if k <= V else rng.integers(0, V, k) for _ in range(B)]).astype(np.int32)
    t = (rng.normal(size=(B, k)) * 2).astype(np.float32)
    if k > 3:
        ids[:, 1] = ids[:, 0]
        ids[::2, 2] = -1
        t[::3, 3] = -INF
    if B > 4:
        ids[3] = -1
        ids[4, -1] = V + 5
    return ids, t


def run(x, mask, ids, t, tau, way, weight=None, vocab=None, stream=None, grad_pad=0, inplace=False):
    import torch
    B = x.shape[0]
    V = x.shape[1] if vocab is None else vocab
    ids, t = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda()
    loss = torch.full((B + 1,), -77.0, device="cuda")
    lse = torch.full((B + 1,), -77.0, device="cuda")
    grad = None
    if way == "loss":
        weight = None
    else:
        weight = torch.from_numpy(weight).cuda()
        grad = x if inplace else torch.full((B + 1, V + grad_pad), 5.0, dtype=x.dtype, device="cuda")
    if way == "grad":
        cg.distill_topk(x, mask, ids, t, tau, loss, lse, vocab=vocab, stream=stream)
        cg.distill_topk_grad(x, mask, ids, t, tau, lse, weight, grad, vocab=vocab, stream=stream)
    else:
        cg.distill_topk(x, mask, ids, t, tau, loss, lse, weight=weight, out_grad=grad, vocab=vocab, stream=stream)
    torch.cuda.synchronize()
    assert float(loss[B]) == -77 and float(lse[B]) == -77
    out = [loss[:B].cpu().numpy().astype(np.float64), lse[:B].cpu().numpy().astype(np.float64), None]
    if way != "loss":
        if not inplace:
            assert bool((grad[B:] == 5).all()) and bool((grad[:, V:] == 5).all())
        out[2] = grad[:B, :V].double().cpu().numpy()
    return out


def check(xs, allowed, ids, t, tau, weight, got, dtype, saved=False):
    """xs: the student's logits as float64."""
    loss, lse, grad = got
    B, V = xs.shape
    tau = float(np.float32(tau))
    step = 2.0 ** -8 if dtype == "bfloat16" else E
    for r in range(B):
        ok = None if allowed is None else allowed[r]
        wl, wz, wg = O.distill_row(xs[r], ok, ids[r], t[r], tau)
        if not math.isfinite(wz):
            assert lse[r] == wz and loss[r] == 0
            assert grad is None or not grad[r].any()
            continue
        le = (2 * math.log(V) + 6) * E
        assert abs(lse[r] - wz) <= abs(wz) * E + le, f"row {r}: lse {lse[r]} for {wz}"
        assert abs(loss[r] - wl) <= tau * tau * le + abs(wl) * E, f"row {r}: loss {loss[r]} for {wl}"
        if grad is None:
            continue
        has = (ids[r] >= 0) & (ids[r] < V) & (t[r] > -INF)
        has[has] = xs[r][ids[r][has]] > -INF
        if ok is not None:
            has[has] = ok[ids[r][has]]
        if not has.any():  # nothing recorded: exactly nothing
            assert not grad[r].any() and loss[r] == 0
            continue
        w = float(weight[r])
        use = np.ones(V, dtype=bool) if ok is None else ok
        with np.errstate(invalid="ignore", over="ignore"):
            z = np.where(use, np.nan_to_num(xs[r], nan=0, posinf=0, neginf=-1e30), 0.0) / tau
        zm = np.max(z[use])
        q = np.where(use, np.exp(np.where(use, z - zm, 0.0)), 0.0)
        q /= q.sum()
        want = w * wg
        p = np.abs(q - wg / tau)  # what the teacher took off
        d = np.where(use, zm - z, 0.0)
        rel = (2 * np.minimum(d, 1e4) + 2 * math.log(V) + 6) * 2 * E + le
        if saved and abs(wz) <= 1024:
            rel = rel + (2 * np.minimum(np.abs(z), 1e4) + 3 * abs(wz)) * 2 * E
        tol = abs(w) * tau * (q * rel + p * E) + step * np.abs(want) + 1e-38
        off = np.abs(grad[r] - want)
        bad = np.flatnonzero(~(off <= tol))
        assert not len(bad), f"row {r} id {bad[0]}: {grad[r][bad[0]]} for {want[bad[0]]} (tol {tol[bad[0]]})"
        assert not grad[r][~use].any()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [1, 2, 63, 65, 700, 2048, 8191, 32000, 50021, 65600, 128256, 131075, 256000])
def test_sizes_and_directions(V, dtype):
    say("distill", dtype, V)
    rng = np.random.default_rng(V)
    B = 6
    for k, tau, way in ((1, 1.0, "both"), (16, 2.0, "grad"), (64, 0.7, "both"), (300, 3.0, "loss"), (1024, 1.3, "both")):
        if V > 60000 and k == 300:
            continue
        x = make(rng, B, V, dtype, 2.0)
        w = rng.uniform(-1, 2, B).astype(np.float32)
        for allowed in (None, masks(rng, B, V)):
            ids, t = teacher(rng, x, allowed, k, V)
            mask = None if allowed is None else pack(allowed)
            check(x.double().cpu().numpy(), allowed, ids, t, tau, w, run(x, mask, ids, t, tau, way, w), dtype, way == "grad")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V,pad,off,gpad", [(1000, 0, 1, 0), (1001, 6, 3, 5), (32000, 24, 5, 3), (40007, 1, 0, 8)])
def test_strides_and_alignment(V, pad, off, gpad, dtype):
    import torch
    say("distill stride", dtype, V, pad, off, gpad)
    rng = np.random.default_rng(V + pad)
    B = 7
    flat = torch.full((B * (V + pad) + off + 64,), math.nan, dtype=getattr(torch, dtype), device="cuda")
    x = flat[off:off + B * (V + pad)].view(B, V + pad)
    x[:, :V] = make(rng, B, V, dtype)
    w = rng.uniform(0, 2, B).astype(np.float32)
    for allowed in (None, masks(rng, B, V)):
        ids, t = teacher(rng, x, allowed, 9, V)
        mask = None if allowed is None else pack(allowed)
        for way in ("both", "grad"):
            check(x[:, :V].double().cpu().numpy(), allowed, ids, t, 1.5, w,
                  run(x, mask, ids, t, 1.5, way, w, vocab=V, grad_pad=gpad), dtype, way == "grad")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [777, 32000, 140000])
def test_gradient_over_the_logits(V, dtype):
    """The gradient written over the logits it is taken of, in both calls."""
    say("distill in place", dtype, V)
    rng = np.random.default_rng(V)
    B = 5
    w = rng.uniform(0.1, 2, B).astype(np.float32)
    allowed = masks(rng, B, V)
    for way in ("both", "grad"):
        x = make(rng, B, V, dtype)
        xs = x.double().cpu().numpy()
        ids, t = teacher(rng, x, allowed, 30, V)
        check(xs, allowed, ids, t, 1.2, w, run(x, pack(allowed), ids, t, 1.2, way, w, inplace=True), dtype, way == "grad")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_special_values(dtype):
    """Anything in masked places; -inf as masked; the lowest value a value; an allowed NaN spreads over its row alone."""
    import torch
    say("distill specials", dtype)
    rng = np.random.default_rng(31)
    B, V, k = 12, 3001, 12
    x = make(rng, B, V, dtype)
    allowed = masks(rng, B, V)
    off = torch.from_numpy(~allowed).cuda()
    x[off] = torch.tensor(rng.choice([np.nan, np.inf, -np.inf], size=(B, V)).astype(np.float32)).cuda().to(x.dtype)[off]
    ids, t = teacher(rng, x, allowed, k, V)
    for r in range(5, B):  # entries the student can take
        ids[r, 4:] = np.flatnonzero(allowed[r])[:k - 4]
    x[5, ids[5, 4]] = -INF
    x[6] = -INF
    low = torch.finfo(x.dtype).min
    x[7][torch.from_numpy(allowed[7]).cuda()] = low
    w = rng.uniform(0.1, 2, B).astype(np.float32)
    xs = x.double().cpu().numpy()
    for way in ("both", "grad"):
        check(xs, allowed, ids, t, 2.0, w, run(x, pack(allowed), ids, t, 2.0, way, w), dtype, way == "grad")
    x[8, int(ids[8, 4])] = math.nan
    got = run(x, pack(allowed), ids, t, 2.0, "both", w)
    assert math.isnan(got[0][8]) and math.isnan(got[1][8])
    assert np.isnan(got[2][8][allowed[8]]).all() and not got[2][8][~allowed[8]].any()
    keep = np.arange(B) != 8
    check(xs[keep], allowed[keep], ids[keep], t[keep], 2.0, w[keep], [g[keep] for g in got], dtype)


def test_gradient_is_the_losses_difference():
    """Central differences of the kernel's own losses.  With step h = 2^-4 on float32 logits the difference is off by
    h^2 / 6 times a third derivative (under tau^2 (2 / tau^3) here) and by the losses' rounding over h."""
    import torch
    say("distill differences")
    rng = np.random.default_rng(41)
    V, k, tau, h = 40, 8, 1.5, 2.0 ** -4
    base = rng.normal(size=V).astype(np.float32)
    ids = np.tile(rng.permutation(V)[:k].astype(np.int32), (2 * V, 1))
    t = np.tile(rng.normal(size=k).astype(np.float32), (2 * V, 1))
    x = np.tile(base, (2 * V, 1))
    for v in range(V):
        x[2 * v, v] += h
        x[2 * v + 1, v] -= h
    hh = np.array([float(x[2 * v, v]) - float(x[2 * v + 1, v]) for v in range(V)])
    loss, _, _ = run(torch.from_numpy(x).cuda(), None, ids, t, tau, "loss")
    diff = (loss[0::2] - loss[1::2]) / hh
    _, _, g = run(torch.from_numpy(base[None]).cuda(), None, ids[:1], t[:1], tau, "both", np.ones(1, np.float32))
    rounding = 2 * (tau * tau * (2 * math.log(V) + 6) * E + np.abs(loss).max() * E) / (2 * h)
    assert np.all(np.abs(diff - g[0]) <= h * h / 6 * (2 / tau) + rounding + 1e-6)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_autograd(dtype):
    """distill_topk_loss: leading shapes, a pad of the vocabulary, strided logits, a weighted mean, and no double gradient."""
    import torch
    say("distill autograd", dtype)
    rng = np.random.default_rng(51)
    V, k, tau = 1003, 10, 2.0
    x = make(rng, 6, V, dtype, pad=5).view(2, 3, V + 5).requires_grad_()
    allowed = masks(rng, 6, V)
    ids, t = teacher(rng, x.view(6, -1), allowed, k, V)
    w = rng.uniform(0.1, 1, 6).astype(np.float32)
    loss = cg.distill_topk_loss(x, torch.from_numpy(ids).cuda().view(2, 3, k), torch.from_numpy(t).cuda().view(2, 3, k),
                                mask=pack(allowed).view(2, 3, -1), temperature=tau, vocab=V)
    assert loss.shape == (2, 3) and loss.dtype == torch.float32
    (loss.view(-1) * torch.from_numpy(w).cuda()).sum().backward()
    assert x.grad.dtype == x.dtype and not x.grad[..., V:].any()
    got = [loss.detach().view(-1).cpu().numpy().astype(np.float64), None, x.grad.view(6, -1)[:, :V].double().cpu().numpy()]
    xs = x.detach().view(6, -1)[:, :V].double().cpu().numpy()
    _, lse, _ = run(x.detach().view(6, -1), pack(allowed), ids, t, tau, "loss", vocab=V)
    check(xs, allowed, ids, t, tau, w, [got[0], lse, got[2]], dtype, saved=True)
    # a transposed view, and a broadcast gradient (mean)
    y = make(rng, V, 4, dtype).t().detach().requires_grad_()
    m = cg.distill_topk_loss(y, torch.from_numpy(ids[:4]).cuda(), torch.from_numpy(t[:4]).cuda(), temperature=tau).mean()
    g, = torch.autograd.grad(m, y)
    ys = y.detach().double().cpu().numpy()
    _, lse, _ = run(y.detach().contiguous(), None, ids[:4], t[:4], tau, "loss")
    ls = cg.distill_topk_loss(y, torch.from_numpy(ids[:4]).cuda(), torch.from_numpy(t[:4]).cuda(), temperature=tau)
    check(ys, None, ids[:4], t[:4], tau, np.full(4, 0.25, np.float32),
          [ls.detach().cpu().numpy().astype(np.float64), lse, g.double().cpu().numpy()], dtype, saved=True)
    one, = torch.autograd.grad(ls.sum(), y, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(one.float().sum(), y)


def test_autograd_in_a_captured_graph():
    """Forward and backward captured together (torch.autograd.grad) and replayed with eager work between."""
    import torch
    say("distill graph")
    rng = np.random.default_rng(61)
    B, V, k = 8, 4000, 16
    xs = [make(rng, B, V, "bfloat16") for _ in range(3)]
    ids, t = teacher(rng, xs[0], None, k, V)
    ids, t = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda()
    w = torch.rand(B, device="cuda")

    def step(x):
        loss = cg.distill_topk_loss(x, ids, t, temperature=2.0)
        return loss, torch.autograd.grad((loss * w).sum(), x)[0]

    want = []
    for v in xs:
        loss, grad = step(v.clone().requires_grad_())
        want.append((loss.detach().clone(), grad.clone()))
        del loss, grad
    x = xs[0].clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad = step(x)
    for n in range(4):
        with torch.no_grad():
            x.copy_(xs[n % 3])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[n % 3][0]) and torch.equal(grad, want[n % 3][1])
        step(xs[1].clone().requires_grad_())


def test_teacher_to_student():
    """The run they are made for: a teacher decodes under the grammar (mask, draw, walk), its top logits are recorded at every
    step, and the student is trained on them under the same masks."""
    import torch
    from logit_masking_amd import workloads as W
    say("teacher to student")
    blob, off = W.make_vocab(3, 8000)
    g = cg.Grammar(W.spec_json(3), blob, off)
    V, B, k, steps_n = g.V, 8, 12, 10
    st = g.new_states(B)
    g.init_state(st)
    steps = torch.zeros(B, dtype=torch.int32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    masks_, ids_, tops_, picks = [], [], [], []
    u = torch.rand((steps_n, B), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    temp = torch.full((B,), 0.8, device="cuda")
    k40 = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    p95 = torch.full((B,), 0.95, device="cuda")
    for s in range(steps_n):
        mask = torch.empty((B, g.W), dtype=torch.int64, device="cuda")
        g.fill_bitmask(st, mask)
        x = W.make_logits(3, s, B, V, "cuda")
        ids = torch.empty(B, dtype=torch.int32, device="cuda")
        lp = torch.empty(B, device="cuda")
        cg.filter_sample(x, mask, temp, k40, p95, None, u[s], None, ids, lp)
        ti = torch.empty((B, k), dtype=torch.int32, device="cuda")
        tl = torch.empty((B, k), device="cuda")
        cg.top_logits(x, mask, None, ti, tl, torch.empty(B, device="cuda"))
        g.advance(st, ids, steps, status)
        assert not bool((status == cg.ROW_REJECTED).any())
        masks_.append(mask), ids_.append(ti), tops_.append(tl), picks.append(ids)
    mask, ti, tl = torch.cat(masks_), torch.cat(ids_), torch.cat(tops_)
    student = (torch.randn((steps_n * B, V), device="cuda", generator=torch.Generator("cuda").manual_seed(4)) * 2).bfloat16()
    xs = student.double().cpu().numpy()
    allowed = np.stack([O.unpack_mask(w, V) for w in mask.cpu().numpy().view(np.uint64)])
    student.requires_grad_()
    loss = cg.distill_topk_loss(student, ti, tl, mask=mask, temperature=2.0)
    loss.mean().backward()
    _, lse, _ = run(student.detach(), mask, ti.cpu().numpy(), tl.cpu().numpy(), 2.0, "loss")
    n = steps_n * B
    check(xs, allowed, ti.cpu().numpy(), tl.cpu().numpy(), 2.0, np.full(n, np.float32(1) / np.float32(n)),
          [loss.detach().cpu().numpy().astype(np.float64), lse, student.grad.double().cpu().numpy()], "bfloat16", saved=True)


def test_binding_refusals():
    import torch
    say("distill refusals")
    x = torch.zeros((4, 128), device="cuda")
    i = torch.zeros((4, 5), dtype=torch.int32, device="cuda")
    t = torch.zeros((4, 5), device="cuda")
    w = torch.zeros(4, device="cuda")
    g = torch.zeros((4, 128), device="cuda")
    cg.distill_topk(x, None, i, t, 1.0, w)
    cg.distill_topk(x, None, i, t, 1.0, w, weight=w.clone(), out_grad=g)
    big = torch.zeros(4 * 128 + 64, device="cuda")
    bad = [dict(weight=w), dict(out_grad=g), dict(weight=w, out_grad=g.bfloat16()), dict(weight=w, out_grad=g[:, :100]),
           dict(weight=w, out_grad=g[:3]), dict(weight=w[:2], out_grad=g), dict(weight=w, out_grad=g.t()), dict(out_lse=w[:1]),
           dict(weight=w, out_grad=g.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            cg.distill_topk(x, None, i, t, 1.0, w, **kw)
    part = big[:512].view(4, 128)
    with pytest.raises(ValueError, match="overlap"):
        cg.distill_topk(part, None, i, t, 1.0, w, weight=w, out_grad=big[64:].view(4, 128))
    for tau in (0.0, -1.0, math.nan, INF):
        with pytest.raises(cg.CgError):
            cg.distill_topk(x, None, i, t, tau, w)
    for args in ((x, None, i[:2], t, 1.0, w), (x, None, i, t[:, :4], 1.0, w), (x, None, i.long(), t, 1.0, w), (x, None, i[0], t, 1.0, w)):
        with pytest.raises(ValueError):
            cg.distill_topk(*args)
    with pytest.raises(ValueError):
        cg.distill_topk_grad(x, None, i, t, 1.0, w[:3], w, g)
    torch.cuda.synchronize()
