"""CPU: the row operators (filtered sampling, top logits, distillation) --
what the C ABI and the binding refuse, and pins of the oracle they are held
to.  No device calls: every refusal is made before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import logit_masking_amd as cg
from oracle import oracle as O

NAN, INF = math.nan, math.inf
P = 1 << 20  # a non-null address that nothing reads


def _err():
    return cg.lib().cg_last_error().decode()


def _sample(dtype=1, batch=2, vocab=100, stride=100, mask=P, words=2, ptrs=(P,) * 5, ws=None, ids=P, lp=P):
    return cg._row_lib().cg_filter_sample(P, dtype, batch, vocab, stride, mask, words, *ptrs, ws, ids, lp, None)


def _top(logits=P, dtype=1, batch=2, vocab=100, stride=100, mask=P, words=2, k=5, ids=P, top=P, lse=P):
    return cg._row_lib().cg_top_logits(logits, dtype, batch, vocab, stride, mask, words, k, None, ids, top, lse, None)


def _distill(logits=P, dtype=1, rows=2, vocab=100, stride=100, mask=P, words=2, tids=P, tl=P, k=4, tau=1.0, loss=P,
             weight=None, grad=None, gs=0):
    return cg._row_lib().cg_distill_topk(logits, dtype, rows, vocab, stride, mask, words, tids, tl, k, tau, loss, None,
                                         weight, grad, gs, None)


def _grad(dtype=1, rows=2, vocab=100, stride=100, mask=P, words=2, k=4, tau=1.0, lse=P, weight=P, grad=P, gs=100):
    return cg._row_lib().cg_distill_topk_grad(P, dtype, rows, vocab, stride, mask, words, P, P, k, tau, lse, weight, grad,
                                              gs, None)


BAD = [
    (_sample, dict(dtype=2)), (_sample, dict(batch=-1)), (_sample, dict(vocab=0)), (_sample, dict(stride=99)),
    (_sample, dict(words=1)), (_sample, dict(vocab=cg.MAX_ROW_VOCAB + 1, stride=1 << 40, words=1 << 20)),
    (_sample, dict(ptrs=(None, P, P, P, P))), (_sample, dict(ptrs=(P, P, P, P, None))), (_sample, dict(ids=None)),
    (_sample, dict(lp=None)),
    (_top, dict(dtype=-1)), (_top, dict(k=0)), (_top, dict(k=cg.MAX_TOP + 1)), (_top, dict(words=1)),
    (_top, dict(stride=50)), (_top, dict(ids=None)), (_top, dict(top=None)), (_top, dict(lse=None)),
    (_top, dict(logits=None)), (_top, dict(vocab=-3)),
    (_distill, dict(dtype=7)), (_distill, dict(k=0)), (_distill, dict(k=cg.MAX_TOP + 1)), (_distill, dict(tau=0.0)),
    (_distill, dict(tau=-1.0)), (_distill, dict(tau=NAN)), (_distill, dict(tau=INF)), (_distill, dict(loss=None)),
    (_distill, dict(tids=None)), (_distill, dict(tl=None)), (_distill, dict(weight=P, grad=P, gs=99)),
    (_distill, dict(grad=P, gs=100)), (_distill, dict(logits=None)), (_distill, dict(rows=-1)),
    (_grad, dict(lse=None)), (_grad, dict(weight=None)), (_grad, dict(grad=None)), (_grad, dict(gs=1)),
    (_grad, dict(tau=INF)), (_grad, dict(words=1)),
]


@pytest.mark.parametrize("call,how", BAD, ids=[f"{c.__name__[1:]}-{i}" for i, (c, _) in enumerate(BAD)])
def test_c_refusals(call, how):
    assert call(**how) == cg.CG_E_ARG
    assert _err()


@pytest.mark.parametrize("tau", [1e-31, 1e-45, 1.1e30])
def test_temperatures_whose_inverse_is_no_float32(tau):
    for call in (_distill, _grad):
        assert call(tau=tau) == cg.CG_E_ARG
        assert "temperature" in _err()


def test_loss_refuses_other_leading_shapes():
    import torch
    x, i, t = torch.zeros(2, 3, 50), torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, 4)
    m = torch.zeros(2, 3, 1, dtype=torch.int64)
    for args in ((x, i[:1], t, m), (x, i, t.reshape(6, 4), m), (x, i, t, m[:, :2]), (x, i.reshape(3, 2, 4), t.reshape(3, 2, 4), None)):
        with pytest.raises(ValueError, match="leading shape"):
            cg.distill_topk_loss(*args)


def test_empty_batches_do_nothing():
    """No rows: CG_OK without touching a pointer; the sizes are still checked."""
    assert _sample(batch=0, ptrs=(None,) * 5, ids=None, lp=None) == cg.CG_OK
    assert _top(batch=0, logits=None, ids=None, top=None, lse=None) == cg.CG_OK
    assert _distill(rows=0, logits=None, tids=None, tl=None, loss=None) == cg.CG_OK
    assert _grad(rows=0, lse=None, weight=None, grad=None) == cg.CG_OK
    assert _top(batch=0, k=0) == cg.CG_E_ARG


def test_workspace_sizes_of_nothing():
    assert cg.filter_workspace_bytes(0, 100) == 0
    assert cg.filter_workspace_bytes(4, 0) == 0
    assert cg.top_workspace_bytes(0, 100, 5) == 0
    assert cg.top_workspace_bytes(4, 100, 0) == 0


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros((2, 64))
    f, i, m = torch.zeros(2), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1), dtype=torch.int64)
    two = torch.zeros((2, 4))
    with pytest.raises(ValueError, match="device"):
        cg.filter_sample(x, m, f, i, f, f, f, None, i, f)
    with pytest.raises(ValueError, match="device"):
        cg.top_logits(x, m, None, two.int(), two, f)
    with pytest.raises(ValueError, match="device"):
        cg.distill_topk(x, m, two.int(), two, 1.0, f)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        cg.filter_sample(x.half(), m, f, i, f, f, f, None, i, f)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        cg.distill_topk_loss(x.double(), two.int(), two)
    with pytest.raises(ValueError, match="leading shape"):
        cg.distill_topk_loss(x, two[:1].int(), two)


# ---- the oracle ------------------------------------------------------------

def test_oracle_order_and_filters():
    x = [1.0, 3.0, -0.0, 3.0, 0.0, -INF, NAN, 2.0]
    assert list(O.ranked(x)) == [1, 3, 7, 0, 2, 4]
    assert list(O.ranked(x, [1, 0, 1, 1, 1, 1, 1, 0])) == [3, 0, 2, 4]
    # four equal candidates: every quarter of [0, 1) is one of them, lowest id first
    for n, u in enumerate((0.0, 0.25, 0.5, 0.75)):
        i, lp, _ = O.filter_sample_row([0, 0, 0, 0], None, 1.0, None, None, None, u)
        assert i == n and lp == -math.log(4)
    # top-p takes ranks while the mass before them is under p: half of four equals is two
    ids = {O.filter_sample_row([0, 0, 0, 0], None, 1.0, None, 0.5, None, u)[0] for u in np.linspace(0, 0.999, 40)}
    assert ids == {0, 1}
    assert {O.filter_sample_row([0, 0, 0, 0], None, 1.0, None, 0.51, None, u)[0] for u in np.linspace(0, 0.999, 40)} == {0, 1, 2}
    # top-k cuts inside equals by id; min-p keeps the weights that reach it
    assert {O.filter_sample_row([0, 0, 0, 0], None, 1.0, 3, None, None, u)[0] for u in np.linspace(0, 0.999, 40)} == {0, 1, 2}
    x = np.log([0.5, 0.25, 0.125, 0.125])
    assert {O.filter_sample_row(x, None, 1.0, None, None, 0.4, u)[0] for u in np.linspace(0, 0.999, 40)} == {0, 1}
    # p = 0 and greedy take the best; a logit of +inf takes everything
    assert O.filter_sample_row(x, None, 1.0, None, 0.0, None, 0.99)[0] == 0
    assert O.filter_sample_row([0, INF, 1], None, 1.0, None, None, None, 0.99)[:2] == (1, 0.0)
    assert O.filter_sample_row([5, 5, 1], None, 0.0, None, None, None, 0.99)[0] == 0
    assert O.filter_sample_row([NAN, -INF], None, 1.0, None, None, None, 0.5)[:2] == (-1, 0.0)


def test_oracle_draw_follows_the_distribution():
    """Counts of an even grid of uniform numbers are the probabilities, to one count a border."""
    rng = np.random.default_rng(7)
    x = rng.normal(size=50) * 2
    n = 20000
    got = np.zeros(50)
    for j in range(0, n, 40):
        got[O.filter_sample_row(x, None, 0.8, 20, 0.9, 0.01, (j + 0.5) / n)[0]] += 40
    w = np.exp((x - x.max()) / np.float32(0.8))
    order = np.argsort(-x)
    keep = order[:20]
    before = np.cumsum(w[keep]) - w[keep]
    keep = keep[(before < np.float32(0.9) * w[keep].sum()) & (w[keep] >= np.float32(0.01))]
    want = np.zeros(50)
    want[keep] = w[keep] / w[keep].sum() * n
    assert np.all(np.abs(got - want) <= 40 + 1e-9)


def test_oracle_top_logits():
    ids, top, lse = O.top_logits_row([1.0, 3.0, 3.0, -INF], [1, 1, 1, 1], 5)
    assert list(ids) == [1, 2, 0, -1, -1] and list(top[:3]) == [3, 3, 1] and np.all(top[3:] == -INF)
    assert abs(lse - math.log(math.e + 2 * math.e ** 3)) < 1e-15 * 10
    assert O.top_logits_row([NAN], None, 2)[2] == -INF


def test_oracle_gradient_is_the_losses_difference():
    rng = np.random.default_rng(3)
    x = rng.normal(size=40) * 2
    allowed = rng.random(40) < 0.8
    ids = np.array([3, 7, 7, -1, 50, 11, 12, 39])  # one id twice, two that are no ids
    t = rng.normal(size=8)
    t[5] = -INF
    loss, _, g = O.distill_row(x, allowed, ids, t, 1.7)
    h = 1e-5  # central difference: error h^2 f'''/6 + 2e-16 f/h, under 1e-9 here
    for v in range(40):
        a, b = x.copy(), x.copy()
        a[v] += h
        b[v] -= h
        d = (O.distill_row(a, allowed, ids, t, 1.7)[0] - O.distill_row(b, allowed, ids, t, 1.7)[0]) / (2 * h)
        assert abs(d - g[v]) < 1e-8, v
        if not allowed[v]:
            assert g[v] == 0
    # equal distributions: no loss, no gradient where the record covers everything
    loss, _, g = O.distill_row(x, None, np.arange(40), x, 2.0)
    assert abs(loss) < 1e-14 and np.all(np.abs(g) < 1e-14)
    assert O.distill_row(x, allowed, [-1, -1], [0.0, 0.0], 1.0)[0] == 0
