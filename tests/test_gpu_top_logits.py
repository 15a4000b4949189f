"""GPU: the k largest masked logits and the normaliser (cg_top_logits) against
the float64 oracle.  Ids and logits are exact; the normaliser is off by half
a float32 step, by the exponentials' rounding (2 ln V + 6 halves of a float32
step: an exponent d below the largest is rounded to d 2^-24 twice, the
exponential itself to two units, and the mean of d under the softmax is at
most ln V)."""
import math

import numpy as np
import pytest

import logit_masking_amd as cg
from oracle import oracle as O
from tests.gpu_util import say
from tests.test_gpu_filter_sample import make, masks, pack

pytestmark = pytest.mark.gpu
INF = math.inf


def run(x, mask, k, vocab=None, stream=None):
    import torch
    B = x.shape[0]
    V = x.shape[1] if vocab is None else vocab
    ids = torch.full((B + 1, k), -77, dtype=torch.int32, device="cuda")
    top = torch.full((B + 1, k), -77.0, dtype=torch.float32, device="cuda")
    lse = torch.full((B + 1,), -77.0, dtype=torch.float32, device="cuda")
    cg.top_logits(x, mask, cg.new_top_workspace(B, V, k), ids, top, lse, vocab=vocab, stream=stream)
    torch.cuda.synchronize()
    assert bool((ids[B] == -77).all()) and bool((top[B] == -77).all()) and float(lse[B]) == -77
    return ids[:B].cpu().numpy(), top[:B].cpu().numpy(), lse[:B].cpu().numpy().astype(np.float64)


def check(x, allowed, k, got, vocab=None):
    ids, top, lse = got
    V = x.shape[1] if vocab is None else vocab
    xs = x[:, :V].float().cpu().numpy().astype(np.float64)
    for r in range(x.shape[0]):
        i, t, l = O.top_logits_row(xs[r], None if allowed is None else allowed[r], k)
        assert np.array_equal(ids[r], i), f"row {r}"
        assert np.array_equal(top[r], t.astype(np.float32)), f"row {r}"
        if math.isfinite(l):
            assert abs(lse[r] - l) <= 2.0 ** -24 * (abs(l) + 2 * math.log(V) + 6), f"row {r}: {lse[r]} for {l}"
        else:
            assert lse[r] == l, f"row {r}"


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [1, 2, 64, 65, 700, 2049, 8191, 32000, 50021, 65537, 128256, 131075, 256000])
def test_sizes(V, dtype):
    say("top_logits", dtype, V)
    rng = np.random.default_rng(V)
    B = 6
    for k in (1, 5, 20, 64, 127, 1000, 1024):
        if V > 60000 and k in (5, 127, 1000):
            continue
        x = make(rng, B, V, dtype, 3.0)
        check(x, None, k, run(x, None, k))
        allowed = masks(rng, B, V)
        check(x, allowed, k, run(x, pack(allowed), k))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V,pad,off", [(1000, 0, 1), (1001, 6, 3), (32000, 24, 5), (40007, 1, 0)])
def test_strides_and_alignment(V, pad, off, dtype):
    import torch
    say("top_logits stride", dtype, V, pad, off)
    rng = np.random.default_rng(V + pad)
    B = 7
    flat = torch.full((B * (V + pad) + off + 64,), INF, dtype=getattr(torch, dtype), device="cuda")
    x = flat[off:off + B * (V + pad)].view(B, V + pad)
    x[:, :V] = make(rng, B, V, dtype)
    allowed = masks(rng, B, V)
    check(x, allowed, 17, run(x, pack(allowed), 17, vocab=V), vocab=V)
    check(x, None, 300, run(x, None, 300, vocab=V), vocab=V)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_ties_and_special_values(dtype):
    import torch
    say("top_logits ties", dtype)
    rng = np.random.default_rng(6)
    B = 20
    for V in (9, 300, 5000, 70001, 140000):
        x = torch.from_numpy(rng.integers(-3, 4, size=(B, V)).astype(np.float32) * 0.5)
        x[::5] = 1.25
        x[1::5][x[1::5] == 0] = -0.0
        x[1::5, ::3] = 0.0
        x[2, ::2] = -INF
        x[3] = -INF
        x[4, ::2] = math.nan
        x[6] = torch.finfo(getattr(torch, dtype)).min
        x[7, V // 2] = INF
        x = x.cuda().to(getattr(torch, dtype))
        allowed = masks(rng, B, V)
        y = x.clone()
        off = torch.from_numpy(~allowed).cuda()
        y[off] = torch.tensor(rng.choice([np.nan, np.inf, -np.inf], size=(B, V)).astype(np.float32)).cuda().to(x.dtype)[off]
        for k in (1, 8, 100, 1024):
            check(x, None, k, run(x, None, k))
            check(y, allowed, k, run(y, pack(allowed), k))


@pytest.mark.parametrize("dtype", ["float32"])
def test_crowded_values(dtype):
    """Float32 logits that agree in their upper bits: the k-th largest among many neighbours."""
    import torch
    say("top_logits crowded")
    rng = np.random.default_rng(8)
    for V in (5000, 60000, 130000):
        x = torch.from_numpy((1.0 + rng.integers(0, 60000, size=(6, V)) * 2.0 ** -23).astype(np.float32)).cuda()
        x[3] = -x[3]
        x[4, 5:] = 1.0
        for k in (1, 33, 1024):
            check(x, None, k, run(x, None, k))


def test_streams_and_graph():
    import torch
    say("top_logits graph")
    rng = np.random.default_rng(23)
    B, V, k = 10, 32000, 20
    xs = [make(rng, B, V, "bfloat16") for _ in range(3)]
    words = pack(masks(rng, B, V))
    want = [run(x, words, k) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, w in zip(xs, want):
        assert all(np.array_equal(a, b) for a, b in zip(run(x, words, k, stream=side), w))
    x = xs[0].clone()
    ids = torch.empty((B, k), dtype=torch.int32, device="cuda")
    top = torch.empty((B, k), device="cuda")
    lse = torch.empty(B, device="cuda")
    ws = cg.new_top_workspace(B, V, k)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cg.top_logits(x, words, ws, ids, top, lse)
    for n in range(4):
        x.copy_(xs[n % 3])
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), want[n % 3][0])
        assert np.array_equal(top.cpu().numpy(), want[n % 3][1])
        assert np.array_equal(lse.cpu().numpy().astype(np.float64), want[n % 3][2])
        run(xs[1], words, k)


def test_binding_refusals():
    import torch
    say("top_logits refusals")
    x = torch.zeros((4, 128), device="cuda")
    m = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    i, t, l = torch.zeros((4, 5), dtype=torch.int32, device="cuda"), torch.zeros((4, 5), device="cuda"), torch.zeros(4, device="cuda")
    cg.top_logits(x, m, None, i, t, l)
    for args in ((x, m, None, i[0], t, l), (x, m, None, i.long(), t, l), (x, m, None, i, t[:, :4], l), (x, m, None, i[:3], t, l),
                 (x, m, None, i, t, l[:2]), (x, m[:2], None, i, t, l), (x, m, None, i.cpu(), t, l)):
        with pytest.raises(ValueError):
            cg.top_logits(*args)
    with pytest.raises(cg.CgError) as e:
        cg.top_logits(x, m, None, torch.zeros((4, 1025), dtype=torch.int32, device="cuda"), torch.zeros((4, 1025), device="cuda"), l)
    assert e.value.code == cg.CG_E_ARG
    torch.cuda.synchronize()
