"""The router and its balance loss against plain implementations in 64 bits
(more_layers_ref.py): choices and counts have to be equal, computed values stay
within bounds that follow from the roundings the operators state."""

import sys

import numpy as np
import pytest
import torch

from tests import more_layers_ref as ref
from tests.layers_ref import ROUND, TINY, to64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402

DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]
INF = float("inf")


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed)).to(dtype).to(DEV)


def router_logits(tokens, experts, seed, dtype, masked=True):
    """With padded tokens, experts that are switched off and tokens with few experts left."""
    l = (1.5 * torch.randn((tokens, experts), generator=gen(seed))).to(dtype)
    if masked:
        l[torch.rand(l.shape, generator=gen(seed + 1)) < 0.15] = -INF
        l[3::7] = -INF
        if tokens > 5:
            l[5, :] = -INF
            l[5, experts // 2] = -3.0
    return l.to(DEV)


def within(got, want, bound, dtype=torch.float32):
    got = to64(got)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    over = np.abs(got - want) - (bound + np.abs(want) * ROUND[dtype] + 2 * TINY[dtype])
    assert (over <= 0).all(), "worst %.3g over its bound at %s" % (
        over.max(), np.unravel_index(over.argmax(), over.shape))


def strided(t, pad, shift):
    rows, cols = t.shape
    buf = torch.empty(rows * (cols + pad) + shift + 16, dtype=t.dtype, device=t.device)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


# tokens, experts, top_k
SIZES = [(1, 1, 1), (4, 8, 2), (1, 64, 8), (7, 13, 3), (33, 32, 32), (65, 33, 5), (100, 64, 8), (64, 65, 2),
         (31, 128, 4), (17, 129, 17), (50, 256, 8), (9, 257, 6), (20, 512, 10), (3, 512, 512), (1000, 16, 2)]


def check_gate(l, top_k, renormalize, choice, weights):
    want, w = ref.gate(to64(l), top_k, renormalize)
    assert choice.dtype == torch.int32 and weights.dtype == torch.float32
    assert np.array_equal(choice.cpu().numpy(), want)
    within(weights, w, w * ref.softmax_error(to64(l))[:, None] + 2.0 ** -120)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,experts,top_k", SIZES)
def test_gate(dtype, tokens, experts, top_k):
    for masked in (False, True):
        l = router_logits(tokens, experts, tokens + experts, dtype, masked)
        for renormalize in (True, False):
            choice, weights = iq.expert_gate(l, top_k, renormalize=renormalize)
            check_gate(l, top_k, renormalize, choice, weights)
            again = iq.expert_gate(strided(l, 3, 1), top_k, renormalize=renormalize)
            assert torch.equal(again[0], choice) and torch.equal(again[1], weights)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("experts", [5, 40, 64, 100, 256, 512])
def test_equal_logits_go_to_the_lowest_expert(dtype, experts):
    l = torch.randint(0, 3, (40, experts), generator=gen(1)).to(dtype)
    l[0] = 0.0
    l[1] = 0.0
    l[1, ::2] = -0.0
    l[2] = torch.finfo(dtype).min
    l[3] = -INF
    l[3, -2:] = torch.finfo(dtype).min            # the lowest value is no mask
    k = min(10, experts)
    for renormalize in (True, False):
        choice, weights = iq.expert_gate(l.to(DEV), k, renormalize=renormalize)
        check_gate(l, k, renormalize, choice, weights)
    assert choice[1].tolist() == list(range(k))
    assert choice[3].tolist()[:3] == [experts - 2, experts - 1, -1]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_logits_far_apart(dtype):
    top = 6e4 if dtype == torch.float16 else 3e38
    l = torch.zeros((6, 48))
    l[0, 7], l[1, 0], l[2, 3] = top, -top, 200.0
    l[3, :] = -top
    l[4, 1], l[4, 2] = top, -top
    l[5] = torch.linspace(-120, 60, 48)
    l = l.to(dtype)
    for renormalize in (True, False):
        choice, weights = iq.expert_gate(l.to(DEV), 4, renormalize=renormalize)
        check_gate(l, 4, renormalize, choice, weights)
    c = choice
    loss, counts, live = iq.expert_balance(l.to(DEV), c)
    want = ref.balance(to64(l), c.cpu().numpy())
    within(loss, np.array(want[0]), ref.balance_bound(want[0], to64(l)))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_what_is_not_a_logit_is_reported(dtype, bad):
    l = router_logits(30, 48, 1, dtype, False)
    l[4, 47], l[9, 0] = bad, bad
    c = torch.randint(0, 48, (30, 2), generator=gen(2)).to(DEV)
    for call in (lambda: iq.expert_gate(l, 3), lambda: iq.expert_balance(l, c)):
        with pytest.raises(iq.IQError) as e:
            call()
        assert e.value.name == "IQ_ERR_NONFINITE"
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    choice, weights = iq.expert_gate(l, 3, status=status, check=False)
    assert int(status) == 5
    clean = l.clone()
    clean[4], clean[9] = -INF, -INF               # such a token has no choices
    check_gate(clean, 3, True, choice, weights)
    status.zero_()
    loss, counts, live = iq.expert_balance(l, c, status=status, check=False)
    assert int(status) == 5 and int(live) == 28
    want = iq.expert_balance(clean, c)
    assert torch.equal(loss, want[0]) and torch.equal(counts, want[1])
    # and no gradient
    one = torch.ones((), device=DEV)
    grad = iq.expert_balance_backward(one, l, counts, live)
    assert torch.equal(grad, iq.expert_balance_backward(one, clean, counts, live))
    g = normal((30, 3), 3)
    grad = iq.expert_gate_backward(g, l, choice, weights, renormalize=False)
    assert not grad[4].any() and not grad[9].any() and torch.isfinite(grad).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,experts,top_k", SIZES)
def test_gate_backward(dtype, tokens, experts, top_k):
    l = router_logits(tokens, experts, tokens * 3 + experts, dtype)
    g = normal((tokens, top_k), 5)
    for renormalize in (True, False):
        choice, weights = iq.expert_gate(l, top_k, renormalize=renormalize)
        got = iq.expert_gate_backward(g, l, choice, weights, renormalize=renormalize)
        want, bound = ref.gate_backward(to64(g), to64(l), choice.cpu().numpy(), to64(weights), renormalize)
        assert got.dtype == dtype
        within(got, want, bound, dtype)
        again = iq.expert_gate_backward(g, strided(l, 3, 1), choice, weights, renormalize=renormalize)
        assert torch.equal(again, got)


@pytest.mark.parametrize("renormalize", [True, False])
def test_gate_backward_of_any_choices(renormalize):
    """The same expert twice, dropped ones, ones out of range."""
    l = router_logits(6, 70, 1, torch.float32, False)
    c = torch.tensor([[3, 3, 69, -1], [-1, -1, -1, -1], [70, 2, -7, 2 ** 31 - 1], [0, 1, 2, 3],
                      [5, 5, 5, 5], [-2 ** 31, 68, 69, 0]], dtype=torch.int32, device=DEV)
    w, g = torch.rand((6, 4), generator=gen(2)).to(DEV), normal((6, 4), 3)
    got = iq.expert_gate_backward(g, l, c, w, renormalize=renormalize)
    want, bound = ref.gate_backward(to64(g), to64(l), c.cpu().numpy(), to64(w), renormalize)
    within(got, want, bound)
    assert not got[1].any()


BALANCES = [(1, 1, 1), (4, 8, 2), (7, 13, 3), (100, 64, 8), (1001, 13, 3), (511, 129, 4), (2000, 256, 8),
            (3000, 512, 2), (20000, 16, 1), (70001, 33, 2)]


def check_balance(l, choice, loss, counts, live):
    want, n, tokens = ref.balance(to64(l), choice.cpu().numpy())
    assert loss.shape == () and live.shape == () and counts.dtype == torch.int32
    assert np.array_equal(counts.cpu().numpy(), n) and int(live) == tokens
    within(loss, np.array(want), ref.balance_bound(want, to64(l)))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,experts,top_k", BALANCES)
def test_balance(dtype, tokens, experts, top_k):
    for masked in (False, True):
        l = router_logits(tokens, experts, tokens + 1, dtype, masked)
        choice, _ = iq.expert_gate(l, top_k)
        loss, counts, live = iq.expert_balance(l, choice)
        check_balance(l, choice, loss, counts, live)
        again = iq.expert_balance(strided(l, 3, 1), choice.long())
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, live)))
        grad = torch.tensor(-0.37, device=DEV)
        got = iq.expert_balance_backward(grad, l, counts, live)
        want, bound = ref.balance_backward(to64(grad), to64(l), counts.cpu().numpy(), int(live))
        assert got.dtype == dtype
        within(got, want, bound, dtype)


def test_balance_of_choices_that_are_not_the_gates():
    l = router_logits(500, 24, 1, torch.float32)
    c = torch.randint(-1, 24, (500, 30), generator=gen(2))       # more choices than experts, some dropped
    loss, counts, live = iq.expert_balance(l, c.to(DEV))
    check_balance(l, c, loss, counts, live)
    c[3, 1], c[400, 29] = 24, -2
    with pytest.raises(iq.IQError) as e:
        iq.expert_balance(l, c.to(DEV))
    assert e.value.name == "IQ_ERR_INDEX"
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, counts, live = iq.expert_balance(l, c.to(DEV), status=status, check=False)
    assert int(status) == 12
    check_balance(l, c, loss, counts, live)                      # they are not counted
    big = c.clone()
    big[3, 1], big[400, 29] = 2 ** 40 + 1, -2 ** 40
    again = iq.expert_balance(l, big.to(DEV), status=status, check=False)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts)


def test_balance_of_nothing():
    none = torch.empty((0, 9), device=DEV)
    for l, c in ((none, torch.empty((0, 2), dtype=torch.int32, device=DEV)),
                 (torch.full((700, 9), -INF, device=DEV), torch.full((700, 2), -1, dtype=torch.int32, device=DEV)),
                 (normal((700, 9), 1), torch.full((700, 2), -1, dtype=torch.int32, device=DEV))):
        loss, counts, live = iq.expert_balance(l, c)
        assert float(loss) == 0 and not counts.any()
        assert int(live) == int(torch.isfinite(l).any(dim=1).sum())
        grad = iq.expert_balance_backward(torch.ones((), device=DEV), l, counts, live)
        assert grad.shape == l.shape and not grad.any()
    choice, weights = iq.expert_gate(none, 2)
    assert choice.shape == weights.shape == (0, 2)
    assert iq.expert_gate_backward(weights, none, choice, weights).shape == (0, 9)


def test_even_use_has_a_loss_of_one():
    l = torch.zeros((64, 8), device=DEV)
    c = (torch.arange(128).view(64, 2) % 8).to(DEV)
    loss, counts, live = iq.expert_balance(l, c)
    assert float(loss) == 1.0 and counts.tolist() == [16] * 8 and int(live) == 64


# ---------------------------------------------------------------------------
# In autograd's graph, on streams, in graphs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients_are_those_of_the_calls(dtype, renormalize):
    l = router_logits(50, 40, 1, dtype)
    g = normal((50, 4), 2)
    choice, weights = iq.expert_gate(l, 4, renormalize=renormalize)
    loss, counts, live = iq.expert_balance(l, choice)
    half = torch.tensor(0.5, device=DEV)
    want = (iq.expert_gate_backward(g, l, choice, weights, renormalize=renormalize)
            + iq.expert_balance_backward(half, l, counts, live))
    leaf = l.clone().requires_grad_()
    c, w = iq.expert_gate(leaf, 4, renormalize=renormalize)
    b, n, t = iq.expert_balance(leaf, c)
    assert w.requires_grad and b.requires_grad and not c.requires_grad and not n.requires_grad
    assert torch.equal(c, choice) and torch.equal(w, weights) and torch.equal(b, loss)
    ((w * g).sum() + 0.5 * b).backward()
    assert leaf.grad.dtype == dtype and torch.equal(leaf.grad, want)
    # the sum's gradient is one value for all
    leaf.grad = None
    iq.expert_gate(leaf, 4, renormalize=renormalize)[1].sum().backward()
    assert torch.equal(leaf.grad, iq.expert_gate_backward(torch.ones_like(w), l, choice, weights,
                                                          renormalize=renormalize))
    # gradients of gradients are refused
    c, w = iq.expert_gate(leaf, 4, renormalize=renormalize)
    (first,) = torch.autograd.grad((w * g).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="has no gradient"):
        first.sum().backward()


def test_gradients_against_differences():
    """Central differences in 64 bits around fp32 logits: the gradient is the formula's, the
    difference off by a third of h^2 times a third derivative below 8 of sums of weights below 8."""
    l = router_logits(6, 12, 4, torch.float32)
    g = normal((6, 3), 5)
    l64, g64, h = to64(l), to64(g), 1e-4
    for renormalize in (True, False):
        leaf = l.clone().requires_grad_()
        c, w = iq.expert_gate(leaf, 3, renormalize=renormalize)
        loss, _, _ = iq.expert_balance(leaf, c)
        ((w * g).sum() + loss).backward()
        got = to64(leaf.grad)
        size = np.abs(g64).sum() + 12
        for i, e in np.ndindex(l64.shape):
            if not np.isfinite(l64[i, e]):
                assert got[i, e] == 0
                continue
            side = []
            for d in (h, -h):
                m = l64.copy()
                m[i, e] += d
                c2, w2 = ref.gate(m, 3, renormalize)
                if not np.array_equal(c2, c.cpu().numpy()):
                    break
                side.append((g64 * w2).sum() + ref.balance(m, c2)[0])
            if len(side) == 2:
                assert abs((side[0] - side[1]) / (2 * h) - got[i, e]) <= 8 * size * h * h + 1e-5


def test_argument_errors():
    l = normal((6, 10), 1)
    c, w = iq.expert_gate(l, 2)
    _, n, t = iq.expert_balance(l, c)
    one = torch.ones((), device=DEV)
    for call in (lambda: iq.expert_gate(l[0], 2), lambda: iq.expert_gate(l.T.contiguous().T, 2),
                 lambda: iq.expert_gate_backward(w[:5], l, c, w), lambda: iq.expert_gate_backward(w, l, c[:5], w),
                 lambda: iq.expert_gate_backward(w.T.contiguous().T, l, c, w),
                 lambda: iq.expert_balance(l, c[:5]), lambda: iq.expert_balance(l, c[:, 0]),
                 lambda: iq.expert_balance_backward(w, l, n, t), lambda: iq.expert_balance_backward(one, l, n[:9], t),
                 lambda: iq.expert_balance_backward(one, l, n, n)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: iq.expert_gate(l.double(), 2), lambda: iq.expert_gate(l, 2.0),
                 lambda: iq.expert_gate(l, 2, renormalize=1), lambda: iq.expert_gate_backward(w, l, c.long(), w),
                 lambda: iq.expert_gate_backward(w.double(), l, c, w), lambda: iq.expert_balance(l, w),
                 lambda: iq.expert_balance_backward(one.double(), l, n, t),
                 lambda: iq.expert_balance_backward(one, l, n.float(), t)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: iq.expert_gate(l, 0), lambda: iq.expert_gate(l, 11), lambda: iq.expert_gate(l, -1),
                 lambda: iq.expert_gate(normal((2, 513), 1), 2),
                 lambda: iq.expert_balance(normal((2, 513), 1), c[:2])):
        with pytest.raises(iq.IQError) as e:
            call()
        assert e.value.name == "IQ_ERR_SHAPE"


@pytest.mark.parametrize("tokens,experts", [(4, 16), (300, 64), (9000, 130)])
def test_on_another_stream_and_in_a_graph(tokens, experts):
    l = router_logits(tokens, experts, 1, torch.bfloat16)
    g, one = normal((tokens, 3), 2), torch.ones((), device=DEV)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        c, w = iq.expert_gate(l, 3, renormalize=False, status=word, check=False)
        loss, n, t = iq.expert_balance(l, c, status=word, check=False)
        return (c, w, loss, n, t, iq.expert_gate_backward(g, l, c, w, renormalize=False),
                iq.expert_balance_backward(one, l, n, t))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                r = step()
            graphs.append((graph, r))
    for i in range(4):
        l.copy_(router_logits(tokens, experts, 30 + i, torch.bfloat16))
        want = [t.clone() for t in step()]
        for graph, r in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert int(word) == 0


# ---------------------------------------------------------------------------
# Together with the experts' products
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 8, 2), (40, 16, 2), (300, 8, 3)])
def test_an_expert_layer_from_its_logits(dtype, tokens, experts, top_k):
    """Router, sort, products with 4-bit weights, combine: against the same in 64 bits."""
    channels, depth = 70, 160
    l = router_logits(tokens, experts, 1, torch.float32)
    x = normal((tokens, depth), 2, dtype)
    q, s = iq.quantize_groups(normal((experts * channels, depth), 3) * 0.1)
    q, s = q.view(experts, channels, -1), s.view(experts, channels, -1)
    choice, weights = iq.expert_gate(l, top_k)
    order, position, offsets = iq.expert_sort(choice, experts)
    y = iq.fp4_expert_linear(x, q, s, offsets, order, top_k=top_k)
    out = iq.expert_combine(y, position, offsets, weights)

    v, x64 = ref.values(q.cpu().numpy(), s.cpu().numpy()), to64(x)
    c, w = ref.gate(to64(l), top_k, True)
    assert np.array_equal(choice.cpu().numpy(), c)
    want, bound = np.zeros((tokens, channels)), np.zeros((tokens, channels))
    rel = ref.softmax_error(to64(l))
    for t in range(tokens):
        for j in range(top_k):
            if c[t, j] < 0:
                continue
            one, size = ref.product(x64[t:t + 1], v[c[t, j]])
            off = ref.product_bound(one, size, depth, dtype)[0]
            want[t] += w[t, j] * one[0]
            # the product's error, the weight's, and combine's product and sum
            bound[t] += w[t, j] * (off + (np.abs(one[0]) + off) * (rel[t] + (top_k + 2) * 2.0 ** -24))
    within(out, want, bound * (1 + ROUND[dtype]), dtype)
    empty = (c < 0).all(axis=1)
    assert not out[torch.from_numpy(empty).to(DEV)].any()


def test_a_training_step_of_the_router():
    """Gate, balance loss, dispatch and combine in one graph: the gradient of the logits is that of
    the weights' path and of the loss together."""
    tokens, experts, top_k, width = 60, 12, 3, 40
    l = router_logits(tokens, experts, 1, torch.float32).requires_grad_()
    x = normal((tokens, width), 2).requires_grad_()
    d = normal((experts, width), 3)
    choice, weights = iq.expert_gate(l, top_k)
    loss, counts, live = iq.expert_balance(l, choice)
    order, position, offsets = iq.expert_sort(choice, experts)
    rows = iq.expert_dispatch(x, position, offsets)
    place = torch.arange(rows.shape[0], device=DEV)
    expert = (place[:, None] >= offsets[None, 1:]).sum(dim=1).clamp(max=experts - 1)
    out = iq.expert_combine(rows * d[expert], position, offsets, weights)
    g = normal((tokens, width), 4)
    ((out * g).sum() + 0.01 * loss).backward()

    c = choice.cpu()
    kept = (c >= 0).double()
    l64 = l.detach().double().cpu().requires_grad_()
    x64 = x.detach().double().cpu().requires_grad_()
    p = torch.where(torch.isfinite(l64).any(dim=1, keepdim=True),
                    torch.softmax(torch.where(torch.isfinite(l64).any(dim=1, keepdim=True), l64, 0.0), dim=1), 0.0)
    chosen = torch.gather(p, 1, c.clamp(min=0).long()) * kept
    w = chosen / chosen.sum(dim=1, keepdim=True).clamp(min=1e-300)
    out64 = (w[:, :, None] * x64[:, None, :] * d.double().cpu()[c.clamp(min=0).long()]).sum(dim=1)
    share = counts.double().cpu() / counts.sum().cpu()
    loss64 = experts * (share * p.sum(dim=0) / int(live)).sum()
    ((out64 * g.double().cpu()).sum() + 0.01 * loss64).backward()
    # a few dozen fp32 roundings of the terms, whose sizes are those of the sums below
    size = (x64.detach().abs()[:, None, :] * d.double().cpu()[c.clamp(min=0).long()].abs()
            * g.double().cpu().abs()[:, None, :]).sum(dim=2).max(dim=1, keepdim=True).values + 1
    assert (out.detach().double().cpu() - out64.detach()).abs().max() <= 64 * 2.0 ** -24 * 20
    assert ((l.grad.double().cpu() - torch.nan_to_num(l64.grad)).abs() <= 128 * 2.0 ** -24 * size).all()
    assert (x.grad.double().cpu() - x64.grad).abs().max() <= 64 * 2.0 ** -24 * 50
    assert l.grad.any() and x.grad.any()


def test_more_choices_than_experts_are_refused_before_room_is_made_for_them():
    l = normal((6, 10), 1)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for top_k in (11, 10 ** 6):
        with pytest.raises(iq.IQError) as e:
            iq.expert_gate(l, top_k)
        assert e.value.name == "IQ_ERR_SHAPE"
    assert torch.cuda.max_memory_allocated() - before < 10 ** 6
