"""The layer operators in autograd's graph: gradients arrive where there are some,
and a backward pass through an operator that has none raises."""

import sys

import pytest
import torch

from tests import layers_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402

DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]
TOKENS, TOP_K, EXPERTS, WIDTH = 23, 3, 5, 130


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed)).to(dtype).to(DEV)


def routing(seed=3, dropped=0.2):
    c = torch.randint(0, EXPERTS, (TOKENS, TOP_K), generator=gen(seed))
    c = torch.where(torch.rand(c.shape, generator=gen(seed + 1)) < dropped, -1, c)
    return iq.expert_sort(c.to(DEV), EXPERTS)


def test_dispatch_and_combine_against_64_bits():
    """A layer whose experts scale each value: dispatch, the scales, combine.

    Roundings in fp32: the answers one for the scale and those of combine; the gradient of x
    that of y (one product), the scale, a sum of top_k; that of the weights the scaled rows and a
    dot product of width terms."""
    _, p, f = routing()
    x, d = normal((TOKENS, WIDTH), 1), normal((TOKENS * TOP_K, WIDTH), 2)
    w = torch.rand((TOKENS, TOP_K), generator=gen(5)).to(DEV)
    g = normal((TOKENS, WIDTH), 6)
    x.requires_grad_(), w.requires_grad_()
    out = iq.expert_combine(iq.expert_dispatch(x, p, f) * d, p, f, w)
    assert out.requires_grad
    out.backward(g)

    kept = (p < f[-1])[:, :, None].double().cpu()
    at = p.long().cpu()
    x64, w64, d64, g64 = (t.detach().double().cpu() for t in (x, w, d, g))
    x64.requires_grad_(), w64.requires_grad_()
    terms = x64[:, None, :] * d64[at] * kept * w64[:, :, None]
    want = terms.sum(dim=1)
    want.backward(g64)
    eps = 2.0 ** -24 * (1 + 2.0 ** -7)
    size = terms.detach().abs().sum(dim=1)
    assert ((out.detach().double().cpu() - want.detach()).abs() <= (TOP_K + 2) * eps * size).all()
    size = (d64[at] * kept * w64.detach()[:, :, None] * g64[:, None, :]).abs().sum(dim=1)
    assert ((x.grad.double().cpu() - x64.grad).abs() <= (TOP_K + 2) * eps * size).all()
    size = (x64.detach()[:, None, :] * d64[at] * kept * g64[:, None, :]).abs().sum(dim=2)
    assert ((w.grad.double().cpu() - w64.grad).abs() <= (WIDTH + 2) * eps * size).all()
    assert x.grad.any() and w.grad.any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gradients_are_those_of_the_calls(dtype):
    _, p, f = routing()
    x, y = normal((TOKENS, WIDTH), 1, dtype), normal((TOKENS * TOP_K, WIDTH), 2, dtype)
    w = torch.rand((TOKENS, TOP_K), generator=gen(5)).to(DEV)
    g, gs = normal((TOKENS, WIDTH), 6, dtype), normal((TOKENS * TOP_K, WIDTH), 7, dtype)
    plain = iq.expert_dispatch(x, p, f), iq.expert_combine(y, p, f, w)
    want = (iq.expert_dispatch_backward(gs, p, f), *iq.expert_combine_backward(g, y, p, f, w))
    x.requires_grad_(), y.requires_grad_(), w.requires_grad_()
    xs, out = iq.expert_dispatch(x, p, f), iq.expert_combine(y, p, f, w)
    assert torch.equal(xs, plain[0]) and torch.equal(out, plain[1])
    xs.backward(gs)
    out.backward(g)
    for got, grad in zip((x.grad, y.grad, w.grad), want):
        assert torch.equal(got, grad)
    # gradients whose values are not consecutive in a row, or the same everywhere
    for grad in (g.t().contiguous().t(), torch.ones((), dtype=dtype, device=DEV).expand(TOKENS, WIDTH)):
        y.grad = w.grad = None
        iq.expert_combine(y, p, f, w).backward(grad)
        gy, gw = iq.expert_combine_backward(grad.contiguous(), y.detach(), p, f, w.detach())
        assert torch.equal(y.grad, gy) and torch.equal(w.grad, gw)
    # only one of the two is wanted
    y.grad = w.grad = None
    iq.expert_combine(y.detach(), p, f, w).backward(g)
    assert torch.equal(w.grad, want[2])
    iq.expert_combine(y, p, f, w.detach()).backward(g)
    assert torch.equal(y.grad, want[1])


def test_gradients_of_gradients():
    _, p, f = routing()
    x, gs = normal((TOKENS, WIDTH), 1), normal((TOKENS * TOP_K, WIDTH), 2)
    x.requires_grad_(), gs.requires_grad_()
    (grad,) = torch.autograd.grad(iq.expert_dispatch(x, p, f), x, gs, create_graph=True)
    assert torch.equal(grad, iq.expert_dispatch_backward(gs.detach(), p, f))
    h = normal((TOKENS, WIDTH), 3)
    (second,) = torch.autograd.grad(grad, gs, h)
    assert torch.equal(second, iq.expert_dispatch(h, p, f))
    y, w = normal((TOKENS * TOP_K, WIDTH), 4).requires_grad_(), torch.ones((TOKENS, TOP_K), device=DEV)
    (grad,) = torch.autograd.grad(iq.expert_combine(y, p, f, w), y, h.requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="expert_combine_backward has no gradient"):
        grad.sum().backward()


def products(x, w_scale):
    """(name, call) of every product, on activations or scales that may require gradients."""
    w = torch.randint(-127, 128, (40, 64), generator=gen(8), dtype=torch.int8).to(DEV)
    q, s = iq.quantize_rows(x)
    f = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=DEV)
    return [("int8_linear", lambda **k: iq.int8_linear(x, w, w_scale, **k)),
            ("int8_matmul", lambda **k: iq.int8_matmul(q, s, w, w_scale, **k)),
            ("int8_expert_matmul", lambda **k: iq.int8_expert_matmul(q, s, w[None], w_scale[None], f, **k))]


def test_products_have_no_gradient():
    x = normal((9, 64), 1, torch.bfloat16)
    scale = torch.rand(40, generator=gen(9)).to(DEV) + 0.1
    plain = [call() for _, call in products(x, scale)]
    scale.requires_grad_()
    for (name, call), want in zip(products(x, scale), plain):
        y = call()
        assert y.requires_grad and torch.equal(y, want)
        with pytest.raises(RuntimeError, match=name + " has no gradient"):
            y.sum().backward()
        with torch.no_grad():
            assert not call().requires_grad
    x.requires_grad_()
    y = products(x, scale.detach())[0][1]()
    with pytest.raises(RuntimeError, match="int8_linear has no gradient"):
        y.sum().backward()
    bad = x.detach().clone()
    bad[2, 3] = float("nan")
    with pytest.raises(iq.IQError):
        iq.int8_linear(bad.requires_grad_(), torch.ones((40, 64), dtype=torch.int8, device=DEV), scale)


def test_codes_are_constants():
    x = normal((9, 64), 1).requires_grad_()
    q, s = iq.quantize_rows(x)
    assert not q.requires_grad and not s.requires_grad


def test_out_is_refused_where_gradients_are_recorded():
    _, p, f = routing()
    x, y = normal((TOKENS, WIDTH), 1), normal((TOKENS * TOP_K, WIDTH), 2)
    w = torch.rand((TOKENS, TOP_K), generator=gen(5)).to(DEV)
    small = normal((9, 64), 1, torch.bfloat16)
    calls = [(lambda out: iq.expert_dispatch(x, p, f, out=out), torch.zeros_like(y)),
             (lambda out: iq.expert_dispatch_backward(y, p, f, out=out), torch.zeros_like(x)),
             (lambda out: iq.expert_combine(y, p, f, w, out=out), torch.zeros_like(x))]
    scale = torch.rand(40, generator=gen(9)).to(DEV)
    for _, call in products(small, scale):
        calls.append((lambda out, call=call: call(out=out), torch.zeros((9, 40), dtype=torch.bfloat16, device=DEV)))
    for t in (x, y, scale):
        t.requires_grad_()
    for call, out in calls:
        with pytest.raises(ValueError, match="out cannot be given"):
            call(out)
        assert not out.any()
        with torch.no_grad():
            assert call(out) is out and out.any()


def test_a_saved_tensor_that_was_written_over_is_noticed():
    _, p, f = routing()
    y = torch.zeros((TOKENS * TOP_K, WIDTH), device=DEV)
    w = torch.ones((TOKENS, TOP_K), device=DEV, requires_grad=True)
    out = iq.expert_combine(y, p, f, w)
    iq.expert_dispatch(normal((TOKENS, WIDTH), 1), p, f, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
