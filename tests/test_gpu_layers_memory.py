"""What the layer operators do with the memory of their arguments: slices of one
buffer side by side are taken, overlapping ones are refused."""

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_results_beside_their_inputs(tokens):
    w, ws = iq.quantize_rows(normal((64, 64), 1))
    x = normal((tokens, 64), 2, torch.bfloat16)
    want = iq.int8_linear(x, w, ws)
    both = torch.zeros((tokens, 128), dtype=torch.bfloat16, device=DEV)
    both[:, :64] = x
    assert torch.equal(iq.int8_linear(both[:, :64], w, ws, out=both[:, 64:]), want)
    assert torch.equal(both[:, :64], x) and torch.equal(both[:, 64:], want)
    # rows of two in every row of the buffer: strides that differ
    if tokens > 1:
        buf = torch.zeros((tokens, 256), dtype=torch.bfloat16, device=DEV)
        held, out = buf[:, :64], buf.view(2 * tokens, 128)[1:tokens + 1, 64:]
        held.copy_(x)
        assert torch.equal(iq.int8_linear(held, w, ws, out=out), want)
        assert torch.equal(held, x)


@pytest.mark.parametrize("tokens", [5, 70])
def test_overlapping_results_are_refused(tokens):
    w, ws = iq.quantize_rows(normal((64, 64), 1))
    x = normal((tokens, 64), 2, torch.bfloat16)
    both = torch.zeros((tokens, 128), dtype=torch.bfloat16, device=DEV)
    p = torch.arange(tokens, dtype=torch.int32, device=DEV)[:, None]
    f = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    one = torch.ones((tokens, 1), device=DEV)
    raw = torch.zeros(tokens * 128, dtype=torch.int8, device=DEV)
    for call in (lambda: iq.int8_linear(x, w, ws, out=x),
                 lambda: iq.int8_linear(both[:, :64], w, ws, out=both[:, 63:127]),
                 lambda: iq.int8_matmul(raw[:tokens * 64].view(tokens, 64), one[:, 0], w, ws,
                                        out=raw.view(torch.bfloat16).view(tokens, 64)),
                 lambda: iq.int8_expert_matmul(raw[tokens * 64:].view(tokens, 64), one[:, 0], w[None], ws[None], f,
                                               out=raw.view(torch.bfloat16).view(tokens, 64)),
                 lambda: iq.expert_dispatch(x, p, f, out=x),
                 lambda: iq.expert_dispatch_backward(x, p, f, out=x),
                 lambda: iq.expert_combine(x, p, f, one, out=x)):
        with pytest.raises(iq.IQError) as e:
            call()
        assert e.value.name == "IQ_ERR_ARG"


def calls_with_out(tokens=6):
    """(call taking out=, a fitting out) of every operator that takes one."""
    w, ws = iq.quantize_rows(normal((64, 64), 1))
    x = normal((tokens, 64), 2, torch.bfloat16)
    q, s = iq.quantize_rows(x)
    p = torch.arange(tokens, dtype=torch.int32, device=DEV)[:, None]
    f = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    one = torch.ones((tokens, 1), device=DEV)
    return [(call, torch.zeros((tokens, 64), dtype=torch.bfloat16, device=DEV)) for call in (
        lambda out: iq.int8_linear(x, w, ws, out=out), lambda out: iq.int8_matmul(q, s, w, ws, out=out),
        lambda out: iq.int8_expert_matmul(q, s, w[None], ws[None], f, out=out),
        lambda out: iq.expert_dispatch(x, p, f, out=out),
        lambda out: iq.expert_dispatch_backward(x, p, f, out=out),
        lambda out: iq.expert_combine(x, p, f, one, out=out))]


def test_writing_a_result_makes_a_new_version():
    for call, out in calls_with_out():
        before = out._version
        assert call(out) is out and out._version > before
    # a tensor that a graph has saved and that was written over since is noticed
    for call, out in calls_with_out():
        leaf = torch.ones((6, 64), device=DEV, requires_grad=True)
        product = leaf * out.float().mul_(1.0)               # saves a copy: not affected
        call(out)
        product.sum().backward()
        loss = (leaf.bfloat16() * out).sum()                 # saves out itself
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_writing_results_in_inference_mode():
    with torch.inference_mode():
        for call, out in calls_with_out():
            assert out.is_inference() and call(out) is out and out.any()
    for call, out in calls_with_out():
        with torch.inference_mode():
            held = torch.zeros_like(out)
        assert call(held) is held and held.any()


def test_negated_views_are_refused():
    """The imaginary part of a conjugate is a view of the values with the other sign."""
    z = torch.complex(normal((12, 1), 1), normal((12, 1), 2))
    x = z.conj().imag
    assert x.is_neg()
    with pytest.raises(ValueError, match="resolve_neg"):
        iq.quantize_rows(x)
    q, _ = iq.quantize_rows(x.resolve_neg())
    assert torch.equal(q.float(), 127 * torch.sign(-z.imag))
