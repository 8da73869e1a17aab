"""What autograd has to know of the 4-bit weights and the router."""

import sys

import pytest
import torch
import torch.autograd.forward_ad as fwd

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


def test_values_are_not_written_into_a_recorded_tensor():
    codes, scale = iq.quantize_groups(normal((6, 64), 1))
    want = iq.dequantize_groups(codes, scale)
    leaf = normal((6, 64), 2).requires_grad_()
    before = leaf.detach().clone()
    computed = leaf * 2.0
    for out in (leaf, computed, computed[:, :64]):
        with pytest.raises(ValueError, match="out cannot be given"):
            iq.dequantize_groups(codes, scale, out=out)
    assert torch.equal(leaf.detach(), before)
    computed.sum().backward()
    assert torch.equal(leaf.grad, torch.full_like(leaf, 2.0))
    # where nothing is recorded they are, as torch's own results
    with torch.no_grad():
        assert iq.dequantize_groups(codes, scale, out=leaf) is leaf
    assert torch.equal(leaf.detach(), want)


def calls():
    """Every call that autograd could record, by one of its floating-point arguments."""
    x, logits = normal((6, 64), 1), normal((6, 8), 2)
    w, s = iq.quantize_groups(normal((10, 64), 3))
    q, qs = iq.quantize_rows(normal((10, 64), 3))
    xq, xs = iq.quantize_rows(x)
    choice, weights = iq.expert_gate(logits, 2)
    order, position, offsets = iq.expert_sort(choice, 8)
    _, counts, live = iq.expert_balance(logits, choice)
    rows, grad, loss_grad = normal((12, 64), 4), normal((6, 2), 5), torch.ones((), device=DEV)
    one = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    return [
        ("expert_gate", lambda v: iq.expert_gate(v, 2), logits),
        ("expert_gate of probabilities", lambda v: iq.expert_gate(v, 2, renormalize=False), logits),
        ("expert_gate_backward", lambda v: iq.expert_gate_backward(v, logits, choice, weights), grad),
        ("expert_gate_backward, logits",
         lambda v: iq.expert_gate_backward(grad, v, choice, weights, renormalize=False), logits),
        ("expert_gate_backward, weights", lambda v: iq.expert_gate_backward(grad, logits, choice, v), weights),
        ("expert_balance", lambda v: iq.expert_balance(v, choice), logits),
        ("expert_balance_backward", lambda v: iq.expert_balance_backward(v, logits, counts, live), loss_grad),
        ("expert_balance_backward, logits",
         lambda v: iq.expert_balance_backward(loss_grad, v, counts, live), logits),
        ("fp4_linear", lambda v: iq.fp4_linear(v, w, s), x),
        ("fp4_linear, out", lambda v: iq.fp4_linear(x, w, s, out=v), normal((6, 10), 6)),
        ("fp4_expert_linear", lambda v: iq.fp4_expert_linear(v, w[None], s[None], one), x),
        ("dequantize_groups, out", lambda v: iq.dequantize_groups(w, s, out=v), normal((10, 64), 7)),
        ("int8_linear", lambda v: iq.int8_linear(v, q, qs), x),
        ("int8_matmul", lambda v: iq.int8_matmul(xq, v, q, qs), xs),
        ("int8_expert_matmul", lambda v: iq.int8_expert_matmul(xq, v, q[None], qs[None], one), xs),
        ("expert_dispatch", lambda v: iq.expert_dispatch(v, position, offsets), x),
        ("expert_dispatch_backward", lambda v: iq.expert_dispatch_backward(v, position, offsets), rows),
        ("expert_combine", lambda v: iq.expert_combine(v, position, offsets, weights), rows),
        ("expert_combine, weights", lambda v: iq.expert_combine(rows, position, offsets, v), weights),
        ("expert_combine_backward",
         lambda v: iq.expert_combine_backward(x, v, position, offsets, weights), rows),
    ]


@pytest.mark.parametrize("recording", [True, False])
def test_tangents_are_refused(recording):
    """No operator has a rule for forward mode; an answer without the tangent would count as
    a constant.  (Forward mode goes on under no_grad, in torch's functions too.)"""
    for name, call, value in calls():
        value = value.clone()
        before = value.clone()
        with torch.set_grad_enabled(recording), fwd.dual_level():
            dual = fwd.make_dual(value, torch.ones_like(value))
            with pytest.raises((NotImplementedError, ValueError)):
                call(dual)
                pytest.fail("%s answered without a tangent" % name)
            assert torch.equal(value, before), name
            # its value alone is an ordinary tensor
            call(fwd.unpack_dual(dual).primal.detach())
        call(value)


@pytest.mark.parametrize("renormalize", [True, False])
def test_logits_written_over_after_the_gate(renormalize):
    """The gradient of renormalized weights does not read the logits: they may be written over
    (masked for the next pass, say) and need not be kept.  That of probabilities does."""
    for dtype in (torch.float32, torch.bfloat16):
        leaf = normal((9, 8), 1, dtype).requires_grad_()
        grad = normal((9, 3), 2)
        _, weights = iq.expert_gate(leaf * 1.0, 3, renormalize=renormalize)
        want, = torch.autograd.grad(weights, leaf, grad)
        logits = leaf * 1.0
        _, weights = iq.expert_gate(logits, 3, renormalize=renormalize)
        logits.masked_fill_(torch.ones((9, 8), dtype=torch.bool, device=DEV), -float("inf"))
        if renormalize:
            got, = torch.autograd.grad(weights, leaf, grad, allow_unused=True)
            assert got is not None and got.dtype == dtype
            # masked_fill_ comes behind the gate in the graph and takes nothing from its gradient
            assert torch.equal(got, want)
        else:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                torch.autograd.grad(weights, leaf, grad)
    # without tokens
    empty = torch.empty((0, 8), device=DEV, requires_grad=True)
    _, weights = iq.expert_gate(empty, 3, renormalize=renormalize)
    weights.sum().backward()
    assert empty.grad.shape == (0, 8)
