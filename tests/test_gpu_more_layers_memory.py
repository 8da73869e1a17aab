"""Whose memory the router's and the 4-bit operators read and write: rows far apart,
results that lie in inputs, results that autograd has saved, views with other signs."""

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402

DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def apart(t):
    """The same rows, the last of which begins beyond 2^32 bytes."""
    ld = 2 ** 32 // ((len(t) - 1) * t.element_size()) + 1027
    return torch.empty((len(t), ld), dtype=t.dtype, device=DEV)[:, :t.shape[1]].copy_(t)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_logits_beyond_32_bits(dtype):
    l = normal((300, 33), 1, dtype)
    far = apart(l)
    for renormalize in (True, False):
        choice, weights = iq.expert_gate(l, 3, renormalize=renormalize)
        got = iq.expert_gate(far, 3, renormalize=renormalize)
        assert torch.equal(got[0], choice) and torch.equal(got[1], weights)
        assert torch.equal(iq.expert_gate_backward(weights, far, choice, weights, renormalize=renormalize),
                           iq.expert_gate_backward(weights, l, choice, weights, renormalize=renormalize))
    loss, counts, live = iq.expert_balance(l, choice)
    got = iq.expert_balance(far, choice)
    assert torch.equal(got[0], loss) and torch.equal(got[1], counts) and torch.equal(got[2], live)
    assert torch.equal(iq.expert_balance_backward(loss, far, counts, live),
                       iq.expert_balance_backward(loss, l, counts, live))


def calls_with_out(tokens=6):
    """(call taking out=, a fitting out) of every operator that takes one."""
    w, s = iq.quantize_groups(normal((64, 64), 1))
    x = normal((tokens, 64), 2, torch.bfloat16)
    f = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    return [(call, torch.zeros((tokens, 64), dtype=torch.bfloat16, device=DEV)) for call in (
        lambda out: iq.fp4_linear(x, w, s, out=out),
        lambda out: iq.fp4_expert_linear(x, w[None], s[None], f, out=out),
        lambda out: iq.dequantize_groups(w[:tokens], s[:tokens], dtype=torch.bfloat16, out=out))]


def test_writing_a_result_makes_a_new_version():
    for call, out in calls_with_out():
        before = out._version
        assert call(out) is out and out._version > before
        leaf = torch.ones((6, 64), device=DEV, requires_grad=True)
        loss = (leaf.bfloat16() * out).sum()                 # saves out
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


def test_results_in_inputs_are_refused():
    w, s = iq.quantize_groups(normal((64, 64), 1))
    x = normal((6, 64), 2, torch.bfloat16)
    both = torch.zeros((6, 130), dtype=torch.bfloat16, device=DEV)
    f = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    for call in (lambda: iq.fp4_linear(x, w, s, out=x),
                 lambda: iq.fp4_linear(both[:, :64], w, s, out=both[:, 63:127]),
                 lambda: iq.fp4_expert_linear(x, w[None], s[None], f, out=x),
                 lambda: iq.fp4_linear(x, w, s, out=w.view(-1)[:768].view(torch.bfloat16).view(6, 64))):
        with pytest.raises(iq.IQError) as e:
            call()
        assert e.value.name == "IQ_ERR_ARG"
    # columns of one buffer beside each other are not
    iq.fp4_linear(both[:, :64], w, s, out=both[:, 64:128])


def test_negated_views_are_refused():
    """The imaginary part of a conjugate is a view of the values with the other sign."""
    x = torch.complex(normal((12, 1), 1), normal((12, 1), 2)).conj().imag
    assert x.is_neg()
    choice = torch.zeros((12, 1), dtype=torch.int32, device=DEV)
    for call in (lambda: iq.expert_gate(x, 1), lambda: iq.expert_balance(x, choice)):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()


def test_two_graphs_share_no_workspace():
    """Two captured products that need a workspace, replayed in turn and on two streams."""
    w, s = iq.quantize_groups(normal((1100, 352), 1))
    xs = [normal((700, 352), seed) for seed in (2, 3)]
    want = [iq.fp4_linear(x, w, s) for x in xs]
    logits = [normal((70000, 16), seed) for seed in (4, 5)]
    choice = [iq.expert_gate(l, 2)[0] for l in logits]
    losses = [iq.expert_balance(l, c)[0] for l, c in zip(logits, choice)]
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    graphs, got = [], []
    for x, l, c in zip(xs, logits, choice):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append((iq.fp4_linear(x, w, s), iq.expert_balance(l, c, status=word, check=False)[0]))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(6):
        for y, loss in got:
            y.zero_()
            loss.zero_()
        torch.cuda.synchronize()
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream if turn % 2 else torch.cuda.current_stream()):
                g.replay()
        torch.cuda.synchronize()
        for (y, loss), a, b in zip(got, want, losses):
            assert torch.equal(y, a) and torch.equal(loss, b)
    assert word.item() == 0
