"""The layer operators where one launch cannot hold the work: 2^32 threads and
more, reached with rows of one value (or rows that are all the same one), and
checked value by value against torch's own elementary operations."""

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
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def small(shape, seed, dtype=torch.float32):
    """Integers within -8..8: their products are exact in every type."""
    return torch.randint(-8, 9, shape, generator=gen(seed), device=DEV, dtype=torch.int8).to(dtype)


def powers(shape, seed):
    """Scales that are powers of two: products with them are exact."""
    return torch.exp2(torch.randint(-3, 4, shape, generator=gen(seed), device=DEV, dtype=torch.int8).float())


def test_quantize_rows():
    rows = 2 ** 26 + 3                        # 64 lanes each
    x = small((rows, 1), 1)
    q, s = iq.quantize_rows(x)
    one = torch.tensor(1.0, device=DEV) / torch.tensor(127.0, device=DEV)
    assert torch.equal(s, x[:, 0].abs() * one)
    # x / (|x| / 127), the scale rounded, is within 2^-23 of 127
    assert torch.equal(q, (torch.sign(x) * 127).to(torch.int8))
    x[rows - 2] = float("nan")
    with pytest.raises(iq.IQError) as e:
        iq.quantize_rows(x)
    assert e.value.name == "IQ_ERR_NONFINITE"


def test_linear():
    rows = 2 ** 26 + 3
    x = small((rows, 1), 2, torch.bfloat16)
    w = torch.full((1, 1), -127, dtype=torch.int8, device=DEV)
    y = iq.int8_linear(x, w, torch.full((1,), 2.0 / 127, device=DEV))
    # five roundings of fp32 on the way, then bf16 values that are exact
    assert torch.equal(y, -2 * x)


@pytest.mark.parametrize("tokens,channels", [(2 ** 28 + 3, 1), (1, 2 ** 28 + 3)])
def test_product(tokens, channels):
    row = small((1, 16), 3, torch.int8)
    x, w = row.expand(tokens, 16), row.expand(channels, 16)
    xs, ws = powers((tokens,), 4), powers((channels,), 5)
    y = iq.int8_matmul(x, xs, w, ws, dtype=torch.float32)
    total = float((row.float() ** 2).sum())
    assert torch.equal(y, total * xs[:, None] * ws)


def test_product_by_expert():
    rows, first = 2 ** 29 + 3, 2 ** 28 + 5
    x, xs = small((rows, 1), 6, torch.int8), powers((rows,), 7)
    w, ws = small((3, 1, 1), 8, torch.int8), powers((3, 1), 9)
    offsets = torch.tensor([0, first, first, rows - 20], dtype=torch.int32, device=DEV)
    y = iq.int8_expert_matmul(x, xs, w, ws, offsets, dtype=torch.float32)[:, 0]
    xs *= x[:, 0]
    of = [float(w[e]) * float(ws[e]) for e in range(3)]
    assert torch.equal(y[:first], xs[:first] * of[0])
    assert torch.equal(y[first:rows - 20], xs[first:rows - 20] * of[2])
    assert not y[rows - 20:].any()


def places(tokens, top_k):
    """Every choice's place, backwards; the last five places are dropped choices."""
    position = torch.arange(tokens * top_k - 1, -1, -1, dtype=torch.int32, device=DEV).view(tokens, top_k)
    return position, torch.tensor([0, tokens * top_k - 5], dtype=torch.int32, device=DEV)


def test_dispatch():
    tokens = 2 ** 28 + 3                      # 16 lanes each
    p, f = places(tokens, 1)
    x = small((tokens, 1), 10, torch.bfloat16)
    y = iq.expert_dispatch(x, p, f)
    x[:5] = 0
    assert torch.equal(y, x.flip(0))


def test_combine_and_the_gradient_of_dispatch():
    tokens = 2 ** 28 + 3
    p, f = places(tokens, 1)
    y, w = small((tokens, 1), 11, torch.bfloat16), powers((tokens, 1), 12)
    out, grad = iq.expert_combine(y, p, f, w), iq.expert_dispatch_backward(y, p, f)
    back = y.flip(0)
    back[:5] = 0
    assert torch.equal(grad, back)
    assert torch.equal(out, (back * w).to(torch.bfloat16))


def test_gradients_of_combine():
    tokens, top_k = 2 ** 26 + 3, 2            # 64 lanes each
    p, f = places(tokens, top_k)
    g, y = small((tokens, 1), 13), small((tokens * top_k, 1), 14)
    w = powers((tokens, top_k), 15)
    gy, gw = iq.expert_combine_backward(g, y, p, f, w)
    kept = torch.ones((tokens, top_k), device=DEV)
    kept.view(-1)[:5] = 0
    assert torch.equal(gw, g * y.flip(0).view(tokens, top_k) * kept)
    assert torch.equal(gy.flip(0).view(tokens, top_k), g * w * kept)
