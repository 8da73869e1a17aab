"""The layer operators against plain implementations in 64 bits (layers_ref.py),
at the sizes, strides, types and masks where they can go wrong.

Codes, scales, orders and copies have to be equal; computed values stay within
bounds that follow from the roundings each operator states.
"""

import sys

import numpy as np
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


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed)).to(dtype).to(DEV)


def codes(shape, seed):
    return torch.randint(-128, 128, shape, generator=gen(seed), dtype=torch.int8).to(DEV)


def scales(shape, seed):
    return (torch.rand(shape, generator=gen(seed)) * 0.02 + 0.001).to(DEV)


def within(got, want, bound):
    got = ref.to64(got)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), "worst %.3g over its bound at %s" % (over.max(), np.unravel_index(over.argmax(), over.shape))


def strided(t, pad, shift):
    """The same values in rows that are `pad` values longer and start `shift` values late."""
    rows, cols = t.shape
    buf = torch.empty(rows * (cols + pad) + shift + 16, dtype=t.dtype, device=t.device)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------
# quantize_rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 257), (7, 1024), (4, 1025), (9, 4096),
                                       (3, 4097), (2, 8192), (2, 20001), (260, 100)])
def test_quantize_rows(dtype, rows, cols):
    x = normal((rows, cols), rows * 10007 + cols, dtype)
    q, s = iq.quantize_rows(x)
    wq, ws = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_quantize_rows_strides(dtype, pad, shift):
    x = normal((6, 515), 11, dtype)
    q, s = iq.quantize_rows(strided(x, pad, shift))
    q0, s0 = iq.quantize_rows(x)
    assert torch.equal(q, q0) and torch.equal(s, s0)


def test_quantize_rows_ties_zeros_and_extremes():
    # 254 * 2^-7 over 127 is a power of two: quotients are exact halves.
    rows = [np.arange(-127, 128) / 2.0, np.zeros(255), np.full(255, 1e-45), np.full(255, 3.4e38),
            np.linspace(-1e-40, 1e-40, 255), np.r_[np.zeros(254), -5.0]]
    x = torch.tensor(np.array(rows, np.float32)).to(DEV)
    q, s = iq.quantize_rows(x)
    wq, ws = ref.quantize(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)
    assert not q[1].any() and s[1] == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_rows_reports_and_blanks_bad_rows(dtype, bad):
    for cols in (33, 5000):
        x = normal((5, cols), 12, dtype)
        x[3, cols - 1] = bad
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        q, s = iq.quantize_rows(x, status=st, check=False)
        assert int(st.item()) == 5
        wq, ws = ref.quantize(x.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
        assert not q[3].any() and s[3] == 0 and q[2].any()
        with pytest.raises(iq.IQError) as e:
            iq.quantize_rows(x)
        assert e.value.name == "IQ_ERR_NONFINITE"
        with pytest.raises(iq.IQError):
            iq.quantize_rows(x, status=torch.zeros(1, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------------
# The products
# ---------------------------------------------------------------------------

def check_product(x, w, dtype, seed=1):
    xs, ws = scales(x.shape[0], seed), scales(w.shape[0], seed + 1)
    y = iq.int8_matmul(x, xs, w, ws, dtype=dtype)
    assert y.dtype == dtype
    want = ref.product(x.cpu().numpy(), xs.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy())
    within(y, want, ref.product_bound(want, dtype))


TOKENS = [1, 2, 3, 15, 16, 17, 31, 33, 64, 65, 100, 129, 257]


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("channels,depth", [(256, 512), (130, 272), (1, 16), (33, 1040), (515, 128)])
def test_product_sizes(tokens, channels, depth):
    check_product(codes((tokens, depth), tokens), codes((channels, depth), channels), torch.float32)


@pytest.mark.parametrize("tokens", [1, 5, 20, 63, 140, 300])
@pytest.mark.parametrize("depth", [1, 2, 15, 17, 100, 129, 1001, 2050])
def test_product_odd_depths(tokens, depth):
    check_product(codes((tokens, depth), tokens), codes((75, depth), depth), torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels", [(1, 1024), (7, 260), (48, 1030), (300, 700), (700, 1200)])
def test_product_types(dtype, tokens, channels):
    check_product(codes((tokens, 768), 3), codes((channels, 768), 4), dtype)


@pytest.mark.parametrize("tokens", [1, 9, 40, 150, 600])
@pytest.mark.parametrize("pad,shift", [(16, 0), (16, 16), (1, 0), (0, 1), (7, 5)])
def test_product_strides(tokens, pad, shift):
    x, w = codes((tokens, 528), 5), codes((290, 528), 6)
    xs, ws = scales(tokens, 7), scales(290, 8)
    plain = iq.int8_matmul(x, xs, w, ws)
    assert torch.equal(plain, iq.int8_matmul(strided(x, pad, shift), xs, w, ws))
    assert torch.equal(plain, iq.int8_matmul(x, xs, strided(w, pad, shift), ws))
    out = strided(torch.zeros_like(plain), pad, shift)
    whole = out.as_strided((out.untyped_storage().nbytes() // out.element_size(),), (1,), 0)
    whole.fill_(7.0)
    assert iq.int8_matmul(x, xs, w, ws, out=out) is out
    assert torch.equal(plain, out)
    out.fill_(7.0)
    assert (whole == 7.0).all()                     # nothing beside the rows was written


# Shapes that take every tile size, with rows, channels and depths that end inside a tile.
LARGE = [(33, 300, 528), (700, 515, 1000), (500, 2049, 528), (700, 2049, 1000), (2600, 515, 2050),
         (1000, 2049, 1000), (2100, 2049, 528), (1300, 4100, 1000), (2600, 2049, 1000), (4100, 2049, 528),
         (4100, 2600, 2050), (190, 4100, 528), (3300, 515, 136), (130, 1540, 1000), (45, 515, 776),
         (70, 1030, 264), (100, 2049, 264), (4265, 403, 144), (978, 5530, 144), (1052, 5530, 144),
         (2366, 5197, 144), (90, 5530, 144), (164, 5530, 528), (127, 4531, 144),
         (9, 10990, 152), (203, 253, 152), (101, 5932, 528)]


def exact_product(x, xs, w, ws):
    """In 64 bits on the GPU: sums of products of 8-bit values are exact there."""
    return (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()


@pytest.mark.parametrize("tokens,channels,depth", LARGE)
@pytest.mark.parametrize("pad", [0, 16], ids=["dense", "padded"])
def test_product_tiles(tokens, channels, depth, pad):
    pad = -depth % 16 + pad if pad else 0            # padded rows start on 16 bytes
    x, w = codes((tokens, depth + pad), 1)[:, :depth], codes((channels, depth + pad), 2)[:, :depth]
    xs, ws = scales(tokens, 3), scales(channels, 4)
    want = ref.to64(exact_product(x, xs, w, ws))
    for dtype in DTYPES:
        within(iq.int8_matmul(x, xs, w, ws, dtype=dtype), want, ref.product_bound(want, dtype))


@pytest.mark.parametrize("tokens,channels,depth", LARGE)
@pytest.mark.parametrize("pad", [0, 16], ids=["dense", "padded"])
def test_expert_product_tiles(tokens, channels, depth, pad):
    experts, top_k = 5, 2
    pad = -depth % 16 + pad if pad else 0
    c = routing(tokens, top_k, experts, tokens, 0.1)
    c[tokens // 2:, 0] = torch.where(c[tokens // 2:, 0] < 0, -1, 2)     # one expert has most rows
    order, position, offsets = (torch.tensor(v).to(DEV) for v in ref.sort(c.numpy(), experts))
    x, w = codes((tokens, depth + pad), 1)[:, :depth], codes((experts, channels, depth + pad), 2)[:, :, :depth]
    xs, ws = scales(tokens, 3), scales((experts, channels), 4)
    want = torch.zeros((tokens * top_k, channels), dtype=torch.float64, device=DEV)
    ends = offsets.tolist()
    for e in range(experts):
        tok = (order[ends[e]:ends[e + 1]] // top_k).long()
        want[ends[e]:ends[e + 1]] = exact_product(x[tok], xs[tok], w[e], ws[e])
    want = ref.to64(want)
    y = iq.int8_expert_matmul(x, xs, w, ws, offsets, order, top_k=top_k, dtype=torch.bfloat16)
    within(y, want, ref.product_bound(want, torch.bfloat16))


def test_product_of_a_broadcast_row():
    x, w = codes((1, 256), 9), codes((140, 256), 10)
    xs, ws = scales(70, 11), scales(140, 12)
    y = iq.int8_matmul(x.expand(70, 256), xs, w, ws, dtype=torch.float32)
    assert torch.equal(y, iq.int8_matmul(x.repeat(70, 1), xs, w, ws, dtype=torch.float32))


@pytest.mark.parametrize("tokens", [1, 30, 200])
def test_product_of_extreme_codes_is_exact(tokens):
    # The largest sums that 32 bits have to hold: -128 * -128 * 131071.
    depth = 131071 if tokens == 1 else 131056
    x = torch.full((tokens, depth), -128, dtype=torch.int8, device=DEV)
    w = torch.full((40, depth), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    one = torch.ones(tokens, device=DEV), torch.ones(40, device=DEV)
    y = iq.int8_matmul(x, one[0], w, one[1], dtype=torch.float32)
    want = np.where(np.arange(40) % 2, -128.0 * 127, 128.0 * 128) * depth
    assert np.array_equal(ref.to64(y), np.broadcast_to(want.astype(np.float32), (tokens, 40)))


@pytest.mark.parametrize("tokens", [3, 40, 200])
def test_product_beyond_32_bit_offsets(tokens):
    stride = (2 ** 32 // tokens // 16 + 16) * 16
    x, w = codes((tokens, 64), 13), codes((20, 64), 14)
    xs, ws = scales(tokens, 15), scales(20, 16)
    plain = iq.int8_matmul(x, xs, w, ws)
    buf = torch.empty(tokens * stride, dtype=torch.int8, device=DEV)
    far = buf.view(tokens, stride)[:, :64]
    far.copy_(x)
    assert torch.equal(plain, iq.int8_matmul(far, xs, w, ws))
    wide = (2 ** 32 // 20 // 16 + 16) * 16
    buf2 = torch.empty(20 * wide, dtype=torch.int8, device=DEV)
    farw = buf2.view(20, wide)[:, :64]
    farw.copy_(w)
    assert torch.equal(plain, iq.int8_matmul(x, xs, farw, ws))
    outs = torch.empty(tokens * (stride // 2), dtype=torch.bfloat16, device=DEV)
    out = outs.view(tokens, stride // 2)[:, :20]
    iq.int8_matmul(x, xs, w, ws, out=out)
    assert torch.equal(plain, out)


def test_product_of_no_tokens():
    y = iq.int8_matmul(codes((0, 64), 1), scales(0, 1), codes((8, 64), 2), scales(8, 2))
    assert y.shape == (0, 8)
    assert iq.int8_linear(normal((0, 64), 1), codes((8, 64), 2), scales(8, 2)).shape == (0, 8)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", [(1, 1024, 4096), (1, 33, 100), (2, 515, 1040), (5, 64, 16),
                                                   (8, 256, 5000), (17, 100, 512), (70, 300, 768),
                                                   (200, 515, 1001), (16, 75, 1024), (16, 75, 1025),
                                                   (4, 64, 4096), (3, 40, 7), (1, 20, 16384),
                                                   (1, 20, 16385), (11, 1, 513), (2, 4097, 8), (8, 50, 1024),
                                                   (2, 40, 4096), (3, 16384, 100), (3, 16385, 100),
                                                   (1, 20, 12345), (8, 50, 1000)])
def test_linear(dtype, tokens, channels, depth):
    x = normal((tokens, depth), tokens + depth, dtype)
    w, ws = iq.quantize_rows(normal((channels, depth), channels))
    y = iq.int8_linear(x, w, ws)
    q, s = ref.quantize(x.float().cpu().numpy())
    want = ref.product(q, s, w.cpu().numpy(), ws.cpu().numpy())
    within(y, want, ref.product_bound(want, dtype))
    # the two calls it stands for give the same bits, and so does any stride
    assert torch.equal(y, iq.int8_matmul(*iq.quantize_rows(x), w, ws, dtype=dtype))
    assert torch.equal(y, iq.int8_linear(strided(x, 3, 1), w, ws))


@pytest.mark.parametrize("tokens", [2, 40])
def test_linear_answers_bad_tokens_with_zeros(tokens):
    x = normal((tokens, 300), 20, torch.bfloat16)
    w, ws = iq.quantize_rows(normal((90, 300), 21))
    good = iq.int8_linear(x, w, ws)
    x[1, 299] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = iq.int8_linear(x, w, ws, status=st, check=False)
    assert int(st.item()) == 5
    assert not y[1].any() and torch.equal(y[0], good[0]) and torch.equal(y[2:], good[2:])
    with pytest.raises(iq.IQError):
        iq.int8_linear(x, w, ws)
    x[1] = 0.0
    assert not iq.int8_linear(x, w, ws)[1].any()


# ---------------------------------------------------------------------------
# The product by expert
# ---------------------------------------------------------------------------

def routing(tokens, top_k, experts, seed, dropped=0.0, kind="even"):
    g = gen(seed)
    c = torch.randint(0, experts, (tokens, top_k), generator=g)
    if kind == "one":                                 # every token to one expert
        c[:] = experts - 1
    elif kind == "few":                               # most experts empty
        c = c % max(1, experts // 8) * 8 % experts
    c = torch.where(torch.rand((tokens, top_k), generator=g) < dropped, -1, c)
    return c.to(torch.int32)


@pytest.mark.parametrize("kind,dropped", [("even", 0.0), ("one", 0.0), ("few", 0.2), ("even", 1.0)])
@pytest.mark.parametrize("tokens,top_k,experts,channels,depth", [
    (1, 1, 1, 16, 16), (1, 2, 16, 130, 256), (5, 3, 13, 75, 100), (16, 2, 16, 256, 512),
    (60, 4, 8, 300, 272), (200, 2, 70, 64, 128), (500, 2, 4, 140, 1040), (333, 3, 5, 515, 129),
    (40, 8, 512, 20, 64)])
def test_expert_product(kind, dropped, tokens, top_k, experts, channels, depth):
    c = routing(tokens, top_k, experts, tokens + experts, dropped, kind)
    order, position, offsets = ref.sort(c.numpy(), experts)
    x, xs = codes((tokens, depth), 1), scales(tokens, 2)
    w, ws = codes((experts, channels, depth), 3), scales((experts, channels), 4)
    o, f = torch.tensor(order).to(DEV), torch.tensor(offsets).to(DEV)
    want = ref.expert_product(x.cpu().numpy(), xs.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy(),
                              order, offsets, top_k)
    for dtype in DTYPES:
        y = iq.int8_expert_matmul(x, xs, w, ws, f, o, top_k=top_k, dtype=dtype)
        within(y, want, ref.product_bound(want, dtype))
    # rows dispatched beforehand, in tensors with strides of their own
    tok = torch.tensor(order // top_k).long().to(DEV)
    wide = torch.empty((experts, channels + 1, depth + 16), dtype=torch.int8, device=DEV)
    wide[:, :channels, :depth] = w
    y2 = iq.int8_expert_matmul(strided(x[tok], 16, 0), xs[tok], wide[:, :channels, :depth], ws, f, dtype=dtype)
    assert torch.equal(y, y2)


def test_expert_product_clamps_what_it_reads_on_the_device():
    x, xs, w, ws = codes((6, 64), 1), scales(6, 2), codes((2, 40, 64), 3), scales((2, 40), 4)
    order = torch.tensor([0, 1, -7, 2 ** 31 - 1, 99, 3], dtype=torch.int32, device=DEV)
    y = iq.int8_expert_matmul(x, xs, w, ws, torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV), order)
    as_read = torch.tensor([0, 1, 5, 5, 5, 3], dtype=torch.int32, device=DEV)
    for off, same in (([0, 3, 6], [0, 3, 6]), ([-5, 3, 1 << 30], [0, 3, 6]), ([4, 2, 6], None), ([0, 9, 9], [0, 6, 6])):
        y = iq.int8_expert_matmul(x, xs, w, ws, torch.tensor(off, dtype=torch.int32, device=DEV), order)
        if same is not None:
            assert torch.equal(y, iq.int8_expert_matmul(
                x, xs, w, ws, torch.tensor(same, dtype=torch.int32, device=DEV), as_read))


def test_expert_product_beyond_32_bit_offsets():
    # Three experts 3 GiB apart.
    far = 3 * 2 ** 30
    buf = torch.empty(2 * far + 64 * 40, dtype=torch.int8, device=DEV)
    w = codes((3, 40, 64), 3)
    for e in range(3):
        buf[e * far:e * far + 64 * 40] = w[e].reshape(-1)
    farw = buf.as_strided((3, 40, 64), (far, 64, 1))
    for tokens in (6, 300):
        x, xs, ws = codes((tokens, 64), 1), scales(tokens, 2), scales((3, 40), 4)
        off = torch.tensor([0, tokens // 3, tokens // 2, tokens], dtype=torch.int32, device=DEV)
        assert torch.equal(iq.int8_expert_matmul(x, xs, farw, ws, off), iq.int8_expert_matmul(x, xs, w, ws, off))


# ---------------------------------------------------------------------------
# The sort
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("tokens,top_k,experts,dropped,kind", [
    (1, 1, 1, 0.0, "even"), (1, 1, 1, 1.0, "even"), (5, 2, 3, 0.3, "even"), (64, 1, 64, 0.0, "one"),
    (100, 3, 13, 0.1, "even"), (1024, 4, 16, 0.0, "few"), (4097, 1, 7, 0.0, "even"),
    (5000, 3, 512, 0.1, "even"), (3000, 8, 64, 0.0, "one"), (2500, 2, 511, 1.0, "even"),
    (150000, 8, 100, 0.05, "even")])
def test_sort(dtype, tokens, top_k, experts, dropped, kind):
    c = routing(tokens, top_k, experts, tokens, dropped, kind)
    got = iq.expert_sort(c.to(dtype).to(DEV), experts)
    for g, w in zip(got, ref.sort(c.numpy(), experts)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w)


def test_sort_of_no_tokens():
    order, position, offsets = iq.expert_sort(torch.empty((0, 4), dtype=torch.int32, device=DEV), 9)
    assert order.shape == (0,) and position.shape == (0, 4) and offsets.tolist() == [0] * 10


@pytest.mark.parametrize("dtype,bad", [(torch.int32, 5), (torch.int32, -2), (torch.int64, 2 ** 40), (torch.int64, -2 ** 40)])
def test_sort_reports_and_drops_bad_choices(dtype, bad):
    for tokens in (10, 3000):
        c = routing(tokens, 2, 5, 3).to(dtype)
        c[7, 1] = bad
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = iq.expert_sort(c.to(DEV), 5, status=st, check=False)
        assert int(st.item()) == 12
        c[7, 1] = -1
        for g, w in zip(got, ref.sort(c.numpy(), 5)):
            assert np.array_equal(g.cpu().numpy(), w)
        c[7, 1] = bad
        with pytest.raises(iq.IQError) as e:
            iq.expert_sort(c.to(DEV), 5)
        assert e.value.name == "IQ_ERR_INDEX"


# ---------------------------------------------------------------------------
# The copies and their gradients
# ---------------------------------------------------------------------------

ROUTES = [(1, 1, 1, 1, 0.0), (1, 2, 4, 7, 0.0), (4, 2, 16, 256, 0.0), (9, 3, 5, 65, 0.3), (33, 8, 13, 130, 0.1),
          (20, 1, 3, 1000, 0.5), (6, 17, 20, 40, 0.2), (3, 2, 2, 4099, 0.0), (7, 3, 4, 64, 1.0)]


def routed(tokens, top_k, experts, dropped, seed=5):
    c = routing(tokens, top_k, experts, seed + tokens, dropped)
    _, position, offsets = ref.sort(c.numpy(), experts)
    return position, offsets, torch.tensor(position).to(DEV), torch.tensor(offsets).to(DEV)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,top_k,experts,width,dropped", ROUTES)
def test_copies(dtype, tokens, top_k, experts, width, dropped):
    position, offsets, p, f = routed(tokens, top_k, experts, dropped)
    rows = tokens * top_k
    x, y = normal((tokens, width), 1, dtype), normal((rows, width), 2, dtype)
    weights = torch.rand((tokens, top_k), generator=gen(3)).to(DEV)
    kept = int(offsets[-1])
    y[kept:] = float("nan")                       # dropped rows are not read
    xs = iq.expert_dispatch(x, p, f)
    assert np.array_equal(ref.to64(xs), ref.dispatch(ref.to64(x), position, offsets))
    w64 = ref.to64(weights)
    out, size = ref.combine(ref.to64(y), position, offsets, w64)
    within(iq.expert_combine(y, p, f, weights), out, ref.combine_bound(out, size, top_k, dtype))
    dx, size = ref.combine(ref.to64(y), position, offsets, np.ones_like(w64))
    within(iq.expert_dispatch_backward(y, p, f), dx, ref.combine_bound(dx, size, top_k, dtype))
    g = normal((tokens, width), 4, dtype)
    gy, gw = iq.expert_combine_backward(g, y, p, f, weights)
    wy, ww, size = ref.combine_backward(ref.to64(g), np.nan_to_num(ref.to64(y)), position, offsets, w64)
    within(gy, wy, ref.combine_bound(wy, np.abs(wy), 1, dtype))
    within(gw, ww, ref.dot_bound(size, width))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("width", [40, 129, 1030])
@pytest.mark.parametrize("pad,shift", [(16, 0), (3, 0), (0, 1), (5, 7)])
def test_copies_strides(dtype, width, pad, shift):
    _, _, p, f = routed(11, 3, 4, 0.2)
    x, y, g = normal((11, width), 1, dtype), normal((33, width), 2, dtype), normal((11, width), 4, dtype)
    weights = torch.rand((11, 3), generator=gen(3)).to(DEV)
    sx, sy, sg = (strided(t, pad, shift) for t in (x, y, g))
    assert torch.equal(iq.expert_dispatch(x, p, f), iq.expert_dispatch(sx, p, f))
    assert torch.equal(iq.expert_combine(y, p, f, weights), iq.expert_combine(sy, p, f, weights))
    assert torch.equal(iq.expert_dispatch_backward(y, p, f), iq.expert_dispatch_backward(sy, p, f))
    for a, b in zip(iq.expert_combine_backward(g, y, p, f, weights),
                    iq.expert_combine_backward(sg, sy, p, f, weights)):
        assert torch.equal(a, b)
    for call, t in ((iq.expert_dispatch, x), (iq.expert_dispatch_backward, y)):
        plain = call(t, p, f)
        out = strided(torch.zeros_like(plain), pad, shift)
        whole = out.as_strided((out.untyped_storage().nbytes() // out.element_size(),), (1,), 0)
        whole.fill_(7.0)
        assert call(t, p, f, out=out) is out and torch.equal(out, plain)
        out.fill_(7.0)
        assert (whole == 7.0).all()


def test_copies_of_rows_larger_than_the_caches():
    """Over 128 MiB of sorted rows: against torch's own indexing, which the copies equal."""
    tokens, top_k, width = 9000, 3, 2603
    c = routing(tokens, top_k, 6, 77, 0.05).to(DEV)
    order, p, f = iq.expert_sort(c, 6)
    kept = int(f[-1])
    x = normal((tokens, width), 1, torch.bfloat16)
    xs = iq.expert_dispatch(x, p, f)
    assert torch.equal(xs[:kept], x[(order[:kept] // top_k).long()]) and not xs[kept:].any()
    w = torch.rand((tokens, top_k), generator=gen(3)).to(DEV)
    gy, gw = iq.expert_combine_backward(x, xs, p, f, w)
    want = (x[(order[:kept] // top_k).long()].float() * w.flatten()[order[:kept].long()][:, None]).bfloat16()
    assert torch.equal(gy[:kept], want) and not gy[kept:].any()
    size = ref.to64(x.float().square().sum(1, dtype=torch.float64))[:, None] * (c >= 0).cpu().numpy()
    within(gw, size, ref.dot_bound(size, width))


def test_copies_skip_places_out_of_range():
    x = normal((4, 24), 1)
    p = torch.tensor([[0, -1], [99, 1], [2, 2 ** 31 - 1], [-2 ** 31, 3]], dtype=torch.int32, device=DEV)
    f = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    out = torch.full((8, 24), 7.0, device=DEV)
    iq.expert_dispatch(x, p, f, out=out)
    assert torch.equal(out[:4], x) and (out[4:] == 7.0).all()
    weights = torch.ones((4, 2), device=DEV)
    y = normal((8, 24), 2)
    assert torch.equal(iq.expert_combine(y, p, f, weights), y[:4])
    gy, gw = iq.expert_combine_backward(x, y, p, f, weights)
    assert torch.equal(gy[:4], x)
    assert gw[0, 1] == 0 and gw[1, 0] == 0 and gw[2, 1] == 0 and gw[3, 0] == 0


def test_nonfinite_rows_reach_their_own_token_only():
    position, offsets, p, f = routed(12, 2, 4, 0.0)
    y = normal((24, 50), 2)
    weights = torch.rand((12, 2), generator=gen(3)).to(DEV)
    good = iq.expert_combine(y, p, f, weights)
    y[position[5, 1], 10] = float("inf")
    y[position[6, 0], 11] = float("nan")
    out = iq.expert_combine(y, p, f, weights)
    assert torch.isinf(out[5, 10]) and torch.isnan(out[6, 11])
    out[5, 10], out[6, 11] = good[5, 10], good[6, 11]
    assert torch.equal(out, good)
    for dtype in (torch.bfloat16, torch.float16):
        assert torch.isnan(iq.expert_combine(y.to(dtype), p, f, weights)[6, 11])


def test_gradients_against_differences():
    """combine is linear in y and in the weights, dispatch in x: a central difference of
    any width is the derivative, up to the roundings of the two passes in fp32."""
    tokens, top_k, width = 9, 3, 70
    _, _, p, f = routed(tokens, top_k, 5, 0.2)
    y, hy = normal((27, width), 1), normal((27, width), 2)
    w, hw = (torch.rand((tokens, top_k), generator=gen(s)).to(DEV) for s in (3, 4))
    g = normal((tokens, width), 5)
    gy, gw = (ref.to64(t) for t in iq.expert_combine_backward(g, y, p, f, w))
    slope = (gy * ref.to64(hy)).sum() + (gw * ref.to64(hw)).sum()
    ends = [ref.to64(iq.expert_combine(y + s * hy, p, f, w + s * hw)) for s in (1.0, -1.0)]
    # |term| <= 10 for |y + hy| <= 10 and weights within (-1, 2); 3 terms and their roundings
    # (inputs, product, sum) in each end, 630 values, gradients below 5
    assert abs((ref.to64(g) * (ends[0] - ends[1])).sum() / 2 - slope) <= 630 * 5 * 3 * 20 * 6 * 2.0 ** -24
    x, hx = normal((tokens, width), 6), normal((tokens, width), 7)
    gs = normal((27, width), 8)
    slope = (ref.to64(iq.expert_dispatch_backward(gs, p, f)) * ref.to64(hx)).sum()
    ends = [ref.to64(iq.expert_dispatch(x + s * hx, p, f)) for s in (1.0, -1.0)]
    assert abs((ref.to64(gs) * (ends[0] - ends[1])).sum() / 2 - slope) <= 1890 * 5 * 20 * 6 * 2.0 ** -24


# ---------------------------------------------------------------------------
# Streams, graphs, repetition, refusals
# ---------------------------------------------------------------------------

def layer(x, choice, weights, w, ws, status):
    order, position, offsets = iq.expert_sort(choice, w.shape[0], status=status, check=False)
    q, s = iq.quantize_rows(x, status=status, check=False)
    y = iq.int8_expert_matmul(q, s, w, ws, offsets, order, top_k=choice.shape[1], dtype=x.dtype)
    return iq.expert_combine(y, position, offsets, weights)


@pytest.mark.parametrize("tokens", [3, 700])
def test_layer_on_streams_and_in_graphs(tokens):
    experts, channels, depth = 8, 160, 272
    w, ws = codes((experts, channels, depth), 1), scales((experts, channels), 2)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sets = []
    for s in range(4):
        sets.append((normal((tokens, depth), 10 + s, torch.bfloat16), routing(tokens, 2, experts, 20 + s, 0.1).to(DEV),
                     torch.rand((tokens, 2), generator=gen(30 + s)).to(DEV)))
    want = [layer(*v, w, ws, status) for v in sets]
    torch.cuda.synchronize()
    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 4
    for i, v in enumerate(sets):
        streams[i % 2].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i % 2]):
            got[i] = layer(*v, w, ws, status)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # a captured graph, replayed with new inputs and eager work in between
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*held, w, ws, status)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(*held, w, ws, status)
    for r in range(8):
        for h, v in zip(held, sets[r % 4]):
            h.copy_(v)
        graph.replay()
        eager = layer(*sets[(r + 1) % 4], w, ws, status)
        torch.cuda.synchronize()
        assert torch.equal(out, want[r % 4]) and torch.equal(eager, want[(r + 1) % 4])
    assert int(status.item()) == 0


def test_repeated_calls_give_the_same_bits():
    x, w = normal((37, 1001), 1, torch.bfloat16), codes((515, 1001), 2)
    ws = scales(515, 3)
    _, _, p, f = routed(500, 3, 7, 0.1)
    y, g, weights = normal((1500, 600), 4), normal((500, 600), 5), torch.rand((500, 3), generator=gen(6)).to(DEV)
    first = iq.int8_linear(x, w, ws), iq.expert_combine(y, p, f, weights), *iq.expert_combine_backward(g, y, p, f, weights)
    for _ in range(5):
        again = iq.int8_linear(x, w, ws), iq.expert_combine(y, p, f, weights), *iq.expert_combine_backward(g, y, p, f, weights)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_binding_refusals():
    x, q, s = normal((4, 32), 1), codes((4, 32), 2), scales(4, 3)
    p, f, wt = torch.zeros((4, 1), dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV), scales((4, 1), 4)
    for kind, call in [
            (TypeError, lambda: iq.quantize_rows(x.double())),
            (TypeError, lambda: iq.quantize_rows(q)),
            (TypeError, lambda: iq.quantize_rows([1.0])),
            (ValueError, lambda: iq.quantize_rows(x[0])),
            (ValueError, lambda: iq.quantize_rows(x.t())),
            (ValueError, lambda: iq.quantize_rows(x.cpu())),
            (TypeError, lambda: iq.int8_matmul(x, s, q, s)),
            (ValueError, lambda: iq.int8_matmul(q, s[:3], q, s)),
            (TypeError, lambda: iq.int8_matmul(q, s.double(), q, s)),
            (ValueError, lambda: iq.int8_matmul(q, s, q[:, :16], s)),
            (TypeError, lambda: iq.int8_matmul(q, s, q, s, dtype=torch.int32)),
            (TypeError, lambda: iq.int8_matmul(q, s, q, s, dtype=torch.float64)),
            (ValueError, lambda: iq.int8_matmul(q, s, q, s, out=torch.empty((4, 5), device=DEV))),
            (ValueError, lambda: iq.int8_linear(x, q[:, :16], s)),
            (TypeError, lambda: iq.int8_linear(x, q, s, out=torch.empty((4, 4), device=DEV, dtype=torch.float16))),
            (TypeError, lambda: iq.int8_linear(x, q, s, status=s)),
            (ValueError, lambda: iq.int8_expert_matmul(q, s, q, s, f)),
            (ValueError, lambda: iq.int8_expert_matmul(q, s, q[None].expand(2, 4, 32), s[None].expand(2, 4), f)),
            (ValueError, lambda: iq.int8_expert_matmul(q, s, q[None], s[None], f)),
            (ValueError, lambda: iq.int8_expert_matmul(q, s, q[None], s[None], f[:2], f[:2])),
            (iq.IQError, lambda: iq.expert_sort(p, 0)),
            (iq.IQError, lambda: iq.expert_sort(p, 513)),
            (TypeError, lambda: iq.expert_sort(p.float(), 2)),
            (ValueError, lambda: iq.expert_sort(p[:, 0], 2)),
            (ValueError, lambda: iq.expert_dispatch(x[:3], p, f)),
            (TypeError, lambda: iq.expert_dispatch(x, p.long(), f)),
            (ValueError, lambda: iq.expert_dispatch_backward(x[:3], p, f)),
            (ValueError, lambda: iq.expert_combine(x, p, f, wt[:3])),
            (TypeError, lambda: iq.expert_combine(x, p, f, wt.half())),
            (ValueError, lambda: iq.expert_combine_backward(x[:3], x, p, f, wt)),
            (TypeError, lambda: iq.expert_combine_backward(x.half(), x, p, f, wt))]:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("fmt", ["iq1_s", "iq2_xs", "iq1_m"])
def test_example_serves_and_trains_an_expert_layer(fmt):
    """Rounding to 8 bits moves a code by at most half a step: an activation or weight of a
    row whose largest is m times its root mean square is off by m / 127 / sqrt(12) of that,
    under 1.2 % for m <= 5; both, and the roundings to bf16 (0.2 % each), stay under 3 %.
    The training step's own gradient is exact up to bf16: three roundings of 2^-9."""
    from examples import expert_layer
    error, train_error, _ = expert_layer.run(experts=4, channels=96, depth=512, tokens=70, top_k=2,
                                             fmt=fmt, repeats=2)
    assert 0.0 < error < 0.03
    assert train_error < 4 * 2.0 ** -9
