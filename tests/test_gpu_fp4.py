"""The 4-bit weights and the products with them against plain implementations in
64 bits (more_layers_ref.py), at the sizes, strides, types and values where they
can go wrong.  Codes and scales have to be equal, and so do products of small
integers, whose sums are exact; others stay within bounds that follow from the
roundings the operators state."""

import sys

import numpy as np
import pytest
import torch

from tests import more_layers_ref as ref
from tests.layers_ref import to64

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


def integers(shape, seed, most=8):
    return torch.randint(-most, most + 1, shape, generator=gen(seed)).float()


def within(got, want, bound):
    got = to64(got)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), "worst %.3g over its bound at %s" % (
        over.max(), np.unravel_index(over.argmax(), over.shape))


def strided(t, pad, shift):
    """The same values in rows that are `pad` values longer and start `shift` values late."""
    rows, cols = t.shape
    buf = torch.empty(rows * (cols + pad) + shift + 16, dtype=t.dtype, device=t.device)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def random_codes(shape, seed, low=0, high=16):
    """Packed codes low..high-1 for [..., depth] values."""
    c = torch.randint(low, high, shape, generator=gen(seed), dtype=torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(DEV)


def random_scale(shape, seed, low, high):
    return torch.randint(low, high, shape, generator=gen(seed), dtype=torch.uint8).to(DEV)


def weight(channels, depth, seed):
    """Codes and scales of a weight as the framework makes them, and their values."""
    w, s = iq.quantize_groups(normal((channels, depth), seed) * 0.02)
    return w, s, ref.values(w.cpu().numpy(), s.cpu().numpy())


# ---------------------------------------------------------------------------
# quantize_groups, dequantize_groups
# ---------------------------------------------------------------------------

SHAPES = [(1, 32), (3, 64), (5, 96), (1, 2048), (2, 2080), (7, 4096), (33, 1024), (2, 8224), (257, 160)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_groups(dtype, rows, cols):
    w = (normal((rows, cols), rows * 7919 + cols) * 0.02).to(dtype)
    w[0, :32] = 0
    codes, scale = iq.quantize_groups(w)
    want, want_scale = ref.quantize(to64(w))
    assert np.array_equal(scale.cpu().numpy(), want_scale)
    assert np.array_equal(codes.cpu().numpy(), ref.pack(want))
    # rows with gaps, from an address that is aligned to the type only
    again = iq.quantize_groups(strided(w, 3, 1))
    assert torch.equal(again[0], codes) and torch.equal(again[1], scale)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_quantize_values_at_the_borders(dtype):
    """Halves between codes and their neighbours, for groups of every size the type has."""
    fi = torch.finfo(dtype)
    m = torch.tensor([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.5, .5, 1, 1.5, 2, 3], dtype=torch.float64)
    near = torch.cat([m, m * (1 - fi.eps)])             # eps / 2 is a step below a power of two
    exponents = range(-151, 126) if dtype != torch.float16 else range(-26, 13)
    rows = []
    for e in exponents:
        v = near * 2.0 ** e
        v[1::2] *= -1
        rows.append(v.to(dtype))
    w = torch.stack(rows).to(DEV)
    codes, scale = iq.quantize_groups(w)
    want, want_scale = ref.quantize(to64(w))
    assert np.array_equal(scale.cpu().numpy(), want_scale)
    assert np.array_equal(codes.cpu().numpy(), ref.pack(want))
    assert len(np.unique(want_scale)) > 30


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_quantize_reports_what_is_not_finite(dtype):
    w = normal((6, 96), 1, dtype)
    w[1, 40], w[4, 95], w[5, 0] = float("nan"), float("inf"), -float("inf")
    with pytest.raises(iq.IQError) as e:
        iq.quantize_groups(w)
    assert e.value.name == "IQ_ERR_NONFINITE"
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scale = iq.quantize_groups(w, status=status, check=False)
    assert int(status) == 5
    want, want_scale = ref.quantize(to64(w))            # the reference zeroes those groups
    assert np.array_equal(codes.cpu().numpy(), ref.pack(want))
    assert np.array_equal(scale.cpu().numpy(), want_scale)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_dequantize_every_code_and_scale(dtype):
    """16 codes twice in each group, one row for each scale byte."""
    c = torch.arange(32, dtype=torch.uint8) % 16
    codes = (c[0::2] | (c[1::2] << 4)).expand(256, 16).contiguous().to(DEV)
    scale = torch.arange(256, dtype=torch.uint8)[:, None].contiguous().to(DEV)
    got = iq.dequantize_groups(codes, scale, dtype=dtype).cpu()
    want = torch.from_numpy(ref.values(codes.cpu().numpy(), scale.cpu().numpy()))
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    want = want.float().to(dtype)
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])
    assert torch.equal(torch.signbit(got[ok]), torch.signbit(want[ok]))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dequantize_groups(dtype, rows, cols):
    codes, scale = random_codes((rows, cols), 1), random_scale((rows, cols // 32), 2, 110, 140)
    want = torch.from_numpy(ref.values(codes.cpu().numpy(), scale.cpu().numpy())).float().to(dtype).to(DEV)
    assert torch.equal(iq.dequantize_groups(codes, scale, dtype=dtype), want)
    out = strided(torch.zeros((rows, cols), dtype=dtype, device=DEV), 5, 3)
    assert iq.dequantize_groups(strided(codes, 3, 1), strided(scale, 2, 1), out=out) is out
    assert torch.equal(out, want)


def test_rows_around_a_result_are_left_as_they_were():
    buf = torch.full((6, 200), 7.0, device=DEV)
    codes, scale = random_codes((4, 160), 1), random_scale((4, 5), 2, 120, 130)
    iq.dequantize_groups(codes, scale, out=buf[1:5, 20:180])
    want = torch.full((6, 200), 7.0, device=DEV)
    want[1:5, 20:180] = iq.dequantize_groups(codes, scale)
    assert torch.equal(buf, want)


# ---------------------------------------------------------------------------
# fp4_linear
# ---------------------------------------------------------------------------

PRODUCTS = [(1, 1, 32), (1, 16, 128), (1, 70, 1056), (2, 33, 96), (5, 257, 160), (15, 64, 512), (16, 100, 64),
            (17, 48, 2080), (31, 130, 256), (33, 65, 1024), (48, 512, 288), (64, 63, 4128), (65, 129, 96),
            (100, 260, 544), (127, 64, 128), (129, 300, 224), (200, 17, 1024), (256, 256, 256),
            (257, 513, 352), (300, 1030, 96), (513, 384, 160), (33, 2050, 32), (9, 4100, 1696),
            (1804, 1100, 352), (1577, 300, 1056), (161, 70, 1280), (1455, 2050, 224), (33, 2050, 1056),
            (1229, 5000, 256), (1, 70, 1280), (9, 2050, 1056)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", PRODUCTS)
def test_linear_of_integers_is_exact(dtype, tokens, channels, depth):
    """Terms are multiples of 1/4 of at most 48 and their sums below 2^22 / 4: exact in any
    order, so the result is the sum rounded once."""
    x = integers((tokens, depth), 1).to(dtype).to(DEV)
    w, s = random_codes((channels, depth), 2), random_scale((channels, depth // 32), 3, 126, 128)
    want = torch.from_numpy(to64(x) @ ref.values(w.cpu().numpy(), s.cpu().numpy()).T).float().to(dtype)
    assert torch.equal(iq.fp4_linear(x, w, s).cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", PRODUCTS)
def test_linear(dtype, tokens, channels, depth):
    x = normal((tokens, depth), 4, dtype)
    w, s, v = weight(channels, depth, 5)
    y, size = ref.product(to64(x), v)
    within(iq.fp4_linear(x, w, s), y, ref.product_bound(y, size, depth, dtype))


@pytest.mark.parametrize("tokens", [1, 20, 300])
def test_every_bit_of_the_activations_counts(tokens):
    """A weight that picks one value of each token: the result is that value.

    The 24 bits of an fp32 value from 2^-110 on reach down to 2^-133 at most, the smallest
    bf16 number, so its three parts hold all of them.  Of a smaller value the bits below 2^-133
    are cut from each part: together less than 2^-133."""
    depth = 160
    x = torch.randint(-2 ** 31, 2 ** 31 - 1, (tokens, depth), generator=gen(6), dtype=torch.int32).view(torch.float32)
    x = torch.where(torch.isfinite(x), x, 1.5).to(DEV)
    code = torch.zeros((depth, depth), dtype=torch.uint8)
    code[torch.arange(depth), torch.arange(depth)] = 2            # 1
    w = (code[:, 0::2] | (code[:, 1::2] << 4)).to(DEV)
    s = torch.full((depth, depth // 32), 127, dtype=torch.uint8, device=DEV)
    for dtype in DTYPES:
        v = x.to(dtype)
        v = torch.where(torch.isfinite(v), v, 1.5)
        got = iq.fp4_linear(v, w, s)
        small = v.abs() < 2.0 ** -110
        assert torch.equal(torch.where(small, 0.0, got), torch.where(small, 0.0, v))
        if dtype == torch.float32:
            assert small.any() and ((got - v).abs()[small] < 2.0 ** -133).all()
        else:
            assert torch.equal(got, v)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens", [3, 40, 260])
def test_scales_of_every_size(dtype, tokens):
    """Each channel one value 1 times a power of two that its one term brings back to range."""
    bytes_ = torch.arange(0, 253, dtype=torch.int64)
    depth, n = 64, len(bytes_)
    code = torch.zeros((n, depth), dtype=torch.uint8)
    code[:, 37] = 2
    w = (code[:, 0::2] | (code[:, 1::2] << 4)).to(DEV)
    s = torch.full((n, 2), 0, dtype=torch.uint8)
    s[:, 1] = bytes_.to(torch.uint8)
    x = torch.zeros((tokens, depth))
    x[:, 37] = torch.tensor([2.0 ** (3 - t % 7) for t in range(tokens)])
    x = x.to(dtype).to(DEV)
    want = torch.from_numpy(np.ldexp(to64(x)[:, 37, None], bytes_.numpy() - 127)).float().to(dtype)
    assert torch.equal(iq.fp4_linear(x, w, s.to(DEV)).cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", [(3, 40, 160), (300, 130, 352)])
def test_offsets_beyond_32_bits(dtype, tokens, channels, depth):
    """Rows so far apart that the last ones begin beyond 2^32 bytes, of one operand at a time."""
    def apart(t):
        ld = 2 ** 32 // ((len(t) - 1) * t.element_size()) + 1027
        far = torch.empty((len(t), ld), dtype=t.dtype, device=DEV)[:, :t.shape[1]]
        return far.copy_(t)

    x = integers((tokens, depth), 1).to(dtype).to(DEV)
    w, s = random_codes((channels, depth), 2), random_scale((channels, depth // 32), 3, 126, 128)
    want = iq.fp4_linear(x, w, s)
    assert torch.equal(iq.fp4_linear(apart(x), w, s), want)
    assert torch.equal(iq.fp4_linear(x, apart(w), s), want)
    assert torch.equal(iq.fp4_linear(x, w, apart(s)), want)
    out = apart(torch.zeros((tokens, channels), dtype=dtype, device=DEV))
    assert torch.equal(iq.fp4_linear(x, w, s, out=out), want)
    order, _, offsets = routing(tokens, 3, 2, 11)
    w, s = random_codes((3, channels, depth), 2), random_scale((3, channels, depth // 32), 3, 126, 128)
    want = iq.fp4_expert_linear(x, w, s, offsets, order, top_k=2)
    assert torch.equal(iq.fp4_expert_linear(apart(x), w, s, offsets, order, top_k=2), want)
    far = [apart(t.view(3, -1)).unflatten(1, t.shape[1:]) for t in (w, s)]
    assert torch.equal(iq.fp4_expert_linear(x, *far, offsets, order, top_k=2), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_groups_beyond_32_bits(dtype):
    x = normal((3, 96), 7, dtype)
    want = iq.quantize_groups(x)
    ld = 2 ** 31 // x.element_size() + 5
    far = torch.empty((3, ld), dtype=dtype, device=DEV)[:, :96]
    far.copy_(x)
    got = iq.quantize_groups(far)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    codes, scale = (torch.empty((3, 2 ** 31 + 5), dtype=torch.uint8, device=DEV)[:, :t.shape[1]].copy_(t)
                    for t in want)
    assert torch.equal(iq.dequantize_groups(codes, scale, dtype=dtype),
                       iq.dequantize_groups(*want, dtype=dtype))


@pytest.mark.parametrize("outside", [None, 103, 141, 255])
@pytest.mark.parametrize("tokens", [1, 5, 30, 100, 700])
def test_weights_at_the_ends_of_fp16(tokens, outside):
    """Scales 104 .. 140 with every code are exact in fp16, and a single channel that has
    another one changes none of the others.  Products by 1/2, 1 and 2 are exact in fp32, the
    results those rounded once."""
    depth, n = 160, 37 * 16
    code = torch.zeros((n, depth), dtype=torch.uint8)
    code[:, 101] = torch.arange(n) % 16
    s = torch.full((n, depth // 32), 120, dtype=torch.uint8)
    s[:, 3] = 104 + torch.arange(n) // 16
    if outside is not None:
        code[200, 101], s[200, 3] = 5, outside
    w = (code[:, 0::2] | (code[:, 1::2] << 4)).to(DEV)
    x = torch.zeros((tokens, depth))
    x[:, 101] = torch.tensor([(1.0, 2.0, 0.5)[t % 3] for t in range(tokens)])
    x = x.half().to(DEV)
    want = torch.from_numpy(to64(x) @ ref.values(w.cpu().numpy(), s.numpy()).T).float().half()
    got = iq.fp4_linear(x, w, s.to(DEV)).cpu()
    assert torch.equal(torch.nan_to_num(got, 1.0), torch.nan_to_num(want, 1.0))
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got).any() == (outside == 255)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", [(1, 40, 160), (7, 40, 160), (40, 70, 224), (300, 130, 352)])
def test_linear_of_slices(dtype, tokens, channels, depth):
    x = integers((tokens, depth), 1).to(dtype).to(DEV)
    w, s = random_codes((channels, depth), 2), random_scale((channels, depth // 32), 3, 126, 128)
    want = iq.fp4_linear(x, w, s)
    for pad, shift in ((1, 0), (7, 1), (8, 8), (32, 3)):
        out = strided(torch.full((tokens, channels), 9.0, dtype=dtype, device=DEV), pad, shift)
        got = iq.fp4_linear(strided(x, pad, shift), strided(w, pad, shift), strided(s, pad, shift), out=out)
        assert got is out and torch.equal(out, want)
    # one row for all tokens
    assert torch.equal(iq.fp4_linear(x[:1].expand(tokens, depth), w, s), want[:1].expand(tokens, channels))
    # rows around the result stay
    buf = torch.full((tokens + 2, channels + 3), 9.0, dtype=dtype, device=DEV)
    iq.fp4_linear(x, w, s, out=buf[1:-1, 1:-2])
    assert torch.equal(buf[1:-1, 1:-2], want)
    buf[1:-1, 1:-2] = 9.0
    assert (buf == 9.0).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens", [1, 9, 50, 270])
def test_what_is_not_finite_passes(dtype, tokens):
    """As a product of floats in any order: NaN where one enters, or where infinities of both
    signs do, or an infinity times 0; other tokens are not touched."""
    channels, depth = 130, 160
    x = integers((tokens, depth), 1).to(dtype)
    x[tokens // 2, 33], x[tokens - 1, 159] = float("inf"), -float("inf")
    if tokens > 3:
        x[1, 7] = float("nan")
        x[0, :] = float("inf")
    w, s = random_codes((channels, depth), 2), random_scale((channels, depth // 32), 3, 126, 128)
    v = ref.values(w.cpu().numpy(), s.cpu().numpy())
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy((to64(x)[:, None, :] * v[None]).sum(axis=2)).float().to(dtype)
    got = iq.fp4_linear(x.to(DEV), w, s).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok]) and torch.isinf(want).any()
    # a NaN of the weight reaches its channel only
    s2 = s.clone()
    s2[5, 2] = 255
    got2 = iq.fp4_linear(x.to(DEV), w, s2).cpu()
    assert torch.isnan(got2[:, 5]).all()
    keep = torch.arange(channels) != 5
    assert torch.equal(torch.nan_to_num(got2[:, keep]), torch.nan_to_num(got[:, keep]))


def test_nan_of_any_payload_stays_nan():
    x = torch.ones((3, 32))
    x.view(torch.int32)[0, 3], x.view(torch.int32)[1, 31], x.view(torch.int32)[2, 0] = 0x7f800001, -0x7fffff, 0x7fc00000
    w, s = random_codes((20, 32), 2), torch.full((20, 1), 127, dtype=torch.uint8, device=DEV)
    assert torch.isnan(iq.fp4_linear(x.to(DEV), w, s)).all()


def test_no_tokens():
    w, s, _ = weight(40, 64, 1)
    for dtype in DTYPES:
        y = iq.fp4_linear(torch.empty((0, 64), dtype=dtype, device=DEV), w, s)
        assert y.shape == (0, 40) and y.dtype == dtype
    codes, scale = iq.quantize_groups(torch.empty((0, 64), device=DEV))
    assert codes.shape == (0, 32) and scale.shape == (0, 2)
    assert iq.dequantize_groups(codes, scale).shape == (0, 64)


# ---------------------------------------------------------------------------
# fp4_expert_linear
# ---------------------------------------------------------------------------

def routing(tokens, experts, top_k, seed, dropped=0.0, favourite=None):
    c = torch.randint(0, experts, (tokens, top_k), generator=gen(seed))
    if favourite is not None:
        c[:, 0] = favourite
    c = torch.where(torch.rand(c.shape, generator=gen(seed + 1)) < dropped, -1, c)
    return iq.expert_sort(c.to(torch.int32).to(DEV), experts)


def expert_reference(x, v, order, offsets, top_k):
    y, size = np.zeros((len(order), v.shape[1])), np.zeros((len(order), v.shape[1]))
    for e in range(v.shape[0]):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        y[rows], size[rows] = ref.product(x[order[rows] // top_k], v[e])
    return y, size


EXPERT_CASES = [
    # tokens, experts, top_k, channels, depth, dropped, favourite
    (1, 8, 2, 40, 96, 0.0, None), (4, 16, 2, 130, 160, 0.0, None), (16, 5, 3, 64, 512, 0.3, None),
    (33, 3, 1, 70, 288, 0.0, 1), (100, 70, 2, 48, 64, 0.1, None), (200, 4, 2, 260, 352, 0.5, 3),
    (300, 8, 2, 300, 128, 0.0, 0), (37, 512, 2, 16, 32, 0.0, None), (600, 3, 2, 129, 224, 0.05, 2),
    (21, 64, 2, 130, 288, 0.0, None), (11, 64, 2, 1100, 32, 0.1, None), (674, 16, 2, 2050, 32, 0.0, 5),
    (82, 16, 2, 130, 32, 0.0, None), (1079, 64, 2, 70, 32, 0.1, None), (19, 3, 2, 2050, 288, 0.0, None),
    (623, 64, 2, 70, 352, 0.0, 7), (38, 64, 2, 1100, 288, 0.0, None), (945, 8, 2, 2050, 32, 0.1, None),
    (98, 2, 2, 70, 416, 0.0, None), (471, 2, 2, 1100, 32, 0.0, None), (47, 3, 1, 2050, 2176, 0.0, None),
    (555, 3, 2, 5000, 64, 0.0, 1), (468, 2, 2, 4100, 160, 0.0, None),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,experts,top_k,channels,depth,dropped,favourite", EXPERT_CASES)
def test_expert_linear(dtype, tokens, experts, top_k, channels, depth, dropped, favourite):
    order, _, offsets = routing(tokens, experts, top_k, 11, dropped, favourite)
    o, f = order.cpu().numpy(), offsets.cpu().numpy()
    # exact sums
    x = integers((tokens, depth), 1).to(dtype).to(DEV)
    w = random_codes((experts, channels, depth), 2)
    s = random_scale((experts, channels, depth // 32), 3, 126, 128)
    v = ref.values(w.cpu().numpy(), s.cpu().numpy())
    y, _ = expert_reference(to64(x), v, o, f, top_k)
    got = iq.fp4_expert_linear(x, w, s, offsets, order, top_k=top_k)
    assert torch.equal(got.cpu(), torch.from_numpy(y).float().to(dtype))
    # rows that are dispatched already
    sorted_x = x[torch.div(order, top_k, rounding_mode="floor").long()]
    assert torch.equal(iq.fp4_expert_linear(sorted_x, w, s, offsets), got)
    # rounded ones, with scales of their own
    x = normal((tokens, depth), 4, dtype)
    s = random_scale((experts, channels, depth // 32), 5, 118, 124)
    v = ref.values(w.cpu().numpy(), s.cpu().numpy())
    y, size = expert_reference(to64(x), v, o, f, top_k)
    within(iq.fp4_expert_linear(x, w, s, offsets, order, top_k=top_k), y,
           ref.product_bound(y, size, depth, dtype))


@pytest.mark.parametrize("tokens,channels", [(3, 40), (40, 130), (700, 300), (500, 4100)])
def test_scales_beyond_fp16(tokens, channels):
    """Of three experts one has scales that fp16 has no room for."""
    order, _, offsets = routing(tokens, 3, 2, 11)
    x = normal((tokens, 352), 4, torch.float16)
    w = random_codes((3, channels, 352), 2)
    s = random_scale((3, channels, 11), 5, 118, 124)
    s[1] = random_scale((channels, 11), 6, 90, 124)
    y, size = expert_reference(to64(x), ref.values(w.cpu().numpy(), s.cpu().numpy()),
                               order.cpu().numpy(), offsets.cpu().numpy(), 2)
    within(iq.fp4_expert_linear(x, w, s, offsets, order, top_k=2), y,
           ref.product_bound(y, size, 352, torch.float16))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens", [3, 60, 400])
def test_expert_linear_of_slices(dtype, tokens):
    experts, top_k, channels, depth = 5, 2, 70, 160
    order, _, offsets = routing(tokens, experts, top_k, 3, 0.2)
    x = integers((tokens, depth), 1).to(dtype).to(DEV)
    w = random_codes((experts, channels, depth), 2)
    s = random_scale((experts, channels, depth // 32), 3, 126, 128)
    want = iq.fp4_expert_linear(x, w, s, offsets, order, top_k=top_k)
    big = torch.zeros((experts, channels + 1, depth // 2 + 3), dtype=torch.uint8, device=DEV)
    big[:, 1:, 3:] = w
    wide = torch.zeros((experts, channels, depth // 32 + 2), dtype=torch.uint8, device=DEV)
    wide[:, :, 1:-1] = s
    out = strided(torch.full((tokens * top_k, channels), 9.0, dtype=dtype, device=DEV), 3, 1)
    got = iq.fp4_expert_linear(strided(x, 3, 1), big[:, 1:, 3:], wide[:, :, 1:-1], offsets, order,
                               top_k=top_k, out=out)
    assert got is out and torch.equal(out, want)
    # one weight for all experts
    one = iq.fp4_expert_linear(x, w[:1].expand(experts, -1, -1), s[:1].expand(experts, -1, -1), offsets, order,
                               top_k=top_k)
    dense = iq.fp4_linear(x[torch.div(order, top_k, rounding_mode="floor").long()], w[0], s[0])
    kept = torch.arange(tokens * top_k, device=DEV)[:, None] < offsets[-1]
    assert torch.equal(one, torch.where(kept, dense, 0.0))


def test_every_choice_dropped():
    choice = torch.full((9, 2), -1, dtype=torch.int32, device=DEV)
    order, _, offsets = iq.expert_sort(choice, 4)
    w, s = random_codes((4, 20, 64), 1), random_scale((4, 20, 2), 2, 120, 130)
    x = torch.full((9, 64), float("nan"), device=DEV)
    y = iq.fp4_expert_linear(x, w, s, offsets, order, top_k=2)
    assert y.shape == (18, 20) and not y.any()


@pytest.mark.parametrize("tokens", [6, 300])
def test_offsets_and_orders_out_of_range_are_bounded(tokens):
    """What is read on the device is clamped: the call ends, and rows of ranges that make
    sense are right."""
    w, s = random_codes((3, 40, 64), 1), random_scale((3, 40, 2), 2, 126, 128)
    x = integers((tokens, 64), 3).to(DEV)
    order = torch.arange(tokens, dtype=torch.int32, device=DEV)
    order[1], order[2] = -5, 10 ** 9                             # clamped to a token
    offsets = torch.tensor([0, 3, 3, 10 ** 9], dtype=torch.int32, device=DEV)
    y = iq.fp4_expert_linear(x, w, s, offsets, order, top_k=1)
    assert torch.equal(y[0], iq.fp4_linear(x, w[0], s[0])[0])
    assert torch.equal(y[3:], iq.fp4_linear(x, w[2], s[2])[3:])
    last = iq.fp4_linear(x, w[0], s[0])[-1]
    assert torch.equal(y[1], last) and torch.equal(y[2], last)


# ---------------------------------------------------------------------------
# How they are called
# ---------------------------------------------------------------------------

def test_argument_errors():
    w, s, _ = weight(40, 64, 1)
    x = normal((4, 64), 2)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for call in (lambda: iq.fp4_linear(x[:, :48], w, s), lambda: iq.fp4_linear(x, w[:, :31], s),
                 lambda: iq.fp4_linear(x, w, s[:, :1]), lambda: iq.fp4_linear(x, w, s[:39]),
                 lambda: iq.fp4_linear(x.T.contiguous().T, w, s), lambda: iq.fp4_linear(x[0], w, s),
                 lambda: iq.fp4_linear(x, w, s, out=torch.empty((4, 41), device=DEV)),
                 lambda: iq.fp4_expert_linear(x, w, s, off), lambda: iq.fp4_expert_linear(x, w[None], s[None], off[:1]),
                 lambda: iq.fp4_expert_linear(x, w[None], s[None, :39], off),
                 lambda: iq.quantize_groups(x[:, :33]), lambda: iq.quantize_groups(x.T.contiguous().T),
                 lambda: iq.dequantize_groups(w, s[:, :1]), lambda: iq.dequantize_groups(w[:, :20], s),
                 lambda: iq.dequantize_groups(w, s[:39])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: iq.fp4_linear(x.double(), w, s), lambda: iq.fp4_linear(x, w.char(), s),
                 lambda: iq.fp4_linear(x, w, s.float()), lambda: iq.quantize_groups(w),
                 lambda: iq.fp4_linear(x, w, s, out=torch.empty((4, 40), device=DEV, dtype=torch.bfloat16)),
                 lambda: iq.dequantize_groups(w, s, dtype=torch.float64), lambda: iq.dequantize_groups(x, s)):
        with pytest.raises(TypeError):
            call()
    raw = torch.zeros(40 * 64 * 4, dtype=torch.uint8, device=DEV)
    for call in (lambda: iq.fp4_linear(x, w, s, out=x[:, :40]),
                 lambda: iq.fp4_expert_linear(x, w[None], s[None], off, out=x[:, 24:]),
                 lambda: iq.dequantize_groups(raw[:1280].view(40, 32), s, out=raw.view(torch.float32).view(40, 64))):
        with pytest.raises(iq.IQError) as e:
            call()
        assert e.value.name == "IQ_ERR_ARG"


def test_products_have_no_gradient():
    w, s, _ = weight(40, 64, 1)
    x = normal((4, 64), 2).requires_grad_()
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for y in (iq.fp4_linear(x, w, s), iq.fp4_expert_linear(x, w[None], s[None], off)):
        assert y.requires_grad
        with pytest.raises(RuntimeError, match="has no gradient"):
            y.sum().backward()
    with pytest.raises(ValueError):
        iq.fp4_linear(x, w, s, out=torch.empty((4, 40), device=DEV))
    with torch.no_grad():
        assert not iq.fp4_linear(x, w, s).requires_grad


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_on_another_stream_and_in_a_graph(dtype, tokens):
    w, s, _ = weight(130, 160, 1)
    we, se = w[None].expand(3, -1, -1).contiguous(), s[None].expand(3, -1, -1).contiguous()
    order, _, offsets = routing(tokens, 3, 2, 5, 0.1)
    x = normal((tokens, 160), 2, dtype)

    def step():
        q, qs = iq.quantize_groups(x, status=word, check=False)
        return (iq.fp4_linear(x, w, s), iq.fp4_expert_linear(x, we, se, offsets, order, top_k=2),
                iq.dequantize_groups(q, qs, dtype=dtype))

    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # two graphs, whose workspaces come from the pools they were captured with
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                r = step()
            graphs.append((g, r))
    for i in range(4):
        x.copy_(normal((tokens, 160), 20 + i, dtype))
        want = [t.clone() for t in step()]
        for g, r in graphs:
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(r, want):
                assert torch.equal(a, b)


def test_results_do_not_change_from_call_to_call():
    w, s, _ = weight(513, 1024, 1)
    for tokens in (1, 24, 100, 700):
        x = normal((tokens, 1024), 2, torch.bfloat16)
        first = iq.fp4_linear(x, w, s)
        for _ in range(5):
            assert torch.equal(iq.fp4_linear(x, w, s), first)


# ---------------------------------------------------------------------------
# Infinite weights
# ---------------------------------------------------------------------------

INF = float("inf")
# Ones whose lower bf16 parts are all 0, ones that have them, and what is not finite.
NEXT_TO_INFINITE = [1.0, 1.00390625, 0.1, 0.0, -1.25, -0.7, 1.5, INF, -INF, float("nan")]


def edge_weight(shape, depth, seed):
    """Small weights [*shape, depth] in whose last group but one value is zero: that has one of
    16 codes and a scale byte of 250 .. 254, where 253 and 254 reach beyond fp32."""
    n = int(np.prod(shape))
    c = torch.randint(0, 16, (n, depth), generator=gen(seed), dtype=torch.uint8)
    s = torch.randint(118, 124, (n, depth // 32), generator=gen(seed + 1), dtype=torch.uint8)
    at, i = depth - 27, torch.arange(n)
    c[:, depth - 32:] = 0
    c[:, at] = (i % 16).to(torch.uint8)
    s[:, -1] = (250 + i // 16 % 5).to(torch.uint8)
    w = (c[:, 0::2] | (c[:, 1::2] << 4)).reshape(*shape, depth // 2)
    s = s.reshape(*shape, depth // 32)
    return w.to(DEV), s.to(DEV), ref.values(w.numpy(), s.numpy())


def edge_tokens(tokens, depth, seed, dtype):
    x = torch.randn((tokens, depth), generator=gen(seed)).to(dtype)
    x[:, depth - 27] = torch.tensor([NEXT_TO_INFINITE[t % 10] for t in range(tokens)]).to(dtype)
    return x.to(DEV)


def edge_product(x, v):
    """The product and the sum of its terms' magnitudes, the one value of the last group apart:
    there 0 and infinity meet as they do in floats."""
    at = x.shape[1] - 27
    rest, last = x.copy(), x[:, at, None]
    rest[:, at] = 0.0
    finite = v.copy()
    finite[:, at] = 0.0
    y, size = ref.product(rest, finite)
    with np.errstate(invalid="ignore"):
        term = last * v[:, at]
        return y + term, size + np.abs(term)


def check_edges(got, y, size, depth, dtype):
    """What is beyond the type's largest value, or not finite, has to be so exactly; the rest is
    within the product's bound.  (No sum is so near to that border that roundings could cross it:
    the large terms are at most 1.875 2^127 or at least 1.125 2^128, the others below 2^10.)"""
    got, most = to64(got), torch.finfo(dtype).max
    with np.errstate(invalid="ignore"):
        y = np.where(np.abs(y) > most, np.sign(y) * np.inf, y)
    assert np.array_equal(np.isnan(got), np.isnan(y))
    inf = np.isinf(y)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], y[inf])
    ok = np.isfinite(y)
    over = np.abs(got[ok] - y[ok]) - ref.product_bound(y[ok], size[ok], depth, dtype)
    assert (over <= 0).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", PRODUCTS)
def test_infinite_weights(dtype, tokens, channels, depth):
    x = edge_tokens(tokens, depth, 4, dtype)
    w, s, v = edge_weight((channels,), depth, 5)
    y, size = edge_product(to64(x), v)
    check_edges(iq.fp4_linear(x, w, s), y, size, depth, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,experts,top_k,channels,depth,dropped,favourite", EXPERT_CASES)
def test_infinite_weights_by_expert(dtype, tokens, experts, top_k, channels, depth, dropped, favourite):
    order, _, offsets = routing(tokens, experts, top_k, 11, dropped, favourite)
    o, f = order.cpu().numpy(), offsets.cpu().numpy()
    x = edge_tokens(tokens, depth, 4, dtype)
    w, s, v = edge_weight((experts, channels), depth, 5)
    y, size = np.zeros((len(o), channels)), np.zeros((len(o), channels))
    for e in range(experts):
        rows = slice(int(f[e]), int(f[e + 1]))
        y[rows], size[rows] = edge_product(to64(x)[o[rows] // top_k], v[e])
    check_edges(iq.fp4_expert_linear(x, w, s, offsets, order, top_k=top_k), y, size, depth, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens", [1, 5, 30, 100, 700])
def test_a_scale_that_is_nan_counts_over_zeros(dtype, tokens):
    """A group of zeros whose scale byte is 255 is a group of NaN, and its channel's results are."""
    channels, depth = 130, 160
    x = integers((tokens, depth), 1).to(dtype).to(DEV)
    w, s = random_codes((channels, depth), 2), random_scale((channels, depth // 32), 3, 126, 128)
    # with any other scale byte it is one of zeros
    w[20:, 64:] = 0
    want = iq.fp4_linear(x, w, s)
    s[20:, 4] = (torch.arange(channels - 20) * 7 % 255).to(torch.uint8).to(DEV)
    assert torch.equal(iq.fp4_linear(x, w, s), want)
    w[5, 32:48], s[5, 2] = 0, 255
    w[77, 64:], s[77, 4] = 0x88, 255                    # -0, a row's last group
    got = iq.fp4_linear(x, w, s)
    assert torch.isnan(got[:, [5, 77]]).all()
    keep = [i for i in range(channels) if i not in (5, 77)]
    assert torch.equal(got[:, keep], want[:, keep])
    off = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    by_expert = iq.fp4_expert_linear(x, w[None], s[None], off)
    assert torch.isnan(by_expert[:, [5, 77]]).all()
    assert torch.equal(by_expert[:, keep], want[:, keep])
