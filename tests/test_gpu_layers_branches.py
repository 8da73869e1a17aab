"""Forms of the layer operators that only certain sizes take: many choices a token
in wide rows, sorted rows beyond the caches, many long rows, sorts of several
chunks, and workspaces on several streams, in graphs and from several threads.

References and bounds as in test_gpu_layers.py.
"""

import sys
import threading

import numpy as np
import pytest
import torch

from tests import layers_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402
from tests.test_gpu_layers import (  # noqa: E402
    DEV, DTYPES, IDS, codes, gen, normal, routed, routing, scales, strided, within)


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


# ---------------------------------------------------------------------------
# Rounding and the layer for a few tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(8193, 1025), (8200, 4096), (8200, 4089)])
def test_quantize_many_long_rows(dtype, rows, cols):
    x = normal((rows, cols), rows + cols, dtype)
    x[rows - 3] = 0
    x[77, 5] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q, s = iq.quantize_rows(x, status=status, check=False)
    assert int(status.item()) == 5
    wq, ws = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,channels,depth", [(16, 75, 512), (16, 4096, 100), (9, 33, 511), (12, 130, 48),
                                                   (16, 17, 1)])
def test_linear_of_9_to_16_tokens(dtype, tokens, channels, depth):
    x = normal((tokens, depth), tokens + depth, dtype)
    w, ws = iq.quantize_rows(normal((channels, depth), channels))
    y = iq.int8_linear(x, w, ws)
    q, s = ref.quantize(x.float().cpu().numpy())
    want = ref.product(q, s, w.cpu().numpy(), ws.cpu().numpy())
    within(y, want, ref.product_bound(want, dtype))
    assert torch.equal(y, iq.int8_matmul(*iq.quantize_rows(x), w, ws, dtype=dtype))
    assert torch.equal(y, iq.int8_linear(strided(x, 3, 1), w, ws))
    x[tokens - 1, depth - 1] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = iq.int8_linear(x, w, ws, status=status, check=False)
    assert int(status.item()) == 5
    assert not bad[tokens - 1].any() and torch.equal(bad[:tokens - 1], y[:tokens - 1])


# ---------------------------------------------------------------------------
# The sort
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("tokens,top_k,experts,dropped,kind", [
    (150001, 2, 64, 0.1, "even"), (125000, 8, 512, 0.05, "even"), (333333, 3, 13, 0.0, "one"),
    (262145, 1, 5, 0.0, "few"), (1048577, 1, 100, 0.1, "even")])
def test_sort_of_several_steps_a_wave(dtype, tokens, top_k, experts, dropped, kind):
    c = routing(tokens, top_k, experts, tokens, dropped, kind)
    for g, w in zip(iq.expert_sort(c.to(dtype).to(DEV), experts), ref.sort(c.numpy(), experts)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w)


# ---------------------------------------------------------------------------
# The copies
# ---------------------------------------------------------------------------

# Rows of a wave or a workgroup, with 5 choices to more than two groups of 8.
ROUTES = [(9, 8, 16, 1100, 0.1), (5, 6, 8, 2056, 0.2), (4, 17, 20, 1300, 0.2), (7, 5, 6, 300, 0.1),
          (6, 9, 12, 600, 0.3), (3, 24, 30, 4099, 0.1), (5, 7, 9, 5120, 0.0)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,top_k,experts,width,dropped", ROUTES)
def test_copies_of_many_choices(dtype, tokens, top_k, experts, width, dropped):
    position, offsets, p, f = routed(tokens, top_k, experts, dropped)
    rows, kept = tokens * top_k, int(offsets[-1])
    x, y, g = normal((tokens, width), 1, dtype), normal((rows, width), 2, dtype), normal((tokens, width), 4, dtype)
    weights = torch.rand((tokens, top_k), generator=gen(3)).to(DEV)
    y[kept:] = float("nan")                       # dropped rows are not read
    assert np.array_equal(ref.to64(iq.expert_dispatch(x, p, f)), ref.dispatch(ref.to64(x), position, offsets))
    w64, y64 = ref.to64(weights), ref.to64(y)
    out, size = ref.combine(y64, position, offsets, w64)
    within(iq.expert_combine(y, p, f, weights), out, ref.combine_bound(out, size, top_k, dtype))
    dx, size = ref.combine(y64, position, offsets, np.ones_like(w64))
    within(iq.expert_dispatch_backward(y, p, f), dx, ref.combine_bound(dx, size, top_k, dtype))
    gy, gw = iq.expert_combine_backward(g, y, p, f, weights)
    wy, ww, size = ref.combine_backward(ref.to64(g), np.nan_to_num(y64), position, offsets, w64)
    within(gy, wy, ref.combine_bound(wy, np.abs(wy), 1, dtype))
    within(gw, ww, ref.dot_bound(size, width))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("top_k", [5, 8, 11])
@pytest.mark.parametrize("width", [515, 1030, 2055])
@pytest.mark.parametrize("pad,shift", [(16, 0), (5, 7)])
def test_copies_of_many_choices_strides(dtype, top_k, width, pad, shift):
    tokens = 6
    _, _, p, f = routed(tokens, top_k, 7, 0.2)
    x, y = normal((tokens, width), 1, dtype), normal((tokens * top_k, width), 2, dtype)
    g, weights = normal((tokens, width), 4, dtype), torch.rand((tokens, top_k), generator=gen(3)).to(DEV)
    sx, sy, sg = (strided(t, pad, shift) for t in (x, y, g))
    assert torch.equal(iq.expert_dispatch(x, p, f), iq.expert_dispatch(sx, p, f))
    assert torch.equal(iq.expert_combine(y, p, f, weights), iq.expert_combine(sy, p, f, weights))
    assert torch.equal(iq.expert_dispatch_backward(y, p, f), iq.expert_dispatch_backward(sy, p, f))
    for a, b in zip(iq.expert_combine_backward(g, y, p, f, weights),
                    iq.expert_combine_backward(sg, sy, p, f, weights)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,top_k,width", [(230000, 3, 101), (60000, 3, 500), (12000, 5, 1204), (3000, 9, 4096)])
def test_sorted_rows_beyond_the_caches(dtype, tokens, top_k, width):
    """Over 128 MiB of them, in 64 bits on the GPU."""
    if dtype == torch.float32:
        tokens = tokens * 2 // 3
    assert tokens * top_k * width * dtype.itemsize > 128 << 20
    c = routing(tokens, top_k, 16, 77, 0.05).to(DEV)
    order, p, f = iq.expert_sort(c, 16)
    kept, token = int(f[-1]), (order // top_k).long()
    x, g = normal((tokens, width), 1, dtype), normal((tokens, width), 2, dtype)
    w = torch.rand((tokens, top_k), generator=gen(3)).to(DEV)
    xs = iq.expert_dispatch(x, p, f)
    assert torch.equal(xs[:kept], x[token[:kept]]) and not xs[kept:].any()
    gy, gw = iq.expert_combine_backward(g, xs, p, f, w)
    want = (g[token[:kept]].float() * w.flatten()[order[:kept].long()][:, None]).to(dtype)
    assert torch.equal(gy[:kept], want) and not gy[kept:].any()
    dots = (x.double() * g.double()).sum(dim=1)[:, None] * (c >= 0)
    sizes = (x.double() * g.double()).abs().sum(dim=1)[:, None] * (c >= 0)
    within(gw, ref.to64(dots), ref.dot_bound(ref.to64(sizes), width))
    # all of a token's kept rows are x: the sums are x times the sum of the weights
    for got, each in ((iq.expert_combine(xs, p, f, w), w.double()), (iq.expert_dispatch_backward(xs, p, f), 1.0)):
        total = ((c >= 0) * each).sum(dim=1, keepdim=True)
        want = x.double() * total
        bound = want.abs() * (ref.ROUND[dtype] + (top_k + 1) * 2.0 ** -24 * (1 + 2.0 ** -7)) + 2 * ref.TINY[dtype]
        assert ((got.double() - want).abs() <= bound).all()


# ---------------------------------------------------------------------------
# Workspaces on streams, in graphs, from threads
# ---------------------------------------------------------------------------

def inputs(seed):
    return (normal((40, 700), seed, torch.bfloat16), routing(5000, 2, 9, seed, 0.1).to(DEV))


def both(x, choice, w, ws, status):
    """A layer whose codes go through a workspace, and a sort whose counts do."""
    report = dict(status=status, check=False)
    return (iq.int8_linear(x, w, ws, **report), *iq.expert_sort(choice, 9, **report))


def test_workspaces_on_streams_and_in_graphs():
    w, ws = codes((300, 700), 1), scales(300, 2)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sets = [inputs(10 + s) for s in range(4)]
    want = [both(*v, w, ws, status) for v in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in sets]
    for _ in range(8):
        for i, v in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(both(*v, w, ws, status))
    torch.cuda.synchronize()
    for results, expected in zip(got, want):
        for result in results:
            assert all(torch.equal(a, b) for a, b in zip(result, expected))
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*held, w, ws, status)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(*held, w, ws, status)
    for r in range(8):
        for h, v in zip(held, sets[r % 4]):
            h.copy_(v)
        graph.replay()
        eager = both(*sets[(r + 1) % 4], w, ws, status)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[r % 4]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[(r + 1) % 4]))
    assert int(status.item()) == 0


@pytest.mark.parametrize("check", [True, False], ids=["waiting", "status"])
def test_calls_from_threads(check):
    w, ws = codes((300, 700), 1), scales(300, 2)
    sets = [inputs(20 + s) for s in range(4)]
    bad = sets[3][0].clone()
    bad[5, 6] = float("nan")
    want = [(iq.int8_linear(x, w, ws), *iq.expert_sort(c, 9)) for x, c in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            x, c = sets[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                status = None if check else torch.zeros(1, dtype=torch.int32, device=DEV)
                for _ in range(20):
                    got = (iq.int8_linear(x, w, ws, status=status, check=check),
                           *iq.expert_sort(c, 9, status=status, check=check))
                    if i == 3 and check:              # this thread's errors are its own
                        with pytest.raises(iq.IQError):
                            iq.int8_linear(bad, w, ws)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except BaseException as e:                    # reported by the test's own thread
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
