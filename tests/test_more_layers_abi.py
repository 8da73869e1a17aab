"""CPU checks of the C-ABI of the 4-bit weights and the router: every function that
include/iq_fp4.h and include/iq_router.h declare is exported, and bad arguments are
refused before any device work."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, ARG = 1, 3, 8
P = ctypes.c_void_p
FAKE = P(0x100000)      # never dereferenced: validation fails before any device access
ODD = P(0x100001)
HALF = P(0x100002)
BASE = 0x100000


@pytest.fixture(scope="module")
def lib():
    import ggml_iq_codebook_amd as iq
    return iq.load(build_if_missing=True)


def test_library_exports_every_declared_symbol(lib):
    found = {}
    for header in ("iq_fp4.h", "iq_router.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        found[header] = sorted(set(re.findall(r"^\s*(?:iq_status_t|int64_t)\s+(iq_\w+)\s*\(", text, flags=re.M)))
    assert found == {
        "iq_fp4.h": sorted(["iq_quantize_groups", "iq_dequantize_groups", "iq_fp4_linear",
                            "iq_fp4_linear_workspace", "iq_fp4_expert_linear",
                            "iq_fp4_expert_linear_workspace"]),
        "iq_router.h": sorted(["iq_expert_gate", "iq_expert_gate_backward", "iq_expert_balance",
                               "iq_expert_balance_workspace", "iq_expert_balance_backward"])}
    for names in found.values():
        for name in names:
            assert hasattr(lib, name), name


# --- the calls, with good arguments by default --------------------------------

def quantize(lib, dt=1, x=FAKE, ldx=64, r=8, c=64, q=FAKE, ldc=32, s=FAKE, lds=2, st=FAKE):
    return lib.iq_quantize_groups(dt, x, ldx, r, c, q, ldc, s, lds, st, None)


def dequantize(lib, q=FAKE, ldc=32, s=FAKE, lds=2, r=8, c=64, dt=1, y=FAKE, ldy=64):
    return lib.iq_dequantize_groups(q, ldc, s, lds, r, c, dt, y, ldy, None)


def linear(lib, dt=1, x=FAKE, ldx=64, w=FAKE, ldw=32, s=FAKE, lds=2, t=8, n=16, k=64, y=FAKE, ldy=16,
           wk=None, wb=0):
    return lib.iq_fp4_linear(dt, x, ldx, w, ldw, s, lds, t, n, k, y, ldy, wk, wb, None)


def expert(lib, dt=1, x=FAKE, ldx=64, t=8, order=FAKE, k=2, off=FAKE, e=3, rows=16, w=FAKE, ldw=32, wst=512,
           s=FAKE, lds=2, sst=32, n=16, d=64, y=FAKE, ldy=16, wk=None, wb=0):
    return lib.iq_fp4_expert_linear(dt, x, ldx, t, order, k, off, e, rows, w, ldw, wst, s, lds, sst, n, d, y,
                                    ldy, wk, wb, None)


def gate(lib, dt=0, l=FAKE, ld=16, t=8, e=16, k=2, rn=1, c=FAKE, w=FAKE, st=FAKE):
    return lib.iq_expert_gate(dt, l, ld, t, e, k, rn, c, w, st, None)


def gate_backward(lib, dt=0, g=FAKE, l=FAKE, ld=16, t=8, e=16, c=FAKE, w=FAKE, k=2, rn=0, o=FAKE, ldo=16):
    return lib.iq_expert_gate_backward(dt, g, l, ld, t, e, c, w, k, rn, o, ldo, None)


def balance(lib, dt=0, l=FAKE, ld=16, t=8, e=16, c=FAKE, cb=4, k=2, loss=FAKE, n=FAKE, live=FAKE, wk=None,
            wb=0, st=FAKE):
    return lib.iq_expert_balance(dt, l, ld, t, e, c, cb, k, loss, n, live, wk, wb, st, None)


def balance_backward(lib, dt=0, g=FAKE, l=FAKE, ld=16, t=8, e=16, n=FAKE, live=FAKE, o=FAKE, ldo=16):
    return lib.iq_expert_balance_backward(dt, g, l, ld, t, e, n, live, o, ldo, None)


CASES = {
    quantize: (["x", "q", "s"],
               [dict(r=-1), dict(c=0), dict(c=48), dict(c=65), dict(ldx=-1), dict(ldc=31), dict(lds=1),
                dict(ldx=1 << 60, r=1 << 20), dict(ldc=1 << 60, r=1 << 20)],
               [dict(dt=3), dict(dt=-1), dict(x=ODD), dict(dt=0, x=HALF), dict(st=HALF)]),
    dequantize: (["q", "s", "y"],
                 [dict(r=-1), dict(c=0), dict(c=48), dict(ldc=-1), dict(lds=-1), dict(ldy=63)],
                 [dict(dt=3), dict(y=ODD), dict(dt=0, y=HALF)]),
    linear: (["x", "w", "s", "y"],
             [dict(t=-1), dict(n=0), dict(k=0), dict(k=40), dict(ldx=-1), dict(ldw=-1), dict(lds=-1),
              dict(ldy=15), dict(t=1 << 31), dict(n=1 << 31), dict(k=1 << 31), dict(ldx=1 << 60)],
             [dict(dt=3), dict(x=ODD), dict(y=ODD), dict(dt=0, y=HALF)]),
    expert: (["x", "off", "w", "s", "y"],
             [dict(t=-1), dict(t=0), dict(k=0), dict(e=0), dict(e=513), dict(rows=-1), dict(rows=1 << 31),
              dict(wst=-1), dict(sst=-1), dict(wst=1 << 60), dict(sst=1 << 60), dict(n=0), dict(d=0),
              dict(d=33), dict(ldy=15), dict(order=None)],
             [dict(dt=3), dict(x=ODD), dict(y=ODD), dict(order=HALF), dict(off=HALF)]),
    gate: (["l", "c", "w"],
           [dict(t=-1), dict(e=0), dict(e=513), dict(k=0), dict(k=17), dict(ld=-1), dict(t=1 << 30, k=2)],
           [dict(dt=3), dict(l=HALF), dict(dt=1, l=ODD), dict(c=HALF), dict(w=HALF), dict(st=HALF)]),
    gate_backward: (["g", "l", "c", "w", "o"],
                    [dict(t=-1), dict(e=0), dict(e=513), dict(k=0), dict(k=17), dict(ld=-1), dict(ldo=15),
                     dict(t=1 << 30, k=2)],
                    [dict(dt=3), dict(l=HALF), dict(o=HALF), dict(c=HALF), dict(w=HALF), dict(g=HALF)]),
    balance: (["l", "c", "loss", "n", "live"],
              [dict(t=-1), dict(e=0), dict(e=513), dict(k=0), dict(ld=-1), dict(t=1 << 30, k=2)],
              [dict(dt=3), dict(l=HALF), dict(c=HALF), dict(cb=2), dict(cb=8, c=P(0x100004)),
               dict(loss=HALF), dict(n=HALF), dict(live=HALF), dict(st=HALF)]),
    balance_backward: (["g", "l", "n", "live", "o"],
                       [dict(t=-1), dict(e=0), dict(e=513), dict(ld=-1), dict(ldo=15)],
                       [dict(dt=3), dict(l=HALF), dict(o=HALF), dict(n=HALF), dict(live=HALF), dict(g=HALF)]),
}


@pytest.mark.parametrize("call", CASES, ids=lambda f: f.__name__)
def test_refusals(lib, call):
    pointers, shapes, args = CASES[call]
    for name in pointers:
        assert call(lib, **{name: None}) == NULL, name
    for bad in shapes:
        assert call(lib, **bad) == SHAPE, bad
    for bad in args:
        assert call(lib, **bad) == ARG, bad


def test_nothing_to_do(lib):
    assert quantize(lib, r=0, x=None, q=None, s=None, st=None) == 0
    assert dequantize(lib, r=0, q=None, s=None, y=None) == 0
    assert linear(lib, t=0, x=None, y=None) == 0
    assert expert(lib, t=0, rows=0, x=None, off=None, y=None) == 0
    assert gate(lib, t=0, l=None, c=None, w=None, st=None) == 0
    assert gate_backward(lib, t=0, g=None, l=None, c=None, w=None, o=None) == 0
    assert balance_backward(lib, t=0, g=None, l=None, n=None, live=None, o=None) == 0


def test_a_workspace_that_is_missing_or_short(lib):
    need = lib.iq_expert_balance_workspace(100000, 64)
    assert need > 0 and lib.iq_expert_balance_workspace(4, 64) == 0
    for bad in ((0, 64), (-1, 64), (8, 0), (8, 513)):
        assert lib.iq_expert_balance_workspace(*bad) == 0
    big = dict(t=100000, e=64, ld=64, l=P(1 << 32), c=P(2 << 32))
    assert balance(lib, **big) == NULL
    assert balance(lib, wk=P(3 << 32), wb=need - 1, **big) == ARG
    assert balance(lib, wk=P((3 << 32) + 4), wb=need, **big) == ARG


# --- overlaps ---------------------------------------------------------------

@pytest.mark.parametrize("call,sizes,outputs", [
    (quantize, dict(x=1024, q=256, s=16, st=4), ["q", "s"]),
    (dequantize, dict(q=256, s=16, y=1024), ["y"]),
    (linear, dict(x=1024, w=512, s=32, y=256), ["y"]),
    (expert, dict(x=1024, order=64, off=16, w=1536, s=96, y=512), ["y"]),
    (gate, dict(l=512, c=64, w=64, st=4), ["c", "w"]),
    (gate_backward, dict(g=64, l=512, c=64, w=64, o=512), ["o"]),
    (balance, dict(l=512, c=64, n=64), ["n"]),
    (balance_backward, dict(l=512, n=64, o=512), ["o"]),
], ids=lambda v: getattr(v, "__name__", None))
def test_overlapping_outputs_are_refused(lib, call, sizes, outputs):
    """Every buffer far from the others, but one pair of an output and another: the second
    begins 8 bytes before the first one's end (a status word has 4), in both orders."""
    names = list(sizes)
    extra = {}
    if call is balance:
        extra = dict(loss=P(0x10), live=P(0x20), st=P(0x30))
    if call is balance_backward:
        extra = dict(g=P(0x10), live=P(0x20))
    for out in outputs:
        for other in names:
            if other == out:
                continue
            for first, second in ((out, other), (other, out)):
                at = {n: BASE + (i + 1) * (1 << 24) for i, n in enumerate(names)}
                at[second] = at[first] + sizes[first] - 8
                assert call(lib, **extra, **{n: P(v) for n, v in at.items()}) == ARG, (out, other, first)


def test_expert_weights_far_apart_may_hold_the_result_between_them(lib):
    """Only the memory of each expert's rows counts, not what lies between."""
    far = dict(wst=1 << 20, w=P(1 << 30), s=P(1 << 32), x=P(1 << 33), order=P(1 << 34), off=P(1 << 35))
    assert expert(lib, y=P((1 << 30) + 256), **far) == ARG
    assert expert(lib, y=P((1 << 30) + (1 << 20) + 256), **far) == ARG
    # between the first two: not refused as an argument (no GPU here, or a different error)
    import torch
    if not torch.cuda.is_available():
        assert expert(lib, y=P((1 << 30) + 4096), **far) not in (ARG, SHAPE, NULL)


def test_one_buffer_for_two_outputs_is_refused(lib):
    assert balance(lib, loss=P(0x100), live=P(0x100), n=P(0x1000), l=P(0x10000), c=P(0x20000)) == ARG
    assert balance(lib, loss=P(0x1000), live=P(0x100), n=P(0x1000), l=P(0x10000), c=P(0x20000)) == ARG
    assert gate(lib, c=P(0x1000), w=P(0x1000), l=P(0x10000), st=P(0x20000)) == ARG


def test_binding_refuses_cpu_tensors():
    import torch

    import ggml_iq_codebook_amd as iq
    x = torch.zeros((2, 32))
    w, s = torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.uint8)
    off, choice = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1), dtype=torch.int32)
    one = torch.zeros((2, 1))
    for call in (lambda: iq.quantize_groups(x), lambda: iq.dequantize_groups(w, s),
                 lambda: iq.fp4_linear(x, w, s), lambda: iq.fp4_expert_linear(x, w[None], s[None], off),
                 lambda: iq.expert_gate(x, 1), lambda: iq.expert_gate_backward(one, x, choice, one),
                 lambda: iq.expert_balance(x, choice),
                 lambda: iq.expert_balance_backward(one, x, torch.zeros(32, dtype=torch.int32), off[0])):
        with pytest.raises(ValueError):
            call()
