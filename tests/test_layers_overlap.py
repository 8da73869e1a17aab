"""CPU checks of what the layer operators refuse about memory: outputs that overlap
inputs or each other.  Only refused calls reach the library here, so the
pointers are never read."""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG = 8
P = ctypes.c_void_p
BASE = 0x100000


@pytest.fixture(scope="module")
def lib():
    import ggml_iq_codebook_amd as iq
    return iq.load(build_if_missing=True)


def refused_alone(call, sizes, outputs):
    """Every buffer far from the others, but one pair of an output and another whose last
    and first bytes are shared, in both orders.  `sizes`: the bytes of each pointer argument."""
    names = list(sizes)
    for out in outputs:
        for other in names:
            if other == out:
                continue
            for first, second in ((out, other), (other, out)):
                at = {n: BASE + (i + 1) * (1 << 24) for i, n in enumerate(names)}
                at[second] = at[first] + sizes[first] - 16
                assert call(**{n: P(v) for n, v in at.items()}) == ARG, (out, other, first)


def test_quantize_rows(lib):
    def f(x, q, s, st):
        return lib.iq_quantize_rows(1, x, 64, 8, 64, q, 64, s, st, None)
    refused_alone(f, dict(x=1024, q=512, s=32, st=16), ["q", "s"])


def test_int8_matmul(lib):
    def f(x, xs, w, ws, y):
        return lib.iq_int8_matmul(x, 64, xs, w, 64, ws, 16, 32, 64, 1, y, 32, None)
    refused_alone(f, dict(x=1024, xs=64, w=2048, ws=128, y=1024), ["y"])


@pytest.mark.parametrize("tokens", [2, 40])
def test_int8_linear(lib, tokens):
    need = lib.iq_int8_linear_workspace(tokens, 64, 64)
    assert (need == 0) == (tokens == 2)

    def f(x, w, ws, y, wk=None):
        return lib.iq_int8_linear(1, x, 64, w, 64, ws, tokens, 64, 64, y, 64, wk, need, P(0x100), None)
    sizes = dict(x=tokens * 128, w=4096, ws=256, y=tokens * 128)
    if need:
        sizes["wk"] = need
    refused_alone(f, sizes, ["y", "wk"] if need else ["y"])
    same = P(BASE)                                           # a square layer on its own input
    assert f(same, P(BASE + (1 << 24)), P(BASE + (2 << 24)), same, P(BASE + (3 << 24)) if need else None) == ARG


def test_int8_expert_matmul(lib):
    def f(x, xs, o, off, w, ws, y):
        return lib.iq_int8_expert_matmul(x, 64, xs, 16, o, 2, off, 3, 32, w, 64, 2048, ws, 32, 64, 1,
                                         y, 32, None)
    refused_alone(f, dict(x=1024, xs=64, o=128, off=16, w=3 * 2048, ws=384, y=2048), ["y"])


def test_expert_sort(lib):
    need = lib.iq_expert_sort_workspace(8192, 3)

    def f(c, o, p, off, wk):
        return lib.iq_expert_sort(c, 4, 4096, 2, 3, o, p, off, wk, need, P(0x100), None)
    refused_alone(f, dict(c=32768, o=32768, p=32768, off=16, wk=need), ["o", "p", "off", "wk"])


def test_routing(lib):
    t, k, d = 16, 2, 32
    small, large = t * d * 2, t * k * d * 2
    refused_alone(lambda x, p, off, y: lib.iq_expert_dispatch(1, x, d, t, d, p, k, off, 3, y, d, None),
                  dict(x=small, p=128, off=16, y=large), ["y"])
    refused_alone(lambda g, p, off, y: lib.iq_expert_dispatch_backward(1, g, d, t, d, p, k, off, 3, y, d, None),
                  dict(g=large, p=128, off=16, y=small), ["y"])
    refused_alone(lambda x, p, off, w, y: lib.iq_expert_combine(1, x, d, t, d, p, k, off, 3, w, y, d, None),
                  dict(x=large, p=128, off=16, w=128, y=small), ["y"])
    refused_alone(lambda g, x, p, off, w, gy, gw: lib.iq_expert_combine_backward(
        1, g, d, x, d, t, d, p, k, off, 3, w, gy, d, gw, None),
        dict(g=small, x=large, p=128, off=16, w=128, gy=large, gw=128), ["gy", "gw"])


SHIM = r"""
#include "overlap.hpp"
extern "C" int overlap_of(uint64_t p, int64_t rows, int64_t cols, int64_t ld, int bytes,
                          uint64_t q, int64_t rows2, int64_t cols2, int64_t ld2, int bytes2)
{
    return iqk::overlap(iqk::region((void*)p, rows, cols, ld, bytes),
                        iqk::region((void*)q, rows2, cols2, ld2, bytes2));
}
"""


@pytest.fixture(scope="module")
def overlap_of(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("overlap")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "ggml_iq_codebook_amd", "csrc"), str(at / "shim.cpp"), "-o",
                    str(at / "shim.so")], check=True)
    f = ctypes.CDLL(str(at / "shim.so")).overlap_of
    i64, u64, c = ctypes.c_int64, ctypes.c_uint64, ctypes.c_int
    f.argtypes = [u64, i64, i64, i64, c] * 2
    return f


def test_overlap_against_every_byte(overlap_of):
    def held(p, rows, cols, ld, bytes):
        return {p + (r * ld) * bytes + b for r in range(rows) for b in range(cols * bytes)}
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(20000):
        ld = rng.randint(0, 12)
        args = []
        for _ in range(2):
            rows, cols, bytes = rng.randint(0, 6), rng.randint(1, 8), rng.choice([1, 2, 4])
            mine = ld if rng.random() < 0.6 else rng.randint(0, 20)
            args.append((rng.randint(1000, 1080), rows, cols, mine, bytes))
        want = bool(held(*args[0]) & held(*args[1]))
        seen[want] += 1
        assert bool(overlap_of(*args[0], *args[1])) == want, args
    assert min(seen) > 3000


def test_overlap_of_large_regions(overlap_of):
    far, rows = 1 << 45, 2 ** 31 - 1
    # two halves of every row of one buffer, and the same moved by one value
    assert not overlap_of(far, rows, 512, 1024, 2, far + 1024, rows, 512, 1024, 2)
    assert overlap_of(far, rows, 512, 1024, 2, far + 1022, rows, 512, 1024, 2)
    assert overlap_of(far, rows, 513, 1024, 2, far + 1024, rows, 512, 1024, 2)
    # a matrix and the buffer right behind it, and its last byte
    assert not overlap_of(far, rows, 64, 64, 4, far + 256 * rows, 5, 7, 9, 4)
    assert overlap_of(far, rows, 64, 64, 4, far + 256 * rows - 1, 5, 7, 9, 1)
    # the widest rows that are accepted
    assert overlap_of(4096, 1, 1 << 61, 1 << 61, 4, 1 << 40, 1, 1, 1, 1)
    assert not overlap_of(1 << 40, 1, 1 << 61, 1 << 61, 4, 4096, 1, 1, 1, 1)
