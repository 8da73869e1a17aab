"""CPU checks of how 8-bit products choose their tile: the tables are what the
measured times give, the choice is as near to the fastest tile as its comments say,
and the GPU tests' shapes take every tile there is."""

import ast
import ctypes
import math
import os
import random
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "perf"))

import tiles  # noqa: E402

NAMES = list(tiles.TABLES)
SHIM = r"""
#include "int8_tiles.hpp"
using namespace iqk;
template <int kN>
static int pick(int64_t rows, int64_t channels, int64_t depth, int experts, int cus, const TileTime (&t)[kN])
{
    return fastest_tile(rows, channels, depth, experts, cus, t);
}
extern "C" int choose(int table, int64_t rows, int64_t channels, int64_t depth, int experts, int cus)
{
    return table == 0 ? pick(rows, channels, depth, experts, cus, kDense)
           : table == 1 ? pick(rows, channels, depth, experts, cus, kByExpert)
                        : pick(rows, channels, depth, experts, cus, kUnaligned);
}
template <int kN>
static int entry(const TileTime (&t)[kN], int i, double* out)
{
    if (i >= kN) return 0;
    const double v[] = {(double)t[i].rows, (double)t[i].channels, t[i].once, t[i].start, t[i].depth,
                        t[i].start_full, t[i].depth_full};
    for (int j = 0; j < 7; ++j) out[j] = v[j];
    return 1;
}
extern "C" int tile(int table, int i, double* out)
{
    return table == 0 ? entry(kDense, i, out) : table == 1 ? entry(kByExpert, i, out) : entry(kUnaligned, i, out);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("tiles")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "ggml_iq_codebook_amd", "csrc"), str(at / "shim.cpp"), "-o",
                    str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(str(at / "shim.so"))
    i64, c = ctypes.c_int64, ctypes.c_int
    lib.choose.argtypes = [c, i64, i64, i64, c, c]
    lib.tile.argtypes = [c, c, ctypes.POINTER(ctypes.c_double)]

    def table(k):
        entries, out = [], (ctypes.c_double * 7)()
        while lib.tile(k, len(entries), out):
            entries.append(list(out))
        return entries
    return lib, [table(k) for k in range(3)]


@pytest.fixture(scope="module")
def data():
    return tiles.measured()


@pytest.mark.parametrize("k", range(3), ids=NAMES)
def test_tables_are_the_fit(rule, data, k):
    constants = tiles.fit(data[NAMES[k]])
    assert [(e[0], e[1]) for e in rule[1][k]] == [tiles.size(t) for t in tiles.TABLES[NAMES[k]]]
    for entry, tile in zip(rule[1][k], tiles.TABLES[NAMES[k]]):
        # rounded to two places, from times with four
        assert all(abs(a - b) < 0.0101 for a, b in zip(entry[2:], constants[tile])), tile


# What the comments state, rounded as there: the average and the worst, in percent.
@pytest.mark.parametrize("k,average,worst", [(0, 0.2, 7), (1, 4, 55), (2, 2, 20)], ids=NAMES)
def test_choice_is_as_near_to_the_fastest_as_stated(rule, data, k, average, worst):
    name = NAMES[k]
    constants = {t: e[2:] for t, e in zip(tiles.TABLES[name], rule[1][k])}
    ratios = tiles.excess(data[name], constants, tiles.TABLES[name])
    assert len(ratios) >= len(data[name]["products"]) - 5
    places = 1 if average < 1 else 0
    assert round(100 * tiles.mean(ratios) - 100, places) == average
    assert round(100 * max(ratios) - 100) == worst


def test_what_the_tiles_with_a_side_of_192_are_worth(rule, data):
    constants = {t: e[2:] for t, e in zip(tiles.TABLES["dense"], rule[1][0])}
    ratios = tiles.excess(data["dense"], constants, [t for t in tiles.TABLES["dense"] if "192" not in t])
    assert round(100 * tiles.mean(ratios) - 100, 1) == 1.5 and round(100 * max(ratios) - 100) == 38
    ratios = tiles.excess(data["dense"], constants, ["128x128"])
    assert round(100 * tiles.mean(ratios) - 100) == 77


@pytest.mark.parametrize("k", range(3), ids=NAMES)
def test_compiled_rule_is_the_fitted_one(rule, k):
    lib, tables = rule
    names = tiles.TABLES[NAMES[k]]
    constants = {t: e[2:] for t, e in zip(names, tables[k])}
    rng = random.Random(k)
    for _ in range(2000):
        rows, channels = (int(math.exp(rng.uniform(0, math.log(70000)))) for _ in range(2))
        depth, experts = rng.randint(1, 16384), rng.randint(1, 512) if k == 1 else 0
        chosen = names[lib.choose(k, rows, channels, depth, experts, 256)]
        times = {t: sum(c * v for c, v in zip(constants[t], tiles.terms(t, rows, channels, depth, experts)))
                 for t in names}
        assert times[chosen] <= min(times.values()) * (1 + 1e-12)


def test_gpu_tests_take_every_tile(rule):
    """LARGE of test_gpu_layers.py, dense and (2 choices, 5 experts) by expert, in rows that
    start on 16 bytes and in rows that do not."""
    lib, tables = rule
    with open(os.path.join(ROOT, "tests", "test_gpu_layers.py")) as f:
        shapes = next(ast.literal_eval(n.value) for n in ast.parse(f.read()).body
                      if isinstance(n, ast.Assign) and n.targets[0].id == "LARGE")
    taken = {k: set() for k in ("dense", "by expert", "dense unaligned", "by expert unaligned")}
    for tokens, channels, depth in shapes:
        taken["dense"].add(lib.choose(0, tokens, channels, depth, 0, 256))
        taken["by expert"].add(lib.choose(1, 2 * tokens, channels, depth, 5, 256))
        if depth % 16:
            taken["dense unaligned"].add(lib.choose(2, tokens, channels, depth, 0, 256))
            taken["by expert unaligned"].add(lib.choose(2, 2 * tokens, channels, depth, 5, 256))
    assert taken == {"dense": set(range(len(tables[0]))), "by expert": set(range(len(tables[1]))),
                     "dense unaligned": set(range(len(tables[2]))),
                     "by expert unaligned": set(range(len(tables[2])))}
