"""CPU checks of how products with 4-bit weights choose their size: the tables are what
the measured times give, the choice is as near to the fastest size as their comments
say, and the GPU tests' shapes take every size there is."""

import ast
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "perf"))

import fp4_sizes  # noqa: E402

CSRC = os.path.join(ROOT, "ggml_iq_codebook_amd", "csrc")
TABLES = {"bf16 dense": "kDenseBf16", "f16 dense": "kDenseF16", "f32 dense": "kDenseF32",
          "bf16 by expert": "kExpertBf16", "f16 by expert": "kExpertF16", "f32 by expert": "kExpertF32"}
DTYPES = {"f32": 0, "bf16": 1, "f16": 2}
SHIM = r"""
#include "fp4_sizes.hpp"
extern "C" int size(int dtype, int64_t rows, int64_t channels, int64_t depth, int experts)
{
    return iqk::fp4_size(dtype, rows, channels, depth, experts);
}
"""


def table(name):
    """The entries of a table in the header, and its comment."""
    text = open(os.path.join(CSRC, "fp4_sizes.hpp")).read()
    before, body = text.split("constexpr Fp4Size %s[] = {" % name)
    comment = " ".join(l[3:] for l in before.splitlines()[-3:] if l.startswith("// "))
    rows = re.findall(r"\{([^{}]+)\}", body.split("};")[0] + "}")
    return [tuple(float(v) for v in r.split(",")) for r in rows], comment


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("sizes")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-I", CSRC, "-I",
                    os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
                    str(at / "shim.cpp"), "-o", str(at / "shim.so")], check=True)
    f = ctypes.CDLL(str(at / "shim.so")).size
    f.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return f


def key(size):
    rows, channels, waves = fp4_sizes.numbers(size)
    return (rows * 1000 + channels) * 100 + waves


@pytest.mark.parametrize("name", TABLES)
def test_tables_are_the_fit(name):
    data = fp4_sizes.measured()[name]
    fitted = fp4_sizes.fit(data)
    want = [(*fp4_sizes.numbers(s), slots, *constants) for s, (slots, constants) in fitted.items()]
    got, comment = table(TABLES[name])
    assert got == [tuple(float(v) for v in w) for w in want]
    ratios = fp4_sizes.excess(data, fitted)
    assert len(ratios) == len(data["products"])
    assert "To %d " % len(ratios) in comment
    assert "%.1f %%" % (100 * fp4_sizes.mean(ratios) - 100) in comment
    assert "%.0f %% at worst" % (100 * max(ratios) - 100) in comment


@pytest.mark.parametrize("name", TABLES)
def test_the_rule_is_the_fits(rule, name):
    data = fp4_sizes.measured()[name]
    fitted = fp4_sizes.fit(data)
    dtype = DTYPES[name.split()[0]]
    for *product, _ in data["products"]:
        assert rule(dtype, *product) == key(fp4_sizes.choice(fitted, data["sizes"], *product)), product
    # beyond what was measured there is a size too
    for product in ((1, 1, 32), (2 ** 31 - 1, 1, 32), (1, 2 ** 30 - 1, 32), (2 ** 31 - 1, 2 ** 30 - 1, 2 ** 30)):
        assert rule(dtype, *product, 512 if "expert" in name else 0) in [key(s) for s in data["sizes"]]


def shapes(name):
    """The list of that name in the GPU tests."""
    tree = ast.parse(open(os.path.join(ROOT, "tests", "test_gpu_fp4.py")).read())
    for node in tree.body:
        if isinstance(node, ast.Assign) and node.targets[0].id == name:
            return ast.literal_eval(node.value)
    raise AssertionError(name)


def test_gpu_tests_take_every_size(rule):
    for kind, dtype in ((k, d) for k in ("dense", "by expert") for d in DTYPES):
        sizes = {key(s) for s in fp4_sizes.measured()["%s %s" % (dtype, kind)]["sizes"]}
        if kind == "dense":
            taken = {rule(DTYPES[dtype], t, n, k, 0) for t, n, k in shapes("PRODUCTS")}
        else:
            taken = {rule(DTYPES[dtype], t * k, n, d, e) for t, e, k, n, d, *_ in shapes("EXPERT_CASES")}
        assert taken >= sizes, (kind, dtype, sorted(sizes - taken))
