"""The tables of ``csrc/fp4_sizes.hpp`` from measured times: how many rows, channels and
waves a workgroup of a product with 4-bit weights has.

``profiles/sizes_fp4.json`` holds the microseconds of every size, "rows x channels
waves" (null: not timed, far from the fastest or beyond the limit in ``taken``) in
products [rows, channels, depth, experts], by type of the activations, dense and by
expert.  They are GPU times in captured graphs on MI355X, 256 compute units, three
weights in turn, the launch that splits fp32 activations included where the size needs
it.  The kernels have changed since (the sizes' header says how), and no program here
takes the times: the library has no way to ask for a size.

    python perf/fp4_sizes.py

prints each table as the fit gives it, and how much longer than the fastest size the
chosen one took: the geometric mean and the worst.
"""

import json
import math
import os

import numpy as np
from scipy.optimize import nnls

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256
SLOTS = (1, 2, 3, 4, 5, 6, 8)


def measured():
    with open(os.path.join(ROOT, "profiles", "sizes_fp4.json")) as f:
        return json.load(f)


def numbers(size):
    """(rows, channels, waves)."""
    tile, waves = size.split()
    return (*(int(v) for v in tile.split("x")), int(waves[:-1]))


def terms(size, slots, rows, channels, depth, experts):
    """What the constants of a size are multiplied with: its expected time is their sum."""
    tall, wide, _ = numbers(size)
    tiles = -(-rows // tall)
    if experts:
        used = experts * (1.0 - math.exp(-rows / experts))
        tiles = max(used, rows / tall + 0.5 * used)
    average = tiles * -(-channels // wide) / CUS
    most, k = math.ceil(average / slots), depth / 1024.0
    return [1.0, most, most * k, average, average * k]


def fit(data):
    """Of every size how many workgroups share a compute unit, as the times say, and the
    constants, rounded to two places: least squares of relative errors, weighted by
    sqrt(fastest / time), without times over twice the fastest, none negative."""
    result = {}
    for i, size in enumerate(data["sizes"]):
        best = None
        for slots in SLOTS:
            a, b = [], []
            for *product, times in data["products"]:
                fastest = min(t for t in times if t)
                if times[i] is None or times[i] > 2 * fastest:
                    continue
                weight = math.sqrt(fastest / times[i])
                a.append([weight * v / times[i] for v in terms(size, slots, *product)])
                b.append(weight)
            constants, left = nnls(np.array(a), np.array(b))
            if best is None or left < best[0] - 1e-9:
                best = left, slots, [round(float(v), 2) for v in constants]
        result[size] = best[1:]
    return result


def taken(size, rows, experts):
    """Sizes of few rows read a weight again for each of their row tiles: up to 12, a limit
    set by hand, beyond which they were hardly timed."""
    tall, wide, _ = numbers(size)
    return wide >= 64 or rows / max(experts, 1) <= 12 * tall


def choice(fitted, sizes, rows, channels, depth, experts):
    def expected(size):
        slots, constants = fitted[size]
        return sum(c * v for c, v in zip(constants, terms(size, slots, rows, channels, depth, experts)))
    return min((s for s in sizes if taken(s, rows, experts)), key=expected)


def excess(data, fitted):
    """Chosen size's time over the fastest size's, where it was timed."""
    ratios = []
    for *product, times in data["products"]:
        t = times[data["sizes"].index(choice(fitted, data["sizes"], *product))]
        if t is not None:
            ratios.append(t / min(v for v in times if v))
    return ratios


def mean(ratios):
    return math.exp(sum(map(math.log, ratios)) / len(ratios))


def main():
    for name, data in measured().items():
        fitted = fit(data)
        print(name)
        for size, (slots, constants) in fitted.items():
            print("    {%s}," % ", ".join(str(v) for v in [*numbers(size), slots, *constants]))
        ratios = excess(data, fitted)
        print("    %d products, chosen size timed in %d: %.1f %% on average, %.0f %% at worst" % (
            len(data["products"]), len(ratios), 100 * mean(ratios) - 100, 100 * max(ratios) - 100))


if __name__ == "__main__":
    main()
