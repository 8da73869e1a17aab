"""The tables of ``csrc/int8_tiles.hpp`` from measured times: which tile an 8-bit
product takes.

``profiles/tiles_int8.json`` holds the microseconds of every tile (null: not timed)
in products [rows, channels, depth, experts]: dense, by expert, and dense with rows
that do not start on 16 bytes.  They are GPU times in captured graphs on MI355X, 256
compute units, codes at random, bf16 results, three or more weights in turn.

    python perf/tiles.py

prints each table as the fit gives it, and how much longer than the fastest tile the
chosen one took: the geometric mean and the worst.
"""

import json
import math
import os

import numpy as np
from scipy.optimize import nnls

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256
# The tiles that the kernels have, of those that were timed.
TABLES = {
    "dense": ["16x16", "32x32", "64x64", "64x128", "64x192", "128x128", "128x192", "192x128", "128x256",
              "192x192", "256x256"],
    "by_expert": ["16x16", "32x64", "32x128", "64x64", "64x128", "64x192", "128x128", "128x192", "192x192",
                  "256x256"],
    "unaligned": ["16x16", "32x32", "64x64", "128x128", "128x256"]}


def measured():
    with open(os.path.join(ROOT, "profiles", "tiles_int8.json")) as f:
        return json.load(f)


def size(tile):
    rows, channels = tile.split()[0].split("x")
    return int(rows), int(channels)


def terms(tile, rows, channels, depth, experts, cus=CUS):
    """What the constants of a tile are multiplied with: its expected time is their sum."""
    tall, wide = size(tile)
    tiles = -(-rows // tall)
    if experts:
        used = experts * (1.0 - math.exp(-rows / experts))
        tiles = max(used, rows / tall + 0.5 * used)
    average = tiles * -(-channels // wide) / cus
    most, k = math.ceil(average), depth / 1024.0
    return [1.0, most, most * k, average, average * k]


def fit(data):
    """The constants of every tile, rounded to two places."""
    constants = {}
    for i, tile in enumerate(data["tiles"]):
        a, b = [], []
        for *product, times in data["products"]:
            fastest = min(t for t in times if t)
            if times[i] is None or times[i] > 2 * fastest:
                continue
            weight = math.sqrt(fastest / times[i])
            a.append([weight * v / times[i] for v in terms(tile, *product)])
            b.append(weight)
        constants[tile] = [round(float(v), 2) for v in nnls(np.array(a), np.array(b))[0]]
    return constants


def choice(constants, tiles, *product):
    return min(tiles, key=lambda t: sum(c * v for c, v in zip(constants[t], terms(t, *product))))


def excess(data, constants, tiles):
    """Chosen tile's time over the fastest tile's, where it was timed."""
    ratios = []
    for *product, times in data["products"]:
        t = times[data["tiles"].index(choice(constants, tiles, *product))]
        if t is not None:
            ratios.append(t / min(v for v in times if v))
    return ratios


def mean(ratios):
    return math.exp(sum(map(math.log, ratios)) / len(ratios))


def main():
    for name, tiles in TABLES.items():
        data = measured()[name]
        constants = fit(data)
        print(name)
        for tile in tiles:
            print("    {%s}," % ", ".join(str(v) for v in [*size(tile), *constants[tile]]))
        ratios = excess(data, constants, tiles)
        print("    %d products, chosen tile timed in %d: %.2f %% on average, %.0f %% at worst" % (
            len(data["products"]), len(ratios), 100 * mean(ratios) - 100, 100 * max(ratios) - 100))


if __name__ == "__main__":
    main()
