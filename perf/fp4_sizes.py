"""The tables of ``csrc/fp4_sizes.hpp`` from measured times: how many rows and
channels a workgroup of a product with 4-bit weights takes.

``profiles/sizes_fp4.json`` holds the microseconds of every size (null: not timed, far
from the fastest) in products [rows, channels, depth, experts], by type of the
activations, dense and by expert.  They are GPU times in captured graphs on MI355X, 256
compute units, three weights in turn, the launch that splits fp16 and fp32 activations
included where the size needs it.  The fit is that of ``tiles.py``.

    python perf/fp4_sizes.py

prints each table as the fit gives it, and how much longer than the fastest size the
chosen one took: the geometric mean and the worst.
"""

import json
import os

import tiles


def measured():
    with open(os.path.join(tiles.ROOT, "profiles", "sizes_fp4.json")) as f:
        return json.load(f)


def main():
    for name, data in measured().items():
        constants = tiles.fit(data)
        print(name)
        for size in data["tiles"]:
            print("    {%s}," % ", ".join(str(v) for v in [*tiles.size(size), *constants[size]]))
        ratios = tiles.excess(data, constants, data["tiles"])
        print("    %d products, chosen size timed in %d: %.1f %% on average, %.0f %% at worst" % (
            len(data["products"]), len(ratios), 100 * tiles.mean(ratios) - 100, 100 * max(ratios) - 100))


if __name__ == "__main__":
    main()
