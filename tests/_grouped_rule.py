"""Which tile the bf16 expert products take for given rows per expert: the rule of
csrc/grouped.hip in plain arithmetic, its tiles and costs read from that file."""
import os
import random
import re

from quantized_mixture_experts_moe_amd import build_lib

CUS = 256  # an MI355X


def _ceil(a, b):
    return -(-a // b)


class Tile:
    def __init__(self, name, bm, bn, wm, wn, stages, cost):
        self.name, self.bm, self.bn, self.cost = name, bm, bn, cost
        lds = stages * (bm + bn) * 128 + wm * wn * 4096 + 2 * bm * 4 + 1028 * 4
        self.per_cu = max(160 * 1024 // lds, 1)

    def tiles(self, counts, N, block_m=16):
        rows = [_ceil(c, block_m) * block_m for c in counts]
        return _ceil(N, self.bn) * sum(_ceil(r, self.bm) for r in rows)


def tiles():
    """{name: Tile} of the source, in its order."""
    with open(os.path.join(build_lib.CSRC, "grouped.hip")) as f:
        text = f.read()
    found = {}
    for name, args, cost in re.findall(
            r"struct (\w+) : Tile<([\d, ]+)> \{\s*static constexpr int ROUND = (\d+);", text):
        found[name] = Tile(name, *map(int, args.split(",")), int(cost))
    for args, name in re.findall(r"typedef Tile<([\d, ]+)> (Half|Low);", text):
        found[name] = Tile(name, *map(int, args.split(",")), None)
    order = re.search(r"launch_tile<TRANS, ACT, F32, (Big[\w, ]+)>", text).group(1).split(", ")
    return {n: found[n] for n in order + ["Half", "Low"]}, order


def choice(counts, N, trans, cus=CUS):
    """(name of the kernel's tile, its tiles, blocks that run at once)."""
    shape, wide = tiles()
    P, E = sum(counts), len(counts)
    mean = P / E
    if not trans and mean <= 8:
        return "rows", 0, 0

    def of(t, slots):
        return t.name, t.tiles(counts, N), slots
    if mean <= 20:
        return of(shape["Low"], cus * shape["Low"].per_cu)
    mid = shape["Mid"]
    one = _ceil(P, mid.bm) if E == 1 else max(mean / mid.bm + 0.5, 1.0)
    if mean <= 44 or one * E * _ceil(N, mid.bn) < cus // 2:
        return of(shape["Half"], cus * shape["Half"].per_cu)
    slots = cus * shape[wide[0]].per_cu

    def rounds(t):
        return _ceil(_ceil(t.tiles(counts, N), 8), slots // 8) * t.cost
    best = min((shape[n] for n in wide), key=rounds)  # (the first of the cheapest)
    return of(best, slots)


def _uneven(E, rows, seed):
    """Rows per expert around `rows`, one expert without any, their sum even."""
    r = random.Random(seed)
    counts = [max(1, round(rows * r.uniform(0.7, 1.3))) for _ in range(E)]
    counts[E // 3] = 0
    counts[-1] += sum(counts) % 2
    return counts


# Tile that is taken, rows per expert, columns: more tiles than blocks that run at once, so
# that blocks take a second one (and a third), with ragged last rows and columns.
ROUNDS = [("Low", _uneven(64, 11, 1), 8208), ("Half", _uneven(32, 36, 2), 8208),
          ("Mid", _uneven(64, 78, 3), 1552), ("Wide", _uneven(32, 140, 4), 3088),
          ("Big", _uneven(64, 200, 5), 1552), ("Broad", _uneven(33, 140, 6), 8208)]
