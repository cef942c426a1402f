"""Calls that take each path of decode, with the path that each is there for:
the kernel's shape, how runs are cut and how partial results are joined.
test_paged_cpu.py holds the choices to this list, test_gpu_paged.py the
results to the oracle."""
import numpy as np


class Path:
    """batch requests of lo to hi keys, `width` block-table entries in all.
    nh: groups of 8 query heads; hw: key/value heads per tile; cost: runs of
    equal cost (else of equal numbers of tiles); join: "none" (one launch),
    "unit" or "cut"; chunks of query heads."""

    def __init__(self, batch, lo, hi, heads, heads_kv, dim, kv, page, width, nh, hw, cost, join, chunks=1):
        self.batch, self.heads, self.heads_kv, self.dim, self.kv, self.page = batch, heads, heads_kv, dim, kv, page
        self.width, self.nh, self.hw, self.cost, self.join, self.chunks = width, nh, hw, cost, join, chunks
        lens = np.random.default_rng(batch + heads + dim).integers(lo, hi + 1, batch)
        lens[0], lens[-1] = hi, lo
        self.lens = [int(x) for x in lens]

    def __str__(self):
        return (f"{self.batch}x{max(self.lens)}-{self.heads}/{self.heads_kv}x{self.dim}-{self.kv}-nh{self.nh}-hw{self.hw}-"
                f"{'cost' if self.cost else 'count'}-{self.join}-{self.chunks}")


PATHS = [
    # ragged batches, runs cut by cost, units in cuts: one, two and four heads per tile
    Path(130, 0, 420, 6, 3, 128, "bf16", 16, 30, 1, 1, True, "cut"),
    Path(130, 0, 420, 12, 6, 128, "bf16", 16, 30, 1, 2, True, "cut"),
    Path(130, 0, 420, 16, 8, 128, "bf16", 16, 30, 1, 4, True, "cut"),
    Path(130, 0, 700, 6, 3, 128, "e4m3", 16, 50, 1, 1, True, "cut"),
    Path(130, 0, 700, 12, 6, 128, "e4m3", 16, 50, 1, 2, True, "cut"),
    Path(130, 0, 700, 16, 8, 128, "e4m3", 16, 50, 1, 4, True, "cut"),
    Path(160, 0, 500, 16, 16, 64, "bf16", 16, 40, 1, 4, True, "cut"),
    Path(160, 0, 900, 16, 16, 64, "e4m3", 16, 60, 1, 4, True, "cut"),
    Path(90, 0, 400, 4, 4, 256, "bf16", 16, 60, 1, 4, True, "cut"),
    Path(200, 0, 900, 8, 4, 256, "e4m3", 16, 80, 1, 4, True, "cut"),
    # the same with 9 to 16 query heads to a key/value head, and with more
    Path(130, 0, 420, 36, 4, 128, "bf16", 16, 60, 2, 2, True, "cut"),
    Path(130, 0, 700, 48, 4, 128, "e4m3", 16, 80, 2, 2, True, "cut"),
    Path(240, 0, 400, 48, 4, 64, "bf16", 16, 60, 2, 4, True, "cut"),
    Path(110, 0, 500, 48, 3, 128, "bf16", 16, 32, 2, 1, True, "cut"),
    Path(110, 0, 800, 60, 3, 64, "bf16", 16, 52, 3, 1, True, "cut"),
    Path(110, 0, 800, 60, 3, 128, "e4m3", 16, 52, 3, 1, True, "cut"),
    Path(110, 0, 800, 96, 3, 64, "bf16", 16, 52, 4, 1, True, "cut"),
    # runs of equal numbers of tiles, units in cuts
    Path(120, 0, 120, 16, 8, 128, "bf16", 16, 300, 1, 4, False, "cut"),
    Path(120, 0, 120, 12, 6, 128, "e4m3", 16, 100, 1, 2, False, "cut"),
    Path(200, 0, 130, 3, 3, 128, "bf16", 16, 10, 1, 1, False, "cut"),
    # few units: combine finds their runs from the lengths
    Path(40, 0, 2500, 8, 4, 128, "bf16", 16, 400, 1, 4, True, "unit"),
    Path(12, 1000, 5000, 8, 4, 128, "e4m3", 16, 4000, 1, 4, True, "unit"),
    Path(5, 0, 300, 8, 4, 128, "bf16", 16, 20, 1, 1, False, "unit"),
    # many units of one or two tiles: four heads per tile without and with combine
    Path(190, 1, 16, 16, 16, 64, "bf16", 16, 1, 1, 4, False, "none"),
    Path(190, 1, 32, 16, 16, 64, "bf16", 16, 2, 1, 4, False, "cut"),
    Path(190, 1, 20, 16, 16, 64, "e4m3", 16, 2, 1, 4, False, "none"),
    Path(190, 1, 64, 16, 16, 64, "e4m3", 16, 4, 1, 4, False, "cut"),
    Path(330, 1, 20, 18, 2, 128, "bf16", 16, 2, 2, 2, False, "none"),
    Path(330, 1, 20, 24, 6, 128, "e4m3", 16, 2, 1, 2, False, "none"),
    # one launch, a head per tile
    Path(30, 0, 64, 4, 2, 128, "bf16", 16, 4, 1, 1, False, "none"),
    # groups of hundreds of query heads
    Path(3, 5, 4000, 300, 1, 128, "bf16", 16, 250, 2, 1, True, "unit", 19),
    Path(3, 5, 900, 300, 1, 128, "e4m3", 16, 60, 3, 1, False, "unit", 13),
    Path(2, 5, 300, 1024, 1, 64, "bf16", 16, 20, 4, 1, False, "unit", 32),
    Path(2, 5, 300, 1024, 1, 64, "e4m3", 16, 20, 4, 1, False, "unit", 32),
    Path(2, 5, 200, 1000, 1, 256, "bf16", 16, 13, 2, 1, False, "cut", 63),
    Path(4, 5, 900, 600, 2, 256, "e4m3", 16, 57, 2, 1, True, "cut", 19),
]
