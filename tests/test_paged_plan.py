"""How single-token attention cuts sequences into items (fa_decode.cuh), run on the host: what the workspace and the
grid are sized by holds for every batch, the largest that the interface takes among them."""
import os
import subprocess

import numpy as np
import pytest

from flash_attention_backward_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
MAX_TILES, MIN_TILES = 1 << 26, 4  # 2^30 positions of 16 keys a tile


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "-I", B.INCLUDE, os.path.join(HERE, "plan_host.cu"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", stdout=subprocess.PIPE, text=True, check=True).stdout
        return [[int(x) for x in row.split()] for row in out.strip().split("\n")]
    return run


def check(R, tiles, row):
    """tiles: (tiles of a sequence, sequences)"""
    n = sum(t for _, t in tiles)
    for chunk, items, slots, split in (row[:4], row[4:]):
        assert MIN_TILES <= chunk <= MAX_TILES, (R, tiles, row)
        live = sum(t for x, t in tiles if x > 0)
        assert live <= items <= R + n and 0 <= split <= min(R, n) and 0 <= slots <= 2 * R, (R, tiles, row)


def test_items_stay_within_the_workspace(plan):
    rng = np.random.default_rng(5)
    cases = []
    for _ in range(3000):
        R = int(np.exp(rng.uniform(0, np.log(608))))
        n = int(np.exp(rng.uniform(0, np.log(400))))
        top = np.exp(rng.uniform(0, np.log(MAX_TILES)))
        tiles = [int(x) for x in np.minimum(np.exp(rng.uniform(-1, np.log(top + 1), n)), MAX_TILES)]
        cases.append((R, [(x, 1) for x in tiles]))
    for (R, tiles), row in zip(cases, plan(["%d %s" % (R, " ".join(str(x) for x, _ in t)) for R, t in cases])):
        check(R, tiles, row)


def test_items_of_the_largest_batches(plan):
    """2^20 sequences of 2^30 positions, few items at a time (many heads): counts of tiles beyond 31 and 45 bits."""
    cases = [(R, [(x, t)]) for R in (1, 2, 3, 76, 608) for x in (1, 5, 4096, MAX_TILES - 1, MAX_TILES) for t in (1, 31, 32, 33, 64, 1 << 12, 1 << 20)]
    cases += [(R, [(MAX_TILES, 40), (0, 100), (7, 1000), (123456, 77)]) for R in (1, 2, 608)]
    for (R, tiles), row in zip(cases, plan(["%d %s" % (R, " ".join("%dx%d" % t for t in ts)) for R, ts in cases])):
        check(R, tiles, row)
