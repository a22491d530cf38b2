"""Whole-prompt attention at the edges of its numbers."""

import math

import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq

from test_gpu_prompt import call, check, config, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    return kvq.load_library()


# ------------------------------------------------------------------ masses
@pytest.mark.parametrize("n", [130, 260, 300])
@pytest.mark.parametrize("g", [3, 5, 6, 7])
@pytest.mark.parametrize("d", [64, 128])
def test_masses_of_low_scores(d, g, n):
    # Every score is -128 (-185 in log2 units).  Query tiles straddle a key
    # tile's border here, and few rows: a stream may hold a key tile that some
    # rows of the query tile do not see at all.
    for t, window in ((32, 0), (64, 0), (128, 0), (64, 9)):
        cfg = config(1, g, d, t)
        q, k, v = rows(cfg, n, 31)
        q.fill_(1.0)
        k.fill_(-128.0 / d)
        check(cfg, q, k, v, [n], window=window, scale=1.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_nan_row_stays_out_of_the_tiles_it_does_not_see(d):
    # token 5 of the first sequence sees tile 0 (of 32 tokens); rows up to
    # token 63 are in the same query tile
    cfg = config(1, 2, d, t=32)
    lens = [100, 40]
    q, k, v = rows(cfg, 140, 32)
    want = call(cfg, q, k, v, lens, 0)[2]
    q[5, 1] = math.nan
    mass = call(cfg, q, k, v, lens, 0)[2]
    assert bool(torch.isnan(mass[0, 0]))
    # the tiles behind it: bit for bit, the row had no weight there
    assert torch.equal(mass[0, 1:], want[0, 1:]) and torch.equal(mass[1], want[1])
