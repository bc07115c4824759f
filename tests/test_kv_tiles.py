"""Attention over caches in which no tile of tokens can be missing, or counted
twice, without showing (tests/kv_tiles.py): whole units, shares and their joins,
tokens that are split, a wave for each request, windows, and tables with room for
more than the requests have.  The first tests, without a GPU, are of that claim."""

import sys

import numpy as np
import pytest

from tests.kv_tiles import Tiled, old_bound_sees
from tests.test_gpu_kv_attention import Setup

CASES = [  # lens, new, q heads, kv heads, dim, page, quant, window, sinks, room
    # a workgroup for a unit
    ([1, 31, 33, 300, 64], [1] * 5, 8, 2, 128, 32, "nf4", 0, 0, 0), ([900, 17], [1, 1], 4, 1, 256, 16, "fp4", 0, 0, 0),
    ([1000, 40], [1, 1], 6, 2, 64, 64, "fp4", 0, 0, 0), ([11 + 7 * i % 90 for i in range(600)], [1] * 600, 2, 1, 256, 16, "nf4", 0, 0, 0),
    ([700, 90], [9, 5], 4, 2, 128, 16, "nf4", 0, 0, 0),
    # shares, cut and joined: few units, units of several blocks of rows, more than 64 units
    ([20011], [1], 8, 2, 128, 64, "nf4", 0, 0, 0), ([12345, 1], [1, 1], 4, 4, 64, 32, "nf4", 0, 0, 0),
    ([2049, 0, 7000], [1, 1, 1], 6, 1, 256, 128, "fp4", 0, 0, 0), ([9000, 350, 4097], [1, 1, 1], 16, 2, 128, 16, "fp4", 0, 0, 0),
    ([9000, 65], [8, 3], 8, 2, 128, 32, "nf4", 0, 0, 0), ([7000], [30], 4, 2, 64, 16, "nf4", 0, 0, 0),
    ([3000] + [37 * i % 2500 for i in range(90)], [1] * 91, 4, 1, 128, 32, "nf4", 0, 0, 0),
    ([5000] + [91 * i % 3000 for i in range(70)], [1] * 71, 2, 2, 256, 64, "nf4", 0, 0, 0),
    # blocks of many rows, whole and with split tokens
    ([700, 300], [150, 97], 256, 256, 64, 16, "nf4", 0, 0, 0), ([900, 33], [130, 33], 256, 256, 128, 32, "fp4", 0, 0, 0),
    ([20000], [97], 2, 2, 128, 64, "nf4", 0, 0, 0), ([9000, 700], [100, 9], 16, 8, 64, 256, "fp4", 0, 0, 0),
    ([6000], [110], 64, 64, 256, 32, "nf4", 0, 0, 0),
    # a wave for a unit
    ([1, 0, 15, 16, 17, 33, 64, 300, 511, 512, 700, 768], [1] * 12, 256, 256, 64, 16, "nf4", 0, 0, 0),
    ([64, 2, 300, 31, 65, 40, 700, 90, 5, 250], [16, 2, 9, 0, 1, 16, 5, 8, 1, 3], 256, 256, 128, 32, "fp4", 0, 0, 0),
    ([64, 3, 300, 31, 65, 40, 700, 90, 5], [3, 1, 3, 2, 1, 3, 2, 1, 1], 1600, 200, 128, 64, "nf4", 0, 0, 0),
    ([300, 2, 65, 31, 32, 40, 700, 90, 5], [1, 1, 2, 0, 1, 1, 2, 1, 1], 160, 160, 256, 16, "fp4", 0, 0, 0),
    # windows and first tokens
    ([9000, 5000, 20], [1, 1, 1], 8, 2, 128, 64, "nf4", 4096, 100, 0), ([3000, 777], [1, 1], 4, 4, 64, 16, "fp4", 1000, 16, 0),
    ([6000], [100], 60, 60, 128, 32, "nf4", 2048, 64, 0), ([9000, 7000], [100, 64], 60, 30, 128, 64, "fp4", 3000, 33, 0),
    # a table with room for more
    ([301], [1], 32, 8, 128, 32, "nf4", 0, 0, 4096), ([301, 20, 5000], [1, 1, 1], 8, 2, 64, 16, "nf4", 0, 0, 100000),
    ([200] * 12, [1] * 12, 256, 256, 64, 16, "fp4", 0, 0, 4096), ([700, 40], [12, 12], 32, 4, 128, 32, "nf4", 0, 0, 65536),
]
IDS = ["%s-%d-%s-%d" % ("+".join(map(str, c[0][:3])), sum(c[1]), c[4], c[7]) for c in CASES]


def heads_of(case):
    return range(case[3]) if case[3] <= 2 else (0, case[3] - 1)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_a_missing_or_doubled_tile_shows(case):
    s = Tiled(None, *case[:7], window=case[7], sinks=case[8], room=case[9], seed=len(case[0]))
    for i in range(len(s.lens)):
        if s.lens[i] and s.new[i]:
            for h in heads_of(case):
                assert s.shows(i, h) > 1, (i, h)


def test_random_entries_do_not_show_them():
    """Why these caches are made as they are: with random entries most tiles of a
    long one are too light for the bound there."""
    random = Setup(None, [12345], [1], 4, 4, 64, 32, "nf4", seed=6)
    hits, of = old_bound_sees(random, 0, 0)
    assert hits < of // 2
    tiled = Tiled(None, [1500], [1], 4, 4, 64, 32, "nf4", seed=6)
    assert tiled.shows(0, 0) > 1


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_every_tile_counts_once(case, request):
    import torch

    from bit_nf4_quantized_04_amd import nf4kv as K

    print("\n[gpu] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    s = Tiled(K, *case[:7], window=case[7], sinks=case[8], room=case[9], seed=len(case[0])).device()
    out = s.run(window=case[7], sinks=case[8])
    s.check_tiles(out, heads_of(case))
    if case[9]:  # the same result whatever the call expects
        exact = s.run(window=case[7], sinks=case[8], max_len=int(np.max(case[0])))
        s.check_tiles(exact, heads_of(case))
    torch.cuda.synchronize()
    assert torch.equal(out, s.run(window=case[7], sinks=case[8]))
