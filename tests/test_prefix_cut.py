"""How the prefix's tiles are cut over the blocks of a call (CPU; prefix_plan)."""
import random

import pytest

from prefix_plan import Plan


@pytest.fixture(scope="module")
def library():
    from head_sparse_decode_b200 import build
    return build.build_test_hooks()


@pytest.mark.parametrize("G", [1, 3, 8, 16])
def test_every_tile_once_with_a_slot_of_its_own(library, G):
    rng = random.Random(G)
    for _ in range(400):
        heads = rng.choice([1, 2, 8, 72, 200, 1000])
        most = rng.choice([1, 5, 40, 300])
        counts = [rng.randint(0, most) if rng.random() < 0.8 else 0 for _ in range(heads)]
        prefix = rng.choice([1, 128, 129, 300, 768, 2000, 4096, 20000])
        Plan(library, counts, G, prefix, 128, share=rng.randint(1, 147)).check()


def test_no_units_use_no_blocks(library):
    p = Plan(library, [0, 0, 0], 4, 500, 64, share=20)
    assert p.used == 0 and p.runs == []


def test_whole_row_tiles_count_only_the_blocks_that_have_some(library):
    """54 row tiles of more than 128 rows on up to 101 blocks: whole ones, on 54 of them."""
    p = Plan(library, [200] * 54, 1, 768, 128, share=101)
    p.check()
    assert p.used == 54 and {run[4] for run in p.runs} == {6}
    # two each, the last block one
    p = Plan(library, [200] * 7, 1, 128, 128, share=5)
    p.check()
    assert p.used == 4
