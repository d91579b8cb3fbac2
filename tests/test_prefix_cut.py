"""How the prefix's tiles are cut over the blocks of a call (CPU; prefix_plan)."""
import random

import pytest

from prefix_plan import SEVERAL_ROW_TILES, Plan
from prefix_reference import Case


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


@pytest.mark.parametrize("args", SEVERAL_ROW_TILES, ids=str)
def test_calls_whose_blocks_take_several_row_tiles(library, args):
    """The calls that the GPU tests make for these blocks do reach them."""
    p = Plan.of(library, Case(*args, seed=args[5]))
    p.check()
    per = p.runs_of_block()
    assert max(per) >= 2 and sum(n >= 2 for n in per) >= p.used // 2
    if p.wide and p.wide < p.row_tiles:          # a paired row tile and another in one block
        kinds = {}
        for block, row_tile, head, _, _, _ in p.runs:
            kinds.setdefault(block, set()).add(row_tile + 1 < p.start[head + 1])
        assert args[4] < args[2] or any(len(k) == 2 for k in kinds.values())
