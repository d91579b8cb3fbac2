"""The ring of key tiles in a shared-prefix block, by its model (CPU; prefix_ring_model)."""
import random

import pytest

from prefix_ring_model import Block, Broken, Tables


@pytest.fixture(scope="module")
def tables():
    from head_sparse_decode_b200 import build
    return Tables(build.build_test_hooks())


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("tiles", [1, 2, 3, 7])
def test_steps_cover_the_keys(tables, tiles, pair):
    """Each stream's steps, for every raggedness of the last tile: a pair's streams take every
    half tile that holds keys, others one each; a tile is given up once by each stream."""
    for rows in (1, 63, 64, 65, 127, 128):
        halves = [(t, h) for t in range(tiles) for h in range(2)
                  if t < tiles - 1 or h == 0 or rows > 64]
        taken = []
        for st in range(2):
            steps, takes_last = tables.steps(pair, tiles, rows, st)
            assert [t for t, _, _ in steps] == sorted(t for t, _, _ in steps)
            given_up = [t for t, _, last in steps if last]
            assert given_up == list(range(tiles if takes_last else tiles - 1))
            taken.append([(t, h) for t, h, _ in steps])
        if pair:
            assert taken == [halves, halves]
        else:
            assert sorted(taken[0] + taken[1]) == halves and len(taken[0]) >= len(taken[1])


@pytest.mark.parametrize("tiles", [1, 2, 5])
def test_ring_positions_are_a_permutation(tables, tiles):
    at = [x for i in range(tiles) for x in tables.ring(i, tiles)]
    assert sorted(at) == list(range(2 * tiles))


# runs of a block: (key tiles, keys of the last one, paired)
RUNS = [
    [(3, 10, False)], [(5, 64, False)], [(16, 10, False)], [(7, 128, False)], [(9, 1, True)],
    [(1, 5, False), (1, 5, False), (1, 70, False), (1, 5, True)],
    [(2, 60, False), (4, 64, False), (3, 30, True), (6, 33, False), (1, 2, False)],
    [(6, 100, True), (6, 100, False), (5, 50, False), (5, 50, True), (2, 128, False)],
]


@pytest.mark.parametrize("bufs", [4, 8])
@pytest.mark.parametrize("runs", RUNS, ids=str)
def test_tiles_are_read_before_they_are_overwritten(tables, runs, bufs):
    rng = random.Random(bufs)
    for _ in range(150):
        Block(tables, runs, bufs).run(rng)


@pytest.mark.parametrize("bufs", [4, 8])
def test_random_runs(tables, bufs):
    rng = random.Random(100 + bufs)
    for _ in range(400):
        runs = [(rng.choice([1, 1, 2, 3, 4, 7]), rng.choice([1, 64, 65, 128]), rng.random() < 0.5)
                for _ in range(rng.randint(1, 6))]
        Block(tables, runs, bufs).run(rng)


@pytest.mark.parametrize("bufs,tiles", [(4, 3), (4, 16), (8, 5), (8, 12)])
def test_a_tile_given_up_before_it_arrived_lets_another_be_overwritten(tables, bufs, tiles):
    """Why a stream without a step in the last tile waits for it: without the wait its release
    counts for the tile that the buffer still holds, and the model finds it overwritten unread."""
    rng = random.Random(7)
    with pytest.raises(Broken):
        for _ in range(3000):
            Block(tables, [(tiles, 10, False)], bufs, release="at once").run(rng)


def test_a_tile_given_up_before_the_last_product_lets_it_read_another(tables):
    """Why that release stands behind the stream's products: a load of the next row tile, two
    rounds of the ring on, takes the phase of the last product's V for one that has gone by."""
    rng = random.Random(8)
    with pytest.raises(Broken):
        for _ in range(3000):
            Block(tables, RUNS[6], 4, release="once arrived").run(rng)
