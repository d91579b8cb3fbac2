"""How a shared-prefix call is cut over its blocks: the library's own cut (its build with test
hooks), fed with the histogram of a selection."""
import ctypes

BLOCKS = 148            # one per SM of a B200


class Plan:
    """counts: units of each head; G query rows a unit; own: stages of 32 own keys of each unit."""

    def __init__(self, library, counts, G, prefix, d, own=(), share=None, blocks=BLOCKS):
        lib = ctypes.CDLL(library)
        lib.sha_test_prefix_share.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong] + \
            [ctypes.c_int] * 2
        per_tile = 256 // G
        self.tiles = -(-prefix // 128)
        start, pairs = [0], [0]
        for n in counts:
            row_tiles = -(-n // per_tile)
            last = n - (row_tiles - 1) * per_tile
            start.append(start[-1] + row_tiles)
            pairs.append(pairs[-1] + (row_tiles - 1 + (last * G > 128) if row_tiles else 0))
        self.row_tiles, self.wide, self.blocks = start[-1], pairs[-1], blocks
        if share is None:
            weights = sum(max(1, s) + 2 for s in own)
            share = lib.sha_test_prefix_share(self.row_tiles, self.wide, self.tiles, weights,
                                              d // 64, blocks)
        self.share = share
        heads = len(counts)
        out = (ctypes.c_int * (6 * (self.row_tiles * 2 + blocks * 2 + 8)))()
        used = ctypes.c_int()
        n = lib.sha_test_prefix_cut((ctypes.c_int * (heads + 1))(*start),
                                    (ctypes.c_int * (heads + 1))(*pairs), heads, self.tiles, share,
                                    blocks, ctypes.byref(used), out)
        self.used = used.value
        self.start = start
        # (block, row tile, head, first tile, tiles, blocks that share it or 0)
        self.runs = [tuple(out[6 * i:6 * i + 6]) for i in range(n)]

    @classmethod
    def of(cls, library, case):
        """That of a prefix_reference.Case."""
        counts = [int((case.idx == h).sum()) for h in range(case.H_kv)]
        box = min(case.page_size, 32)
        key0 = case.prefix // box * box
        own = [-(-(int(n) - key0) // 32) for n in case.lens for _ in range(case.idx.shape[1])]
        return cls(library, counts, case.G, case.prefix, case.d, own)

    def runs_of_block(self):
        per = [0] * self.blocks
        for run in self.runs:
            per[run[0]] += 1
        return per

    def check(self):
        taken, blocks_of, slots = set(), {}, set()
        for block, row_tile, head, first, n, sharers in self.runs:
            assert 0 <= block < self.used <= self.share
            assert self.start[head] <= row_tile < self.start[head + 1]
            assert n >= 1 and first >= 0 and first + n <= self.tiles
            for tile in range(first, first + n):
                assert (row_tile, tile) not in taken
                taken.add((row_tile, tile))
            blocks_of.setdefault(row_tile, []).append(block)
            slots.add(row_tile + block)
        assert len(taken) == self.row_tiles * self.tiles
        assert len(slots) == len(self.runs) and all(s < self.row_tiles + self.blocks for s in slots)
        for block, row_tile, head, first, n, sharers in self.runs:
            if first == 0:                       # the slots of a row tile follow one another
                assert blocks_of[row_tile] == list(range(block, block + sharers))
        # every block that counts as in use has work; the others take the rows' own keys
        assert self.used == len({run[0] for run in self.runs})


# Calls whose blocks take several row tiles each (their own keys, too many for the prefix to
# get a block for each row tile): arguments of prefix_reference.Case
SEVERAL_ROW_TILES = [
    (3, 300, 300, 64, 200, 300, 400, 32, "fp16"),        # narrow row tiles, some split
    (2, 260, 260, 128, 260, 330, 600, 16, "fp16"),
    (2, 160, 160, 128, 160, 1025, 300, 32, "fp16"),      # nine key tiles, the last of one key
    (2, 160, 160, 64, 160, 1070, 150, 8, "bf16"),
    (1, 1000, 1000, 128, 1000, 40, 60, 8, "fp16"),       # one key tile: whole row tiles
    (40, 800, 100, 64, 100, 300, 130, 16, "bf16"),       # wide row tiles between narrow ones
    (40, 800, 100, 128, 40, 340, 130, 32, "bf16"),
    (36, 400, 100, 64, 100, 100, 90, 8, "fp16"),
]
