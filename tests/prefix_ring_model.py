"""The pipeline of a shared-prefix block as a model: its warps as they wait, arrive and issue, run
in random orders.

Barriers count arrivals and complete phases as the hardware's do: an arrival counts for the phase
that is current when it comes, whoever sends it, and a wait names only a phase's parity, so that
one that has gone by twice looks like one not yet begun.  Copies land and products execute at any
time after they were issued, products of one stream in order.  Every product checks that its
buffer holds the tile it is meant to read, and every copy that nobody reads its buffer any more.

The tables of steps and ring positions are the library's own (its build with test hooks); the
order of waits and arrivals in each warp is that of sha_prefix_kernel.
"""
import ctypes


class Broken(Exception):
    """A tile was read in the wrong place, or overwritten before it was read."""


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


class Tables:
    def __init__(self, library):
        self.lib = ctypes.CDLL(library)

    def steps(self, pair, tiles, rows, st):
        """([(tile, half, last of the tile)], whether the stream has a step in the last tile)."""
        out = (ctypes.c_int * (3 * 2 * tiles + 1))()
        n = self.lib.sha_test_prefix_steps(int(pair), tiles, rows, st, out)
        return [(out[3 * i], out[3 * i + 1], bool(out[3 * i + 2])) for i in range(n)], bool(out[3 * n])

    def ring(self, i, n):
        out = (ctypes.c_int * 2)()
        self.lib.sha_test_prefix_ring(i, n, out)
        return out[0], out[1]


class Block:
    """One block over `runs`: (tiles, keys in the last tile, whether its row tile is a pair's)."""

    def __init__(self, tables, runs, bufs, release="behind products"):
        # how a stream gives up a tile without a step of its own: "behind products", once the
        # tile has arrived; "once arrived" alone; or "at once"
        self.t, self.runs, self.bufs, self.release = tables, runs, bufs, release
        self.full = [Barrier(1) for _ in range(bufs)]
        self.empty = [Barrier(2) for _ in range(bufs)]
        self.q_full, self.q_seen = Barrier(2), Barrier(2)
        self.s_full, self.s_free, self.p_full, self.pv_done = (
            [Barrier(1), Barrier(1)] for _ in range(4))
        self.holds = [None] * bufs              # ring position in each buffer
        self.landing = {}                       # copies on their way: position -> buffer
        self.readers = {}                       # reads still to come of each ring position
        self.queue = [[], []]                   # products and commits issued, by stream
        self.at_barrier = [0, 0]                # softmax: runs begun
        base = 0
        for tiles, rows, pair in runs:
            for st in range(2):
                for tile, _, _ in tables.steps(pair, tiles, rows, st)[0]:
                    k, v = tables.ring(tile, tiles)
                    for pos in (base + k, base + v):
                        self.readers[pos] = self.readers.get(pos, 0) + 1
            base += 2 * tiles

    # Each warp yields a condition to wait for (None: it may just go on).
    def loader(self, is_k):
        base = 0
        for tiles, _, _ in self.runs:
            for i in range(tiles):
                pos = base + self.t.ring(i, tiles)[0 if is_k else 1]
                buf, phase = pos % self.bufs, pos // self.bufs
                yield lambda b=buf, p=phase: self.empty[b].passed((p & 1) ^ 1)
                if phase and self.readers[pos - self.bufs]:
                    raise Broken(f"position {pos} overwrites {pos - self.bufs} before it was read")
                if buf in self.landing.values():
                    raise Broken(f"two copies into buffer {buf}")
                self.holds[buf] = None
                self.landing[pos] = buf
                yield None
            base += 2 * tiles

    def products(self, st):
        base, q_parity, s_parity, p_parity = 0, 0, 0, 0
        for tiles, rows, pair in self.runs:
            yield lambda p=q_parity: self.q_full.passed(p)
            q_parity ^= 1
            self.q_seen.arrive()
            steps, takes_last = self.t.steps(pair, tiles, rows, st)

            def scores(step):
                tile, _, last = steps[step]
                pos = base + self.t.ring(tile, tiles)[0]
                yield lambda: self.full[pos % self.bufs].passed((pos // self.bufs) & 1)
                self.queue[st] += [("read", pos), ("arrive", self.s_full[st])]
                if last:
                    self.queue[st].append(("arrive", self.empty[pos % self.bufs]))

            if steps:
                yield from scores(0)
            for step in range(len(steps)):
                if step + 1 < len(steps):
                    yield lambda p=s_parity: self.s_free[st].passed(p)
                    yield from scores(step + 1)
                s_parity ^= 1
                tile, _, last = steps[step]
                pos = base + self.t.ring(tile, tiles)[1]
                yield lambda: self.full[pos % self.bufs].passed((pos // self.bufs) & 1)
                yield lambda p=p_parity: self.p_full[st].passed(p)
                p_parity ^= 1
                self.queue[st] += [("read", pos), ("arrive", self.pv_done[st])]
                if last:
                    self.queue[st].append(("arrive", self.empty[pos % self.bufs]))
            if not takes_last:
                for pos in (base + x for x in self.t.ring(tiles - 1, tiles)):
                    if self.release != "at once":
                        yield lambda: self.full[pos % self.bufs].passed((pos // self.bufs) & 1)
                    if self.release == "behind products":
                        self.queue[st].append(("arrive", self.empty[pos % self.bufs]))
                    else:
                        self.empty[pos % self.bufs].arrive()
                    yield None
            base += 2 * tiles

    def softmax(self, st):
        base, s_parity, pv_parity = 0, 0, 0
        for r, (tiles, rows, pair) in enumerate(self.runs):
            self.at_barrier[st] += 1
            yield lambda n=r + 1: self.at_barrier[st ^ 1] >= n
            if r > 0:
                yield lambda p=(r - 1) & 1: self.q_seen.passed(p)
            self.q_full.arrive()
            steps, _ = self.t.steps(pair, tiles, rows, st)
            for step, (tile, half, _) in enumerate(steps):
                yield lambda p=s_parity: self.s_full[st].passed(p)
                s_parity ^= 1
                self.s_free[st].arrive()
                left = (rows if tile == tiles - 1 else 128) - 64 * half
                if left < 64:                   # zeroes V past the keys: it has to be there
                    pos = base + self.t.ring(tile, tiles)[1]
                    yield lambda: self.full[pos % self.bufs].passed((pos // self.bufs) & 1)
                    if self.holds[pos % self.bufs] != pos:
                        raise Broken(f"V at {pos} is zeroed elsewhere")
                if step > 0:
                    yield lambda p=pv_parity: self.pv_done[st].passed(p)
                    pv_parity ^= 1
                self.p_full[st].arrive()
            if steps:
                yield lambda p=pv_parity: self.pv_done[st].passed(p)
                pv_parity ^= 1
            base += 2 * tiles

    def land(self, rng):
        pos = rng.choice(list(self.landing))
        self.holds[self.landing[pos]] = pos
        self.full[self.landing.pop(pos)].arrive()

    def execute(self, st):
        what, x = self.queue[st].pop(0)
        if what == "arrive":
            x.arrive()
            return
        if self.holds[x % self.bufs] != x:
            raise Broken(f"stream {st} reads position {x}, its buffer holds "
                         f"{self.holds[x % self.bufs]}")
        self.readers[x] -= 1

    def run(self, rng):
        """To the end, in an order drawn from rng: the agents' paces differ by up to 1000."""
        agents = [self.loader(True), self.loader(False), self.products(0), self.products(1),
                  self.softmax(0), self.softmax(1)]
        wants = [next(a, StopIteration) for a in agents]
        pace = [10.0 ** rng.uniform(-3, 0) for _ in range(len(agents) + 3)]
        while True:
            ready = [i for i, w in enumerate(wants)
                     if w is not StopIteration and (w is None or w())]
            if self.landing:
                ready.append(len(agents))
            ready += [len(agents) + 1 + st for st in range(2) if self.queue[st]]
            if not ready:
                break
            i = rng.choices(ready, [pace[r] for r in ready])[0]
            if i < len(agents):
                wants[i] = next(agents[i], StopIteration)
            elif i == len(agents):
                self.land(rng)
            else:
                self.execute(i - len(agents) - 1)
        if any(w is not StopIteration for w in wants) or any(self.readers.values()):
            raise Broken("stands still")
