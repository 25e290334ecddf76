"""The barriers of query attention's kernel as a simulation: its warps as coroutines that a random
scheduler steps, copies and products as events that land some time after they are issued.

It holds who waits for what and who arrives how often, as the kernel does, and checks that
  - no phase of a barrier gets more arrivals than it counts;
  - no wait by parity passes before its phase, or finds itself two phases behind;
  - everything read (a tile, Q, what is present of a block, scores, exponentials, O, a piece) is
    what its reader expects, whatever may already write there;
  - everything ends.
An AssertionError names what does not hold."""
from __future__ import annotations

import random
from dataclasses import dataclass


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.phase, self.bytes = name, count, count, 0, 0

    def arrive(self, times=1, expect=0):
        assert self.pending >= times, f"{self.name}: {times} arrivals where {self.pending} are due"
        self.bytes += expect
        self.pending -= times
        self.turn()

    def landed(self, count):
        self.bytes -= count
        self.turn()

    def turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count


@dataclass
class Sizes:
    """tiles of rows, halves of a block, and the kernel's constants"""
    tiles: int
    parts: int
    stages: int
    info: int
    turns: int
    ring: int


@dataclass
class Piece:
    blocks: int
    two: bool          # both tiles of rows
    cut: list          # for each block, whether a box of its V comes row by row
    counted: bool      # a whole unit from the counter


class Kernel:
    """mode: 'boxes' (TMA), 'rows' (cp.async, made visible by a warp of its own) or 'registers'
    (e4m3).  without: names of waits that are left out, for a test of this simulation."""

    def __init__(self, seed, sizes, mode, pieces, without=()):
        self.r, self.z, self.mode, self.pieces, self.without = random.Random(seed), sizes, mode, pieces, set(without)
        z, relayed = sizes, mode == "rows"
        self.soft_warps = 4 * z.tiles
        self.q_boxes = self.r.random() < 0.6
        self.bars = {}

        def bars(name, n, count):
            for i in range(n):
                self.bars[name, i] = Barrier(f"{name}[{i}]", count)
        bars("full", z.stages, 128)
        bars("empty", z.stages, 1)
        bars("ready", z.stages, 1)
        bars("known", z.info, 4)
        bars("q", 2, 1 if self.q_boxes else 4)
        bars("scores", 2, 1)
        bars("exps", 4, 4)
        bars("pv", 4, 1)
        bars("last", 1, 1)
        bars("group", 1, 4)
        bars("other", 1, 4)
        bars("added", 1, 4)
        bars("piece", z.ring, 1)
        bars("taken", z.ring, self.soft_warps + 5 + relayed)
        self.pipe, self.later = [], []            # products, in order; copies, in any
        self.tile = [[None, None] for _ in range(z.stages)]       # by box, row by row
        self.q = [[None] * 4 for _ in range(2)]                   # of each warp's rows
        self.sums = [None] * 4                                    # in the place of the second tile's Q
        self.there, self.offs = [None] * z.info, [[None] * 4 for _ in range(2)]
        self.s, self.p, self.o = [None] * 2, [[None] * 4 for _ in range(2)], [None] * 2
        self.ring = [None] * z.ring
        self.reads = {}

    # ---- what every role uses
    def wait(self, name, i, nth):
        """Until phase nth (from 0) of the barrier has ended, as far as its parity shows."""
        b = self.bars[name, i]
        if name in self.without:
            return
        while (b.phase & 1) == (nth & 1):
            yield
        assert b.phase > nth, f"{b.name}: a wait for phase {nth} passes in phase {b.phase}"

    def arrive(self, name, i=0, times=1, expect=0):
        self.bars[name, i].arrive(times, expect)

    def take(self, role):
        """The next piece's number, or None."""
        n = self.reads.get(role, 0)
        slot = n % self.z.ring
        yield from self.wait("piece", slot, n // self.z.ring)
        yield
        assert self.ring[slot] == n, f"{role} finds piece {self.ring[slot]} in place of {n}"
        self.reads[role] = n + 1
        self.arrive("taken", slot)
        return n if n < len(self.pieces) else None

    # ---- roles
    def planner(self):
        z = self.z
        for i in range(len(self.pieces) + 1):
            counted = i < len(self.pieces) and self.pieces[i].counted or i == len(self.pieces) and self.pieces[-1].counted
            for ahead in (z.ring, 1) if counted else (z.ring,):
                if i >= ahead:
                    j = i - ahead
                    yield from self.wait("taken", j % z.ring, j // z.ring)
            self.ring[i % z.ring] = i
            yield
            self.arrive("piece", i % z.ring)

    def copier(self, w):
        z, blk, turns = self.z, 0, 0

        def together():
            nonlocal turns
            yield
            self.arrive("group")
            yield from self.wait("group", 0, turns)
            turns += 1

        def empty(t):
            if t >= z.stages:
                yield from self.wait("empty", t % z.stages, t // z.stages - 1)

        def known(p, x):
            self.there[blk % z.info] = (p, x)
            yield

        def offsets(x):
            self.offs[blk & 1][w] = x
            yield

        def use_offsets(b, x):
            assert self.offs[b & 1] == [x] * 4, f"places {self.offs[b & 1]} in place of {x}"

        while True:
            n = yield from self.take(("copy", w))
            if n is None:
                break
            p = self.pieces[n]
            if self.mode == "boxes":
                for x in range(p.blocks):
                    if blk % z.turns == w:
                        yield from known(n, x)
                        self.arrive("known", blk % z.info, 4)
                        for kv in range(2):
                            t = 2 * blk + kv
                            yield from empty(t)
                            st, cut = t % z.stages, kv == 1 and p.cut[x]
                            self.arrive("full", st, 1, expect=100)
                            yield
                            if not cut:
                                self.arrive("full", st, 127)

                            def land(st=st, v=(n, x, kv), cut=cut):
                                self.tile[st][0] = v
                                if not cut:
                                    self.tile[st][1] = v
                                self.bars["full", st].landed(100)
                            self.later.append(land)
                            if cut:
                                yield
                                self.tile[st][1] = (n, x, kv)
                                yield
                                self.arrive("full", st, 127)
                    blk += 1
                    yield
            elif self.mode == "rows":
                for x in range(p.blocks):
                    yield from offsets((n, x))
                    if w == 0:
                        yield from known(n, x)
                    self.arrive("known", blk % z.info)
                    yield from together()
                    for kv in range(2):
                        t = 2 * blk + kv
                        yield from empty(t)
                        use_offsets(blk, (n, x))

                        def land(st=t % z.stages, v=(n, x, kv)):
                            self.tile[st] = [v, v]
                            self.arrive("full", st, 32)
                        self.later.append(land)
                        yield
                    blk += 1
            else:
                def place(b, x, kv):
                    t = 2 * b + kv
                    yield from empty(t)
                    self.tile[t % z.stages] = [(n, x, kv)] * 2
                    yield
                    self.arrive("full", t % z.stages, 32)
                for x in range(p.blocks + 1):
                    if x < p.blocks:
                        yield from offsets((n, x))
                        if w == 0:
                            yield from known(n, x)
                        self.arrive("known", blk % z.info)
                        yield from together()
                        use_offsets(blk, (n, x))
                    if x > 0:
                        yield from place(blk - 1, x - 1, 1)
                    if x == p.blocks:
                        break
                    yield
                    use_offsets(blk, (n, x))
                    yield from place(blk, x, 0)
                    blk += 1

    def relay(self):
        t = 0
        while True:
            n = yield from self.take("relay")
            if n is None:
                return
            for _ in range(2 * self.pieces[n].blocks):
                yield from self.wait("full", t % self.z.stages, t // self.z.stages)
                yield
                self.arrive("ready", t % self.z.stages)
                t += 1

    def products(self):
        z, landed = self.z, "ready" if self.mode == "rows" else "full"
        used, blk, twos, count = [0, 0], 0, 0, 0
        while True:
            n = yield from self.take("products")
            if n is None:
                break
            p = self.pieces[n]
            steps = p.blocks * (2 if p.two else 1)
            block = lambda s: s >> 1 if p.two else s  # noqa: E731

            def have(t):
                yield from self.wait(landed, t % z.stages, t // z.stages)

            def product(x, b, t, n=n, p=p):
                def run():
                    assert self.tile[t % z.stages] == [(n, b, 0)] * 2, f"K: {self.tile[t % z.stages]} in place of {(n, b)}"
                    rows = x if p.two else 0
                    assert self.q[rows] == [n] * 4, f"Q of {self.q[rows]} in place of {n}"
                    self.s[x] = (n, b)
                self.pipe.append(run)
                self.pipe.append(lambda: self.arrive("scores", x))
                if not p.two or x == 1:
                    self.pipe.append(lambda: self.arrive("empty", t % z.stages))

            def product_v(x, s, b, t, n=n, p=p):
                for part in range(z.parts):
                    yield from self.wait("exps", 2 * part + x, used[x] + (s >> 1))

                    def run(part=part):
                        assert self.tile[t % z.stages] == [(n, b, 1)] * 2, f"V: {self.tile[t % z.stages]} in place of {(n, b)}"
                        mine = self.p[x]
                        assert all(m is not None and m[:2] == (n, b) and m[2] >= part for m in mine), f"P: {mine}, {(n, b, part)}"
                        self.o[x if z.tiles == 2 else 0] = (n, b, part)
                    self.pipe.append(run)
                    self.pipe.append(lambda part=part: self.arrive("pv", 2 * part + x))
                if not p.two or x == 1:
                    self.pipe.append(lambda: self.arrive("empty", t % z.stages))

            for s in range(-2, steps):
                x, more = s & 1, s + 2 < steps
                if s == -2:
                    yield from self.wait("q", 0, count)
                    count += 1
                if s == -1 and p.two:
                    yield from self.wait("q", 1, twos)
                    twos += 1
                k, v = 2 * (blk + block(s + 2)), 2 * (blk + block(s)) + 1
                if not p.two or x == 0:
                    if s >= 0:
                        yield from have(v)
                    if p.two and more:
                        yield from have(k)
                if s >= 0:
                    yield from product_v(x, s, block(s), v)
                if more:
                    if not p.two:
                        yield from have(k)
                    product(x, block(s + 2), k)
                yield
            used[0] += (steps + 1) >> 1
            used[1] += steps >> 1
            blk += p.blocks
        self.pipe.append(lambda: self.arrive("last"))
        yield from self.wait("last", 0, 0)

    def softmax(self, tile, w):
        z, r = self.z, self.r
        used, blk, shares, n, now = [0, 0], 0, 0, None, None
        while True:
            blocks, two = (now.blocks, now.two) if now else (0, False)
            shared = z.tiles == 2 and not two
            j0, each = (tile, 2) if shared else (0, 1)
            way = lambda j: tile if z.tiles == 2 else j & 1  # noqa: E731
            nth = lambda j: used[0] + (j >> 1 if shared else j) if z.tiles == 2 else used[j & 1] + (j >> 1)  # noqa: E731
            o = tile if z.tiles == 2 else 0
            for j in range(j0, blocks, each):
                i, x = blk + j, way(j)
                yield from self.wait("known", i % z.info, i // z.info)
                assert self.there[i % z.info] == (n, j), f"present: {self.there[i % z.info]} in place of {(n, j)}"
                yield from self.wait("scores", x, nth(j))
                yield
                assert self.s[x] == (n, j), f"scores of {self.s[x]} in place of {(n, j)}"
                assert self.there[i % z.info] == (n, j), "present: overwritten"
                for part in range(z.parts):
                    if (j > j0 or part > 0) and r.random() < 0.3:      # a reference moves, O with it
                        last, half = (j, 0) if part > 0 else (j - each, z.parts - 1)
                        yield from self.wait("pv", 2 * half + way(last), nth(last))
                        assert self.o[o] == (n, last, half), f"O of {self.o[o]} in place of {(n, last, half)}"
                    yield
                    self.p[x][w] = (n, j, part)
                    yield
                    self.arrive("exps", 2 * part + x)
            mine = len(range(j0, blocks, each))
            j1 = j0 + (mine - 1) * each
            last, last_nth = way(j1), nth(j1)
            used[0] += mine if z.tiles == 2 else (blocks + 1) >> 1
            used[1] += blocks if two else blocks >> 1
            blk += blocks
            was, early, following = n, not (shared and tile == 1), None

            def begin():
                if shared and blocks > 1 and blocks % 2 == 0 and tile == 0:
                    yield from self.wait("scores", 1, used[1] - 1)
                m = yield from self.take(("softmax", tile, w))
                if m is None or not (tile == 0 or self.pieces[m].two):
                    return m
                if self.q_boxes:
                    if w == 0:
                        def land():
                            self.q[tile] = [m] * 4
                            if tile == 1:
                                self.sums = [None] * 4
                            self.bars["q", tile].landed(100)
                        self.arrive("q", tile, expect=100)
                        self.later.append(land)
                else:
                    self.q[tile][w] = m
                    if tile == 1:
                        self.sums[w] = None
                    yield
                    self.arrive("q", tile)
                return m

            if early:
                following = yield from begin()
            if mine:
                yield from self.wait("pv", 2 * (z.parts - 1) + last, last_nth)
                assert self.o[o] == (was, j1, z.parts - 1), f"O of {self.o[o]} in place of {(was, j1)}"
            if shared and blocks:
                if tile == 1:
                    yield
                    self.sums[w] = was
                    self.q[1][w] = None
                    self.arrive("other")
                    yield from self.wait("added", 0, shares)
                else:
                    yield from self.wait("other", 0, shares)
                    yield
                    assert self.sums[w] == was, f"sums of {self.sums[w]} in place of {was}"
                shares += 1
            if not early:
                following = yield from begin()
            if blocks and tile == 0 or blocks and two:
                yield                             # the epilogue reads O
                assert self.o[o][0] == was, f"O of {self.o[o]} in place of {was}"
                if shared:
                    if blocks > 1:
                        assert self.o[1][0] == was, f"the other set's O is of {self.o[1]} in place of {was}"
                    self.arrive("added")
            if following is None:
                return
            n, now = following, self.pieces[following]

    def run(self):
        z, r = self.z, self.r
        roles = [self.copier(w) for w in range(4)] + [self.planner(), self.products()]
        roles += [self.relay()] if self.mode == "rows" else []
        roles += [self.softmax(t, w) for t in range(z.tiles) for w in range(4)]
        # each role at a pace of its own, copies and products too
        pace = [r.choice((0.03, 0.3, 1.0)) for _ in roles]
        pipe, later = (r.choice((0.03, 0.3, 1.0)) for _ in range(2))
        alive, steps = list(range(len(roles))), 0
        while alive or self.pipe or self.later:
            steps += 1
            assert steps < 1_000_000, f"stuck: {alive}"
            if self.pipe and r.random() < pipe:
                self.pipe.pop(0)()
            if self.later and r.random() < later:
                self.later.pop(r.randrange(len(self.later)))()
            if alive:
                i = r.choice(alive)
                if r.random() < pace[i]:
                    try:
                        next(roles[i])
                    except StopIteration:
                        alive.remove(i)


def pieces_of(seed, tiles):
    """Some pieces: in chunks, as whole units, or (a prefix call) first the one, then the other."""
    r = random.Random(seed)
    n = r.randint(1, 9)
    first = r.choice((0, n, r.randint(0, n)))
    res = []
    for i in range(n):
        blocks = r.choice((1, 1, 2, 3, 4, 7, 12, 20))
        res.append(Piece(blocks, tiles == 2 and r.random() < 0.5, [r.random() < 0.3 for _ in range(blocks)], i >= first))
    return res
