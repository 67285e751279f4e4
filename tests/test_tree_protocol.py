"""Barrier protocols of the tcgen05 tree-attention kernels (tree_context_sm100.cu; Rows and Split: the two forms of
tree_rows_sm100.cu), on randomised schedules (CPU only).

Roles: a loading warp (segments through a ring of four, then K0, K1, V0, K2, V1, ... through a ring of tiles), a thread
that issues the products (S of the next tile before PV of this one), and softmax groups that share S, P^T and O by
columns.  Same model and checks as the training kernels': no wait outside the one-phase window that a parity wait can
tell apart, every buffer holds what its reader expects, every role finishes; and a wait left out is caught.
"""

import pytest

from test_kernel_protocols import Bar, Core, Hazard

RING = 4


class Tree(Core):
    def __init__(self, segs, seed, stages=5, bufs=2, groups=2, drop=None):
        names = ([f"full{i}" for i in range(stages)] + [f"empty{i}" for i in range(stages)] +
                 ["q_full", "s_full", "s_free", "p_ready0", "p_ready1", "p_free0", "p_free1", "o_done"] +
                 [f"seg_full{i}" for i in range(RING)] + [f"seg_empty{i}" for i in range(RING)])
        super().__init__(seed, names)
        for n in ("q_full", "s_free", "p_ready0", "p_ready1"):
            self.B[n] = Bar(groups)
        for i in range(RING):
            self.B[f"seg_empty{i}"] = Bar(groups + 1)
        self.segs, self.stages, self.bufs, self.groups, self.drop = segs, stages, bufs, groups, drop
        self.ring = [None] * stages
        self.info = [None] * RING
        self.Q = [None] * groups
        self.S, self.S_unread = None, 0
        self.P = [[None] * groups for _ in range(bufs)]
        self.PV = -1                      # the last tile whose second product has executed
        self.O, self.O_unread = None, 0
        self.has_rows = [self.rng.random() < 0.8 or g == 0 for g in range(groups)]

    def w(self, bar, n, name):
        if self.drop != name and n >= 0:
            yield from self.wait(bar, n)

    # ---------------------------------------------------------------- the loading warp
    def loader(self):
        c = 0
        for s in range(len(self.segs) + 1):
            yield from self.w(f"seg_empty{s % RING}", s // RING - 1, "seg_empty")
            self.info[s % RING] = s
            self.B[f"seg_full{s % RING}"].arrive()
            if s == len(self.segs):
                return
            n = self.segs[s]
            order = [("K", 0)]
            for j in range(n):
                order += ([("K", j + 1)] if j + 1 < n else []) + [("V", j)]
            for kind, j in order:
                slot = c % self.stages
                yield from self.w(f"empty{slot}", c // self.stages - 1, "empty")
                self.load(f"full{slot}", lambda a=(slot, (kind, s, j)): self.land(*a))
                c += 1
                yield

    def land(self, slot, x):
        self.check(self.ring[slot] is None, f"{x} lands on {self.ring[slot]}")
        self.ring[slot] = x

    # ---------------------------------------------------------------- the products
    def products(self):
        c, t = 0, 0

        def scores(s, j, t, slot):
            self.check(self.ring[slot] == ("K", s, j), "K")
            self.check(all(q == s for q in self.Q), "Q")
            self.check(self.S_unread == 0, "S overwritten before it was read")
            self.ring[slot] = None
            self.S, self.S_unread = t, self.groups

        def second(s, j, t, slot):
            self.check(self.ring[slot] == ("V", s, j), "V")
            self.check(all(p == t for p, r in zip(self.P[t % self.bufs], self.has_rows) if r), "P")
            self.check(self.O == (s, j - 1) if j else self.O_unread == 0, "O")
            self.ring[slot] = None
            self.PV = t
            self.O, self.O_unread = (s, j), self.groups

        def issue_s(s, j, t):
            nonlocal c
            yield from self.w("s_free", t - 1, "s_free")
            yield from self.w(f"full{c % self.stages}", c // self.stages, "K full")
            self.mma(lambda a=(s, j, t, c % self.stages): scores(*a))
            self.commit(f"empty{c % self.stages}")
            self.commit("s_full")
            c += 1

        for s in range(len(self.segs) + 1):
            yield from self.w(f"seg_full{s % RING}", s // RING, "seg_full")
            self.check(self.info[s % RING] == s, "segment")
            if s == len(self.segs):
                return
            self.B[f"seg_empty{s % RING}"].arrive()
            yield from self.w("q_full", s, "q_full")
            yield from issue_s(s, 0, t)
            for j in range(self.segs[s]):
                if j + 1 < self.segs[s]:
                    yield from issue_s(s, j + 1, t + 1)
                yield from self.w(f"p_ready{t % 2}", t // 2, "p_ready")
                yield from self.w(f"full{c % self.stages}", c // self.stages, "V full")
                self.mma(lambda a=(s, j, t, c % self.stages): second(*a))
                self.commit(f"empty{c % self.stages}")
                self.commit(f"p_free{t % 2}")
                self.commit("o_done")
                c, t = c + 1, t + 1
                yield

    # ---------------------------------------------------------------- a softmax group
    def done(self, i):
        if self.drop == "one barrier":
            yield from self.wait("o_done", i)
        else:
            yield from self.w(f"p_free{i % 2}", i // 2, "p_free")

    def group(self, g):
        def open_(s):
            yield from self.w(f"seg_full{s % RING}", s // RING, "seg_full")
            self.check(self.info[s % RING] == s, "segment")

        t, ring0 = 0, 0
        yield from open_(0)
        self.Q[g] = 0
        self.B["q_full"].arrive()
        for s, n in enumerate(self.segs):
            for j in range(n):
                yield from self.w("s_full", t, "s_full")
                self.check(self.S == t, "S")
                if j + 1 == n:
                    yield from open_(s + 1)
                    if self.drop != "early Q":
                        self.Q[g] = s + 1
                elif self.drop == "early Q" and j + 2 == n:
                    self.Q[g] = s + 1
                if j and self.has_rows[g] and self.rng.random() < 0.3:     # a reference moves: O is rescaled
                    yield from self.done(t - 1)
                    self.check(self.O == (s, j - 1), "O rescaled")
                yield
                self.S_unread -= 1
                self.B["s_free"].arrive()
                if t >= self.bufs:
                    yield from self.done(t - self.bufs)
                    self.check(self.PV >= t - self.bufs, "P rewritten before it was read")
                self.P[t % self.bufs][g] = t
                yield
                if g == 0 and self.rng.random() < 0.4:                     # V rows are zeroed
                    i = ring0 + (2 * j + 2 if j + 1 < n else 2 * j + 1)
                    yield from self.w(f"full{i % self.stages}", i // self.stages, "V zeroed")
                    self.check(self.ring[i % self.stages] == ("V", s, j), "V zeroed")
                self.B[f"p_ready{t % 2}"].arrive()
                t += 1
            ring0 += 2 * n
            if s + 1 < len(self.segs):
                self.B["q_full"].arrive()
            yield from self.done(t - 1)
            self.check(self.O == (s, n - 1), "O read")
            self.O_unread -= 1
            self.B[f"seg_empty{s % RING}"].arrive()
            yield

    def go(self):
        roles = {"loader": self.loader(), "products": self.products()}
        roles.update({f"group{g}": self.group(g) for g in range(self.groups)})
        self.run(roles)


SEGS = [[1], [2, 1], [1, 1, 1, 1, 1, 1, 1], [7], [3, 1, 4, 1, 5], [9, 2, 6]]


@pytest.mark.parametrize("stages,bufs,groups", [(5, 2, 2), (3, 1, 4), (5, 1, 2), (8, 2, 1), (4, 2, 4)])
def test_tree_protocol(stages, bufs, groups):
    for seed in range(60):
        Tree(SEGS[seed % len(SEGS)], seed, stages, bufs, groups).go()


# (waits that another one implies are not listed: full before the zeroing of V and before the products order different
# things, but K's arrival is only ever seen by the products)
@pytest.mark.parametrize("drop", ["seg_empty", "empty", "s_free", "K full", "V full", "p_ready", "s_full", "p_free", "q_full",
                                  "one barrier", "early Q", "V zeroed"])
def test_a_missing_wait_is_caught(drop):
    for seed in range(400):
        try:
            Tree(SEGS[seed % len(SEGS)], seed, 8 if drop == "seg_empty" else 5, 2, 2, drop).go()
        except Hazard:
            return
    pytest.fail(f"no schedule shows the hazard that {drop} guards")


class Rows(Core):
    """tree_rows_sm100.cu: one or two row tiles a segment (nx), each with a softmax group of its own; K0, V0, K1, ..."""

    def __init__(self, segs, seed, stages=5, drop=None):
        names = ([f"full{i}" for i in range(stages)] + [f"empty{i}" for i in range(stages)] + ["q_full"] +
                 [f"{n}{x}" for n in ("s_full", "p_ready", "o_full") for x in range(2)] +
                 [f"seg_full{i}" for i in range(RING)] + [f"seg_empty{i}" for i in range(RING)])
        super().__init__(seed, names)
        self.B["q_full"] = Bar(2)
        for i in range(RING):
            self.B[f"seg_empty{i}"] = Bar(3)
        self.segs, self.stages, self.drop = segs, stages, drop     # segs: (tiles, nx)
        self.ring, self.info = [None] * stages, [None] * RING
        self.Q, self.S, self.O, self.unread = [None] * 2, [None] * 2, [None] * 2, [False] * 2

    w, land = Tree.w, Tree.land

    def loader(self):
        c = 0
        for s in range(len(self.segs) + 1):
            yield from self.w(f"seg_empty{s % RING}", s // RING - 1, "seg_empty")
            self.info[s % RING] = s
            self.B[f"seg_full{s % RING}"].arrive()
            if s == len(self.segs):
                return
            for j in range(self.segs[s][0]):
                for kind in "KV":
                    slot = c % self.stages
                    yield from self.w(f"empty{slot}", c // self.stages - 1, "empty")
                    self.load(f"full{slot}", lambda a=(slot, (kind, s, j)): self.land(*a))
                    c += 1
                    yield

    def products(self):
        c, np = 0, [0, 0]

        def scores(x, s, j, slot, last):
            self.check(self.ring[slot] == ("K", s, j) and self.Q[x] == s, "K or Q")
            self.check(self.S[x] is None, "S overwritten")
            self.S[x] = ("S", s, j)
            if last:
                self.ring[slot] = None

        def second(x, s, j, slot, last):
            self.check(self.ring[slot] == ("V", s, j), "V")
            self.check(self.S[x] == ("P", s, j), "P")
            self.check(self.O[x] == (s, j - 1) if j else not self.unread[x], "O")
            self.S[x], self.O[x], self.unread[x] = None, (s, j), True
            if last:
                self.ring[slot] = None

        for s in range(len(self.segs) + 1):
            yield from self.w(f"seg_full{s % RING}", s // RING, "seg_full")
            self.check(self.info[s % RING] == s, "segment")
            if s == len(self.segs):
                return
            tiles, nx = self.segs[s]
            self.B[f"seg_empty{s % RING}"].arrive()
            yield from self.w("q_full", s, "q_full")
            full = lambda i, n: self.w(f"full{i % self.stages}", i // self.stages, n)  # noqa: E731
            yield from full(c, "K full")
            for x in range(nx):
                self.mma(lambda a=(x, s, 0, c % self.stages, x == nx - 1): scores(*a))
                self.commit(f"s_full{x}")
            self.commit(f"empty{c % self.stages}")
            for j in range(tiles):
                v, k = c + 2 * j + 1, c + 2 * j + 2
                for x in range(nx):
                    yield from self.w(f"p_ready{x}", np[x], "p_ready")
                    np[x] += 1
                    if x == 0:
                        yield from full(v, "V full")
                    self.mma(lambda a=(x, s, j, v % self.stages, x == nx - 1): second(*a))
                    if x == nx - 1:
                        self.commit(f"empty{v % self.stages}")
                    if j + 1 < tiles:
                        if x == 0:
                            yield from full(k, "K full")
                        self.mma(lambda a=(x, s, j + 1, k % self.stages, x == nx - 1): scores(*a))
                        self.commit(f"s_full{x}")
                        if x == nx - 1:
                            self.commit(f"empty{k % self.stages}")
                    else:
                        self.commit(f"o_full{x}")
                yield
            c += 2 * tiles

    def group(self, x):
        def open_(s):
            yield from self.w(f"seg_full{s % RING}", s // RING, "seg_full")
            self.check(self.info[s % RING] == s, "segment")

        ns, no, ring0 = 0, 0, 0
        yield from open_(0)
        self.Q[x] = 0
        self.B["q_full"].arrive()
        for s, (tiles, nx) in enumerate(self.segs):
            more = s + 1 < len(self.segs)
            if x >= nx:
                yield from open_(s + 1)
                yield from self.w("o_full0", s, "skip")
                if more:
                    self.Q[x] = s + 1
                    self.B["q_full"].arrive()
            else:
                for j in range(tiles):
                    yield from self.w(f"s_full{x}", ns, "s_full")
                    ns += 1
                    self.check(self.S[x] == ("S", s, j), "S")
                    if j + 1 == tiles:
                        yield from open_(s + 1)
                        self.Q[x] = s + 1
                    if j:
                        self.check(self.O[x] == (s, j - 1), "O rescaled")
                    yield
                    if x == 0 and self.rng.random() < 0.4:
                        i = ring0 + 2 * j + 1
                        yield from self.w(f"full{i % self.stages}", i // self.stages, "V zeroed")
                        self.check(self.ring[i % self.stages] == ("V", s, j), "V zeroed")
                    self.S[x] = ("P", s, j)
                    self.B[f"p_ready{x}"].arrive()
                if more:
                    self.B["q_full"].arrive()
                yield from self.w(f"o_full{x}", no, "o_full")
                no += 1
                self.check(self.O[x] == (s, tiles - 1), "O read")
                self.unread[x] = False
            ring0 += 2 * tiles
            self.B[f"seg_empty{s % RING}"].arrive()
            yield

    def go(self):
        self.run({"loader": self.loader(), "products": self.products(), "group0": self.group(0), "group1": self.group(1)})


class Split(Core):
    """tree_rows_sm100.cu with one row tile: two softmax groups take key tiles in turn, each with scores and an O of its
    own; both join the Os when the segment ends.  K0, K1, V0, K2, V1, ..."""

    def __init__(self, segs, seed, stages=6, drop=None):
        names = ([f"full{i}" for i in range(stages)] + [f"empty{i}" for i in range(stages)] + ["q_full", "joined", "left"] +
                 [f"{n}{x}" for n in ("s_full", "p_ready", "o_full") for x in range(2)] +
                 [f"seg_full{i}" for i in range(RING)] + [f"seg_empty{i}" for i in range(RING)])
        super().__init__(seed, names)
        self.B["joined"] = Bar(2)      # the groups' named barrier, its two uses a segment
        self.B["left"] = Bar(2)
        for i in range(RING):
            self.B[f"seg_empty{i}"] = Bar(3)
        self.segs, self.stages, self.drop = segs, stages, drop     # segs: tiles
        self.ring, self.info = [None] * stages, [None] * RING
        self.Q, self.S, self.O, self.readers = None, [None] * 2, [None] * 2, [0, 0]

    w, land, loader = Tree.w, Tree.land, Tree.loader

    def products(self):
        c, np = 0, [0, 0]

        def scores(x, s, j, slot):
            self.check(self.ring[slot] == ("K", s, j) and self.Q == s, "K or Q")
            self.check(self.S[x] is None, "S overwritten")
            self.S[x], self.ring[slot] = ("S", s, j), None

        def second(x, s, j, slot):
            self.check(self.ring[slot] == ("V", s, j), "V")
            self.check(self.S[x] == ("P", s, j), "P")
            self.check(self.O[x] == (s, j - 2) if j > 1 else not self.readers[x], "O")
            self.S[x], self.O[x], self.readers[x], self.ring[slot] = None, (s, j), 2, None

        def next_(f, x, s, j, name):
            slot = c % self.stages
            yield from self.w(f"full{slot}", c // self.stages, name)
            self.mma(lambda: f(x, s, j, slot))

        for s in range(len(self.segs) + 1):
            yield from self.w(f"seg_full{s % RING}", s // RING, "seg_full")
            self.check(self.info[s % RING] == s, "segment")
            if s == len(self.segs):
                return
            tiles = self.segs[s]
            self.B[f"seg_empty{s % RING}"].arrive()
            yield from self.w("q_full", s, "q_full")
            for j in range(min(tiles, 2)):
                yield from next_(scores, j, s, j, "K full")
                self.commit(f"s_full{j}")
                self.commit(f"empty{c % self.stages}")
                c += 1
            for j in range(tiles):
                x = j % 2
                yield from self.w(f"p_ready{x}", np[x], "p_ready")
                np[x] += 1
                yield from next_(second, x, s, j, "V full")
                self.commit(f"empty{c % self.stages}")
                c += 1
                if j + 2 < tiles:
                    yield from next_(scores, x, s, j + 2, "K full")
                    self.commit(f"s_full{x}")
                    self.commit(f"empty{c % self.stages}")
                    c += 1
                else:
                    self.commit(f"o_full{x}")
                yield

    def group(self, x):
        def open_(s):
            yield from self.w(f"seg_full{s % RING}", s // RING, "seg_full")
            self.check(self.info[s % RING] == s, "segment")

        ns, no, ring0 = 0, 0, 0
        yield from open_(0)
        if x == 0:
            self.Q = 0
            self.B["q_full"].arrive()
        for s, tiles in enumerate(self.segs):
            more, mine = s + 1 < len(self.segs), (tiles - 1) % 2 == x or self.drop == "early Q"
            for j in range(x, tiles, 2):
                yield from self.w(f"s_full{x}", ns, "s_full")
                ns += 1
                self.check(self.S[x] == ("S", s, j), "S")
                if j + 1 == tiles or (self.drop == "early Q" and j + 2 == tiles):
                    yield from open_(s + 1)
                    self.Q = s + 1
                if j > 1:
                    self.check(self.O[x] == (s, j - 2), "O rescaled")
                yield
                if self.rng.random() < 0.4:
                    i = ring0 + 2 * j + (2 if j + 1 < tiles else 1)
                    yield from self.w(f"full{i % self.stages}", i // self.stages, "V zeroed")
                    self.check(self.ring[i % self.stages] == ("V", s, j), "V zeroed")
                self.S[x] = ("P", s, j)
                self.B[f"p_ready{x}"].arrive()
            if (tiles - 1) % 2 != x:
                yield from open_(s + 1)
            elif more:
                self.B["q_full"].arrive()
            if x < tiles:
                yield from self.w(f"o_full{x}", no, "o_full")
                no += 1
            self.B["joined"].arrive()
            yield from self.w("joined", s, "joined")
            for y in range(min(tiles, 2)):
                self.check(self.O[y] == (s, tiles - 1 - (tiles - 1 - y) % 2), "O read")
                yield
                self.readers[y] -= 1
            ring0 += 2 * tiles
            self.B[f"seg_empty{s % RING}"].arrive()
            self.B["left"].arrive()
            yield from self.w("left", s, "left")

    def go(self):
        self.run({"loader": self.loader(), "products": self.products(), "group0": self.group(0), "group1": self.group(1)})


SPLIT_SEGS = [[1], [2, 1], [1, 1, 1, 1, 2, 1], [7], [3, 1, 4, 1, 5], [1] * 6 + [2] * 3, [6, 5]]


@pytest.mark.parametrize("stages", [5, 6, 8])
def test_split_protocol(stages):
    for seed in range(80):
        Split(SPLIT_SEGS[seed % len(SPLIT_SEGS)], seed, stages).go()


@pytest.mark.parametrize("drop", ["seg_empty", "empty", "K full", "V full", "p_ready", "s_full", "q_full", "o_full", "joined",
                                  "left", "early Q", "V zeroed"])
def test_a_missing_wait_of_the_split_form_is_caught(drop):
    for seed in range(400):
        try:
            Split(SPLIT_SEGS[seed % len(SPLIT_SEGS)], seed, 8 if drop == "seg_empty" else 5, drop).go()
        except Hazard:
            return
    pytest.fail(f"no schedule shows the hazard that {drop} guards")


ROW_SEGS = [[(1, 2)], [(2, 1), (1, 2)], [(1, 1), (1, 2), (1, 1), (1, 1), (2, 2), (1, 2)], [(7, 2)],
            [(3, 2), (1, 1), (4, 2), (1, 2), (5, 1)], [(1, 1)] * 6 + [(2, 2)] * 3]


@pytest.mark.parametrize("stages", [4, 5, 8])
def test_rows_protocol(stages):
    for seed in range(80):
        Rows(ROW_SEGS[seed % len(ROW_SEGS)], seed, stages).go()


@pytest.mark.parametrize("drop", ["seg_empty", "empty", "K full", "V full", "p_ready", "s_full", "q_full", "o_full", "skip",
                                  "V zeroed"])
def test_a_missing_wait_of_the_rows_kernel_is_caught(drop):
    for seed in range(400):
        try:
            Rows(ROW_SEGS[seed % len(ROW_SEGS)], seed, 8 if drop == "seg_empty" else 5, drop).go()
        except Hazard:
            return
    pytest.fail(f"no schedule shows the hazard that {drop} guards")
