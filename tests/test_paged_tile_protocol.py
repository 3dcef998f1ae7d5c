"""Model check of the paged tile kernel's synchronisation protocol (no GPU).

The model of tests/protocol_model.py, restated for csrc/sa_paged_tiles.cu: a
producer of tile entries, Q rows, key words and K stages, another of V stages;
per half one warp issuing, for each chunk and 64-key part, O += P V of the
chunk before and then S = Q K; four softmax warps per half that take S, may
correct O, write P over it and read O out at the tile's end.  The tensor pipe
runs MMAs in the order of their issue, so S may be issued over a P that an
earlier MMA still has to read: S and P change hands when an MMA completes, not
when it is issued.  A tile's first P, of all four warps, also says that they
have read the last tile's O out: the kernel's own wait for that is left out
here.  Half 1 may have no rows or, for SA, only some of a tile's chunks; a
tile's last chunk may have one part.
"""

from __future__ import annotations

from dataclasses import dataclass

import pytest

from protocol_model import Accumulator, Barrier, Buffer, ProtocolError, arrive, copy, mma, simulate, wait
from protocol_model import call as do


@dataclass
class Tile:
    chunks: int
    halves: tuple  # ((a, b), (a, b)): each half's chunks
    last_parts: int = 2

    def parts(self, c):
        return self.last_parts if c == self.chunks - 1 else 2


@dataclass
class Mutation:
    waits_k_free: bool = True
    waits_v_free: bool = True
    waits_q_free: bool = True
    waits_seg_free: bool = True
    key_slots: int = 8
    pv_waits_p: bool = True
    epilogue_waits_pv: bool = True
    pv_before_qk: bool = True


class Then:
    """What an MMA does when it completes."""

    def __init__(self, fn):
        self.arrive = fn


class Model:
    def __init__(self, tiles, ns, mut=None):
        self.tiles, self.ns, self.mut = tiles, ns, mut or Mutation()
        B = Barrier
        self.q_full, self.q_free = B("Qfull", 1), B("Qfree", 2)
        self.k_full, self.k_free = [B(f"Kfull{s}", 1) for s in range(ns)], [B(f"Kfree{s}", 2) for s in range(ns)]
        self.v_full, self.v_free = [B(f"Vfull{s}", 1) for s in range(ns)], [B(f"Vfree{s}", 2) for s in range(ns)]
        two = lambda name, count: [[B(f"{name}{h}.{u}", count) for u in range(2)] for h in range(2)]
        self.s_full, self.p_full, self.pv_done = two("Sfull", 1), two("Pfull", 4), two("PVdone", 1)
        self.seg_full, self.seg_free = [B(f"SegFull{i}", 1) for i in range(4)], [B(f"SegFree{i}", 10) for i in range(4)]
        self.q = Buffer("Q")
        self.k, self.v = [Buffer(f"K{s}") for s in range(ns)], [Buffer(f"V{s}") for s in range(ns)]
        self.keys = [Buffer(f"keys{i}") for i in range(self.mut.key_slots)]
        self.seg = [Buffer(f"seg{i}") for i in range(4)]
        self.sp = [[[Buffer(f"S/P{h}.{u}.{w}") for w in range(4)] for u in range(2)] for h in range(2)]
        self.o = [[Accumulator(f"O{h}.{w}") for w in range(4)] for h in range(2)]

    # ------------------------------------------------------------ roles
    def produce_k(self):
        n = 0
        for x, t in enumerate(self.tiles):
            if x > 3 and self.mut.waits_seg_free:
                z = (x >> 2) - 1
                yield wait(self.seg_free[x & 3], z & 1, z)
            yield do(lambda x=x: self.seg[x & 3].write("K producer", x))
            yield arrive(self.seg_full[x & 3])
            if x > 0 and self.mut.waits_q_free:
                yield wait(self.q_free, (x - 1) & 1, x - 1)
            yield copy([(self.q, x)], f"loadQ{x}", self.q_full, "arrive")
            for _ in range(t.chunks):
                st, z = n % self.ns, n // self.ns - 1
                yield do(lambda n=n: self.keys[n % self.mut.key_slots].write("K producer", n))
                if n >= self.ns and self.mut.waits_k_free:
                    yield wait(self.k_free[st], z & 1, z)
                yield copy([(self.k[st], n)], f"loadK{n}", self.k_full[st], "arrive")
                n += 1

    def produce_v(self):
        for n in range(sum(t.chunks for t in self.tiles)):
            st, z = n % self.ns, n // self.ns - 1
            if n >= self.ns and self.mut.waits_v_free:
                yield wait(self.v_free[st], z & 1, z)
            yield copy([(self.v[st], n)], f"loadV{n}", self.v_full[st], "arrive")

    def issue(self, h):
        who = f"mma{h}"
        n = 0
        taken = [0, 0]  # P of each part taken so far

        def pv(x, n, u, first):
            z = taken[u]
            taken[u] += 1
            if self.mut.pv_waits_p:
                yield wait(self.p_full[h][u], z & 1, z)

            def begin():
                for w in range(4):
                    self.o[h][w].begin_mma(f"{who} PV{n}.{u}", ("O", x), first)

            def done():
                for w in range(4):
                    self.sp[h][u][w].read(f"{who} PV{n}.{u}", ("P", n))
                    self.sp[h][u][w].write(f"{who} PV{n}.{u}", "taken")
                    self.o[h][w].end_mma()
            yield do(begin)
            yield mma([(self.v[n % self.ns], n)], [], f"{who} PV{n}.{u}", [Then(done), self.pv_done[h][u]])

        def qk(x, n, u):
            def done():
                for w in range(4):
                    b = self.sp[h][u][w]
                    if b.content not in (None, "taken"):
                        raise ProtocolError(f"{who}: S of chunk {n}.{u} over {b.content}")
                    b.write(f"{who} QK{n}.{u}", ("S", n))
            yield mma([(self.q, x), (self.k[n % self.ns], n)], [], f"{who} QK{n}.{u}", [Then(done), self.s_full[h][u]])

        for x, t in enumerate(self.tiles):
            a, b = t.halves[h]
            yield wait(self.seg_full[x & 3], (x >> 2) & 1, x >> 2)
            yield do(lambda x=x: self.seg[x & 3].read(who, x))
            yield arrive(self.seg_free[x & 3])
            yield wait(self.q_full, x & 1, x)
            for c in range(t.chunks):
                last = n - 1
                if c > 0:
                    yield wait(self.v_full[last % self.ns], (last // self.ns) & 1, last // self.ns)
                    yield do(lambda last=last: self.keys[last % self.mut.key_slots].read(who, last))
                yield wait(self.k_full[n % self.ns], (n // self.ns) & 1, n // self.ns)
                yield do(lambda n=n: self.keys[n % self.mut.key_slots].read(who, n))
                for u in range(2):
                    steps = []
                    if a < c <= b:
                        steps.append(pv(x, last, u, u == 0 and c - 1 == a))
                    if a <= c < b and u < t.parts(c):
                        steps.append(qk(x, n, u))
                    for s in steps if self.mut.pv_before_qk else steps[::-1]:
                        yield from s
                commits = [self.v_free[last % self.ns]] if c > 0 else []
                commits += [self.k_free[n % self.ns]] + ([self.q_free] if c == t.chunks - 1 else [])
                yield mma([], [], who, commits)
                n += 1
            last = n - 1
            yield wait(self.v_full[last % self.ns], (last // self.ns) & 1, last // self.ns)
            if b > a and b == t.chunks:
                for u in range(t.last_parts):
                    yield from pv(x, last, u, u == 0 and t.chunks - 1 == a)
            yield mma([], [], who, [self.v_free[last % self.ns]])

    def softmax(self, h, w):
        who = f"softmax{h}.{w}"
        k, nbase = [0, 0], 0
        ob = self.o[h][w]
        for x, t in enumerate(self.tiles):
            a, b = t.halves[h]
            yield wait(self.seg_full[x & 3], (x >> 2) & 1, x >> 2)
            yield do(lambda x=x: self.seg[x & 3].read(who, x))
            yield arrive(self.seg_free[x & 3])
            for c in range(a, b):
                for u in range(t.parts(c)):
                    n = nbase + c
                    yield wait(self.s_full[h][u], k[u] & 1, k[u])
                    yield do(lambda n=n: self.keys[n % self.mut.key_slots].read(who, n))
                    if (c > a or u > 0) and (n + u + w) % 3 == 0:  # the reference rises: O is corrected
                        z = k[0] - 1 if u == 1 else k[1] - 1
                        yield wait(self.pv_done[h][u ^ 1], z & 1, z)
                        yield do(lambda x=x: ob.read(who, ("O", x)))

                    def passes(n=n, u=u):
                        self.sp[h][u][w].read(who, ("S", n))
                        self.sp[h][u][w].write(who, ("P", n))
                    yield do(passes)
                    yield arrive(self.p_full[h][u])
                    k[u] += 1
                    last_u = u
            nbase += t.chunks
            if b > a:
                if self.mut.epilogue_waits_pv:
                    yield wait(self.pv_done[h][last_u], (k[last_u] - 1) & 1, k[last_u] - 1)
                yield do(lambda x=x: ob.read(who, ("O", x)))

    def run(self, seed):
        roles = {"K": self.produce_k(), "V": self.produce_v(), "mma0": self.issue(0), "mma1": self.issue(1)}
        for h in range(2):
            for w in range(4):
                roles[f"softmax{h}.{w}"] = self.softmax(h, w)
        return simulate(roles, seed)


whole = lambda n, parts=2: Tile(n, ((0, n), (0, n)), parts)
one_half = lambda n, parts=2: Tile(n, ((0, n), (0, 0)), parts)
GEOMETRIES = {
    "one_chunk": ([whole(1) for _ in range(7)], 2),
    "one_part": ([whole(1, 1) for _ in range(7)], 2),
    "odd_ends": ([whole(2, 1), whole(3), whole(1, 1), whole(2), whole(1), whole(4, 1)], 2),
    "half_without_rows": ([one_half(1, 1), whole(2), one_half(3), whole(1, 1), one_half(2, 1), whole(2)], 4),
    "few_rows": ([one_half(1, 1 + x % 2) for x in range(10)], 2),
    "long": ([whole(9, 1), whole(7)], 4),
    # SA: a half's chunks begin and end inside the tile
    "sa": ([Tile(5, ((0, 3), (2, 5))), Tile(4, ((0, 2), (2, 4))), Tile(3, ((0, 3), (0, 3))), Tile(2, ((0, 2), (0, 0))),
            Tile(6, ((0, 2), (4, 6))), Tile(1, ((0, 1), (0, 1))), Tile(3, ((0, 1), (1, 3)))], 2),
}


@pytest.mark.parametrize("geo", sorted(GEOMETRIES))
def test_paged_tile_protocol_has_no_race_deadlock_or_parity_alias(geo):
    for seed in range(60):
        Model(*GEOMETRIES[geo]).run(seed)


MUTANTS = {
    "K stage refilled before both halves' S MMAs": (Mutation(waits_k_free=False), "odd_ends"),
    "V stage refilled before both halves' O MMAs": (Mutation(waits_v_free=False), "odd_ends"),
    "Q overwritten before the tile's last S MMA": (Mutation(waits_q_free=False), "one_chunk"),
    "tile entry overwritten before all have read it": (Mutation(waits_seg_free=False), "few_rows"),
    "key words overwritten before the softmax": (Mutation(key_slots=2), "long"),
    "O MMA does not wait for P": (Mutation(pv_waits_p=False), "odd_ends"),
    "O read out before the last O MMA": (Mutation(epilogue_waits_pv=False), "one_chunk"),
    "S over a P not yet read": (Mutation(pv_before_qk=False), "long"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_planted_paged_tile_protocol_mistakes_are_caught(name):
    mut, geo = MUTANTS[name]
    for seed in range(300):
        try:
            Model(*GEOMETRIES[geo], mut).run(seed)
        except ProtocolError:
            return
    pytest.fail(f"the model did not catch: {name}")
