"""CPU model of the whole-prompt forward's barriers with every wait in it: the
producer and its two tile records, the q warp, the two issuers and their turns,
the eight softmax warps, and roles that give up.

A wait names the phase it means; the model passes it by the phase's parity, as
the hardware does, and checks that it was that phase.  Random interleavings look
for deadlocks, phases mistaken for others, and buffers refilled or overwritten
before their readers are done.  With `give_up`, a wait runs out in the middle
although what it waits for may still come: every role has to return all the
same.
"""
import os
import random
import re

import pytest

from tests.test_shared_protocol import Barrier

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAGES, WORK = 5, 2


class Forward:
    def __init__(self, tiles, rnd):
        """tiles: (n0, n1, whether rows of V behind the sequence are cleared); n1 is 0, n0 or n0 + 1, or n0 is 0."""
        self.tiles, self.rnd = tiles, rnd
        self.bar, self.landing, self.abort = {}, {}, False
        for name, count, n in (("q_full", 1, 2), ("q_empty", 1, 2), ("kv_full", 1, 2 * STAGES),
                               ("kv_empty", 2, STAGES), ("s_full", 1, 2), ("p_half", 4, 2), ("lo_done", 1, 2),
                               ("p_full", 4, 2), ("o_full", 1, 2), ("o_empty", 4, 2), ("turn", 1, 2), ("done", 2, 1),
                               ("work_full", 1, WORK), ("work_empty", 11, WORK)):
            for i in range(n):
                self.bar[name, i] = Barrier(count)
        self.work = [None] * WORK
        self.stage, self.qbuf = {}, [-1, -1]         # what has landed: ring place, the group's tile number
        self.reads, self.qreads = {}, {}             # products still to read it
        self.scores, self.products, self.lows = [0, 0], [0, 0], [0, 0]  # q k^T, P V and their first halves done
        self.weights = [[0] * 4, [0] * 4]            # blocks that each warp has written P of
        self.tile_of_o, self.o_read = [0, 0], [[0] * 4, [0] * 4]
        at, count = 0, [0, 0]
        for n0, n1, _ in tiles:
            for i in range(max(n0, n1)):
                self.reads[at + 2 * i] = self.reads[at + 2 * i + 1] = (i < n0) + (i < n1)
            for h, n in ((0, n0), (1, n1)):
                if n:
                    self.qreads[h, count[h]] = n
                    count[h] += 1
            at += 2 * max(n0, n1)

    # ------------------------------------------------------------ machinery
    def check(self, ok, what):
        assert ok or self.abort, f"{what}: {self.tiles}"

    def arrive(self, name, i=0, times=1):
        for _ in range(times):
            self.bar[name, i].arrive()

    def later(self, source, fn):
        self.landing.setdefault(source, []).append(fn)

    def ready(self, w):
        return (self.bar[w[0], w[1]].phases - 1) & 1 == w[2] & 1

    def kv_full(self, place):
        return "kv_full", place % (2 * STAGES), place // (2 * STAGES)

    def run(self, give_up=False):
        roles = {"prod": self.producer(), "q": self.queries()}
        roles.update({("mma", h): self.issuer(h) for h in range(2)})
        roles.update({("soft", h, w): self.softmax(h, w) for h in range(2) for w in range(4)})
        waits = {k: None for k in roles}
        steps, limit = 0, self.rnd.randint(1, 60 * sum(max(t[:2]) for t in self.tiles)) if give_up else None
        while roles or any(self.landing.values()):
            steps += 1
            can = [k for k in roles if waits[k] is None or self.ready(waits[k])]
            stuck = [k for k in roles if k not in can and len(waits[k]) == 3]  # (a drain does not look at the abort)
            if give_up and stuck and (self.abort or steps >= limit):
                can += [k for k in stuck if self.abort] or [self.rnd.choice(stuck)]
            lands = [s for s, v in self.landing.items() if v]
            assert can or lands, f"deadlock: {self.tiles} {waits}"
            k = self.rnd.choice(can + lands)
            if k not in roles:
                self.landing[k].pop(0)()
                continue
            ok = True
            if waits[k] is not None:
                ok = self.ready(waits[k])
                if ok:
                    self.check(self.bar[waits[k][:2]].phases > waits[k][2], f"{k} took another phase of {waits[k]}")
                else:
                    self.abort = True
            try:
                waits[k] = roles[k].send(None if waits[k] is None else ok)
            except StopIteration:
                del roles[k], waits[k]
        if not self.abort:
            assert all(v == 0 for v in self.reads.values()) and all(v == 0 for v in self.qreads.values())

    # ---------------------------------------------------------------- roles
    def next_tile(self, taken):
        if not (yield "work_full", taken % WORK, taken // WORK):
            return None
        number, tile = self.work[taken % WORK]
        self.check(number == taken, "another tile's record")
        self.arrive("work_empty", taken % WORK)
        return tile

    def producer(self):
        at, ok = 0, True
        for k, tile in enumerate(self.tiles + [None]):
            if not (yield "work_empty", k % WORK, k // WORK - 1):
                break
            self.work[k % WORK] = (k, tile)
            self.arrive("work_full", k % WORK)
            for _ in range(2 * max(tile[:2]) if tile else 0):
                ok = yield "kv_empty", at % STAGES, at // STAGES - 1
                if not ok:
                    break
                self.check(at < STAGES or self.reads[at - STAGES] == 0, "stage refilled early")

                def land(x=at):
                    self.stage[x % STAGES] = x
                    self.arrive(*self.kv_full(x)[:2])
                self.later(("kv", at % STAGES), land)
                at += 1
            if not ok:
                break
        for x in range(max(0, at - STAGES), at):
            yield self.kv_full(x) + ("drain",)

    def queries(self):
        ok, taken, n = True, 0, [0, 0]
        while ok:
            tile = yield from self.next_tile(taken)
            if tile is None:
                break
            taken += 1
            for h in range(2):
                if not tile[h]:
                    continue
                ok = yield "q_empty", h, n[h] - 1
                if not ok:
                    break
                self.check(n[h] == 0 or self.qreads[h, n[h] - 1] == 0, "q refilled early")

                def land(h=h, x=n[h]):
                    self.qbuf[h] = x
                    self.arrive("q_full", h)
                self.later(("q", h), land)
                n[h] += 1
        for h in range(2):
            if n[h]:
                yield "q_full", h, n[h] - 1, "drain"

    def issuer(self, h):
        ok, place, taken, np, nt, turns = True, 0, 0, 0, 0, 0
        while ok:
            tile = yield from self.next_tile(taken)
            if tile is None:
                break
            taken += 1
            n, blocks, both = tile[h], max(tile[:2]), min(tile[:2]) > 0
            start = place
            for i in range((blocks if both else n) + 1):
                if i > n or n == 0:
                    if not both:
                        break
                    if h == 1 or turns > 0:
                        ok = yield "turn", h, turns if h else turns - 1
                    turns += 1
                    if not ok:
                        break
                    self.arrive("turn", h ^ 1)
                    continue
                alone_v = (i - 1 >= tile[0]) if h else not both
                alone_k = (i >= tile[0]) if h else not both
                vp = kp = None
                if i > 0:
                    vp, place = place, place + 1
                    ok = yield self.kv_full(vp)
                if ok and i < n:
                    kp, place = place, place + 1
                    ok = yield self.kv_full(kp)
                if ok and i == 0:
                    ok = yield "q_full", h, nt
                if ok and i == 1 and nt > 0:
                    ok = yield "o_empty", h, nt - 1
                if ok and i > 0:
                    ok = yield "p_half", h, np
                if ok and both:
                    if h == 1 or turns > 0:
                        ok = yield "turn", h, turns if h else turns - 1
                    turns += 1
                if not ok:
                    break
                if i > 0:
                    def low(vp=vp, block=np, first=i == 1, tiles=nt):
                        self.check(self.stage[vp % STAGES] == vp, "another V")
                        self.check(not first or min(self.o_read[h]) == tiles, "O overwritten before it was read")
                        self.check(min(self.weights[h]) >= block + 0.5, "P V before P's first half")
                        self.lows[h] += 1
                        self.arrive("lo_done", h)
                    self.later(("pipe", h), low)
                    ok = yield "p_full", h, np
                    np += 1
                    if not ok:
                        break

                def done(vp=vp, kp=kp, block=np - 1, i=i, n=n, alone_v=alone_v, alone_k=alone_k, tiles=nt):
                    if i > 0:
                        self.check(min(self.weights[h]) >= block + 1, "P V before P")
                        self.check(self.stage[vp % STAGES] == vp, "V gone")
                        self.products[h] += 1
                        self.reads[vp] -= 1
                        if i == n:
                            self.tile_of_o[h] += 1
                            self.arrive("o_full", h)
                    if i < n:
                        self.check(self.stage[kp % STAGES] == kp and self.qbuf[h] == tiles, "another q or K")
                        self.check(self.products[h] == self.scores[h], "S overwritten before its product")
                        self.scores[h] += 1
                        self.reads[kp] -= 1
                        self.qreads[h, tiles] -= 1
                        self.arrive("s_full", h)
                        self.arrive("kv_empty", kp % STAGES, 2 if alone_k else 1)
                        if i == n - 1:
                            self.arrive("q_empty", h)
                    if i > 0:
                        self.arrive("kv_empty", vp % STAGES, 2 if alone_v else 1)
                self.later(("pipe", h), done)
                if both:
                    self.arrive("turn", h ^ 1)
                yield None
            place = start + 2 * blocks
            nt += n > 0
        self.later(("pipe", h), lambda: self.arrive("done"))
        yield "done", 0, 0, "drain"

    def softmax(self, h, warp):
        ok, at, ns, no, taken = True, 0, 0, 0, 0
        while ok:
            tile = yield from self.next_tile(taken)
            if tile is None:
                break
            taken += 1
            n, start = tile[h], at
            at += 2 * max(tile[:2])
            if n == 0:
                continue
            for i in range(n):
                ok = yield "s_full", h, ns
                if not ok:
                    break
                self.check(self.scores[h] == ns + 1, "another block's scores")
                self.check(self.products[h] == ns, "O rescaled while a product writes it")
                if tile[2] and i == n - 1:
                    place = start + 2 * i + 1
                    ok = yield self.kv_full(place)
                    if not ok:
                        break
                    self.check(self.stage[place % STAGES] == place, "rows cleared in another block's stage")
                self.weights[h][warp] = ns + 0.5
                self.arrive("p_half", h)
                yield None
                if self.rnd.random() < 0.2:  # the second half raises the reference
                    ok = yield "lo_done", h, ns
                    if not ok:
                        break
                    self.check(self.lows[h] == ns + 1, "O rescaled before the first half's product")
                ns += 1
                self.weights[h][warp] = ns
                self.arrive("p_full", h)
            if not ok:
                break
            ok = yield "o_full", h, no
            if not ok:
                break
            no += 1
            self.check(self.tile_of_o[h] == no, "another tile's O")
            self.o_read[h][warp] = no
            self.arrive("o_empty", h)


def random_tiles(r):
    tiles = []
    for _ in range(r.randint(1, 8)):
        n0 = r.choice([1, 1, 2, 3, r.randint(1, 9), r.randint(8, 25)])
        n1 = r.choice([0, 0, n0, n0, n0 + 1])
        if n1 == 0 and r.random() < 0.5:  # a tile of one half that the second group has
            n0, n1 = 0, n0
        tiles.append((n0, n1, r.random() < 0.5))
    return tiles


@pytest.mark.parametrize("seed", range(40))
def test_every_order_ends(seed):
    r = random.Random(seed)
    for _ in range(4):
        Forward(random_tiles(r), r).run()


def test_a_group_that_passes_over_long_tiles():
    """One barrier per stage would be enough only while no role is two uses behind: here group 1 has nothing of tiles
    many rounds of the ring long."""
    r = random.Random(7)
    for _ in range(20):
        Forward([(2, 3, True), (23, 0, True), (1, 1, False), (12, 0, False), (9, 10, True)], r).run()
        Forward([(2, 3, True), (0, 23, True), (1, 0, False), (0, 12, True), (11, 0, False), (9, 9, True)], r).run()


@pytest.mark.parametrize("seed", range(40))
def test_every_role_returns_when_one_gives_up(seed):
    r = random.Random(1000 + seed)
    for _ in range(6):
        Forward(random_tiles(r), r).run(give_up=True)


def test_the_model_is_the_source():
    src = open(os.path.join(ROOT, "block_sparse_attention_builder_gb300", "csrc", "prompt.cu")).read()
    assert re.search(r"kRStages = 5, kRWork = 2;", src)
    for name, count in (("work_empty", 11), ("o_empty", 4), ("p_half", 4), ("p_full", 4), ("kv_empty", 2),
                        ("lo_done", 1), ("turn", 1)):
        assert re.search(rf"mbar_init\(&c\.{name}\[i\], {count}\);", src), name
