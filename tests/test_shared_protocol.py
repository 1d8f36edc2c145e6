"""CPU model of the shared-prefix forward's barriers with every wait in it: the
issuers' turns, the eight softmax warps one by one, the groups' own barrier in
a tile with copies, and roles that give up.

A wait names the phase it means; the model passes it by the phase's parity, as
the hardware does, and checks that it was that phase.  Random interleavings
look for deadlocks, phases mistaken for others, and buffers refilled or
overwritten before their readers are done.  With `give_up`, a wait runs out in
the middle although what it waits for may still come: every role has to return
all the same.  The groups' barrier knows no limit: a warp that leaves arrives
there once, and whoever is let through looks at the abort.
"""
import os
import random
import re

import pytest

from tests.test_shared_models import STAGES, WINDOW, WINDOWS, WORK, place_k, place_v

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phases = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phases = 0, self.phases + 1


class Forward:
    def __init__(self, tiles, rnd, leave=True):
        """tiles: (blocks, keys, edge); keys: 0 two halves, 1 one half, 2 or 4 one half with copies of its rows."""
        self.tiles, self.rnd, self.leave = tiles, rnd, leave
        self.bar, self.landing, self.abort = {}, {}, False
        for name, count, n in (("q_full", 1, 4), ("q_empty", 2, 2), ("kv_full", 1, 2 * STAGES),
                               ("kv_empty", 2, STAGES), ("s_full", 1, 2), ("p_half", 4, 2), ("p_full", 4, 2),
                               ("o_full", 1, 2), ("o_empty", 4, 2), ("turn", 1, 2), ("group", 4, 2), ("done", 2, 1),
                               ("work_full", 1, WORK), ("work_empty", 10, WORK), ("win_full", 1, WINDOWS),
                               ("win_empty", 1, WINDOWS)):
            for i in range(n):
                self.bar[name, i] = Barrier(count)
        self.work, self.win = [None] * WORK, [None] * WINDOWS
        self.stage, self.qbuf = {}, {}               # what has landed: ring place, q number
        self.reads, self.qreads = {}, {}             # products still to read it
        self.scores, self.products = [0, 0], [0, 0]  # q k^T and P V completed
        self.weights = [[0] * 4, [0] * 4]            # blocks that each warp has written P of
        self.tile_of_o, self.o_read = [0, 0], [[0] * 4, [0] * 4]
        self.turns = []
        at = qn = 0
        for n, keys, _ in tiles:
            for i in range(n):
                self.reads[at + place_k(i)] = self.reads[at + place_v(i, n)] = 1 if keys else 2
            for x in range(1 if keys else 2):
                self.qreads[qn + x] = n
            at, qn = at + 2 * n, qn + (1 if keys else 2)

    # ------------------------------------------------------------ machinery
    def check(self, ok, what):
        assert ok or self.abort, f"{what}: {self.tiles}"

    def arrive(self, name, i=0, times=1):
        for _ in range(times):
            self.bar[name, i].arrive()

    def later(self, source, fn):
        self.landing.setdefault(source, []).append(fn)

    def ready(self, w):
        b = self.bar[w[0], w[1]]
        return b.phases > w[2] if w[0] == "group" else (b.phases - 1) & 1 == w[2] & 1

    def kv_full(self, place):
        return "kv_full", place % (2 * STAGES), place // (2 * STAGES)

    def q_full(self, x):
        return "q_full", x & 3, x >> 2

    def run(self, give_up=False):
        roles = {"sched": self.scheduler(), "prod": self.producer()}
        roles.update({("mma", h): self.issuer(h) for h in range(2)})
        roles.update({("soft", h, w): self.softmax(h, w) for h in range(2) for w in range(4)})
        waits = {k: None for k in roles}
        steps, limit = 0, self.rnd.randint(1, 60 * sum(t[0] for t in self.tiles)) if give_up else None
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
            assert all(a != b for a, b in zip(self.turns, self.turns[1:])), "a group took two turns"

    # ---------------------------------------------------------------- roles
    def next_tile(self, taken):
        if not (yield "work_full", taken % WORK, taken // WORK):
            return None
        number, tile = self.work[taken % WORK]
        self.check(number == taken, "another tile's record")
        self.arrive("work_empty", taken % WORK)
        return tile

    def scheduler(self):
        wn = qn = 0
        for k, tile in enumerate(self.tiles + [None]):
            if not (yield "work_empty", k % WORK, k // WORK - 1):
                break
            self.work[k % WORK] = (k, tile)
            self.arrive("work_full", k % WORK)
            n, keys = tile[:2] if tile else (0, 0)
            i, size, ok = 0, (n - 1) % WINDOW + 1 if n else 0, True
            while ok:
                ok = yield "win_empty", wn % WINDOWS, wn // WINDOWS - 1
                if not ok:
                    break
                self.win[wn % WINDOWS] = (wn, size, i == 0, i + size >= n)
                self.arrive("win_full", wn % WINDOWS)
                wn += 1
                for _ in range((1 if keys else 2) if i == 0 and n else 0):
                    ok = yield "q_empty", qn & 1, (qn >> 1) - 1
                    if not ok:
                        break
                    self.check(qn < 2 or self.qreads[qn - 2] == 0, "q refilled early")

                    def land(x=qn):
                        self.qbuf[x & 1] = x
                        self.arrive("q_full", x & 3)
                    self.later(("q", qn & 1), land)
                    qn += 1
                i, size = i + size, WINDOW
                if i >= n:
                    break
            if not ok or tile is None:
                break
            if not (yield "win_empty", wn % WINDOWS, wn // WINDOWS - 1):
                break
        for x in range(max(0, qn - 2), qn):
            yield self.q_full(x) + ("drain",)

    def producer(self):
        at = w = block = 0
        order = [(k, x) for k, (n, _, _) in enumerate(self.tiles) for x in range(2 * n)]

        def load(kv, b):
            nonlocal at
            if not (yield "kv_empty", at % STAGES, at // STAGES - 1):
                return False
            self.check(at < STAGES or self.reads[at - STAGES] == 0, "stage refilled early")
            k, x = order[at]
            b -= sum(t[0] for t in self.tiles[:k])
            self.check(x == (place_k(b) if kv == "k" else place_v(b, self.tiles[k][0])), "another block's place")

            def land(x=at):
                self.stage[x % STAGES] = x
                self.arrive(*self.kv_full(x)[:2])
            self.later(("kv", at % STAGES), land)
            at += 1
            return True

        ok = True
        while ok:
            ok = yield "win_full", w % WINDOWS, w // WINDOWS
            if not ok:
                break
            number, n, first, last = self.win[w % WINDOWS]
            self.check(number == w, "another window")
            if n == 0:
                break
            for i in range(n):
                if i == n - 1:
                    self.arrive("win_empty", w % WINDOWS)
                ok = yield from load("k", block)
                if ok and (i or not first):
                    ok = yield from load("v", block - 1)
                if not ok:
                    break
                block += 1
            if ok and last:
                ok = yield from load("v", block - 1)
            w += 1
        for x in range(max(0, at - STAGES), at):
            yield self.kv_full(x) + ("drain",)

    def issuer(self, h):
        ok, at, qn, taken, np, no, nt, owed = True, 0, 0, 0, 0, 0, 0, None

        def wait_v():
            place, first = owed[:2]
            ok = yield self.kv_full(place)
            self.check(not ok or self.stage[place % STAGES] == place, "another V")
            if ok and first and no:
                ok = yield "o_empty", h, no - 1
            return ok

        def start_pv():
            if not (yield "p_half", h, np):
                return False
            block, tiles, first = np, no, owed[1]

            def low(place=owed[0]):
                self.check(not first or min(self.o_read[h]) == tiles, "O overwritten before it was read")
                self.check(min(self.weights[h]) >= block + 0.5, "P V before P's first half")
                self.check(self.stage[place % STAGES] == place, "V gone")
            self.later(("pipe", h), low)
            return (yield "p_full", h, np)

        def rest_pv():
            place, _, last, keys = owed
            frees = not (last and keys > 1)  # (with copies the softmax frees the tile's last V)

            def done(block=np):
                self.check(min(self.weights[h]) >= block + 1, "P V before P")
                self.products[h] += 1
                if frees:
                    self.reads[place] -= 1
                    self.arrive("kv_empty", place % STAGES, 2 if keys else 1)
                if last:
                    self.tile_of_o[h] += 1
                    self.arrive("o_full", h)
            self.later(("pipe", h), done)

        while ok:
            tile = yield from self.next_tile(taken)
            if tile is None:
                break
            taken += 1
            n, keys, _ = tile
            stride = 2 if keys else 1
            half, qp = (h ^ (qn & 1), qn) if keys else (0, qn + h)
            for i in range(half, n, stride):
                kp = at + place_k(i)
                if owed:
                    ok = yield from wait_v()
                alone = i == half or not self.ready(self.kv_full(kp))
                if ok and not keys:
                    if h == 1 or nt > 0:
                        ok = yield "turn", h, nt if h else nt - 1
                    nt += 1
                if ok and owed:
                    ok = yield from start_pv()
                    if ok and alone:
                        rest_pv()
                        np, no, owed = np + 1, no + owed[2], None
                if ok and not owed:
                    if i == half:
                        ok = yield self.q_full(qp)
                    if ok:
                        ok = yield self.kv_full(kp)
                if not ok:
                    break
                self.check(self.qbuf[qp & 1] == qp and self.stage[kp % STAGES] == kp, "another q or K")
                last = i + stride >= n
                if owed:
                    rest_pv()

                def done(kp=kp, qp=qp, last=last, keys=keys):
                    self.check(self.products[h] == self.scores[h], "S overwritten before its product")
                    self.scores[h] += 1
                    self.reads[kp] -= 1
                    self.qreads[qp] -= 1
                    self.arrive("s_full", h)
                    self.arrive("kv_empty", kp % STAGES, 2 if keys else 1)
                    if last:
                        self.arrive("q_empty", qp & 1, 1 if keys else 2)
                self.later(("pipe", h), done)
                if not keys:
                    self.turns.append(h)
                    self.arrive("turn", h ^ 1)
                if owed:
                    np, no = np + 1, no + owed[2]
                owed = (at + place_v(i, n), i == half, int(last), keys)
                yield None
            if ok and half >= n:
                if owed:
                    ok = (yield from wait_v()) and (yield from start_pv())
                    if not ok:
                        break
                    rest_pv()
                    np, no, owed = np + 1, no + owed[2], None
                ok = yield self.q_full(qp)
                if not ok:
                    break
                self.later(("pipe", h), lambda qp=qp: self.arrive("q_empty", qp & 1))
            at, qn = at + 2 * n, qn + (1 if keys else 2)
        if ok and owed:
            if (yield from wait_v()) and (yield from start_pv()):
                rest_pv()
        self.later(("pipe", h), lambda: self.arrive("done"))
        yield "done", 0, 0, "drain"

    def softmax(self, h, warp):
        ok, at, ns, no, qn, taken, syncs = True, 0, 0, 0, 0, 0, 0
        while ok:
            tile = yield from self.next_tile(taken)
            if tile is None:
                break
            taken += 1
            n, keys, edge = tile
            half = h ^ (qn & 1) if keys else 0
            qn += 1 if keys else 2
            mine = False
            for i in range(half, n, 2 if keys else 1):
                ok = yield "s_full", h, ns
                if not ok:
                    break
                self.check(self.scores[h] == ns + 1, "another block's scores")
                if edge and i in (0, n - 1):
                    place = at + place_v(i, n)
                    ok = yield self.kv_full(place)
                    if not ok:
                        break
                    self.check(self.stage[place % STAGES] == place, "rows cleared in another block's stage")
                self.check(self.products[h] == ns, "O rescaled while a product writes it")
                self.weights[h][warp] = ns + 0.5
                self.arrive("p_half", h)
                yield None
                ns += 1
                self.weights[h][warp] = ns
                self.arrive("p_full", h)
                mine = True
            at += 2 * n
            if not ok or not mine:
                continue
            ok = yield "o_full", h, no
            if not ok:
                break
            no += 1
            self.check(self.tile_of_o[h] == no, "another tile's O")
            if keys > 1:  # the copies joined in the last V's stage
                place = at - 2 * n + place_v(((n - 1 - half) & ~1) + half, n)
                for _ in range(6):
                    self.check(self.stage[place % STAGES] == place, "the join's memory is another block's")
                    self.arrive("group", h)
                    yield "group", h, syncs, "no limit"
                    syncs += 1
                    yield None
                    ok = not self.abort
                    if not ok:
                        break
                if not ok:
                    break
                if warp == 0:
                    self.reads[place] -= 1
                    self.arrive("kv_empty", place % STAGES, 2)
            self.o_read[h][warp] = no
            self.arrive("o_empty", h)
        yield None
        if self.abort and self.leave:
            self.arrive("group", h)


def random_tiles(r):
    tiles = [(r.choice([1, 1, 2, 3, r.randint(1, 9), r.randint(8, 20)]), r.choice([0, 0, 1, 2, 4, 4]), r.random() < 0.5)
             for _ in range(r.randint(1, 7))]
    return [(1, k, True) for k in r.sample([0, 1, 4], r.randint(0, 3))] + tiles


@pytest.mark.parametrize("seed", range(40))
def test_every_order_ends(seed):
    r = random.Random(seed)
    for _ in range(4):
        Forward(random_tiles(r), r).run()


@pytest.mark.parametrize("seed", range(40))
def test_every_role_returns_when_one_gives_up(seed):
    r = random.Random(1000 + seed)
    for _ in range(6):
        Forward(random_tiles(r), r).run(give_up=True)


def test_a_warp_that_left_without_arriving_would_be_waited_for():
    """The model sees it: warps that give up at the wait before the groups' barrier, while others pass that wait."""
    def hangs(seed):
        r = random.Random(seed)
        try:
            Forward([(2, 4, False)] * 3 + [(3, 2, False)], r, leave=False).run(give_up=True)
        except AssertionError as e:
            return "deadlock" in str(e)
        return False

    assert any(hangs(s) for s in range(600))


def test_the_forward_arrives_as_it_leaves():
    src = open(os.path.join(ROOT, "block_sparse_attention_builder_gb300", "csrc", "shared.cu")).read()
    assert len(re.findall(r"bar\.sync", src)) == 1 and len(re.findall(r"bar\.arrive", src)) == 1
    assert re.search(r"bar\.sync[^\n]*\n\s*return hwarp_all\(\*abort_flag == 0\);", src)
