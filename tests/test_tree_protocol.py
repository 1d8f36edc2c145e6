"""CPU model of the barriers of the trees' one-launch forward: the producer and
its ring, of whose blocks the two groups take every other one, the issuers, the
softmax warps, and roles that give up.  Waits pass by parity, as the hardware's
do, and the model checks that it was the phase that was meant (see
test_prompt_protocol.py).
"""
import os
import random
import re

import pytest

from tests.test_shared_protocol import Barrier

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAGES = 5


class Forward:
    def __init__(self, blocks, rnd):
        self.blocks, self.rnd = blocks, rnd
        self.bar, self.landing, self.abort = {}, {}, False
        for name, count, n in (("found", 1, 1), ("q_full", 1, 1), ("kv_full", 1, 2 * STAGES), ("kv_empty", 1, STAGES),
                               ("s_full", 1, 2), ("p_half", 4, 2), ("lo_done", 1, 2), ("p_full", 4, 2),
                               ("o_full", 1, 2), ("done", 2, 1)):
            for i in range(n):
                self.bar[name, i] = Barrier(count)
        self.stage, self.reads = {}, {p: 1 for p in range(2 * blocks)}
        self.scores, self.products, self.lows, self.weights = [0, 0], [0, 0], [0, 0], [[0] * 4, [0] * 4]

    def check(self, ok, what):
        assert ok or self.abort, f"{what}: {self.blocks}"

    def later(self, source, fn):
        self.landing.setdefault(source, []).append(fn)

    def ready(self, w):
        return (self.bar[w[0], w[1]].phases - 1) & 1 == w[2] & 1

    def kv_full(self, place):
        return "kv_full", place % (2 * STAGES), place // (2 * STAGES)

    def run(self, give_up=False):
        roles = {"prod": self.producer()}
        roles.update({("mma", h): self.issuer(h) for h in range(2)})
        roles.update({("soft", h, w): self.softmax(h, w) for h in range(2) for w in range(4)})
        waits = {k: None for k in roles}
        steps, limit = 0, self.rnd.randint(1, 40 * self.blocks + 20) if give_up else None
        while roles or any(self.landing.values()):
            steps += 1
            can = [k for k in roles if waits[k] is None or self.ready(waits[k])]
            stuck = [k for k in roles if k not in can and len(waits[k]) == 3]
            if give_up and stuck and (self.abort or steps >= limit):
                can += [k for k in stuck if self.abort] or [self.rnd.choice(stuck)]
            lands = [s for s, v in self.landing.items() if v]
            assert can or lands, f"deadlock: {self.blocks} {waits}"
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
            assert all(v == 0 for v in self.reads.values())

    def producer(self):
        self.bar["found", 0].arrive()
        self.later("q", lambda: self.bar["q_full", 0].arrive())
        at = 0
        for at in range(2 * self.blocks):
            if not (yield "kv_empty", at % STAGES, at // STAGES - 1):
                break
            self.check(at < STAGES or self.reads[at - STAGES] == 0, "stage refilled early")

            def land(x=at):
                self.stage[x % STAGES] = x
                self.bar[self.kv_full(x)[:2]].arrive()
            self.later(("kv", at), land)  # (copies may land in any order)
            at += 1
        for x in range(max(0, at - STAGES), at):
            yield self.kv_full(x) + ("drain",)
        yield "q_full", 0, 0, "drain"

    def issuer(self, h):
        ok = yield "found", 0, 0
        n = (self.blocks - h + 1) // 2 if ok and self.blocks > h else 0
        if n:
            ok = yield "q_full", 0, 0
        for i in range(n + 1 if n and ok else 0):
            vp, kp = 2 * (2 * (i - 1) + h) + 1, 2 * (2 * i + h)
            if i > 0:
                ok = yield self.kv_full(vp)
                if ok:
                    ok = yield "p_half", h, i - 1
                if not ok:
                    break

                def low(i=i, vp=vp):
                    self.check(self.stage[vp % STAGES] == vp, "another V")
                    self.check(min(self.weights[h]) >= i - 0.5, "P V before P's first half")
                    self.lows[h] += 1
                    self.bar["lo_done", h].arrive()
                self.later(("pipe", h), low)
                ok = yield "p_full", h, i - 1
                if not ok:
                    break

                def high(i=i, vp=vp):
                    self.check(min(self.weights[h]) >= i and self.stage[vp % STAGES] == vp, "P V before P")
                    self.products[h] += 1
                    self.reads[vp] -= 1
                    self.bar["kv_empty", vp % STAGES].arrive()
                    if i == n:
                        self.bar["o_full", h].arrive()
                self.later(("pipe", h), high)
            if i < n:
                ok = yield self.kv_full(kp)
                if not ok:
                    break

                def scores(i=i, kp=kp):
                    self.check(self.stage[kp % STAGES] == kp, "another K")
                    self.check(self.products[h] == i, "S overwritten before its product")
                    self.scores[h] += 1
                    self.reads[kp] -= 1
                    self.bar["s_full", h].arrive()
                    self.bar["kv_empty", kp % STAGES].arrive()
                self.later(("pipe", h), scores)
            yield None
        self.later(("pipe", h), lambda: self.bar["done", 0].arrive())
        yield "done", 0, 0, "drain"

    def softmax(self, h, warp):
        ok = yield "found", 0, 0
        n = (self.blocks - h + 1) // 2 if ok and self.blocks > h else 0
        for i in range(n):
            ok = yield "s_full", h, i
            if not ok:
                return
            self.check(self.scores[h] == i + 1 and self.products[h] == i, "another block's scores")
            if 2 * i + h == self.blocks - 1:  # V rows behind the sequence
                place = 2 * (2 * i + h) + 1
                ok = yield self.kv_full(place)
                if not ok:
                    return
                self.check(self.stage[place % STAGES] == place, "rows cleared in another block's stage")
            self.weights[h][warp] = i + 0.5
            self.bar["p_half", h].arrive()
            yield None
            if self.rnd.random() < 0.2:
                ok = yield "lo_done", h, i
                if not ok:
                    return
                self.check(self.lows[h] == i + 1, "O rescaled before the first half's product")
            self.weights[h][warp] = i + 1
            self.bar["p_full", h].arrive()
        if n:
            yield "o_full", h, 0


@pytest.mark.parametrize("seed", range(30))
def test_every_order_ends(seed):
    r = random.Random(seed)
    for blocks in (0, 1, 2, 3, r.randint(4, 12), r.randint(12, 40)):
        Forward(blocks, r).run()


@pytest.mark.parametrize("seed", range(30))
def test_every_role_returns_when_one_gives_up(seed):
    r = random.Random(100 + seed)
    for blocks in (1, 2, r.randint(3, 12), r.randint(12, 30)):
        Forward(blocks, r).run(give_up=True)


def test_the_model_is_the_source():
    src = open(os.path.join(ROOT, "block_sparse_attention_builder_gb300", "csrc", "tree.cu")).read()
    assert "kTStages = 5;" in src
    for name, count in (("p_half", 4), ("p_full", 4), ("kv_empty", 1), ("lo_done", 1)):
        assert re.search(rf"mbar_init\(&c\.{name}\[i\], {count}\);", src), name
