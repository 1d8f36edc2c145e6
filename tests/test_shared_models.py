"""CPU models of the dense path over shared prefixes (mxsa_dense_shared_fwd).

The plan: jobs, tiles and their chunks restated in Python; random problems
check that every visible (token, key) pair lies in exactly one tile, that a
row's partials are distinct and that the bounds on tiles, partial rows and
partials of one row that size the workspace hold.

The forward's protocol (producer, two MMA issuers, two softmax groups, five
K/V stages, two q buffers, the ring of tiles) under random interleavings: no
deadlock, and no buffer is refilled or overwritten before its readers are
done.
"""
import random

import pytest

from tests.test_barrier_models import Bar

MAXC, WR, WK, TILE, STAGES, WORK = 160, 8, 4, 10, 5, 4
WINDOWS, WINDOW = 2, 3
PER_CTA, ONE_CHUNK = 2, 24


def cdiv(a, b):
    return -(-a // b)


def plan(p):
    """p: cu, lens, gp, prefix, hkv, hq, causal, ctas.  Returns (tiles, partial rows)."""
    G = p["hq"] // p["hkv"]
    T, B, cu = 128 // G, len(p["lens"]), p["cu"]
    seq_group, prefix = [-1] * B, []
    for j, P in enumerate(p["prefix"]):
        members = range(p["gp"][j], p["gp"][j + 1])
        P = min([max(P, 0)] + [p["lens"][s] for s in members if cu[s + 1] > cu[s]])
        prefix.append(P if len(members) > 1 else 0)
        for s in members:
            seq_group[s] = j if prefix[j] > 0 else -1
    jobs = []
    for j, P in enumerate(prefix):
        on = P > 0
        jobs.append(dict(tok0=cu[p["gp"][j]] if on else 0, ntok=cu[p["gp"][j + 1]] - cu[p["gp"][j]] if on else 0, lo=0,
                         hi=P, own=False))
    for s in range(B):
        jobs.append(dict(tok0=cu[s], ntok=cu[s + 1] - cu[s], lo=prefix[seq_group[s]] if seq_group[s] >= 0 else 0,
                         hi=p["lens"][s], own=True))
    total = 0
    for j in jobs:
        j["nb"] = cdiv(j["hi"], 128) - j["lo"] // 128 if j["ntok"] > 0 and j["hi"] > j["lo"] else 0
        rem = j["ntok"] % (2 * T)
        j["nrt"] = cdiv(j["ntok"], 2 * T) if j["nb"] else 0
        keys = int(0 < rem <= T)
        j["w"] = WR if j["nrt"] > keys else WK
        if j["nb"]:
            total += p["hkv"] * ((j["nrt"] - keys) * (j["nb"] * WR + TILE) + keys * (j["nb"] * WK + TILE))
    share = max(cdiv(total, p["ctas"]), 1)
    tiles = []
    for j in jobs:
        whole = cdiv(share, j["w"])
        nb = j["nb"]
        c = min(whole if whole <= ONE_CHUNK else cdiv(whole, PER_CTA), max(nb, 1))
        nch = max((nb + c // 2) // c, 1) if nb else 0
        c = cdiv(nb, nch) if nch else 1
        j["chunk"], j["nch"] = c, nch
        j["tile0"] = len(tiles)
        for g in range(p["hkv"]):
            for ch in range(j["nch"]):
                for rt in range(j["nrt"]):
                    ntok = min(2 * T, j["ntok"] - rt * 2 * T)
                    end = cdiv(j["hi"], 128)
                    if p["causal"] and j["own"]:
                        end = min(end, cdiv(max(j["hi"] - j["ntok"] + rt * 2 * T + ntok, 0), 128))
                    b0 = j["lo"] // 128 + ch * c
                    tiles.append(dict(tok0=j["tok0"] + rt * 2 * T, ntok=ntok, g=g, lo=j["lo"], hi=j["hi"], b0=b0,
                                      n=max(min(b0 + c, end) - b0, 0), keys=ntok <= T, job=j))
    part = 0
    for t in tiles:
        t["part0"] = part
        if t["n"]:
            part += t["ntok"] * G * (2 if t["keys"] else 1)
    return tiles, part


def random_problem(r):
    hq, hkv = r.choice([(8, 1), (16, 2), (12, 4), (4, 4), (128, 1), (10, 2)])
    B = r.choice([1, 2, 5, 17, 40])
    tq = [r.choice([0, 1, 1, 1, 3, r.randint(1, 90)]) for _ in range(B)]
    off = r.randint(0, 2)
    cu = [off]
    for x in tq:
        cu.append(cu[-1] + x)
    lens = [r.choice([0, 1, 127, 128, 129, r.randint(1, 6000)]) for _ in range(B)]
    ng = r.randint(0, min(B, 4))
    gp = sorted(r.randint(0, B) for _ in range(ng + 1)) if ng else [0]
    prefix = [r.choice([0, 1, 128, r.randint(-3, 7000)]) for _ in range(ng)]
    return dict(hq=hq, hkv=hkv, cu=cu, lens=lens, gp=gp, prefix=prefix, causal=r.random() < 0.5,
                ctas=r.choice([1, 3, 148, 152, 160]), total_q=cu[-1] + r.randint(0, 3))


@pytest.mark.parametrize("seed", range(60))
def test_plan_covers_every_key_once_within_its_bounds(seed):
    p = random_problem(random.Random(seed))
    G, B = p["hq"] // p["hkv"], len(p["lens"])
    T = 128 // G
    tiles, part = plan(p)
    triples = p["hkv"] * (2 * (p["total_q"] // (2 * T)) + 2 * B)
    blocks = max(1, cdiv(max(p["lens"]), 128))
    by_cost = PER_CTA * 2 * MAXC
    extra = min(by_cost, triples * (blocks - 1))
    assert len(tiles) <= triples + extra
    assert part <= 4 * p["total_q"] * p["hq"] + min(256, 2 * p["total_q"] * G) * extra
    assert all(t["ntok"] * G * (2 if t["keys"] else 1) <= 256 for t in tiles)
    # tokens: the key blocks of its tiles, masked, make up its visible keys
    for s in range(B):
        for tok in range(p["cu"][s], p["cu"][s + 1]):
            L = p["lens"][s]
            see = max(L - (p["cu"][s + 1] - tok) + 1, 0) if p["causal"] else L
            for g in {0, p["hkv"] - 1}:
                got, parts = [], 0
                for t in tiles:
                    if t["g"] == g and t["tok0"] <= tok < t["tok0"] + t["ntok"] and t["n"]:
                        got.append((max(t["b0"] * 128, t["lo"]), min((t["b0"] + t["n"]) * 128, t["hi"], see)))
                        parts += min(t["n"], 2) if t["keys"] else 1
                assert parts <= 2 * min(2 + by_cost // p["hkv"], 2 * blocks + 2)
                got = sorted(x for x in got if x[1] > x[0])
                at = 0
                for lo, hi in got:
                    assert lo == at
                    at = hi
                assert at == min(see, L)


def place_k(i):
    return 0 if i == 0 else 2 * i - 1


def place_v(i, n):
    return 2 * i + 2 if i < n - 1 else 2 * n - 1


@pytest.mark.parametrize("n", range(1, 9))
def test_ring_places_are_the_producers_order(n):
    order = [place_k(i) if kv == 0 else place_v(i - 1, n) for i in range(n + 1) for kv in range(2)
             if not (kv == 0 and i >= n) and not (kv == 1 and i == 0)]
    assert order == list(range(2 * n))


def run_protocol(segs, seed):
    """segs: (blocks, keys, edge) of the CTA's tiles; keys: 0 two halves, 1 one half, 4 one half with copies; edge: the groups wait for V to clear rows of it."""
    rnd = random.Random(seed)
    B, pending = {}, {}

    def bar(n, c=1):
        B[n] = Bar(n, c)

    for i in range(2):
        for n in ("s_full", "p_half", "p_full", "o_full", "o_empty"):
            bar(f"{n}{i}")
        bar(f"q_empty{i}", 2)
    for i in range(4):
        bar(f"q_full{i}")
    for i in range(WORK):
        bar(f"work_full{i}")
        bar(f"work_empty{i}", 4)
    work = [None] * WORK

    def tiles_of():
        """The tiles as a role sees them, through the ring."""
        k = 0
        while True:
            yield ("wait", B[f"work_full{k % WORK}"], (k // WORK) & 1)
            got = work[k % WORK]
            B[f"work_empty{k % WORK}"].arrive()
            k += 1
            assert got[0] == k - 1, "another tile's record"
            yield ("tile", got[1])
            if got[1] is None:
                return
    for i in range(STAGES):
        bar(f"kv_full{i}")
        bar(f"kv_full{i + STAGES}")
        bar(f"kv_empty{i}", 2)

    def q_full(x):
        return ("wait", B[f"q_full{x & 3}"], (x >> 2) & 1)

    def kv_full(x):
        return ("wait", B[f"kv_full{x % (2 * STAGES)}"], (x // (2 * STAGES)) & 1)

    def later(src, cb):
        pending.setdefault(src, []).append(cb)

    stage, qbuf = {}, {}          # landed place / q number
    reads = {}                    # place -> products still to come that read it
    qreads = {}
    S, O = [None, None], [None, None]
    finished = [0, 0]

    for i in range(WINDOWS):
        bar(f"win_full{i}")
        bar(f"win_empty{i}")
    win = [None] * WINDOWS

    def scheduler():
        wn = qn = 0
        for k, tile in enumerate(segs + [None]):
            yield ("wait", B[f"work_empty{k % WORK}"], ((k // WORK) & 1) ^ 1)
            work[k % WORK] = (k, tile)
            B[f"work_full{k % WORK}"].arrive()
            n, keys = tile[:2] if tile else (0, 0)
            i, size = 0, (n - 1) % WINDOW + 1 if n else 0
            while True:
                yield ("wait", B[f"win_empty{wn % WINDOWS}"], ((wn // WINDOWS) & 1) ^ 1)
                win[wn % WINDOWS] = (wn, size, i == 0, i + size >= n)
                B[f"win_full{wn % WINDOWS}"].arrive()
                wn += 1
                for _h in range((1 if keys else 2) if i == 0 and n else 0):
                    b = qn & 1
                    yield ("wait", B[f"q_empty{b}"], ((qn >> 1) & 1) ^ 1)
                    assert qn < 2 or qreads[qn - 2] == 0, "q refilled early"

                    def land(b=b, qn=qn):
                        qbuf[b] = qn
                        B[f"q_full{qn & 3}"].arrive()
                    later(f"q{b}", land)
                    qn += 1
                i, size = i + size, WINDOW
                if i >= n:
                    break
            if tile is None:
                return
            yield ("wait", B[f"win_empty{wn % WINDOWS}"], ((wn // WINDOWS) & 1) ^ 1)

    def producer():
        at = w = 0
        order = [(k, x) for k, (n, _, _) in enumerate(segs) for x in range(2 * n)]
        block = 0  # of the windows so far

        def load(kv):
            nonlocal at
            st = at % STAGES
            yield ("wait", B[f"kv_empty{st}"], ((at // STAGES) & 1) ^ 1)
            assert at < STAGES or reads[at - STAGES] == 0, "stage refilled early"
            k, x = order[at]
            n, b = segs[k][0], block - sum(t[0] for t in segs[:k])
            assert x == (place_k(b) if kv == "k" else place_v(b, n)), "another block's place"

            def land(st=st, at=at):
                stage[st] = at
                B[f"kv_full{at % (2 * STAGES)}"].arrive()
            later(f"kv{st}", land)
            at += 1

        while True:
            yield ("wait", B[f"win_full{w % WINDOWS}"], (w // WINDOWS) & 1)
            num, n, first, last = win[w % WINDOWS]
            assert num == w, "another window"
            if n == 0:
                assert at == len(order)
                return
            for i in range(n):
                if i == n - 1:
                    win[w % WINDOWS] = None
                    B[f"win_empty{w % WINDOWS}"].arrive()
                yield from load("k")
                if i or not first:
                    block -= 1
                    yield from load("v")
                    block += 1
                block += 1
            if last:
                block -= 1
                yield from load("v")
                block += 1
            w += 1

    def issuer(h):
        at = qn = npv = no = 0
        owed = None

        def wait_v():
            pl, first, _, _ = owed
            yield kv_full(pl)
            assert stage[pl % STAGES] == pl
            if first and no:
                yield ("wait", B[f"o_empty{h}"], (no - 1) & 1)
                assert O[h] == "read", "O overwritten before it was read"

        def start_pv():
            yield ("wait", B[f"p_half{h}"], npv & 1)
            pl = owed[0]

            def low():
                assert S[h][0] in ("half", "P") and stage[pl % STAGES] == pl
                O[h] = "acc"
            later(f"mma{h}", low)
            yield ("wait", B[f"p_full{h}"], npv & 1)
            assert S[h][0] == "P"

        def rest_pv():
            pl, _, last, alone = owed

            def done():
                assert S[h][0] == "P"
                S[h] = ("used",)
                O[h] = "done" if last else "acc"
                reads[pl] -= 1
                if not (alone > 1 and last):  # (with copies the softmax frees the tile's last V)
                    for _x in range(2 if alone else 1):
                        B[f"kv_empty{pl % STAGES}"].arrive()
                else:
                    reads[pl] += 1
                if last:
                    B[f"o_full{h}"].arrive()
            later(f"mma{h}", done)

        for got in tiles_of():
            if got[0] == "wait":
                yield got
                continue
            if got[1] is None:
                break
            n, keys, _ = got[1]
            half = h ^ (qn & 1) if keys else 0
            qp = qn if keys else qn + h
            for i in range(half, n, 2 if keys else 1):
                kp = at + place_k(i)
                st = kp % STAGES
                if owed:
                    yield from wait_v()
                    alone = i == half or not kv_full(kp)[1].ready(kv_full(kp)[2])
                    yield from start_pv()
                    if alone:
                        rest_pv()
                        npv, no, owed = npv + 1, no + owed[2], None
                if not owed:
                    if i == half:
                        yield q_full(qp)
                    yield kv_full(kp)
                assert qbuf[qp & 1] == qp and stage[st] == kp
                last = i + (2 if keys else 1) >= n
                if owed:
                    rest_pv()

                def done(qp=qp, kp=kp, st=st, last=last, keys=keys):
                    assert S[h] is None or S[h][0] == "used", "S overwritten before its product"
                    S[h] = ("S",)
                    reads[kp] -= 1
                    qreads[qp] -= 1
                    B[f"s_full{h}"].arrive()
                    for _x in range(2 if keys else 1):
                        B[f"kv_empty{st}"].arrive()
                    for _x in range((1 if keys else 2) if last else 0):
                        B[f"q_empty{qp & 1}"].arrive()
                later(f"mma{h}", done)
                if owed:
                    npv, no = npv + 1, no + owed[2]
                owed = (at + place_v(i, n), i == half, int(last), keys)
                yield None
            if half >= n:
                if owed:
                    yield from wait_v()
                    yield from start_pv()
                    rest_pv()
                    npv, no, owed = npv + 1, no + owed[2], None
                yield q_full(qp)
                later(f"mma{h}", lambda qp=qp: B[f"q_empty{qp & 1}"].arrive())
            at += 2 * n
            qn += 1 if keys else 2
        if owed:
            yield from wait_v()
            yield from start_pv()
            rest_pv()

    def softmax(h):
        at = ns = no = qn = 0
        for got in tiles_of():
            if got[0] == "wait":
                yield got
                continue
            if got[1] is None:
                break
            n, keys, edge = got[1]
            mine = False
            half = h ^ (qn & 1) if keys else 0
            qn += 1 if keys else 2
            for i in range(half, n, 2 if keys else 1):
                yield ("wait", B[f"s_full{h}"], ns & 1)
                ns += 1
                assert S[h] == ("S",)
                if edge and i in (0, n - 1):
                    pl = at + place_v(i, n)
                    yield kv_full(pl)
                    assert stage[pl % STAGES] == pl, "rows cleared in another block's stage"
                if mine:
                    assert O[h] == "acc", "O rescaled while a product writes it"
                S[h] = ("half",)
                B[f"p_half{h}"].arrive()
                yield None
                S[h] = ("P",)
                B[f"p_full{h}"].arrive()
                mine = True
            at += 2 * n
            if mine:
                yield ("wait", B[f"o_full{h}"], no & 1)
                no += 1
                assert O[h] == "done"
                O[h] = "read"
                if keys > 1:  # the copies joined in the last V's stage
                    yield None
                    pl = at - 2 * n + place_v(((n - 1 - half) & ~1) + half, n)
                    assert stage[pl % STAGES] == pl
                    reads[pl] -= 1
                    for _x in range(2):
                        B[f"kv_empty{pl % STAGES}"].arrive()
                B[f"o_empty{h}"].arrive()
                finished[h] += 1

    # products still to read a place or a q buffer, by number
    at = qn = 0
    for n, keys, _ in segs:
        for i in range(n):
            reads[at + place_k(i)] = reads[at + place_v(i, n)] = 1 if keys else 2
        for x in range(1 if keys else 2):
            qreads[qn + x] = n
        at += 2 * n
        qn += 1 if keys else 2
    roles = {"c": scheduler(), "p": producer(), "m0": issuer(0), "m1": issuer(1), "s0": softmax(0), "s1": softmax(1)}
    blocked = dict.fromkeys(roles)
    while roles or any(pending.values()):
        ready = [k for k in roles if blocked[k] is None or blocked[k][1].ready(blocked[k][2])]
        sources = [k for k, v in pending.items() if v]
        assert ready or sources, f"deadlock: {segs} {blocked}"
        k = rnd.choice(ready + sources)
        if k in sources and k not in roles:
            pending[k].pop(0)()
            continue
        try:
            blocked[k] = next(roles[k])
        except StopIteration:
            del roles[k]
    assert sum(finished) >= len(segs) and all(v == 0 for v in reads.values())


@pytest.mark.parametrize("seed", range(40))
def test_forward_protocol(seed):
    r = random.Random(seed)
    for x in range(8):
        segs = [(r.choice([1, 1, 2, 3, r.randint(1, 9), r.randint(8, 26)]), r.choice([0, 0, 1, 4, 4]), r.random() < 0.5)
                for _ in range(r.randint(1, 7))]
        run_protocol([(1, 0, True), (1, 2, True), (1, 4, True)] + segs, seed * 100 + x)  # (the tiles before the plan)
