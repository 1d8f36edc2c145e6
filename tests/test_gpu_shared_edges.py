"""mxsa_dense_shared_fwd at its edges: values that are not finite, and the plan
that its workspace holds after a call against the model of it."""
import numpy as np
import pytest
import torch

from tests.test_gpu_shared import CASES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["decode", "two_row_tiles", "decode_aligned"])
def test_an_infinity_in_v_stays_in_its_column(name):
    """A prefix key's V holds an infinity: that column of the kv head's rows is not finite, nothing else changes."""
    c = Case(**CASES[name], seed=1).run().check()
    good, lse = c.out.clone(), c.lse.clone()
    page, off = (x[50] for x in c.slots[0])
    c.v[page, 0, off, 7] = float("inf")
    c.run()
    torch.cuda.synchronize()
    G = c.hq // c.hkv
    assert not c.out[:, :G, 7].isfinite().any()
    same = torch.ones_like(c.out, dtype=torch.bool)
    same[:, :G, 7] = False
    assert torch.equal(c.out[same], good[same]) and torch.equal(c.lse, lse)


def words(ws, at, count, dtype=torch.int32):
    return ws[at:at + count * dtype.itemsize].view(dtype).cpu().tolist()


@pytest.mark.parametrize("name", list(CASES))
def test_the_plan_is_its_models(name):
    """Tiles, pieces, tokens and queues in the workspace against tests/test_shared_models.py's plan."""
    from tests.test_shared_models import MAXC, TILE, WK, WR, plan
    from tests.test_shared_workspace import layout

    c = Case(**CASES[name], seed=1).run()
    torch.cuda.synchronize()
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, MAXC)
    p = dict(cu=c.cu, lens=c.lens, gp=c.gp or [0], prefix=c.prefix or [], hq=c.hq, hkv=c.hkv, causal=c.causal,
             ctas=ctas, total_q=c.total)
    tiles, part = plan(p)
    L, G = layout(c.prob), c.hq // c.hkv
    T2 = 2 * (128 // G)
    assert part <= L["row_cap"] and len(tiles) <= L["tile_cap"]

    def row_of(job):
        if job["own"]:
            return max(s for s in range(c.B) if c.cu[s] == job["tok0"])
        return next(a for a, b in zip(c.gp, c.gp[1:]) if c.cu[b] > c.cu[a] == job["tok0"])

    want = [[], []]
    pieces = []
    for t in tiles:
        keys = t["keys"]
        pieces += [t["part0"], t["tok0"], t["ntok"], min(t["n"], 2 if keys else 1)]
        if t["n"]:
            rows = t["ntok"] * G
            copies = 0 if not keys else 1 if t["ntok"] > 8 or rows > 64 else 2 if rows > 32 else 4
            want[keys].append([t["tok0"], t["ntok"], t["g"], row_of(t["job"]), t["lo"], t["hi"], t["b0"], t["n"],
                               t["part0"], 0, copies])
    assert words(c.ws, L["pieces"], len(pieces)) == pieces
    count = words(c.ws, L["hdr"], 6)
    assert count[:2] == [len(want[0]), len(want[1])]
    for k in range(2):
        q = words(c.ws, L["queue"] + 48 * L["tile_cap"] * k, 12 * len(want[k]))
        assert [q[i:i + 11] for i in range(0, len(q), 12)] == want[k]
    # CTAs that begin with each queue
    cost = [0, 0]
    for j in {id(t["job"]): t["job"] for t in tiles}.values():
        keys = int(0 < j["ntok"] % T2 <= T2 // 2)
        cost[0] += c.hkv * (j["nrt"] - keys) * (j["nb"] * WR + TILE)
        cost[1] += c.hkv * keys * (j["nb"] * WK + TILE)
    with1 = min(max(cost[1] * ctas * 5 // 8 // max(sum(cost), 1), 1), ctas - 1)
    with1 = 0 if not want[1] else ctas if not want[0] else with1
    assert count[4:] == [ctas - with1, with1]
    # tokens
    got = words(c.ws, L["tok"], 8 * c.total)
    jobs = {(t["job"]["own"], row_of(t["job"])): t["job"] for t in tiles}
    for i in range(c.total):
        inside = c.cu[0] <= i < c.cu[-1]
        s = max((s for s in range(c.B) if c.cu[s] <= i), default=-1) if inside else -1
        expect = [-1] + [0] * 7
        if s >= 0:
            seen = min(max(c.lens[s] - (c.cu[s + 1] - i) + 1, 0), c.lens[s]) if c.causal else c.lens[s]
            expect[:2] = [s, seen]
            group = next((a for a, b in zip(p["gp"], p["gp"][1:]) if a <= s < b), -1)
            for at, key in ((2, (True, s)), (5, (False, group))):
                j = jobs.get(key)
                if j:
                    expect[at:at + 3] = [j["tile0"] + (i - j["tok0"]) // T2, j["nch"], j["nrt"]]
        assert got[8 * i:8 * i + 8] == expect, i
